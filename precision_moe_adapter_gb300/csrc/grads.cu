// grads.cu -- the global norm of a list of gradients and clipping by it.
//
//   norm = sqrt(sum over all tensors of g^2)      coef = min(1, max_norm / (norm + 1e-6))
//   dst = g coef
//
// Bound by HBM: the norm reads every gradient once, the clip reads it again
// and writes it.  (The coefficient needs the last gradient's square before the
// first one can be scaled, so two reads it is, but for what the L2 still holds.)  906 MB
// of f32 in two tensors take 421 us, 6.5 TB/s of these 2.7 GB (0.95 of a copy's rate); 691 MB
// in 60 tensors, half of them BF16, 261 us.  Chunks go round the CTAs in turn, as BF16 ones
// take longer: with a run of chunks for each CTA the latter took 300 us.
#include <algorithm>
#include <cmath>
#include <vector>

#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace pmoe {
namespace gr {

// A list entry as the kernels read it; chunk0 is the number of chunks before it
struct Entry {
    const void *src;
    void *dst;
    int64_t n;
    int64_t chunk0;
    int32_t dtype;
    int32_t pad;
};
constexpr int kThreads = 256;
constexpr int kVecs = 8;                                  // 16-byte loads a thread has in flight
constexpr int64_t kChunkBytes = kThreads * kVecs * 16;    // 32 KB
constexpr int kCtasPerSm = 4;                             // (64 registers a thread)
constexpr int kMaxParts = 4096;                           // partial sums in the workspace
constexpr size_t kWsBytes = kHdrBytes + kMaxParts * sizeof(double);

__host__ __device__ inline int64_t chunk_elems(int dtype) { return kChunkBytes / (dtype == PMOE_GRAD_F32 ? 4 : 2); }
__host__ __device__ inline int64_t chunks_of(int64_t n, int dtype) { return cdiv(n, chunk_elems(dtype)); }

// Entry that holds chunk c, the last one with chunk0 <= c (entries without elements have
// no chunk): a whole warp looks at 32 entries at a time
__device__ __forceinline__ int find(const Entry *e, int n, int64_t c)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n;
    while (len > 1) {
        const int step = (len + 31) / 32, at = lane * step;
        const uint32_t b = __ballot_sync(0xffffffffu, at < len && e[lo + min(at, len - 1)].chunk0 <= c);
        const int last = b ? 31 - __clz((int)b) : 0;   // (the first one always is)
        len = min(step, len - last * step);
        lo += last * step;
    }
    return lo;
}

template <bool BF16>
__device__ __forceinline__ void unpack(uint4 u, float *x)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            x[i] = __uint_as_float(w[i]);
        }
    }
}

// Whether a sum of squares formed in FP32 stands: it neither overflowed nor is it so
// small that its terms may have lost bits below the normal range
__device__ __forceinline__ bool stands(float s) { return s >= 8.0779357e-28f && s < __int_as_float(0x7f800000); }   // 2^-90
// Sum of a vector's squares; where FP32 does not do, in FP64 (the products of FP32
// numbers are exact there)
template <int N>
__device__ __forceinline__ float squares32(const float *x)
{
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(x[i], x[i], s);
    return s;
}
template <int N>
__device__ __forceinline__ double squares(const float *x)
{
    const float s = squares32<N>(x);
    if (stands(s)) return (double)s;
    double d = 0.;
#pragma unroll
    for (int i = 0; i < N; ++i) d = fma((double)x[i], (double)x[i], d);
    return d;
}

// Sum over the CTA in a fixed order; valid in thread 0
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double sh[kThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = threadIdx.x < kThreads / 32 ? sh[threadIdx.x] : 0.;
#pragma unroll
        for (int o = kThreads / 64; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}

template <bool BF16>
__device__ __forceinline__ double chunk_squares(const void *src, int64_t at, int64_t n)
{
    constexpr int kE = BF16 ? 8 : 4;   // elements of a vector
    const int64_t left = n - at;
    const uint4 *p = (const uint4 *)((const uint8_t *)src + at * (BF16 ? 2 : 4));
    double d = 0.;
    float x[kE];
    if (left >= (int64_t)kThreads * kVecs * kE) {
        uint4 u[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) u[i] = p[i * kThreads + threadIdx.x];
        // one FP64 addition for the thread's 8 vectors (one for each made the kernel
        // FP64-bound: 906 MB took 180 us, the FP64 units having 2 lanes an SM)
        float s[kVecs];
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            unpack<BF16>(u[i], x);
            s[i] = squares32<kE>(x);
            any |= u[i].x | u[i].y | u[i].z | u[i].w;
        }
#pragma unroll
        for (int h = kVecs / 2; h; h /= 2) {
#pragma unroll
            for (int i = 0; i < h; ++i) s[i] += s[i + h];
        }
        if (stands(s[0])) return (double)s[0];
        if ((any & (BF16 ? 0x7fff7fffu : 0x7fffffffu)) == 0) return 0.;
#pragma unroll 1
        for (int i = 0; i < kVecs; ++i) {   // (read again: rare, and it keeps the registers free)
            unpack<BF16>(p[i * kThreads + threadIdx.x], x);
            d += squares<kE>(x);
        }
        return d;
    }
    const int nv = (int)(left / kE);   // whole vectors, then single elements
    for (int i = threadIdx.x; i < nv; i += kThreads) {
        unpack<BF16>(p[i], x);
        d += squares<kE>(x);
    }
    const int e = nv * kE + threadIdx.x;
    if (e < left) {
        const float v = BF16 ? bf2f(((const uint16_t *)src)[at + e]) : ((const float *)src)[at + e];
        d = fma((double)v, (double)v, d);
    }
    return d;
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) k_grad_squares(const Entry *__restrict__ list, int n, int64_t chunks,
                                                           double *__restrict__ parts)
{
    grid_wait();
    grid_go();
    double d = 0.;
    int64_t end = 0;
    Entry e{};
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        if (c >= end) {
            e = list[find(list, n, c)];
            end = e.chunk0 + chunks_of(e.n, e.dtype);
        }
        const int64_t at = (c - e.chunk0) * chunk_elems(e.dtype);
        d += e.dtype == PMOE_GRAD_F32 ? chunk_squares<false>(e.src, at, e.n) : chunk_squares<true>(e.src, at, e.n);
    }
    d = block_sum(d);
    if (threadIdx.x == 0) parts[blockIdx.x] = d;
}

// The norm from the partial sums, in the same order in every CTA
__device__ __forceinline__ double norm_of(const double *parts, int nparts)
{
    __shared__ double total;
    double d = 0.;
    for (int i = threadIdx.x; i < nparts; i += kThreads) d += __ldcg(parts + i);
    d = block_sum(d);
    if (threadIdx.x == 0) total = sqrt(d);
    __syncthreads();
    return total;
}

__global__ void __launch_bounds__(kThreads) k_grad_norm(const double *__restrict__ parts, int nparts,
                                                        float *__restrict__ norm)
{
    grid_wait();
    grid_go();
    const double v = norm_of(parts, nparts);
    if (threadIdx.x == 0) *norm = (float)v;
}

template <bool BF16>
__device__ __forceinline__ uint4 scaled(uint4 u, float c)
{
    float x[BF16 ? 8 : 4];
    unpack<BF16>(u, x);
    if constexpr (BF16)
        return make_uint4(pack_bf2(x[0] * c, x[1] * c), pack_bf2(x[2] * c, x[3] * c), pack_bf2(x[4] * c, x[5] * c),
                          pack_bf2(x[6] * c, x[7] * c));
    else
        return make_uint4(__float_as_uint(x[0] * c), __float_as_uint(x[1] * c), __float_as_uint(x[2] * c),
                          __float_as_uint(x[3] * c));
}
template <bool BF16>
__device__ __forceinline__ void chunk_scale(const void *src, void *dst, int64_t at, int64_t n, float coef)
{
    constexpr int kE = BF16 ? 8 : 4;
    const int64_t left = n - at;
    const uint4 *p = (const uint4 *)((const uint8_t *)src + at * (BF16 ? 2 : 4));
    uint4 *q = (uint4 *)((uint8_t *)dst + at * (BF16 ? 2 : 4));
    if (left >= (int64_t)kThreads * kVecs * kE) {
        uint4 u[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) u[i] = __ldcs(p + i * kThreads + threadIdx.x);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) __stcs(q + i * kThreads + threadIdx.x, scaled<BF16>(u[i], coef));
        return;
    }
    const int nv = (int)(left / kE);
    for (int i = threadIdx.x; i < nv; i += kThreads) q[i] = scaled<BF16>(p[i], coef);
    const int e = nv * kE + threadIdx.x;
    if (e < left) {
        if constexpr (BF16) ((uint16_t *)dst)[at + e] = f2bf(bf2f(((const uint16_t *)src)[at + e]) * coef);
        else ((float *)dst)[at + e] = ((const float *)src)[at + e] * coef;
    }
}

// The chunks from the last one back: what k_grad_squares read last may still be in the L2
__global__ void __launch_bounds__(kThreads, kCtasPerSm) k_grad_scale(const Entry *list, int n, int64_t chunks,
                                                         const double *__restrict__ parts, int nparts, float max_norm,
                                                         float *__restrict__ norm)
{
    grid_wait();
    grid_go();
    const double v = norm_of(parts, nparts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
    const double ratio = (double)max_norm / (v + 1e-6);
    const float coef = ratio >= 1. ? 1.f : (float)ratio;   // (a NaN stays one)
    int64_t first = chunks;
    Entry e{};
    for (int64_t c = chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
        if (c < first) {
            e = list[find(list, n, c)];
            first = e.chunk0;
        }
        if (coef == 1.f && e.src == e.dst) continue;
        const int64_t at = (c - e.chunk0) * chunk_elems(e.dtype);
        if (e.dtype == PMOE_GRAD_F32) chunk_scale<false>(e.src, e.dst, at, e.n, coef);
        else chunk_scale<true>(e.src, e.dst, at, e.n, coef);
    }
}

static int grid_of(int64_t chunks)
{
    return (int)std::max<int64_t>(1, std::min<int64_t>({chunks, (int64_t)gemm_num_sms() * kCtasPerSm, kMaxParts}));
}
static bool list_ok(const pmoe_grad_list &l)
{
    return l.n >= 0 && l.chunks >= 0 && (l.n == 0 ? l.chunks == 0 : l.table != nullptr) && ((uintptr_t)l.table & 15) == 0;
}
static pmoe_status check(const pmoe_grad_list &l, const float *norm, const void *ws, size_t ws_bytes)
{
    if (!list_ok(l) || !norm || ((uintptr_t)norm & 3)) return PMOE_ERR_INVALID_ARG;
    if (!ws || ws_bytes < kWsBytes || ((uintptr_t)ws & 15)) return PMOE_ERR_WORKSPACE;
    return PMOE_OK;
}
static bool launch_squares(const pmoe_grad_list &l, double *parts, cudaStream_t st)
{
    return launch_chained<k_grad_squares>((unsigned)grid_of(l.chunks), kThreads, 0, 1, st, (const Entry *)l.table, l.n,
                                          l.chunks, parts);
}

}  // namespace gr
}  // namespace pmoe

using namespace pmoe;

extern "C" {

size_t grad_list_bytes(int32_t n) { return n < 0 ? 0 : std::max<size_t>(16, (size_t)n * sizeof(gr::Entry)); }

pmoe_status grad_list_fill(int32_t n, const pmoe_grad *grads, void *table, size_t bytes, pmoe_grad_list *list)
{
    if (n < 0 || !list || (n > 0 && (!grads || !table))) return PMOE_ERR_INVALID_ARG;
    if (bytes < grad_list_bytes(n)) return PMOE_ERR_WORKSPACE;
    struct Span {
        uintptr_t a, b;
        int32_t i;
    };
    std::vector<Span> dst;
    try {
        dst.reserve((size_t)n);
    } catch (...) {
        return PMOE_ERR_WORKSPACE;
    }
    for (int32_t i = 0; i < n; ++i) {
        const pmoe_grad &g = grads[i];
        if (g.dtype != PMOE_GRAD_F32 && g.dtype != PMOE_GRAD_BF16) return PMOE_ERR_INVALID_ARG;
        if (g.n < 0 || g.n > (1ll << 40) || (g.n > 0 && (!g.src || !g.dst))) return PMOE_ERR_INVALID_ARG;
        if (((uintptr_t)g.src & 15) || ((uintptr_t)g.dst & 15)) return PMOE_ERR_INVALID_ARG;
        const uintptr_t size = (uintptr_t)g.n * (g.dtype == PMOE_GRAD_F32 ? 4 : 2);
        if (size) dst.push_back({(uintptr_t)g.dst, (uintptr_t)g.dst + size, i});
    }
    // a result may lie where its own gradient is, and nowhere else on a gradient
    // or another result
    std::sort(dst.begin(), dst.end(), [](const Span &x, const Span &y) { return x.a < y.a; });
    for (size_t j = 1; j < dst.size(); ++j)
        if (dst[j].a < dst[j - 1].b) return PMOE_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i) {
        const uintptr_t a = (uintptr_t)grads[i].src;
        const uintptr_t b = a + (uintptr_t)grads[i].n * (grads[i].dtype == PMOE_GRAD_F32 ? 4 : 2);
        if (a == b) continue;
        auto it = std::upper_bound(dst.begin(), dst.end(), a, [](uintptr_t v, const Span &s) { return v < s.b; });
        for (; it != dst.end() && it->a < b; ++it)
            if (it->i != i || it->a != a) return PMOE_ERR_INVALID_ARG;
    }
    gr::Entry *e = (gr::Entry *)table;
    int64_t chunks = 0;
    for (int32_t i = 0; i < n; ++i) {
        e[i] = {grads[i].src, grads[i].dst, grads[i].n, chunks, grads[i].dtype, 0};
        chunks += gr::chunks_of(grads[i].n, grads[i].dtype);
    }
    list->table = nullptr;
    list->chunks = chunks;
    list->n = n;
    return PMOE_OK;
}

size_t grad_ws_bytes(void) { return gr::kWsBytes; }

pmoe_status grad_norm(pmoe_grad_list list, float *norm, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    const pmoe_status s = gr::check(list, norm, ws, ws_bytes);
    if (s != PMOE_OK) return s;
    double *parts = (double *)((uint8_t *)ws + kHdrBytes);
    return gr::launch_squares(list, parts, stream) &&
                   launch_chained<gr::k_grad_norm>(1, gr::kThreads, 0, 1, stream, (const double *)parts,
                                                   gr::grid_of(list.chunks), norm)
               ? PMOE_OK
               : PMOE_ERR_CUDA;
}

pmoe_status grad_clip(pmoe_grad_list list, float max_norm, float *norm, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    if (!(max_norm > 0.f) || !std::isfinite(max_norm)) return PMOE_ERR_INVALID_ARG;
    const pmoe_status s = gr::check(list, norm, ws, ws_bytes);
    if (s != PMOE_OK) return s;
    double *parts = (double *)((uint8_t *)ws + kHdrBytes);
    const int grid = gr::grid_of(list.chunks);
    return gr::launch_squares(list, parts, stream) &&
                   launch_chained<gr::k_grad_scale>((unsigned)grid, gr::kThreads, 0, 1, stream,
                                                    (const gr::Entry *)list.table, list.n, list.chunks,
                                                    (const double *)parts, grid, max_norm, norm)
               ? PMOE_OK
               : PMOE_ERR_CUDA;
}

}  // extern "C"
