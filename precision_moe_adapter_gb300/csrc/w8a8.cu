// w8a8.cu -- 8-bit linear layers: quantisation per row and block of 128 columns,
// the transposed weight of the gradient, the product's launches and the dense
// layer with the orthogonal adapter around them (w8a8_gemm.cuh has the product).
#include <cstring>

#include "w8a8_gemm.cuh"

namespace pmoe {
namespace tc {
bool make_rows_tmap(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int box_rows);
bool make_bytes_tmap(CUtensorMap *m, const void *base, int64_t rows, int64_t row_bytes, int box_bytes, int box_rows,
                     int swizzle_bytes, int l2_promote = 256);
bool make_f32_tmap(CUtensorMap *m, const void *base, int64_t planes, int64_t rows, int64_t cols);
void take_wait_hook(uint64_t &wait_ns, int &skip_item);
}  // namespace tc
namespace w8 {

constexpr int kSms = 152;   // SMs of a GB300

// ------------------------------------------------------------------ quantisation
// Bound by HBM: 2 bytes read and 1 written per element.  A half-warp holds one
// block of a row, 8 values a lane.
//
// q is the exact quotient 448 x / a rounded to E4M3.  x and a are BF16 numbers, so a
// quotient that is not one of E4M3's rounding midpoints is at least 2^-13 of itself
// away from all of them (their products with a are integers of at most 12 bits on one
// scale): the FP32 product with 448 / a, two roundings from it, is rounded to 16
// bits first, which takes it back to a midpoint that it stands for, and across none.
constexpr int kQThreads = 256;
constexpr int kQBlocks = 4;   // blocks a half-warp has in flight

__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t x)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x & 0x7FFF7FFFu));
    return r;
}
__device__ __forceinline__ float to_16_bits(float p)
{
    return __uint_as_float((__float_as_uint(p) + 0x80u) & 0xFFFFFF00u);
}
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1), "f"(x0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3), "f"(x2));
    return (uint32_t)lo | (uint32_t)hi << 16;
}

template <bool POW2>
__global__ void __launch_bounds__(kQThreads) k_fp8_quantize(int rows, int K, int KB, const uint16_t *__restrict__ X,
                                                            uint8_t *__restrict__ q, float *__restrict__ s)
{
    grid_wait();
    grid_go();
    const int lane = threadIdx.x & 15;
    const uint32_t nblk = (uint32_t)rows * KB;   // (< 2^31: more would not fit the memory)
    const uint32_t per = gridDim.x * (kQThreads / 16);
    for (uint32_t b0 = blockIdx.x * (kQThreads / 16) + threadIdx.x / 16; b0 < ((nblk + 1) & ~1u);
         b0 += per * kQBlocks) {
        uint4 u[kQBlocks];
        int64_t row[kQBlocks];
        int kb[kQBlocks];
#pragma unroll
        for (int i = 0; i < kQBlocks; ++i) {
            const uint32_t b = b0 + i * per;
            row[i] = b / (uint32_t)KB;
            kb[i] = (int)(b % (uint32_t)KB);
            const int c = kb[i] * 128 + lane * 8;
            u[i] = make_uint4(0, 0, 0, 0);
            if (b < nblk && c < K) u[i] = __ldcs((const uint4 *)(X + row[i] * K + c));
        }
#pragma unroll
        for (int i = 0; i < kQBlocks; ++i) {
            uint32_t m = absmax2(absmax2(u[i].x & 0x7FFF7FFFu, u[i].y), absmax2(u[i].z & 0x7FFF7FFFu, u[i].w));
#pragma unroll
            for (int o = 8; o; o >>= 1) m = absmax2(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = absmax2(m, m >> 16 | m << 16);
            float a = __uint_as_float(m << 16);
            a = a < 7.8886091e-31f ? 7.8886091e-31f : a;   // 2^-100; a NaN stays
            float sc = a / 448.f, r;
            if constexpr (POW2) {
                // (a / 448 in FP32 is a power of two only where the quotient is: 448 = 7 * 2^6)
                const uint32_t e = (__float_as_uint(sc) + 0x7FFFFFu) & 0x7F800000u;
                sc = a <= 3.4e38f ? __uint_as_float(e) : a;
                r = 1.f / sc;
            } else {
                r = 448.f / a;
            }
            if (!(a <= 3.4e38f)) sc = __int_as_float(0x7fffffff);   // an infinity makes its block NaN too
            const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = to_16_bits(__uint_as_float(w[j] << 16) * r);
                v[2 * j + 1] = to_16_bits(__uint_as_float(w[j] & 0xFFFF0000u) * r);
            }
            const uint32_t b = b0 + i * per;
            const int c = kb[i] * 128 + lane * 8;
            if (b < nblk && c < K) {
                *(uint2 *)(q + row[i] * K + c) = make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
                if (lane == 0) s[(int64_t)kb[i] * rows + row[i]] = sc;
            }
        }
    }
}

// ------------------------------------------------------------------ transpose
// 64 x 64 codes at a time through shared memory (once per weight)
__global__ void __launch_bounds__(256) k_fp8_transpose(int N, int K, const uint8_t *__restrict__ q,
                                                       const float *__restrict__ s, uint8_t *__restrict__ qt,
                                                       float *__restrict__ st)
{
    __shared__ uint8_t tile[64][68];
    const int n0 = blockIdx.y * 64, k0 = blockIdx.x * 64;
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
        const int n = i / 16, k = i % 16 * 4;
        uint32_t v = 0;
        if (n0 + n < N && k0 + k < K) v = *(const uint32_t *)(q + (int64_t)(n0 + n) * K + k0 + k);
        *(uint32_t *)&tile[n][k] = v;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
        const int k = i / 16, n = i % 16 * 4;
        if (k0 + k < K && n0 + n < N)
            *(uint32_t *)(qt + (int64_t)(k0 + k) * N + n0 + n) =
                (uint32_t)tile[n][k] | (uint32_t)tile[n + 1][k] << 8 | (uint32_t)tile[n + 2][k] << 16 |
                (uint32_t)tile[n + 3][k] << 24;
    }
    if (threadIdx.x == 0 && n0 % 128 == 0 && k0 % 128 == 0) {
        const int KB = (K + 127) / 128, NB = (N + 127) / 128;
        st[(int64_t)(k0 / 128) * NB + n0 / 128] = s[(int64_t)(n0 / 128) * KB + k0 / 128];
    }
}

// ------------------------------------------------------------------ product
// out = sum of the splits' FP32 sums, in order; a thread 4 columns
template <bool F32>
__global__ void __launch_bounds__(256) k_w8_sum(int64_t n, int splits, const float *__restrict__ part,
                                                void *__restrict__ out)
{
    grid_wait();
    grid_go();
    const int64_t i = (blockIdx.x * 256ll + threadIdx.x) * 4;
    if (i >= n) return;
    float4 a = *(const float4 *)(part + i);
#pragma unroll 4
    for (int s = 1; s < splits; ++s) {
        const float4 x = *(const float4 *)(part + s * n + i);
        a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    }
    if constexpr (F32) *(float4 *)((float *)out + i) = a;
    else *(uint2 *)((uint16_t *)out + i) = make_uint2(hg::bf2(a.x, a.y), hg::bf2(a.z, a.w));
}

struct Tiling {
    int ctas, mt, nt, gm, splits, kper;
};
static Tiling tiling(int64_t M, int64_t N, int64_t ksteps)
{
    Tiling t;
    t.ctas = cdiv(M, 256) * cdiv(N, 256) >= kSms / 2 && M > 128 ? 2 : 1;
    t.mt = (int)cdiv(M, 128 * t.ctas);
    t.nt = (int)cdiv(N, 128 * t.ctas);
    // m tiles that run together: their rows of A stay in the L2 while the n tiles pass
    const int64_t stripe = 128ll * t.ctas * ksteps * kStep;
    const int64_t most = std::max<int64_t>(8, (48ll << 20) / std::max<int64_t>(stripe, 1));
    t.gm = (int)cdiv(t.mt, cdiv(t.mt, most));
    // few tiles: the blocks of K are shared out, so that every SM streams a part of W
    const int64_t tiles = (int64_t)t.mt * t.nt;
    const int64_t want = std::max<int64_t>(1, std::min(kSms / t.ctas / tiles, cdiv(ksteps, 4)));
    t.kper = (int)cdiv(ksteps, want);
    t.splits = (int)cdiv(ksteps, t.kper);
    return t;
}
static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
// Most FP32 values of the splits' sums, for up to `rows` rows: there are at most
// kSms items of 128 x 128, and one for every four blocks of K
static size_t part_elems(int64_t rows, int64_t N, int64_t K)
{
    const int64_t splits = std::min<int64_t>(kSms, cdiv(cdiv(K, kStep), 4));
    return splits < 2 ? 0 : (size_t)std::min<int64_t>(splits * rows * N, (int64_t)kSms * 128 * 128);
}

template <int CTAS, int BN>
static bool launch_as(const CUtensorMap &ma, const CUtensorMap &mt, const CUtensorMap &mb, const CUtensorMap &mo,
                      const Args &a, cudaStream_t st)
{
    constexpr auto kern = k_w8_gemm<CTAS, BN>;
    if (!set_attribute<kern, cudaFuncAttributeMaxDynamicSharedMemorySize>(smem_of(BN))) return false;
    const int64_t items = (int64_t)a.mt * a.nt * a.splits;
    const int64_t clusters = std::min<int64_t>(items, gemm_num_sms() / CTAS);
    return launch_chained<kern>((unsigned)(clusters * CTAS), threads_of(BN), smem_of(BN), CTAS, st, ma, mt, mb, mo, a);
}

static bool product(int rows, int N, int K, const void *A, const float *As, const void *W, const float *Ws, void *out,
                    bool out_f32, float *part, DevErr *err, cudaStream_t st)
{
    const int ksteps = (int)cdiv(K, kStep);
    const Tiling t = tiling(rows, N, ksteps);
    Args a{};
    a.M = rows;
    a.N = N;
    a.mt = t.mt;
    a.nt = t.nt;
    a.gm = t.gm;
    a.ksteps = ksteps;
    a.splits = t.splits;
    a.kper = t.kper;
    a.tail = rows % 128;
    a.abytes = rows < 128 ? (int)cdiv(a.tail, 8) * 1024 : kOpBytes;
    a.stages = std::min(kMaxStages, kRingBytes / (kOpBytes + a.abytes));
    a.As = As;
    a.Ws = Ws;
    a.f32_out = t.splits > 1 || out_f32;
    a.err = err;
    tc::take_wait_hook(a.wait_ns, a.skip_item);
    CUtensorMap ma, mt, mb, mo;
    memset(&ma, 0, sizeof ma);
    memset(&mt, 0, sizeof mt);
    if (rows >= 128 && !tc::make_bytes_tmap(&ma, A, rows, K, kStep, 128, 128)) return false;
    if (a.tail && !tc::make_bytes_tmap(&mt, A, rows, K, kStep, a.tail, 128)) return false;
    if (!tc::make_bytes_tmap(&mb, W, N, K, kStep, 128, 128)) return false;
    float *f32 = t.splits > 1 ? part : (float *)out;
    if (a.f32_out ? !tc::make_f32_tmap(&mo, f32, t.splits, rows, N) : !tc::make_rows_tmap(&mo, out, rows, N, 32))
        return false;
    if (!(t.ctas == 2 ? launch_as<2, 256>(ma, mt, mb, mo, a, st) : launch_as<1, 128>(ma, mt, mb, mo, a, st))) return false;
    if (t.splits == 1) return true;
    const int64_t n = (int64_t)rows * N;
    const unsigned grid = (unsigned)cdiv(n, 1024);
    return out_f32 ? launch_chained<k_w8_sum<true>>(grid, 256, 0, 1, st, n, t.splits, (const float *)part, out)
                   : launch_chained<k_w8_sum<false>>(grid, 256, 0, 1, st, n, t.splits, (const float *)part, out);
}

static bool quantize(int rows, int K, const void *X, bool pow2, void *q, float *s, cudaStream_t st)
{
    const int KB = (int)cdiv(K, 128);
    const int64_t ctas = cdiv((int64_t)rows * KB, kQThreads / 16 * (int64_t)kQBlocks);
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(ctas, (int64_t)gemm_num_sms() * 32));
    return pow2 ? launch_chained<k_fp8_quantize<true>>(grid, kQThreads, 0, 1, st, rows, K, KB, (const uint16_t *)X,
                                                       (uint8_t *)q, s)
                : launch_chained<k_fp8_quantize<false>>(grid, kQThreads, 0, 1, st, rows, K, KB, (const uint16_t *)X,
                                                        (uint8_t *)q, s);
}

static bool dim_ok(int64_t v) { return v > 0 && v <= (1 << 20) && v % 16 == 0; }
static bool shape_ok(int rows, int N, int K)
{
    return rows >= 0 && rows <= (1 << 24) && dim_ok(N) && dim_ok(K) && (int64_t)rows * cdiv(std::max(N, K), 128) < (1ll << 30);
}
static bool block_ok(int b) { return b == 16 || b == 32 || b == 64 || b == 128; }
static bool a16(const void *p) { return ((uintptr_t)p & 15) == 0; }

struct Ws {
    DevErr *err;
    uint8_t *q;      // [rows][max(N, K)]
    float *s;        // [blocks][rows]
    float *part;     // the splits' sums, of either direction
    float *buf;      // adapter: x~ (BF16) or dx~ (FP32), [rows][K]
    size_t bytes;
};
static Ws carve(void *ws, int64_t rows, int64_t N, int64_t K, bool dense, bool adapter)
{
    Ws w;
    uint8_t *base = (uint8_t *)ws;
    size_t off = kHdrBytes;
    auto take = [&](size_t bytes) {
        uint8_t *p = base ? base + off : nullptr;
        off = up256(off + bytes);
        return p;
    };
    w.err = (DevErr *)ws;
    const int64_t most = std::max(N, K);
    w.q = dense ? take((size_t)rows * most) : nullptr;
    w.s = dense ? (float *)take((size_t)rows * cdiv(most, 128) * 4) : nullptr;
    size_t parts = part_elems(rows, N, K);
    if (dense) parts = std::max(parts, part_elems(rows, K, N));
    w.part = (float *)take(parts * 4);
    w.buf = adapter ? (float *)take((size_t)rows * K * 4) : nullptr;
    w.bytes = off;
    return w;
}
static RotCall rotation(int b, bool trans, const void *src, bool src_f32, const void *R, int rows, int K, void *out)
{
    RotCall c{};
    c.b = b;
    c.trans = trans;
    c.src = src;
    c.src_f32 = src_f32;
    c.src_ld = K;
    c.k = 1;
    c.R = (const uint16_t *)R;
    c.dim = K;
    c.out = out;
    c.out_ld = K;
    c.nrows = rows;
    return c;
}
// Checks of the dense layer's calls; PMOE_OK to go on
static pmoe_status check_dense(const void *q, const float *s, int N, int K, int block, const void *R, int rows)
{
    if (!shape_ok(rows, N, K) || !q || !s || !a16(q) || !a16(s) || !a16(R)) return PMOE_ERR_INVALID_ARG;
    if (R && (!block_ok(block) || K % block || K % 64)) return PMOE_ERR_INVALID_ARG;
    return PMOE_OK;
}

}  // namespace w8
}  // namespace pmoe

using namespace pmoe;

extern "C" {

pmoe_status fp8_quantize(int32_t rows, int32_t K, const void *X, int pow2, void *q, float *s, cudaStream_t stream)
{
    if (!w8::shape_ok(rows, 16, K) || (rows > 0 && (!X || !q || !s)) || !w8::a16(X) || !w8::a16(q) || !w8::a16(s))
        return PMOE_ERR_INVALID_ARG;
    if (rows == 0) return PMOE_OK;
    return w8::quantize(rows, K, X, pow2 != 0, q, s, stream) ? PMOE_OK : PMOE_ERR_CUDA;
}

pmoe_status fp8_transpose(int32_t N, int32_t K, const void *q, const float *s, void *qt, float *st, cudaStream_t stream)
{
    if (!w8::shape_ok(0, N, K) || !q || !s || !qt || !st || !w8::a16(q) || !w8::a16(s) || !w8::a16(qt) || !w8::a16(st) ||
        q == qt || s == st)
        return PMOE_ERR_INVALID_ARG;
    w8::k_fp8_transpose<<<dim3((unsigned)cdiv(K, 64), (unsigned)cdiv(N, 64)), 256, 0, stream>>>(
        N, K, (const uint8_t *)q, s, (uint8_t *)qt, st);
    note_launch();
    return cudaPeekAtLastError() == cudaSuccess ? PMOE_OK : PMOE_ERR_CUDA;
}

size_t fp8_gemm_ws_bytes(int32_t rows, int32_t N, int32_t K)
{
    return w8::shape_ok(rows, N, K) ? w8::carve(nullptr, rows, N, K, false, false).bytes : 0;
}

pmoe_status fp8_gemm(int32_t rows, int32_t N, int32_t K, const void *A, const float *As, const void *W, const float *Ws,
                     void *Y, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    if (!w8::shape_ok(rows, N, K) || !W || !Ws || (rows > 0 && (!A || !As || !Y)) || !w8::a16(A) || !w8::a16(As) ||
        !w8::a16(W) || !w8::a16(Ws) || !w8::a16(Y))
        return PMOE_ERR_INVALID_ARG;
    const w8::Ws w = w8::carve(ws, rows, N, K, false, false);
    if (!ws || ws_bytes < w.bytes || !w8::a16(ws)) return PMOE_ERR_WORKSPACE;
    if (rows == 0) return PMOE_OK;
    return w8::product(rows, N, K, A, As, W, Ws, Y, false, w.part, w.err, stream) ? PMOE_OK : PMOE_ERR_CUDA;
}

size_t dense_w8a8_ws_bytes(int32_t rows, int32_t N, int32_t K, int adapter)
{
    return w8::shape_ok(rows, N, K) ? w8::carve(nullptr, rows, N, K, true, adapter != 0).bytes : 0;
}

pmoe_status dense_w8a8_forward(const void *q, const float *s, int32_t N, int32_t K, int32_t block, const void *R,
                               int32_t rows, const void *X, int pow2, void *Y, void *ws, size_t ws_bytes,
                               cudaStream_t stream)
{
    const pmoe_status e = w8::check_dense(q, s, N, K, block, R, rows);
    if (e != PMOE_OK) return e;
    if ((rows > 0 && (!X || !Y)) || !w8::a16(X) || !w8::a16(Y)) return PMOE_ERR_INVALID_ARG;
    const w8::Ws w = w8::carve(ws, rows, N, K, true, R != nullptr);
    if (!ws || ws_bytes < w.bytes || !w8::a16(ws)) return PMOE_ERR_WORKSPACE;
    if (rows == 0) return PMOE_OK;
    if (R) {
        launch_rotate_tc(w8::rotation(block, false, X, false, R, rows, K, w.buf), stream);
        X = w.buf;
    }
    return w8::quantize(rows, K, X, pow2 != 0, w.q, w.s, stream) &&
                   w8::product(rows, N, K, w.q, w.s, q, s, Y, false, w.part, w.err, stream) &&
                   cudaPeekAtLastError() == cudaSuccess
               ? PMOE_OK
               : PMOE_ERR_CUDA;
}

pmoe_status dense_w8a8_backward(const void *qt, const float *st, int32_t N, int32_t K, int32_t block, const void *R,
                                int32_t rows, const void *X, const void *dY, int pow2, void *dX, float *dR, void *ws,
                                size_t ws_bytes, cudaStream_t stream)
{
    const pmoe_status e = w8::check_dense(qt, st, N, K, block, R, rows);
    if (e != PMOE_OK) return e;
    if ((R && !dR) || (rows > 0 && (!dY || !dX || (R && !X))) || !w8::a16(X) || !w8::a16(dY) || !w8::a16(dX) ||
        !w8::a16(dR))
        return PMOE_ERR_INVALID_ARG;
    const w8::Ws w = w8::carve(ws, rows, N, K, true, R != nullptr);
    if (!ws || ws_bytes < w.bytes || !w8::a16(ws)) return PMOE_ERR_WORKSPACE;
    if (rows == 0)
        return !R || cudaMemsetAsync(dR, 0, (size_t)K * block * sizeof(float), stream) == cudaSuccess ? PMOE_OK
                                                                                                      : PMOE_ERR_CUDA;
    // dx~ in FP32 where an adapter follows, as in dense_linear_backward
    if (!w8::quantize(rows, N, dY, pow2 != 0, w.q, w.s, stream) ||
        !w8::product(rows, K, N, w.q, w.s, qt, st, R ? (void *)w.buf : dX, R != nullptr, w.part, w.err, stream))
        return PMOE_ERR_CUDA;
    if (R) {
        launch_outer_tc(1, rows, K, block, (const uint16_t *)X, K, false, nullptr, 1, w.buf, true, K, nullptr, dR, stream);
        launch_rotate_tc(w8::rotation(block, true, w.buf, true, R, rows, K, dX), stream);
    }
    return cudaPeekAtLastError() == cudaSuccess ? PMOE_OK : PMOE_ERR_CUDA;
}

}  // extern "C"
