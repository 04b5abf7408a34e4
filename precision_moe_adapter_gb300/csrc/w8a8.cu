// w8a8.cu -- 8-bit linear layers: quantisation per row and block of 128 columns,
// the transposed weight of the gradient, the product's launches and the dense
// layer with the orthogonal adapter around them (w8a8_gemm.cuh has the product).
#include <atomic>
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

constexpr int kSms = 152;       // SMs of a GB300
constexpr int kMaxSplits = 8;   // CTAs that share a tile: a portable cluster

// ------------------------------------------------------------------ quantisation
// Bound by HBM: 2 bytes read and 1 written per element.  Eight lanes hold one block of a
// row, 16 values each (with 16 lanes of 8 values the work per block, its maximum and scale,
// made the kernel issue-bound: 15.3 instructions an element, 18.9 us for 4096 x 7168).
//
// q is the exact quotient 448 x / a rounded to E4M3.  x and a are BF16 numbers, so a
// quotient that is not one of E4M3's rounding midpoints is at least 2^-13 of itself
// away from all of them (their products with a are integers of at most 13 bits on one
// scale).  The FP32 product with an approximate 448 / a (2^-21), 2^-16 above it, is cut
// to 16 bits: that takes it back to a midpoint that it stands for, and across none.
constexpr int kQThreads = 256;
constexpr int kQBlocks = 2;   // blocks that eight lanes have in flight

// max(|a|, |b|) of two BF16 pairs, signs left to chance; NaN if either is
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float cut16(float p) { return __uint_as_float(__float_as_uint(p) & 0xFFFFFF00u); }
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1), "f"(x0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3), "f"(x2));
    return (uint32_t)lo | (uint32_t)hi << 16;
}
// Codes of four values, given as two BF16 pairs
__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, float r)
{
    return e4m3x4(cut16(__uint_as_float(a << 16) * r), cut16(__uint_as_float(a & 0xFFFF0000u) * r),
                  cut16(__uint_as_float(b << 16) * r), cut16(__uint_as_float(b & 0xFFFF0000u) * r));
}
// a / 448, correctly rounded: the remainder of a first quotient is exact, as a has 8
// bits (checked for every BF16 number)
__device__ __forceinline__ float over_448(float a)
{
    constexpr float r = 1.f / 448.f;
    const float q = a * r;
    return fmaf(fmaf(-q, 448.f, a), r, q);
}

template <bool POW2>
__global__ void __launch_bounds__(kQThreads) k_fp8_quantize(int rows, int K, int KB, const uint16_t *__restrict__ X,
                                                            uint8_t *__restrict__ q, float *__restrict__ s)
{
    grid_wait();
    grid_go();
    const uint32_t l = threadIdx.x & 7;
    const uint32_t nblk = (uint32_t)rows * KB;   // (< 2^30)
    const uint32_t per = gridDim.x * (kQThreads / 8) * kQBlocks;
    // (all of a warp make the same turns)
    for (uint32_t w0 = (blockIdx.x * (kQThreads / 8) + threadIdx.x / 32 * 4) * kQBlocks; w0 < nblk; w0 += per) {
        const uint32_t b0 = w0 + (threadIdx.x / 8 & 3) * kQBlocks;
        const uint32_t row0 = b0 / (uint32_t)KB, kb0 = b0 % (uint32_t)KB;
        uint4 u[kQBlocks], v[kQBlocks];   // columns 8 l .. and 64 + 8 l .. of the block
        uint32_t row = row0, kb = kb0;
#pragma unroll
        for (int i = 0; i < kQBlocks; ++i) {
            const uint32_t c = kb * 128 + l * 8;
            const uint16_t *p = X + (int64_t)row * K + c;
            u[i] = v[i] = make_uint4(0, 0, 0, 0);
            if (b0 + i < nblk && c < (uint32_t)K) u[i] = __ldcs((const uint4 *)p);
            if (b0 + i < nblk && c + 64 < (uint32_t)K) v[i] = __ldcs((const uint4 *)(p + 64));
            if (++kb == (uint32_t)KB) kb = 0, ++row;
        }
        row = row0, kb = kb0;
#pragma unroll
        for (int i = 0; i < kQBlocks; ++i) {
            uint32_t m = absmax2(absmax2(absmax2(u[i].x, u[i].y), absmax2(u[i].z, u[i].w)),
                                 absmax2(absmax2(v[i].x, v[i].y), absmax2(v[i].z, v[i].w)));
#pragma unroll
            for (int o = 4; o; o >>= 1) m = absmax2(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = absmax2(m, m >> 16) & 0x7FFFu;
            float a = __uint_as_float(m << 16), r;
            a = a < 7.8886091e-31f ? 7.8886091e-31f : a;   // 2^-100; a NaN stays
            float sc = over_448(a);
            if constexpr (POW2) {
                // (a / 448 in FP32 is a power of two only where the quotient is: 448 = 7 * 2^6)
                sc = __uint_as_float((__float_as_uint(sc) + 0x7FFFFFu) & 0x7F800000u);
                r = __uint_as_float(0x7F000000u - __float_as_uint(sc));
            } else {
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(sc));   // (sc and 1 / sc are normal numbers)
            }
            r *= 1.0000152587890625f;                               // 1 + 2^-16
            if (!(a <= 3.4e38f)) sc = __int_as_float(0x7fffffff);   // an infinity makes its block NaN too
            const uint32_t c = kb * 128 + l * 8;
            uint8_t *p = q + (int64_t)row * K + c;
            if (b0 + i < nblk) {
                if (c < (uint32_t)K) *(uint2 *)p = make_uint2(codes4(u[i].x, u[i].y, r), codes4(u[i].z, u[i].w, r));
                if (c + 64 < (uint32_t)K) *(uint2 *)(p + 64) = make_uint2(codes4(v[i].x, v[i].y, r), codes4(v[i].z, v[i].w, r));
                if (l == 0) s[(int64_t)kb * rows + row] = sc;
            }
            if (++kb == (uint32_t)KB) kb = 0, ++row;
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
struct Tiling {
    int ctas, mt, nt, gm, splits, kper;
};
// Clusters of `size` CTAs of the product that run at once (they lie within a GPC, so
// fewer than SMs / size)
static int active_clusters(int size)
{
    static std::atomic<int> known[kMaxSplits + 1];
    int n = known[size].load(std::memory_order_relaxed);
    if (n) return n;
    constexpr auto kern = k_w8_gemm<1, 128>;
    if (!set_attribute<kern, cudaFuncAttributeMaxDynamicSharedMemorySize>(kSmem)) return 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = size;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) return 0;
    if (n > 0) known[size].store(n, std::memory_order_relaxed);
    return n;
}
static Tiling tiling(int64_t M, int64_t N, int64_t ksteps, bool one_order)
{
    Tiling t;
    // Pairs on 256 x 256 read each operand half as often; a step of theirs takes 7/4 of one
    // of a single CTA on 128 x 128, so it is the rounds of the GPU that decide.  us for
    // quantisation and product, singles and pairs: 512 x 4096 (K 2048, one round each) 12.7
    // and 13.8; 1024 x 4864 (two, one) 18.1 and 16.8; 2048 x 4864 (four, two) 28.2 and 26.7;
    // 1024 x 4096 (K 7168; two, one) 41.1 and 36.3.
    t.ctas = M > 128 && 7 * cdiv(cdiv(M, 256) * cdiv(N, 256), kSms / 2) <= 4 * cdiv(cdiv(M, 128) * cdiv(N, 128), kSms) ? 2 : 1;
    t.mt = (int)cdiv(M, 128 * t.ctas);
    t.nt = (int)cdiv(N, 128 * t.ctas);
    // m tiles that run together: their rows of A stay in the L2 while the n tiles pass.
    // 16384 rows, N = K = 7168: 727 us; with all of them together 800, in groups of 8 729 to 745.
    const int64_t stripe = 128ll * t.ctas * ksteps * kStep;
    const int64_t most = std::max<int64_t>(8, (48ll << 20) / std::max<int64_t>(stripe, 1));
    t.gm = (int)cdiv(t.mt, cdiv(t.mt, most));
    // Few tiles: the blocks of K are shared out among the CTAs of a cluster.  A step takes
    // 0.24 us (one row, while HBM keeps up), the join 1 us and 0.3 a CTA, and 1.5 more where there are several tiles of rows.
    // us (W in the L2 in part), shared and not: 1 x 4096 x 7168 (rows x N x K; by 4) 9.1 and 17.5; 64 x 7168 x 7168
    // (by 2) 15.9 and 21.3; 16 x 512 x 18432 (by 8) 10.1 and 37.6; 128 x 2048 x 2048 (by 4) 8.5,
    // by 8 8.9, not 9.3; and 32 x 128 x 512 (by 2) 6.0 and 5.1; 333 x 1104 x 2064 (by 5) 11.7 and 10.3.
    t.splits = 1;
    t.kper = (int)ksteps;
    const int64_t tiles = (int64_t)t.mt * t.nt;
    double least = 0.24 * ksteps;
    for (int s = 2; s <= kMaxSplits && t.ctas == 1 && !one_order; ++s) {
        const int64_t per = cdiv(ksteps, s);
        const double us = 0.24 * per + 1 + 0.3 * s + (t.mt > 1 ? 1.5 : 0);
        if (us >= least || tiles * s > kSms || cdiv(ksteps, per) != s || tiles > active_clusters(s)) continue;
        least = us;
        t.splits = s;
        t.kper = (int)per;
    }
    return t;
}
static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

template <int CTAS, int BN>
static bool launch_as(const CUtensorMap &ma, const CUtensorMap &mt, const CUtensorMap &mb, const CUtensorMap &mo,
                      const Args &a, cudaStream_t st)
{
    constexpr auto kern = k_w8_gemm<CTAS, BN>;
    if (!set_attribute<kern, cudaFuncAttributeMaxDynamicSharedMemorySize>(kSmem)) return false;
    const int64_t items = (int64_t)a.mt * a.nt * a.splits;
    const int64_t clusters = a.splits > 1 ? items : std::min<int64_t>(items, gemm_num_sms() / CTAS);
    return launch_chained<kern>((unsigned)(clusters * CTAS), kThreads, kSmem, CTAS * a.splits, st, ma, mt, mb, mo,
                                a);
}

static bool product(int rows, int N, int K, const void *A, const float *As, const void *W, const float *Ws, void *out,
                    bool out_f32, bool w_early, bool one_order, DevErr *err, cudaStream_t st)
{
    const int ksteps = (int)cdiv(K, kStep);
    const Tiling t = tiling(rows, N, ksteps, one_order);
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
    a.f32_out = out_f32;
    a.out = out;
    a.w_early = w_early;
    a.err = err;
    tc::take_wait_hook(a.wait_ns, a.skip_item);
    CUtensorMap ma, mt, mb, mo;
    memset(&ma, 0, sizeof ma);
    memset(&mt, 0, sizeof mt);
    if (rows >= 128 && !tc::make_bytes_tmap(&ma, A, rows, K, kStep, 128, 128)) return false;
    if (a.tail && !tc::make_bytes_tmap(&mt, A, rows, K, kStep, a.tail, 128)) return false;
    if (!tc::make_bytes_tmap(&mb, W, N, K, kStep, 128, 128)) return false;
    memset(&mo, 0, sizeof mo);
    if (t.splits == 1 &&
        !(out_f32 ? tc::make_f32_tmap(&mo, out, 1, rows, N) : tc::make_rows_tmap(&mo, out, rows, N, 32)))
        return false;
    return t.ctas == 2 ? launch_as<2, 256>(ma, mt, mb, mo, a, st) : launch_as<1, 128>(ma, mt, mb, mo, a, st);
}

static bool quantize(int rows, int K, const void *X, bool pow2, void *q, float *s, cudaStream_t st)
{
    const int KB = (int)cdiv(K, 128);
    const int64_t ctas = cdiv((int64_t)rows * KB, kQThreads / 8 * (int64_t)kQBlocks);
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
    float *buf;      // adapter: x~ (BF16) or dx~ (FP32), [rows][K]
    size_t bytes;
};
static Ws carve(void *ws, int64_t rows, int64_t N, int64_t K, bool adapter)
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
    w.q = take((size_t)rows * most);
    w.s = (float *)take((size_t)rows * cdiv(most, 128) * 4);
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

// The entry points; one_order: no sharing of a tile's blocks of K, so that they are added
// in the same order whatever the rows of the call.  The layer's forward in a graph, each weight
// read from HBM, shared and in one order: 1 x 4096 x 7168 11.1 and 17.9 us, 64 x 7168 x 7168
// 16.1 and 21.3, 128 x 4096 x 4096 11.1 and 13.9; the same where nothing is shared.
static pmoe_status gemm(int32_t rows, int32_t N, int32_t K, const void *A, const float *As, const void *W, const float *Ws,
                        void *Y, void *ws, size_t ws_bytes, bool one_order, cudaStream_t stream)
{
    if (!shape_ok(rows, N, K) || !W || !Ws || (rows > 0 && (!A || !As || !Y)) || !a16(A) || !a16(As) || !a16(W) ||
        !a16(Ws) || !a16(Y))
        return PMOE_ERR_INVALID_ARG;
    if (!ws || ws_bytes < kHdrBytes || !a16(ws)) return PMOE_ERR_WORKSPACE;
    if (rows == 0) return PMOE_OK;
    return product(rows, N, K, A, As, W, Ws, Y, false, false, one_order, (DevErr *)ws, stream) ? PMOE_OK : PMOE_ERR_CUDA;
}

static pmoe_status forward(const void *q, const float *s, int32_t N, int32_t K, int32_t block, const void *R,
                           int32_t rows, const void *X, int pow2, void *Y, void *ws, size_t ws_bytes, bool one_order,
                           cudaStream_t stream)
{
    const pmoe_status e = check_dense(q, s, N, K, block, R, rows);
    if (e != PMOE_OK) return e;
    if ((rows > 0 && (!X || !Y)) || !a16(X) || !a16(Y)) return PMOE_ERR_INVALID_ARG;
    const Ws w = carve(ws, rows, N, K, R != nullptr);
    if (!ws || ws_bytes < w.bytes || !a16(ws)) return PMOE_ERR_WORKSPACE;
    if (rows == 0) return PMOE_OK;
    if (R) {
        launch_rotate_tc(rotation(block, false, X, false, R, rows, K, w.buf), stream);
        X = w.buf;
    }
    return quantize(rows, K, X, pow2 != 0, w.q, w.s, stream) &&
                   product(rows, N, K, w.q, w.s, q, s, Y, false, true, one_order, w.err, stream) &&
                   cudaPeekAtLastError() == cudaSuccess
               ? PMOE_OK
               : PMOE_ERR_CUDA;
}

static pmoe_status backward(const void *qt, const float *st, int32_t N, int32_t K, int32_t block, const void *R,
                            int32_t rows, const void *X, const void *dY, int pow2, void *dX, float *dR, void *ws,
                            size_t ws_bytes, bool one_order, cudaStream_t stream)
{
    const pmoe_status e = check_dense(qt, st, N, K, block, R, rows);
    if (e != PMOE_OK) return e;
    if ((R && !dR) || (rows > 0 && (!dY || !dX || (R && !X))) || !a16(X) || !a16(dY) || !a16(dX) || !a16(dR))
        return PMOE_ERR_INVALID_ARG;
    const Ws w = carve(ws, rows, N, K, R != nullptr);
    if (!ws || ws_bytes < w.bytes || !a16(ws)) return PMOE_ERR_WORKSPACE;
    if (rows == 0)
        return !R || cudaMemsetAsync(dR, 0, (size_t)K * block * sizeof(float), stream) == cudaSuccess ? PMOE_OK
                                                                                                      : PMOE_ERR_CUDA;
    // dx~ in FP32 where an adapter follows, as in dense_linear_backward
    if (!quantize(rows, N, dY, pow2 != 0, w.q, w.s, stream) ||
        !product(rows, K, N, w.q, w.s, qt, st, R ? (void *)w.buf : dX, R != nullptr, true, one_order, w.err, stream))
        return PMOE_ERR_CUDA;
    if (R) {
        launch_outer_tc(1, rows, K, block, (const uint16_t *)X, K, false, nullptr, 1, w.buf, true, K, nullptr, dR, stream);
        launch_rotate_tc(rotation(block, true, w.buf, true, R, rows, K, dX), stream);
    }
    return cudaPeekAtLastError() == cudaSuccess ? PMOE_OK : PMOE_ERR_CUDA;
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
    return w8::shape_ok(rows, N, K) ? kHdrBytes : 0;
}

pmoe_status fp8_gemm(int32_t rows, int32_t N, int32_t K, const void *A, const float *As, const void *W, const float *Ws,
                     void *Y, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    return w8::gemm(rows, N, K, A, As, W, Ws, Y, ws, ws_bytes, false, stream);
}

pmoe_status fp8_gemm_one_order(int32_t rows, int32_t N, int32_t K, const void *A, const float *As, const void *W,
                               const float *Ws, void *Y, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    return w8::gemm(rows, N, K, A, As, W, Ws, Y, ws, ws_bytes, true, stream);
}

size_t dense_w8a8_ws_bytes(int32_t rows, int32_t N, int32_t K, int adapter)
{
    return w8::shape_ok(rows, N, K) ? w8::carve(nullptr, rows, N, K, adapter != 0).bytes : 0;
}

pmoe_status dense_w8a8_forward(const void *q, const float *s, int32_t N, int32_t K, int32_t block, const void *R,
                               int32_t rows, const void *X, int pow2, void *Y, void *ws, size_t ws_bytes,
                               cudaStream_t stream)
{
    return w8::forward(q, s, N, K, block, R, rows, X, pow2, Y, ws, ws_bytes, false, stream);
}

pmoe_status dense_w8a8_forward_one_order(const void *q, const float *s, int32_t N, int32_t K, int32_t block, const void *R,
                                         int32_t rows, const void *X, int pow2, void *Y, void *ws, size_t ws_bytes,
                                         cudaStream_t stream)
{
    return w8::forward(q, s, N, K, block, R, rows, X, pow2, Y, ws, ws_bytes, true, stream);
}

pmoe_status dense_w8a8_backward(const void *qt, const float *st, int32_t N, int32_t K, int32_t block, const void *R,
                                int32_t rows, const void *X, const void *dY, int pow2, void *dX, float *dR, void *ws,
                                size_t ws_bytes, cudaStream_t stream)
{
    return w8::backward(qt, st, N, K, block, R, rows, X, dY, pow2, dX, dR, ws, ws_bytes, false, stream);
}

pmoe_status dense_w8a8_backward_one_order(const void *qt, const float *st, int32_t N, int32_t K, int32_t block, const void *R,
                                          int32_t rows, const void *X, const void *dY, int pow2, void *dX, float *dR, void *ws,
                                          size_t ws_bytes, cudaStream_t stream)
{
    return w8::backward(qt, st, N, K, block, R, rows, X, dY, pow2, dX, dR, ws, ws_bytes, true, stream);
}

}  // extern "C"
