// head_gemm.cuh -- the tensor-core products of the vocabulary head (tcgen05 +
// TMEM + TMA), one kernel for the four of a training step:
//
//   HG_FWD   Z = X W^T              epilogue: softmax partials, target logits
//   HG_GRAD  Z = X W^T again        epilogue: G = c (softmax(Z) - q), BF16
//   HG_DX    dX = G W               epilogue: FP32 partial sums, or BF16 dX
//   HG_DW    dW = G^T X             epilogue: BF16 dW
//
// D[m, n] = sum_k A[m, k] B[n, k] with both operands BF16 in shared memory:
// K-major tiles where k is contiguous in memory (X, W and G as rows of k),
// MN-major tiles where m or n is (W as [k = v][n = d], G as [k = t][m = v],
// X as [k = t][n = d]); nothing is transposed in memory.
//
// Roles (CTAS CTAs of one cluster work on one CTAS*128 x BN tile; persistent
// over the tiles):
//   warp 0      TMA producer of this CTA's 128 rows of A and BN/CTAS of B
//   warp 1      MMA issuer (CTA 0 of the cluster only), K steps of 64
//   warp 2      TMEM allocator
//   warps 4..   epilogue, one warp per 32 TMEM lanes and 128 columns: a
//               thread owns one row's 128 columns, in registers
//
// The tensor cores' FP32 accumulation truncates: its error grows linearly
// with the number of K steps (about one part in 2^24 per 16 columns).  Every
// run of kChunk K steps is therefore summed in its own TMEM buffer and added
// to the tile's FP32 sum in registers (round to nearest), which holds the
// relative error near 5e-7 at any length.  The two buffers alternate, so the
// tensor cores work on the next chunk while one is drained, and on the next
// tile's first two chunks during the epilogue proper.
//
// G is the BF16 operand of two products.  Where a token's distribution is
// concentrated, the few large entries of G carry the whole gradient, and
// their rounding to 8 bits would be its error.  A 128 x 128 block of G that
// holds an entry |p - q| >= kLarge therefore keeps the rounding's remainder
// too (a second BF16, 16 bits together), and is flagged; the products run a
// second K step on the remainders of flagged blocks only (a token has at most
// 1 / kLarge such entries of p, spread over the vocabulary).
//
// Every element's sum runs over k in the same order whatever the tile shape,
// and the softmax partials cover 128 aligned columns: the results do not
// depend on the number of tokens in the call.
#pragma once

#include "gemm_tc.cuh"

namespace pmoe {
namespace hg {

using tc::kBK;
using tc::mbar_arrive;
using tc::mbar_expect_tx;
using tc::mbar_init;
using tc::mbar_wait;
using tc::smem_u32;
using tc::tc_fence_after;
using tc::tc_fence_before;

enum Epi { HG_FWD = 0, HG_GRAD = 1, HG_DX = 2, HG_DW = 3 };

constexpr int kUnit = 128;               // columns per softmax partial and per epilogue thread
constexpr int kStages = 6;               // 32 KB each: 16 KB of A, 16 KB of B
constexpr int kOpBytes = 128 * kBK * 2;  // one operand tile of a stage
constexpr int kStageBytes = 2 * kOpBytes;
constexpr int kOutBytes = 128 * 128;     // one staged output box: 128 rows of 128 bytes
constexpr int kChunk = 8;                // K steps summed in one TMEM buffer
constexpr float kLarge = 0.125f;         // entries of p - q whose block keeps its remainder
constexpr int kThreads0 = 128;           // producer, MMA and allocator warps

constexpr int epi_warps(int BN) { return BN / kUnit * 4; }
constexpr int threads_of(int BN) { return kThreads0 + 32 * epi_warps(BN); }
// 1024 bytes of slack to align the swizzled tiles, 256 for the barriers
constexpr int smem_of(int BN) { return kStages * kStageBytes + BN / kUnit * kOutBytes + 256 + 1024; }

struct Args {
    int M, N;                // output rows and columns of this launch
    int n0;                  // GRAD: first vocabulary column; FWD: 0
    int mt, nt, gm;          // tiles, and m tiles that run together
    int splits, ksteps, kper;   // K steps of 64 in all and per split
    int kb0;                 // first k coordinate of B (A: 0)
    int arows;               // rows of A's tensor map: the row past its end
    int V;                   // FWD, GRAD: number of vocabulary entries
    float c;                 // FWD, GRAD: scale * log2(e)
    int NU;                  // FWD: partials per token
    float2 *part;            // FWD: [T][NU] (max, sum) in base 2
    float *zt;               // FWD: [T][K] raw logits of the target entries
    const int32_t *ids;      // FWD, GRAD: [T][K] target entries, ascending
    const float *q;          // GRAD: [T][K] their probabilities, or NULL: 1
    int K;
    const float *lse;        // GRAD: [T]
    const float *coef;       // GRAD: [T] factor of the row (0: no gradient)
    uint8_t *fl, *flt;       // flagged blocks of G: [token block][fs], and transposed
    int fs, fst;             // [vocabulary block][fst]; row strides, multiples of 4
    int accumulate;          // DX: add to the FP32 partials
    int bf16_out;            // DX: the output map is the BF16 dX itself
    DevErr *err;
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t cta_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Address of this CTA's shared-memory location in CTA 0 of the cluster
__device__ __forceinline__ uint32_t map_leader(uint32_t addr)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <int CTAS>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap *tm, int x, int y, uint32_t bar)
{
    if constexpr (CTAS == 2)   // the barrier may be the other CTA's
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"((uint64_t)tm), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        tc::tma_load_2d(dst, tm, x, y, bar);
}
__device__ __forceinline__ void store_3d(const CUtensorMap *tm, uint32_t src, int x, int y, int z, bool add)
{
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                         (uint64_t)tm),
                     "r"(x), "r"(y), "r"(z), "r"(src)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                         (uint64_t)tm),
                     "r"(x), "r"(y), "r"(z), "r"(src)
                     : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void store_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void bar_group(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool bar_group_and(int id, bool v)
{
    uint32_t r;
    asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %2, 0;\n"
                 "barrier.cta.red.and.pred q, %1, 128, p; selp.u32 %0, 1, 0, q; }"
                 : "=r"(r)
                 : "r"(id), "r"((uint32_t)v)
                 : "memory");
    return r != 0;
}
__device__ __forceinline__ bool bar_group_or(int id, bool v) { return !bar_group_and(id, !v); }
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int CTAS>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum)
{
    if constexpr (CTAS == 2)
        asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(accum)
                     : "memory");
    else
        asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(accum)
                     : "memory");
}
// The barrier (of both CTAs of a pair) completes when the MMAs issued so far have
template <int CTAS>
__device__ __forceinline__ void commit(uint32_t bar)
{
    if constexpr (CTAS == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                bar),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
}
// Shared-memory descriptor of a 128 x 64 operand tile, 128-byte swizzle.
// K-major: 8-row groups 1024 bytes apart.  MN-major: two boxes of 64 mn x 64
// k rows (8 KB), so the next 64 mn are 8192 bytes on and the next 8 k 1024.
template <bool MN>
__device__ __forceinline__ uint64_t desc_of(uint32_t saddr)
{
    if constexpr (!MN) return tc::sdesc(saddr);
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(8192 >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Value j of a register array (j varies between the lanes)
__device__ __forceinline__ float pick(const float (&v)[kUnit], int j)
{
    float r = 0.f;
#pragma unroll
    for (int i = 0; i < kUnit; ++i) r = i == j ? v[i] : r;
    return r;
}
// First of the K ascending ids that is >= v
__device__ __forceinline__ int lower_bound(const int32_t *ids, int K, int v)
{
    int lo = 0, n = K;
    while (n > 0) {
        const int h = n >> 1;
        if (ids[lo + h] < v) {
            lo += h + 1;
            n -= h + 1;
        } else {
            n = h;
        }
    }
    return lo;
}

struct Item {
    int m, n, s;   // m tile, n tile, split
};
__device__ __forceinline__ Item item_of(const Args &a, int i)
{
    Item t;
    const int per = a.mt * a.nt;
    t.s = i / per;
    i -= t.s * per;
    const int gsz = a.gm * a.nt, g = i / gsz;
    i -= g * gsz;
    const int gm = min(a.gm, a.mt - g * a.gm);   // the last group may be smaller
    t.n = i / gm;
    t.m = g * a.gm + i - t.n * gm;
    return t;
}

// ------------------------------------------------------------------ kernel
template <int CTAS, int BN, int EPI>
__global__ void __launch_bounds__(threads_of(BN), 1) k_head_gemm(const __grid_constant__ CUtensorMap tmA,
                                                                 const __grid_constant__ CUtensorMap tmB,
                                                                 const __grid_constant__ CUtensorMap tmOut,
                                                                 const __grid_constant__ CUtensorMap tmLo,
                                                                 const Args a)
{
    constexpr bool kAMn = EPI == HG_DW, kBMn = EPI == HG_DX || EPI == HG_DW;
    constexpr int kEpi = epi_warps(BN);
    static_assert(BN / CTAS == 128, "one 128-row operand tile of B per CTA");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t s0 = smem_u32(smem);
    const uint32_t out0 = s0 + kStages * kStageBytes;
    const uint32_t bar0 = out0 + BN / kUnit * kOutBytes;
    auto full = [&](uint32_t s) { return bar0 + 8 * s; };
    auto empty = [&](uint32_t s) { return bar0 + 8 * (kStages + s); };
    auto tfull = [&](uint32_t b) { return bar0 + 8 * (2 * kStages + b); };
    auto tempty = [&](uint32_t b) { return bar0 + 8 * (2 * kStages + 2 + b); };
    const uint32_t slot = bar0 + 8 * (2 * kStages + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 2 ? cta_rank() : 0u;
    const int n_items = a.mt * a.nt * a.splits;
    const int first = blockIdx.x / CTAS, step = gridDim.x / CTAS;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), CTAS * kEpi);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tc::fence_proxy_async();
    }
    if (warp == 2) {
        if constexpr (CTAS == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                         "r"(2 * BN)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                         "r"(2 * BN)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CTAS == 2) cluster_sync();   // the peer's barriers are ready too
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot));

    // K steps of an item
    auto krange = [&](const Item &t, int &k0, int &k1) {
        k0 = t.s * a.kper;
        k1 = min(k0 + a.kper, a.ksteps);
    };
    // DX, DW: the flags of the next kChunk K steps of A's row blocks, a byte per
    // 128 k, one word per CTA of the cluster
    constexpr bool kLo = EPI == HG_DX || EPI == HG_DW;
    static_assert(kChunk == 8 && kBK == 64, "a chunk is four flag bytes");
    auto flags = [&](const Item &t, int k, uint32_t (&w)[CTAS]) {
#pragma unroll
        for (int r = 0; r < CTAS; ++r) {
            w[r] = 0;
            if constexpr (kLo) {
                const int mb = t.m * CTAS + r;
                const uint8_t *f = EPI == HG_DX ? a.fl + (int64_t)mb * a.fs : a.flt + (int64_t)mb * a.fst;
                if (k < a.ksteps && mb * 128 < a.M) w[r] = *(const uint32_t *)(f + (k >> 1));
            }
        }
    };
    auto flag_at = [](uint32_t w, int j) { return ((w >> ((j >> 1) * 8)) & 1u) != 0; };
    bool ok = true;
    // The epilogue's 128 sums a thread need more registers than an even split
    // of 384 threads gives (168): the first four warps hand theirs over.  Of
    // the launch's 384 x 168 = 64512: 128 x 40 + 256 x 232, and where the
    // producer and the MMA issuer follow flags 128 x 72 + 256 x 216.
    if (warp >= 4) {
        // ---------------- epilogue
        if constexpr (kEpi == 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLo ? 216 : 232));
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const int rl = quad * 32 + lane;   // row of the CTA's 128
        const uint32_t tld = tmem + ((uint32_t)(quad * 32) << 16) + half * kUnit;
        const uint32_t ob = out0 + half * kOutBytes;
        uint32_t gc = 0;
        for (int i = first; ok && i < n_items; i += step) {
            const Item t = item_of(a, i);
            int k0, k1;
            krange(t, k0, k1);
            float acc[kUnit];
#pragma unroll
            for (int j = 0; j < kUnit; ++j) acc[j] = 0.f;
            for (int c0 = k0; c0 < k1; c0 += kChunk, ++gc) {
                const uint32_t b = gc & 1;
                // (warp-uniform: every lane sees the same outcome before the aligned loads)
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(tfull(b), (gc >> 1) & 1, a.err, 4, tc::kWaitNs))))
                    break;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < kUnit; j += 16) {
                    float v[16];
                    tc::tmem_ld16(tld + b * BN + j, v);
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[j + e] += v[e];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CTAS == 2) arrive_cluster(map_leader(tempty(b)));
                    else mbar_arrive(tempty(b));
                }
            }
            // the group's four warps leave together (the barriers below are unbounded)
            if (EPI != HG_FWD) ok = bar_group_and(1 + half, ok);
            if (!ok) break;
            const int mrow = (t.m * CTAS + (int)rank) * 128;
            const int row = mrow + rl;
            const int cb = a.n0 + t.n * BN + half * kUnit;   // first column
            bool lo = false;   // GRAD: this block's remainders are kept
            if constexpr (EPI == HG_FWD || EPI == HG_GRAD) {
                const int nv = min(kUnit, a.V - cb);         // valid columns (may be <= 0)
                const bool live = row < a.M && nv > 0;
                const int32_t *ids = a.ids + (int64_t)row * a.K;
                int pos = 0, id = 0x7fffffff;
                if (live) {
                    pos = a.K > 1 ? lower_bound(ids, a.K, cb) : 0;
                    if (pos < a.K) id = ids[pos];
                    if (id < cb) id = 0x7fffffff;   // K == 1: an earlier column, or no target
                }
                if constexpr (EPI == HG_FWD) {
                    while (__any_sync(0xffffffffu, id - cb < nv)) {
                        const bool has = id - cb < nv;
                        const float z = pick(acc, has ? id - cb : -1);
                        if (has) {
                            a.zt[(int64_t)row * a.K + pos] = z;
                            ++pos;
                            id = pos < a.K ? ids[pos] : 0x7fffffff;
                        }
                    }
                    if (live) {
                        if (nv < kUnit) {
#pragma unroll
                            for (int j = 0; j < kUnit; ++j)
                                if (j >= nv) acc[j] = -__int_as_float(0x7f800000);
                        }
                        float mx[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx[e] = acc[e];
#pragma unroll
                        for (int j = 4; j < kUnit; ++j) mx[j & 3] = fmaxf(mx[j & 3], acc[j]);
                        const float m2 = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.c;
                        float sm[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int j = 0; j < kUnit; ++j) sm[j & 3] += ex2(fmaf(acc[j], a.c, -m2));
                        a.part[(int64_t)row * a.NU + cb / kUnit] =
                            make_float2(m2, (sm[0] + sm[1]) + (sm[2] + sm[3]));
                    }
                } else {
                    const float l2 = row < a.M ? a.lse[row] * 1.4426950408889634f : 0.f;
                    const float cf = row < a.M ? a.coef[row] : 0.f;
#pragma unroll
                    for (int j = 0; j < kUnit; ++j) acc[j] = ex2(fmaf(acc[j], a.c, -l2));
                    while (__any_sync(0xffffffffu, id - cb < nv)) {
                        const bool has = id - cb < nv;
                        const int j0 = has ? id - cb : -1;
                        const float qv = !has ? 0.f : a.q ? a.q[(int64_t)row * a.K + pos] : 1.f;
#pragma unroll
                        for (int j = 0; j < kUnit; ++j) acc[j] = j == j0 ? acc[j] - qv : acc[j];
                        if (has) {
                            ++pos;
                            id = pos < a.K ? ids[pos] : 0x7fffffff;
                        }
                    }
                    bool big = false;
#pragma unroll
                    for (int j = 0; j < kUnit; ++j) {
                        big |= j < nv && fabsf(acc[j]) >= kLarge;
                        acc[j] = j < nv ? acc[j] * cf : 0.f;
                    }
                    lo = bar_group_or(1 + half, big && cf != 0.f);
                    if (quad == 0 && lane == 0 && mrow < a.M) {
                        const int tb = mrow >> 7, vb = (t.n * BN >> 7) + half;
                        a.fl[(int64_t)tb * a.fs + vb] = lo;
                        a.flt[(int64_t)vb * a.fst + tb] = lo;
                    }
                }
            }
            if constexpr (EPI != HG_FWD) {
                // through shared memory (128-byte rows, 128-byte swizzle) to TMA
                // stores, which clip rows and columns past the output's end
                const int xc = t.n * BN + half * kUnit;
                const bool f32 = EPI == HG_DX && !a.bf16_out;
                const uint32_t srow = ob + rl * 128;
                auto box = [&](const CUtensorMap *tm, int x) {   // the group's staged box goes out at column x
                    tc::fence_proxy_async();
                    bar_group(1 + half);
                    if (quad == 0 && lane == 0) store_3d(tm, ob, x, mrow, t.s, a.accumulate != 0);
                };
                auto reuse = [&]() {      // the group's previous box has been read
                    if (quad == 0 && lane == 0) store_wait_read();
                    bar_group(1 + half);
                };
                if (f32) {
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                        reuse();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int e = q4 * 32 + j * 4;
                            tc::st_shared_v4(srow + ((j ^ (rl & 7)) << 4),
                                             make_uint4(__float_as_uint(acc[e]), __float_as_uint(acc[e + 1]),
                                                        __float_as_uint(acc[e + 2]), __float_as_uint(acc[e + 3])));
                        }
                        if (xc + q4 * 32 < a.N) box(&tmOut, xc + q4 * 32);
                    }
                } else {
#pragma unroll
                    for (int q2 = 0; q2 < 2; ++q2) {
                        reuse();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int e = q2 * 64 + j * 8;
                            tc::st_shared_v4(srow + ((j ^ (rl & 7)) << 4),
                                             make_uint4(pack_bf2(acc[e], acc[e + 1]), pack_bf2(acc[e + 2], acc[e + 3]),
                                                        pack_bf2(acc[e + 4], acc[e + 5]),
                                                        pack_bf2(acc[e + 6], acc[e + 7])));
                        }
                        if (xc + q2 * 64 < a.N) box(&tmOut, xc + q2 * 64);
                    }
                    if (EPI == HG_GRAD && lo) {
#pragma unroll
                        for (int j = 0; j < kUnit; ++j) acc[j] -= bf2f(f2bf(acc[j]));   // exact
#pragma unroll
                        for (int q2 = 0; q2 < 2; ++q2) {
                            reuse();
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int e = q2 * 64 + j * 8;
                                tc::st_shared_v4(
                                    srow + ((j ^ (rl & 7)) << 4),
                                    make_uint4(pack_bf2(acc[e], acc[e + 1]), pack_bf2(acc[e + 2], acc[e + 3]),
                                               pack_bf2(acc[e + 4], acc[e + 5]), pack_bf2(acc[e + 6], acc[e + 7])));
                            }
                            if (xc + q2 * 64 < a.N) box(&tmLo, xc + q2 * 64);
                        }
                    }
                }
            }
        }
        if (EPI != HG_FWD && quad == 0 && lane == 0) store_wait_all();
    } else {
        if constexpr (kEpi == 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLo ? 72 : 40));
        if (warp == 0) {
            // ---------------- producer
            if (lane == 0) {
                uint32_t g = 0;
                for (int i = first; ok && i < n_items; i += step) {
                    const Item t = item_of(a, i);
                    int k0, k1;
                    krange(t, k0, k1);
                    const int ma = (t.m * CTAS + (int)rank) * 128;
                    const int nb = a.n0 + t.n * BN + (int)rank * 128;
                    // one K step; `mine`: A holds data (else it is filled with zeros, from
                    // past its last row)
                    auto load = [&](const CUtensorMap *tma, int k, bool mine) {
                        const uint32_t s = g % kStages;
                        if (!(ok = mbar_wait(empty(s), ((g / kStages) & 1) ^ 1, a.err, 1, tc::kWaitNs))) return;
                        if (rank == 0) mbar_expect_tx(full(s), CTAS * kStageBytes);
                        const uint32_t fb = CTAS == 2 ? map_leader(full(s)) : full(s);
                        const uint32_t sa = s0 + s * kStageBytes, sb = sa + kOpBytes;
                        const int ka = k * kBK, kb = a.kb0 + k * kBK;
                        if constexpr (kAMn) {
                            load_2d<CTAS>(sa, tma, ma, mine ? ka : a.arows, fb);
                            load_2d<CTAS>(sa + 8192, tma, ma + 64, mine ? ka : a.arows, fb);
                        } else {
                            load_2d<CTAS>(sa, tma, ka, mine ? ma : a.arows, fb);
                        }
                        if constexpr (kBMn) {
                            load_2d<CTAS>(sb, &tmB, nb, kb, fb);
                            load_2d<CTAS>(sb + 8192, &tmB, nb + 64, kb, fb);
                        } else {
                            load_2d<CTAS>(sb, &tmB, kb, nb, fb);
                        }
                        ++g;
                    };
                    uint32_t w[CTAS], wn[CTAS];
                    flags(t, k0, w);
                    for (int c0 = k0; ok && c0 < k1; c0 += kChunk) {
                        flags(t, c0 + kChunk, wn);
                        const int c1 = min(c0 + kChunk, k1);
                        for (int k = c0; ok && k < c1; ++k) {
                            load(&tmA, k, true);
                            if (ok && kLo && flag_at(w[0] | w[CTAS - 1], k - c0)) load(&tmLo, k, flag_at(w[rank], k - c0));
                        }
    #pragma unroll
                        for (int r = 0; r < CTAS; ++r) w[r] = wn[r];
                    }
                }
            }
        } else if (warp == 1) {
            // ---------------- MMA issuer
            if (lane == 0 && rank == 0) {
                const uint32_t idesc = tc::idesc_bf16(CTAS * 128, BN, kAMn) | ((uint32_t)kBMn << 16);
                constexpr uint32_t kAStep = kAMn ? 2048 >> 4 : 32 >> 4;   // 16 k
                constexpr uint32_t kBStep = kBMn ? 2048 >> 4 : 32 >> 4;
                const uint64_t da0 = desc_of<kAMn>(s0), db0 = desc_of<kBMn>(s0 + kOpBytes);
                uint32_t g = 0, gc = 0;
                for (int i = first; ok && i < n_items; i += step) {
                    const Item t = item_of(a, i);
                    int k0, k1;
                    krange(t, k0, k1);
                    uint32_t w[CTAS], wn[CTAS];
                    flags(t, k0, w);
                    for (int c0 = k0; ok && c0 < k1; c0 += kChunk, ++gc) {
                        flags(t, c0 + kChunk, wn);
                        const uint32_t b = gc & 1;
                        if (!(ok = mbar_wait(tempty(b), ((gc >> 1) & 1) ^ 1, a.err, 2, tc::kWaitNs))) break;
                        tc_fence_after();
                        const int c1 = min(c0 + kChunk, k1);
                        auto kstep = [&](bool add) {
                            const uint32_t s = g % kStages;
                            if (!(ok = mbar_wait(full(s), (g / kStages) & 1, a.err, 3, tc::kWaitNs))) return;
                            tc_fence_after();
                            const uint64_t da = da0 + s * (kStageBytes >> 4), db = db0 + s * (kStageBytes >> 4);
    #pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mma<CTAS>(tmem + b * BN, da + j * kAStep, db + j * kBStep, idesc, add || j > 0);
                            commit<CTAS>(empty(s));
                            ++g;
                        };
                        for (int k = c0; ok && k < c1; ++k) {
                            kstep(k > c0);
                            if (ok && kLo && flag_at(w[0] | w[CTAS - 1], k - c0)) kstep(true);
                        }
                        if (ok) commit<CTAS>(tfull(b));
    #pragma unroll
                        for (int r = 0; r < CTAS; ++r) w[r] = wn[r];
                    }
                }
            }
        }
    }
    // After a wait that ran out, copies or MMAs may still be in flight: give
    // them a millisecond to land before shared memory and TMEM go.
    if (!ok) {
        const uint64_t t0 = tc::globaltimer();
        while (tc::globaltimer() - t0 < 1000000ull) __nanosleep(1000);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (CTAS == 2) cluster_sync();   // no CTA leaves while its peer still signals it
    tc_fence_after();
    if (warp == 2) {
        if constexpr (CTAS == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN));
    }
}

}  // namespace hg
}  // namespace pmoe
