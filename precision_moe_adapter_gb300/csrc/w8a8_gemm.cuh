// w8a8_gemm.cuh -- the product of two E4M3 operands with FP32 scales per block of
// 128 along K (tcgen05 + TMEM + TMA):
//
//   D[r, n] = sum_b As[b][r] Ws[n / 128][b] (sum_{k in block b} A[r, k] W[n, k])
//
// Both operands are K-major; a K step is one block, 128 bytes of a row, one
// 128-byte swizzle row.  The tensor cores sum one block into a TMEM buffer of its
// own, the epilogue warps scale it and add it to the tile's FP32 sums, which stay in
// registers: a thread owns 128 (or 64) columns of a row, so that its scale is one
// number a block, As[b][row] Ws[n / 128][b].
//
// Few tiles: a cluster of up to 8 CTAs shares a tile's blocks of K.  Their sums meet
// through distributed shared memory and are added in order, each CTA a share of the
// rows, so that neither a second kernel nor FP32 sums in memory are needed.
//
// What bounds it.  Many rows: 16384 rows, N = K = 7168 take 670 us (2.5 PFLOP/s, 1.46 times the
// BF16 rate that the card sustains), as much as without the drain of the TMEM buffers; for seconds
// on end 689 us at the card's power limit, which takes 6% off the SM clock (1366 W, 1942 MHz of
// 2070).  Shorter products: 4096 x 4096 x 7168 takes 115 us (2.1 PFLOP/s, 3.4 rounds
// of tiles taking 4, the tensor pipe 54% active); without the drain (8 loads of 16 columns
// and 128 multiply-adds a thread and step) forward and dX are 22% faster.  Few rows: a step of a CTA,
// 16 KB of W, takes 0.24 us at one row and 0.27 at 64 while up to 56 CTAs run, a rate of the CTA
// and not of the memory; with 112 CTAs 0.27 at one row, 6.8 TB/s, and 0.35 at 64, 5.3 TB/s.
// Beside the steps stand some 5 us of launches, of the wait for the codes of A and of the join
// (64 rows, N = K = 7168, the layer in a graph: 16.1 us where W comes from HBM, of which at a
// copy's rate it is 7.6; 15.3 with two weights, which the L2 holds in part).
// Kept from what was tried: the buffer is released before the last columns are added; eight
// epilogue warps; W's first stages on their way before the kernel before is done (0.2 to 0.4
// us).  Not kept: pairs of sums in one instruction (fma.rn.f32x2: 1943 us against 1438 for
// 16384 rows both ways, the pairs take moves); loads of 32 or 64 columns (the same); A's codes
// made by the product's own producer warp up to 16 rows (one row 11.1 us against 9.1).
//
// Roles as in the head's products (head_gemm.cuh): warps 0 and 3 load A and W,
// warp 1 issues the MMAs, warp 2 allocates TMEM, warps 4.. are the epilogue; CTAS CTAs
// of a cluster work on one CTAS*128 x BN tile.
#pragma once

#include "head_gemm.cuh"

namespace pmoe {
namespace w8 {

using hg::kMaxStages;
using hg::kOpBytes;
using hg::kRingBytes;
using hg::kUnit;
using hg::kWarpOut;
using tc::mbar_arrive;
using tc::mbar_init;
using tc::mbar_wait;
using tc::smem_u32;
using tc::tc_fence_after;
using tc::tc_fence_before;

constexpr int kStep = 128;                     // K of a step: a block
constexpr int kThreads0 = 128;
// eight epilogue warps: each takes 32 rows and half of the tile's columns
constexpr int kEpi = 8;
constexpr int kThreads = kThreads0 + 32 * kEpi;
constexpr int bufs_of(int BN) { return 512 / BN; }   // all of TMEM
constexpr int kSmem = kRingBytes + kEpi * kWarpOut + 512 + 1024;

struct Args {
    int M, N;
    int mt, nt, gm;          // tiles, and m tiles that run together
    int ksteps, splits, kper;   // K steps of a tile; CTAs (of a cluster) that share it, kper each
    int stages, abytes;      // the ring: stages, and bytes of A in one
    int tail;                // rows of tmAt's boxes: the M % 128 last rows of A
    const float *As;         // [ksteps][M]
    const float *Ws;         // [ceil(N/128)][ksteps]
    int f32_out;             // the output is FP32
    void *out;               // splits > 1: [M][N]
    int w_early;             // W was complete before the kernel before started
    uint64_t wait_ns;
    int skip_item;           // test hook (-1: none)
    DevErr *err;
};

struct Item {
    int m, n, s, k0, k1;
};
__device__ __forceinline__ bool item_of(const Args &a, int i, Item &t)
{
    const int tile = i / a.splits;   // (shared tiles: one item a CTA, the cluster's ranks in order)
    if (tile >= a.mt * a.nt) return false;
    t.s = i - tile * a.splits;
    t.k0 = t.s * a.kper;
    t.k1 = min(t.k0 + a.kper, a.ksteps);
    i = tile;
    const int gsz = a.gm * a.nt, g = i / gsz;
    i -= g * gsz;
    const int gm = min(a.gm, a.mt - g * a.gm);
    t.n = i / gm;
    t.m = g * a.gm + i - t.n * gm;
    return true;
}
// Place of 4 columns of a row among a CTA's sums of 128 x 128 (no bank conflicts by
// rows or by columns)
__device__ __forceinline__ uint32_t sum_at(int row, int j) { return (uint32_t)(row * 512 + ((j ^ (row & 31)) << 4)); }
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, uint32_t rank)
{
    float4 v;
    asm volatile("{ .reg .b32 r; mapa.shared::cluster.u32 r, %4, %5;\n"
                 "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [r]; }"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

// A K step of 128: four MMAs of K = 32, the first one overwriting, and the
// commits of the stage and of the TMEM buffer
template <int CTAS>
__device__ __forceinline__ void mma_step_warp(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t bar)
{
    constexpr uint32_t sa = 32 >> 4;
    if constexpr (CTAS == 2)
        asm volatile(
            "{ .reg .pred e, p, t; elect.sync _|e, 0xffffffff; setp.ne.b32 p, %9, %9; setp.eq.b32 t, %9, %9;\n"
            "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %5, %9, p;\n"
            "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %2, %6, %9, t;\n"
            "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %3, %7, %9, t;\n"
            "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %4, %8, %9, t;\n"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%10], %11; }" ::"r"(
                d),
            "l"(da), "l"(da + sa), "l"(da + 2 * sa), "l"(da + 3 * sa), "l"(db), "l"(db + sa), "l"(db + 2 * sa),
            "l"(db + 3 * sa), "r"(idesc), "r"(bar), "h"((uint16_t)3)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred e, p, t; elect.sync _|e, 0xffffffff; setp.ne.b32 p, %9, %9; setp.eq.b32 t, %9, %9;\n"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %5, %9, p;\n"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %2, %6, %9, t;\n"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %3, %7, %9, t;\n"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %4, %8, %9, t;\n"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%10]; }" ::"r"(d),
            "l"(da), "l"(da + sa), "l"(da + 2 * sa), "l"(da + 3 * sa), "l"(db), "l"(db + sa), "l"(db + 2 * sa),
            "l"(db + 3 * sa), "r"(idesc), "r"(bar)
            : "memory");
}
// Instruction descriptor, kind::f8f6f4: E4M3 A and B (both K-major), FP32 D, M x N
__device__ __forceinline__ uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_issue16(uint32_t taddr, float *v)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
                   "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait16(float *v)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])::"memory");
}

// Quads f0, f0 + 32 kEpi, ... < f1 of a shared tile: the sum over the cluster's CTAs
// in their order, kU quads at a time
template <int kS, int kU>
__device__ __forceinline__ void join(const Args &a, const Item &t, uint32_t sums, int f0, int f1)
{
    for (; f0 < f1; f0 += kU * 32 * kEpi) {
        float4 x[kU][kS];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int f = f0 + u * 32 * kEpi;
#pragma unroll
            for (int q = 0; q < kS; ++q)
                if (f < f1 && q < a.splits) x[u][q] = ld_cluster(sums + sum_at(f >> 5, f & 31), (uint32_t)q);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int f = f0 + u * 32 * kEpi, c = t.n * 128 + (f & 31) * 4;
            float4 v = x[u][0];
#pragma unroll
            for (int q = 1; q < kS; ++q)
                if (q < a.splits) v.x += x[u][q].x, v.y += x[u][q].y, v.z += x[u][q].z, v.w += x[u][q].w;
            if (f >= f1 || c >= a.N) continue;
            const int64_t at = (int64_t)(t.m * 128 + (f >> 5)) * a.N + c;
            if (a.f32_out) *(float4 *)((float *)a.out + at) = v;
            else *(uint2 *)((uint16_t *)a.out + at) = make_uint2(hg::bf2(v.x, v.y), hg::bf2(v.z, v.w));
        }
    }
}

template <int CTAS, int BN>
__global__ void __launch_bounds__(kThreads, 1) k_w8_gemm(const __grid_constant__ CUtensorMap tmA,
                                                               const __grid_constant__ CUtensorMap tmAt,
                                                               const __grid_constant__ CUtensorMap tmB,
                                                               const __grid_constant__ CUtensorMap tmOut, const Args a)
{
    constexpr int kBufs = bufs_of(BN), kCols = BN / 2;   // (columns of an epilogue thread)
    static_assert(BN / CTAS == 128, "one 128-row operand tile of W per CTA");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t s0 = smem_u32(smem);
    const uint32_t out0 = s0 + kRingBytes;
    const uint32_t bar0 = out0 + kEpi * kWarpOut;
    auto full = [&](uint32_t s) { return bar0 + 8 * s; };
    auto empty = [&](uint32_t s) { return bar0 + 8 * (kMaxStages + s); };
    auto tfull = [&](uint32_t b) { return bar0 + 8 * (2 * kMaxStages + b); };
    auto tempty = [&](uint32_t b) { return bar0 + 8 * (2 * kMaxStages + kBufs + b); };
    const uint32_t slot = bar0 + 8 * (2 * kMaxStages + 2 * kBufs);
    const uint32_t stages = (uint32_t)a.stages, stage_bytes = kOpBytes + (uint32_t)a.abytes;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 2 ? hg::cta_rank() : 0u;
    const int first = blockIdx.x / CTAS, step = gridDim.x / CTAS;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < kBufs; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), CTAS * kEpi);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tc::fence_proxy_async();
    }
    if (warp == 2) {
        if constexpr (CTAS == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(512)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(512)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CTAS == 2) hg::cluster_sync();   // the peer's barriers are ready too
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot));

    // W may be on its way before the wait (a.w_early): the kernel before neither writes
    // it nor lets this one start before its own wait is over
    if (warp != 3 || !a.w_early) {
        grid_wait();
        grid_go();
    }
    bool ok = true;
    // registers: 384 x 168 = 128 x 40 + 256 x 232
    if (warp >= 4) {
        // ---------------- epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const int rl = quad * 32 + lane;   // row of the CTA's 128
        const uint32_t tld = tmem + ((uint32_t)(quad * 32) << 16) + half * kCols;
        const uint32_t ob = out0 + (warp - 4) * kWarpOut, orow = ob + lane * 128;
        const int NB = (int)cdiv(a.N, kUnit);
        uint32_t gc = 0;
        Item t;
        for (int i = first; ok && item_of(a, i, t); i += step) {
            const int mrow = (t.m * CTAS + (int)rank) * 128;
            const int row = mrow + rl, unit = (t.n * BN + half * kCols) / kUnit;
            const bool live = row < a.M && unit < NB, used = mrow + quad * 32 < a.M;
            const float *ap = a.As + (live ? row : 0), *wp = a.Ws + (int64_t)(live ? unit : 0) * a.ksteps;
            // the scales of two steps on their way
            constexpr int kAhead = 2;
            float sa[kAhead], sw[kAhead];
            auto fetch = [&](int u, int k) {
                if (k < t.k1) {
                    sa[u] = live ? __ldg(ap + (int64_t)k * a.M) : 0.f;
                    sw[u] = __ldg(wp + k);
                }
            };
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                sa[u] = sw[u] = 0.f;
                fetch(u, t.k0 + u);
            }
            float acc[kCols];
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] = 0.f;
#pragma unroll 1
            for (int k = t.k0; ok && k < t.k1; k += kAhead) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (k + u >= t.k1) break;
                    const uint32_t b = gc % kBufs;
                    // (warp-uniform: every lane sees the same outcome before the aligned loads)
                    if (!(ok = __all_sync(0xffffffffu,
                                          mbar_wait(tfull(b), (gc / kBufs) & 1, a.err, 4, a.wait_ns))))
                        break;
                    tc_fence_after();
                    const float s = sa[u] * sw[u];
                    fetch(u, k + u + kAhead);
                    auto release = [&]() {   // all of the buffer is in registers
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if constexpr (CTAS == 2) hg::arrive_cluster(hg::map_leader(tempty(b)));
                            else mbar_arrive(tempty(b));
                        }
                    };
                    if (CTAS == 1 && !used) {   // (no row of the warp's 32 exists)
                        release();
                        ++gc;
                        continue;
                    }
                    // 16 columns are on their way while the 16 before are added.  (All 64 of a
                    // single CTA's at once: 20.1 us against 15.8 at 64 rows, N = K = 7168.)
                    const uint32_t at = tld + b * BN;
                    float v[2][16];
                    tmem_issue16(at, v[0]);
#pragma unroll
                    for (int j = 0; j < kCols / 16; ++j) {
                        tmem_wait16(v[j & 1]);
                        if (j + 1 < kCols / 16) tmem_issue16(at + (j + 1) * 16, v[(j + 1) & 1]);
                        else release();
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[j * 16 + e] = fmaf(v[j & 1][e], s, acc[j * 16 + e]);
                    }
                    ++gc;
                }
            }
            if (!ok) break;
            if (CTAS == 1 && a.splits > 1) {   // (every MMA has read the ring: it holds the sums now)
                if (row < a.M) {
#pragma unroll
                    for (int j = 0; j < kCols / 4; ++j)
                        tc::st_shared_v4(s0 + sum_at(rl, half * (kCols / 4) + j),
                                         make_uint4(__float_as_uint(acc[4 * j]), __float_as_uint(acc[4 * j + 1]),
                                                    __float_as_uint(acc[4 * j + 2]), __float_as_uint(acc[4 * j + 3])));
                }
                continue;
            }
            // through shared memory (the warp's 32 rows of 128 bytes, 128-byte swizzle)
            // to TMA stores, which clip rows and columns past the end
            const int xc = t.n * BN + half * kCols, yr = mrow + quad * 32;
            auto put = [&](int x) {
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0 && x < a.N && yr < a.M) hg::store_3d(&tmOut, ob, x, yr, 0, false);
            };
            auto reuse = [&]() {   // the previous box has been read
                if (lane == 0) hg::store_wait_read();
                __syncwarp();
            };
            if (a.f32_out) {
#pragma unroll
                for (int q = 0; q < kCols; q += 32) {
                    reuse();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int e = q + j * 4;
                        tc::st_shared_v4(orow + ((j ^ (lane & 7)) << 4),
                                         make_uint4(__float_as_uint(acc[e]), __float_as_uint(acc[e + 1]),
                                                    __float_as_uint(acc[e + 2]), __float_as_uint(acc[e + 3])));
                    }
                    put(xc + q);
                }
            } else {
#pragma unroll
                for (int q = 0; q < kCols; q += 64) {
                    reuse();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int e = q + j * 8;
                        tc::st_shared_v4(orow + ((j ^ (lane & 7)) << 4),
                                         make_uint4(hg::bf2(acc[e], acc[e + 1]), hg::bf2(acc[e + 2], acc[e + 3]),
                                                    hg::bf2(acc[e + 4], acc[e + 5]), hg::bf2(acc[e + 6], acc[e + 7])));
                    }
                    put(xc + q);
                }
            }
        }
        if (lane == 0) hg::store_wait_all();
        if (CTAS == 1 && a.splits > 1) {
            __syncwarp();
            hg::cluster_sync();   // the cluster's sums are there
            item_of(a, blockIdx.x, t);
            const int n4 = min(128, a.M - t.m * 128) * 32;   // quads of the tile's rows
            const int f0 = n4 * t.s / a.splits + threadIdx.x - kThreads0, f1 = n4 * (t.s + 1) / a.splits;
            if (a.splits <= 4) join<4, 4>(a, t, s0, f0, f1);   // (as many loads on their way as registers allow)
            else join<8, 2>(a, t, s0, f0, f1);
            __syncwarp();
            hg::cluster_sync();   // no CTA leaves while its sums are read
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0 || warp == 3) {
            // ---------------- producers (whole warps): A, and W
            const bool isA = warp == 0;
            uint32_t s = 0, ph = 1;   // stage, and the parity of its last release
            Item t;
            for (int i = first; ok && item_of(a, i, t); i += step) {
                const int ma = (t.m * CTAS + (int)rank) * 128;
                const int nb = t.n * BN + (int)rank * 128;
                auto arows = [&](int r) {   // rows of A that each CTA of the cluster loads
                    const int left = a.M - (t.m * CTAS + r) * 128;
                    return left >= 128 ? 128 : left > 0 ? a.tail : 0;
                };
                const uint32_t bytes = CTAS * kOpBytes + (arows(0) + (CTAS == 2 ? arows(1) : 0)) * 128u;
                const int mine = arows(rank);
                for (int k = t.k0; k < t.k1; ++k) {
                    const uint32_t fb = CTAS == 2 ? hg::map_leader(full(s)) : full(s);
                    const uint32_t sb = s0 + s * stage_bytes, sa = sb + kOpBytes;
                    if (!(ok = __all_sync(0xffffffffu, mbar_wait(empty(s), ph, a.err, 1, a.wait_ns)))) break;
                    if (isA) {
                        if (rank == 0) hg::expect_tx_warp(full(s), bytes);
                        if (mine) hg::load_2d_warp<CTAS>(sa, mine == 128 ? &tmA : &tmAt, k * kStep, ma, fb);
                    } else {
                        hg::load_2d_warp<CTAS>(sb, &tmB, k * kStep, nb, fb);
                    }
                    __syncwarp();
                    if (++s == stages) s = 0, ph ^= 1;
                }
            }
        } else if (warp == 1) {
            // ---------------- MMA issuer
            if (rank == 0) {
                const uint32_t idesc = idesc_e4m3(CTAS * 128, BN);
                const uint64_t db0 = tc::sdesc(s0), da0 = tc::sdesc(s0 + kOpBytes);
                uint32_t s = 0, ph = 0, gc = 0;
                Item t;
                for (int i = first; ok && item_of(a, i, t); i += step) {
                    for (int k = t.k0; k < t.k1; ++k, ++gc) {
                        const uint32_t b = gc % kBufs;
                        ok = __all_sync(0xffffffffu,
                                        mbar_wait(tempty(b), ((gc / kBufs) & 1) ^ 1, a.err, 2, a.wait_ns) &&
                                            mbar_wait(full(s), ph, a.err, 3, a.wait_ns));
                        if (!ok) break;
                        tc_fence_after();
                        mma_step_warp<CTAS>(tmem + b * BN, da0 + s * (stage_bytes >> 4), db0 + s * (stage_bytes >> 4),
                                            idesc, empty(s));
                        // (withheld by the test hook: the epilogue's bounded wait runs out)
                        if (i != a.skip_item) hg::commit_warp<CTAS>(tfull(b));
                        if (++s == stages) s = 0, ph ^= 1;
                    }
                }
            }
        }
        if (CTAS == 1 && a.splits > 1) {   // (the epilogue's two meetings)
            __syncwarp();
            hg::cluster_sync();
            hg::cluster_sync();
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
    if constexpr (CTAS == 2) hg::cluster_sync();   // no CTA leaves while its peer still signals it
    tc_fence_after();
    if (warp == 2) {
        if constexpr (CTAS == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

}  // namespace w8
}  // namespace pmoe
