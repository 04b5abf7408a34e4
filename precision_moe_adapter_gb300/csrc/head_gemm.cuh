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
//   warps 0, 3  TMA producers of this CTA's 128 rows of A, and of its BN/CTAS
//               rows of B (one warp for both would bound the
//               smaller tiles by the rate at which it issues copies)
//   warp 1      MMA issuer (CTA 0 of the cluster only), K steps of 64
//   warp 2      TMEM allocator
//   warps 4..   epilogue, one warp per 32 TMEM lanes and 128 columns: a
//               thread owns one row's 128 columns, in registers
//
// The tensor cores' FP32 accumulation truncates: its error grows linearly
// with the number of K steps (about one part in 2^24 per 16 columns).  Every
// run of chunk_of(EPI) K steps is therefore summed in its own TMEM buffer and
// added to the tile's FP32 sum in registers (round to nearest), which bounds
// the error at any length.  (DX and DW end with the extra steps described below
// in their last run.  At most T / 8 of them meet in one tile, and the four MMAs of
// each lose up to 2^-24 of that run's sum: 6e-5 of dW at any T, should all tokens
// have all their 8 entries in one block of the vocabulary, for results that are
// rounded to 2^-9.)  The forward's values are FP32 outputs:
// runs of 512 columns, relative error about 5e-7; GRAD takes the same runs, so
// that its logits are the forward's bit for bit and p - 1 of a confident token
// does not see their error.  The other results are rounded to BF16, so longer
// runs do.  (Runs of 256 columns in FWD and GRAD cost a step at
// T = 4096, d = 2048, V = 131072 1 to 2%.)
// The two buffers alternate, so the tensor cores work on the next chunk while
// one is drained, and on the next tile's first two chunks during the epilogue
// proper: 91 to 97% of the tensor pipe's cycles are busy at T = 4096, d = 2048,
// V = 32768, and a step at T = 8192, d = 7168, V = 131072 runs its three
// products at 1.65 to 1.72 PFLOP/s (27 to 28 ms), the card's sustained rate.
// Exponentials are ex2.approx, whose relative error PTX bounds by about 2^-22;
// their arguments are rounded once, 2^-24 of their size.
//
// G is the BF16 operand of two products.  Where a token's distribution is
// concentrated, a few large entries of G carry the whole gradient, and their
// rounding to 8 bits would be its error.  GRAD lists the entries with
// |p - q| >= kLarge (a token has at most 8, as sum |p - q| <= 2; with a single
// target y, |p - q| >= kLarge (1 - p_y): at most 5), and the products run
// extra K steps of 64 such entries each on the roundings' remainders (a second
// BF16, 16 bits together): A holds one remainder per column (built by head.cu,
// one list per 256 output rows), B the matching rows of W or X, gathered by
// TMA.  That is a few steps per tile of the hundreds the product has;
// remainders of whole tiles would double the steps of every tile that holds a
// large entry.  (Where the vocabulary is so small that the lists would be long,
// all remainders are kept beside G and the products run over both: head.cu,
// `terms`.)  A teacher that is spread over many entries has none that large, and
// its gradient takes the rounding of G's entries to 8 bits beside its own: dX at
// T = 4096, d = 2048, V = 131072, K = 64 (the largest q about 0.16) is 1.95e-3 from
// FP64, 1.66e-3 being dX's own rounding.  Listing from 1/16 (up to 32 entries a
// token) gives 1.78e-3 and from 1/32 1.72e-3, for 0 and 3% of that step but 26 and
// 94% of one at T = 1024, d = 512, V = 32000, K = 16 with both gradients.
//
// Anchors: where a token's target (or an entry of the teacher) holds much of
// the probability, the value and G there are differences of nearly equal
// numbers, and the tensor cores' error of z (5e-7 relative, biased) would be
// 1e-6 and more of them.  The logits of the target, or of teacher entries
// with q >= 1/4 (at most 4), are therefore computed in FP32 by head.cu: FWD leaves
// these columns out of its sums, so that what is left of the probability keeps
// its own relative accuracy, and GRAD is given these entries of G.
//
// Every logit's sum runs over k in the same order whatever the tile shape, and
// the softmax partials cover 128 aligned columns: the forward's results do not
// depend on the number of tokens in the call.  (A row of dX may, in its last
// bits: the pieces of the vocabulary, the cuts along K and the choice between
// lists and whole remainders go by T.)
#pragma once

#include "gemm_tc.cuh"
#include "pdl.cuh"

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
constexpr int kOpBytes = 128 * kBK * 2;  // one operand tile of a stage (16 KB)
// The ring of stages, each B's tile and then A's: 6 of 32 KB; where A has few
// rows its tiles are that much smaller and the ring deeper (11 stages for up
// to 8 tokens), which is what streaming W needs.  The MMA then reads past A's
// rows into the next stage: those rows of the result are not stored.
constexpr int kRingBytes = 6 * 2 * kOpBytes;
constexpr int kMaxStages = 11;
static_assert(kMaxStages * (kOpBytes + 1024) <= kRingBytes, "deepest ring");
constexpr int kWarpOut = 32 * 128;       // a warp's staged output box: 32 rows of 128 bytes
// K steps summed in one TMEM buffer
constexpr int chunk_of(int epi) { return epi == HG_FWD || epi == HG_GRAD ? 8 : 32; }
constexpr int32_t kNoId = 0x7fffffff;
constexpr float kLarge = 0.25f;          // entries of |p - q| that keep their remainder
constexpr int kMaxLarge = 8;             // of a token
constexpr int kListRows = 256;           // output rows that share a list of remainders
constexpr int kThreads0 = 128;           // producer, MMA and allocator warps

constexpr int epi_warps(int BN) { return BN / kUnit * 4; }
constexpr int threads_of(int BN) { return kThreads0 + 32 * epi_warps(BN); }
// 1024 bytes of slack to align the swizzled tiles, 256 for the barriers
constexpr int smem_of(int BN) { return kRingBytes + epi_warps(BN) * kWarpOut + 256 + 1024; }

struct Args {
    int M, N;                // output rows and columns of this launch
    int n0;                  // GRAD: first vocabulary column; FWD: 0
    int mt, nt, gm;          // tiles, and m tiles that run together
    int ksteps;              // K steps of 64 of a tile
    int whole;               // tiles taken whole; each of the others is cut into
    int splits, kper;        // `splits` items of kper K steps
    int kb0;                 // first k coordinate of B (A: 0)
    int stages, abytes;      // the ring: stages, and bytes of A in one
    int tail;                // FWD, GRAD, DX: rows of tmAt's boxes, the M % 128 last rows of A
                             // (a box with rows past the tensor's end loads slowly)
    int V;                   // FWD, GRAD: number of vocabulary entries
    float scale, c;          // GRAD: the logits' factor; FWD: that times log2(e)
    int NU;                  // FWD, GRAD: units of the vocabulary
    float2 *part;            // FWD: [T][NU] (largest z, sum of 2^(c z - its c z))
    // the target entries of FWD and GRAD: one per token with probability 1 (an
    // anchor), or up to K per token, in vocabulary order
    const int32_t *target;   // [T], or NULL
    const uint16_t *tab;     // [T][NU]: 0 where the unit has none, else 256 + place of its first
    const uint4 *mask;       // [T][NU]: the unit's columns that have one (where tab is not 0)
    const float *q;          // GRAD: [T][K] probabilities
    float *zt;               // FWD: [T][K] raw logits of a teacher's entries (out)
    int K;
    const float *lse;        // GRAD: [T]
    const float2 *coef;      // GRAD: [T] factor of the row (0: no gradient) and least |G| of an
                             // entry that keeps its remainder
    const int4 *anchor;      // [T] vocabulary ids of the row's anchors (-1: none; FWD: without
    const float4 *anchor_g;  // targets) and, GRAD, their entries of G
    int terms;               // 2: G's remainders are kept in whole, aoff columns to the right of
    int aoff;                // G, and no entries are listed; DX, DW: K runs over both, kone
    int kone;                // steps each
    int *cnt;                // GRAD: [T] large entries of each token, listed in
    int2 *large;             // [T][kMaxLarge] as (vocabulary column - n0, remainder)
    uint8_t *fl;             // GRAD: [vocabulary block of 256][fs] 1 where a block of 128
    int fs;                  // tokens holds a large entry (NULL: not wanted)
    const int2 *lists;       // DX, DW: per 256 rows (first step, number of steps) of remainders
    const int32_t *lidx;     // DX, DW: [step][64] row of B
    int lb0;                 // DX, DW: offset of these rows
    int beside;              // DW: launched right behind DX
    int accumulate;          // DX: add to the FP32 partials
    int bf16_out;            // DX: the output map is the BF16 dX itself
    uint64_t wait_ns;        // limit of every wait
    int skip_item;           // test hook: work item whose accumulator-full signals are withheld (-1: none)
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
// (what it orders are TMEM reads, which tcgen05's own fence covers; a release
// at cluster scope would also wait for the warp's global stores)
__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The calls named *_warp are made by a whole converged warp, so that their
// operands stay in uniform registers; one elected lane issues.  (Issued from
// a branch on the lane, each MMA or copy first moves its operands there: a K
// step then takes the same time whatever the tile's size.)
template <int CTAS>
__device__ __forceinline__ void load_2d_warp(uint32_t dst, const CUtensorMap *tm, int x, int y, uint32_t bar)
{
    if constexpr (CTAS == 2)   // the barrier may be the other CTA's
        asm volatile(
            "{ .reg .pred e; elect.sync _|e, 0xffffffff;\n"
            "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3}], [%4]; }" ::"r"(dst),
            "l"((uint64_t)tm), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred e; elect.sync _|e, 0xffffffff;\n"
            "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3}], [%4]; }" ::"r"(dst),
            "l"((uint64_t)tm), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void expect_tx_warp(uint32_t bar, uint32_t bytes)
{
    asm volatile("{ .reg .pred e; elect.sync _|e, 0xffffffff;\n"
                 "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1; }" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}
// Rows r.x .. r.w of a map whose boxes are one row of 128 bytes, from column x
template <int CTAS>
__device__ __forceinline__ void gather4(uint32_t dst, const CUtensorMap *tm, int x, int4 r, uint32_t bar)
{
    if constexpr (CTAS == 2)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2 "
            "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
            "l"((uint64_t)tm), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
            "l"((uint64_t)tm), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
            : "memory");
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
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A K step of 64: four MMAs of K = 16, da and db advancing by sa and sb, and
// the commit of `bar` (of both CTAs of a pair), which completes when the MMAs
// issued so far have
template <int CTAS>
__device__ __forceinline__ void mma_step_warp(uint32_t d, uint64_t da, uint64_t db, uint32_t sa, uint32_t sb,
                                              uint32_t idesc, uint32_t accum, uint32_t bar)
{
    if constexpr (CTAS == 2)
        asm volatile(
            "{ .reg .pred e, p, t; elect.sync _|e, 0xffffffff; setp.ne.b32 p, %10, 0; setp.eq.b32 t, %10, %10;\n"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %5, %9, p;\n"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %2, %6, %9, t;\n"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %3, %7, %9, t;\n"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %4, %8, %9, t;\n"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%11], %12; }" ::"r"(
                d),
            "l"(da), "l"(da + sa), "l"(da + 2 * sa), "l"(da + 3 * sa), "l"(db), "l"(db + sb), "l"(db + 2 * sb),
            "l"(db + 3 * sb), "r"(idesc), "r"(accum), "r"(bar), "h"((uint16_t)3)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred e, p, t; elect.sync _|e, 0xffffffff; setp.ne.b32 p, %10, 0; setp.eq.b32 t, %10, %10;\n"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %5, %9, p;\n"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %6, %9, t;\n"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %7, %9, t;\n"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %8, %9, t;\n"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%11]; }" ::"r"(d),
            "l"(da), "l"(da + sa), "l"(da + 2 * sa), "l"(da + 3 * sa), "l"(db), "l"(db + sb), "l"(db + 2 * sb),
            "l"(db + 3 * sb), "r"(idesc), "r"(accum), "r"(bar)
            : "memory");
}
template <int CTAS>
__device__ __forceinline__ void commit_warp(uint32_t bar)
{
    if constexpr (CTAS == 2)
        asm volatile(
            "{ .reg .pred e; elect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1; }" ::"r"(
                bar),
            "h"((uint16_t)3)
            : "memory");
    else
        tc::umma_commit_warp(bar);
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

// 32 TMEM columns of the warp's lanes; complete after tmem_wait on the same registers
__device__ __forceinline__ void tmem_issue32(uint32_t taddr, float *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait(float *v)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                   "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]),
                   "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]),
                   "+f"(v[29]), "+f"(v[30]), "+f"(v[31])::"memory");
}
__device__ __forceinline__ uint32_t bf2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

struct Item {
    int m, n, s;   // m tile, n tile, split
    int part;      // s > 0: place among the further parts of the cut tiles
    int k0, k1;    // K steps
};
// Work item i (the whole tiles, then the others' first parts, their second
// parts, ...); false past the last one
__device__ __forceinline__ bool item_of(const Args &a, int i, Item &t)
{
    t.s = 0;
    t.k0 = 0;
    t.k1 = a.ksteps;
    if (i >= a.whole) {
        const int cut = a.mt * a.nt - a.whole;
        if (i - a.whole >= cut * a.splits) return false;
        t.s = (i - a.whole) / cut;
        i -= t.s * cut;
        t.part = (t.s - 1) * cut + i - a.whole;
        t.k0 = t.s * a.kper;
        t.k1 = min(t.k0 + a.kper, a.ksteps);
    }
    const int gsz = a.gm * a.nt, g = i / gsz;
    i -= g * gsz;
    const int gm = min(a.gm, a.mt - g * a.gm);   // the last group may be smaller
    t.n = i / gm;
    t.m = g * a.gm + i - t.n * gm;
    return true;
}

// ------------------------------------------------------------------ kernel
template <int CTAS, int BN, int EPI>
__global__ void __launch_bounds__(threads_of(BN), 1) k_head_gemm(const __grid_constant__ CUtensorMap tmA,
                                                                 const __grid_constant__ CUtensorMap tmAt,
                                                                 const __grid_constant__ CUtensorMap tmB,
                                                                 const __grid_constant__ CUtensorMap tmOut,
                                                                 const __grid_constant__ CUtensorMap tmPart,
                                                                 const __grid_constant__ CUtensorMap tmLoA,
                                                                 const __grid_constant__ CUtensorMap tmLoB,
                                                                 const Args a)
{
    constexpr bool kAMn = EPI == HG_DW, kBMn = EPI == HG_DX || EPI == HG_DW;
    constexpr int kEpi = epi_warps(BN);
    static_assert(BN / CTAS == 128, "one 128-row operand tile of B per CTA");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t s0 = smem_u32(smem);
    const uint32_t out0 = s0 + kRingBytes;
    const uint32_t bar0 = out0 + kEpi * kWarpOut;
    auto full = [&](uint32_t s) { return bar0 + 8 * s; };
    auto empty = [&](uint32_t s) { return bar0 + 8 * (kMaxStages + s); };
    auto tfull = [&](uint32_t b) { return bar0 + 8 * (2 * kMaxStages + b); };
    auto tempty = [&](uint32_t b) { return bar0 + 8 * (2 * kMaxStages + 2 + b); };
    const uint32_t slot = bar0 + 8 * (2 * kMaxStages + 4);
    const uint32_t stages = (uint32_t)a.stages, stage_bytes = kOpBytes + (uint32_t)a.abytes;

    // (through a shuffle: the compiler then knows the warp's number to be uniform)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 2 ? cta_rank() : 0u;
    const int first = blockIdx.x / CTAS, step = gridDim.x / CTAS;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
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

    // DW after DX: its inputs were complete when DX started, so it runs beside
    // DX and waits for it at the end only (whatever comes next waits for both)
    if (EPI != HG_DW || !a.beside) grid_wait();
    grid_go();
    // DX, DW: the item's extra K steps on remainders (with a tile's first K step)
    constexpr bool kLo = EPI == HG_DX || EPI == HG_DW;
    constexpr int kChunk = chunk_of(EPI);
    auto extra = [&](const Item &t) {
        if constexpr (kLo)
            if (t.k0 == 0 && a.terms == 1) return __ldcg(a.lists + t.m * CTAS * 128 / kListRows);
        return make_int2(0, 0);
    };
    bool ok = true;
    // The epilogue's 128 sums a thread need more registers than an even split
    // of 384 threads gives (168): the first four warps hand theirs over.  Of
    // the launch's 384 x 168 = 64512: 128 x 40 + 256 x 232, and where the
    // producer and the MMA issuer run extra steps 128 x 72 + 256 x 216.
    if (warp >= 4) {
        // ---------------- epilogue
        if constexpr (kEpi == 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLo ? 216 : 232));
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const int rl = quad * 32 + lane;   // row of the CTA's 128
        const uint32_t tld = tmem + ((uint32_t)(quad * 32) << 16) + half * kUnit;
        const uint32_t ob = out0 + (warp - 4) * kWarpOut, orow = ob + lane * 128;
        const float inf = __int_as_float(0x7f800000);
        uint32_t gc = 0;
        Item t;
        for (int i = first; ok && item_of(a, i, t); i += step) {
            const int k0 = t.k0, k1 = t.k1;
            const int mrow = (t.m * CTAS + (int)rank) * 128;
            const int row = mrow + rl;
            const int cb = a.n0 + t.n * BN + half * kUnit;   // first column
            const int nv = min(kUnit, a.V - cb);             // FWD, GRAD: valid columns (may be <= 0)
            const bool live = row < a.M && nv > 0;
            // the row's target entries among the columns (a bit each) and the place
            // of the first, its normaliser and factor: fetched while the tensor
            // cores work
            uint32_t mw[kUnit / 32] = {0, 0, 0, 0};
            int64_t pos = (int64_t)row * a.K;
            float lse = 0.f;
            float2 cf = make_float2(0.f, 0.f);   // factor, least large entry
            int an[4] = {-1, -1, -1, -1};        // anchors and their entries of G
            float ag[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (EPI == HG_FWD || EPI == HG_GRAD) {
                if (EPI == HG_FWD && live) {
                    if (a.target) {
                        an[0] = a.target[row];
                    } else {
                        const int4 i4 = a.anchor[row];
                        an[0] = i4.x, an[1] = i4.y, an[2] = i4.z, an[3] = i4.w;
                    }
                }
                if (live && !a.target) {
                    const int64_t at = (int64_t)row * a.NU + cb / kUnit;
                    const int e = a.tab[at];
                    if (e) {
                        const uint4 m = a.mask[at];
                        mw[0] = m.x, mw[1] = m.y, mw[2] = m.z, mw[3] = m.w;
                        pos += e - 256;
                    }
                }
                if (EPI == HG_GRAD && row < a.M) {
                    lse = a.lse[row];
                    cf = a.coef[row];
                    const int4 i4 = a.anchor[row];
                    const float4 g4 = a.anchor_g[row];
                    an[0] = i4.x, an[1] = i4.y, an[2] = i4.z, an[3] = i4.w;
                    ag[0] = g4.x, ag[1] = g4.y, ag[2] = g4.z, ag[3] = g4.w;
                }
            }
            float acc[kUnit];
            for (int c0 = k0; c0 < k1; c0 += kChunk, ++gc) {
                const uint32_t b = gc & 1;
                // (warp-uniform: every lane sees the same outcome before the aligned loads)
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(tfull(b), (gc >> 1) & 1, a.err, 4, a.wait_ns))))
                    break;
                tc_fence_after();
                if constexpr (kLo) {   // (16 columns at a time: fewer registers)
                    if (c0 == k0) {
#pragma unroll
                        for (int j = 0; j < kUnit; ++j) acc[j] = 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < kUnit; j += 16) {
                        float v[16];
                        tc::tmem_ld16(tld + b * BN + j, v);
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[j + e] += v[e];
                    }
                } else if (c0 == k0) {
#pragma unroll
                    for (int j = 0; j < kUnit; j += 32) tmem_issue32(tld + b * BN + j, acc + j);
#pragma unroll
                    for (int j = 0; j < kUnit; j += 32) tmem_wait(acc + j);
                } else {
#pragma unroll
                    for (int j = 0; j < kUnit; j += 32) {
                        float v[32];
                        tmem_issue32(tld + b * BN + j, v);
                        tmem_wait(v);
#pragma unroll
                        for (int e = 0; e < 32; ++e) acc[j + e] += v[e];
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CTAS == 2) arrive_cluster(map_leader(tempty(b)));
                    else mbar_arrive(tempty(b));
                }
            }
            if (!ok) break;
            if constexpr (EPI == HG_FWD) {
#pragma unroll
                for (int q = 0; q < kUnit; q += 32) {
                    if (__any_sync(0xffffffffu, mw[q / 32] != 0)) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (mw[q / 32] >> j & 1u) a.zt[pos++] = acc[q + j];
                    }
                    // the anchors stay out of the sum: the combine adds them
                    uint32_t out = 0;
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const uint32_t j = (uint32_t)an[n] - (uint32_t)(cb + q);
                        out |= j < 32u ? 1u << j : 0u;
                    }
                    if (__any_sync(0xffffffffu, out != 0)) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (out >> j & 1u) acc[q + j] = -inf;
                    }
                }
                if (nv < kUnit) {
#pragma unroll
                    for (int j = 0; j < kUnit; ++j)
                        if (j >= nv) acc[j] = -inf;
                }
                float mx[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = acc[e];
#pragma unroll
                for (int j = 4; j < kUnit; ++j) mx[j & 3] = fmaxf(mx[j & 3], acc[j]);
                // (logits of -inf only sum to zero, and a NaN among them to NaN)
                const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), m2 = m == -inf ? 0.f : m * a.c;
                float sm[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < kUnit; ++j) sm[j & 3] += ex2(fmaf(acc[j], a.c, -m2));
                if (live)
                    a.part[(int64_t)row * a.NU + cb / kUnit] = make_float2(m, (sm[0] + sm[1]) + (sm[2] + sm[3]));
            } else {
                // through shared memory (the warp's 32 rows of 128 bytes, 128-byte
                // swizzle) to TMA stores, which clip rows and columns past the end
                const int xc = t.n * BN + half * kUnit, yr = mrow + quad * 32;
                auto put = [&](int x, int xoff = 0) {   // the staged box goes out at column x (+ xoff)
                    tc::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0 && x < a.N && yr < a.M) {
                        if (EPI == HG_DX && t.s > 0)    // a tile of its own
                            store_3d(&tmPart, ob, x - t.n * BN, yr - t.m * CTAS * 128, t.part, a.accumulate != 0);
                        else store_3d(&tmOut, ob, x + xoff, yr, 0, a.accumulate != 0);
                    }
                };
                auto reuse = [&]() {                             // the previous box has been read
                    if (lane == 0) store_wait_read();
                    __syncwarp();
                };
                auto stage16 = [&](int e0) {                     // columns e0 .. e0 + 63 in BF16
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int e = e0 + j * 8;
                        tc::st_shared_v4(orow + ((j ^ (lane & 7)) << 4),
                                         make_uint4(bf2(acc[e], acc[e + 1]), bf2(acc[e + 2], acc[e + 3]),
                                                    bf2(acc[e + 4], acc[e + 5]), bf2(acc[e + 6], acc[e + 7])));
                    }
                };
                if constexpr (EPI == HG_GRAD) {
                    uint32_t large[kUnit / 32], any = 0;   // the columns to list
#pragma unroll
                    for (int q = 0; q < kUnit; q += 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)   // (the difference is exact near p = 1)
                            acc[q + j] = ex2((__fmul_rn(acc[q + j], a.scale) - lse) * 1.4426950408889634f) * cf.x;
                        if (__any_sync(0xffffffffu, mw[q / 32] != 0)) {
#pragma unroll
                            for (int j0 = 0; j0 < 32; j0 += 8) {   // (eight loads on their way at once)
                                float v[8];
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    v[j] = 0.f;
                                    if (mw[q / 32] >> (j0 + j) & 1u) v[j] = a.q[pos++];
                                }
#pragma unroll
                                for (int j = 0; j < 8; ++j) acc[q + j0 + j] = fmaf(v[j], -cf.x, acc[q + j0 + j]);
                            }
                        }
                        const int e0 = cb + q;
                        auto in = [&](int id) { return (unsigned)(id - e0) < 32u; };
                        if (__any_sync(0xffffffffu, in(an[0]) || in(an[1]) || in(an[2]) || in(an[3]))) {
#pragma unroll 1
                            for (int n = 0; n < 4; ++n) {
                                const int j0 = (n == 0 ? an[0] : n == 1 ? an[1] : n == 2 ? an[2] : an[3]) - e0;
                                const float gv = n == 0 ? ag[0] : n == 1 ? ag[1] : n == 2 ? ag[2] : ag[3];
#pragma unroll
                                for (int j = 0; j < 32; ++j) acc[q + j] = j == j0 ? gv : acc[q + j];
                            }
                        }
                        if (nv < kUnit) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (q + j >= nv) acc[q + j] = 0.f;
                        }
                        float big = 0.f;
#pragma unroll
                        for (int j = 0; j < 32; ++j) big = fmaxf(big, fabsf(acc[q + j]));
                        const bool keep = big >= cf.y && cf.x != 0.f && a.terms == 1;
                        large[q / 32] = 0;
                        if (__any_sync(0xffffffffu, keep)) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                large[q / 32] |= keep && fabsf(acc[q + j]) >= cf.y ? 1u << j : 0u;
                        }
                        any |= large[q / 32];
                        // a row without gradient stays zero, whatever its hidden state holds
                        if (__any_sync(0xffffffffu, cf.x == 0.f)) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) acc[q + j] = cf.x == 0.f ? 0.f : acc[q + j];
                        }
                        if (q & 32) {
                            reuse();
                            stage16(q - 32);
                            put(xc + q - 32);
                        }
                    }
                    if (a.terms == 2) {
#pragma unroll
                        for (int q = 0; q < kUnit; q += 64) {
#pragma unroll
                            for (int j = 0; j < 64; ++j) acc[q + j] -= bf2f(f2bf(acc[q + j]));   // exact
                            reuse();
                            stage16(q);
                            put(xc + q, a.aoff);
                        }
                    }
                    if (__any_sync(0xffffffffu, any != 0)) {
                        int n = 0;
                        if (any) {
#pragma unroll
                            for (int q = 0; q < kUnit / 32; ++q) n += __popc(large[q]);
                            n = atomicAdd(&a.cnt[row], n);
                            if (a.fl) a.fl[(int64_t)((cb - a.n0) / kListRows) * a.fs + (row >> 7)] = 1;
                        }
#pragma unroll
                        for (int q = 0; q < kUnit; q += 32) {
                            while (__any_sync(0xffffffffu, large[q / 32] != 0)) {
                                const int j0 = __ffs(large[q / 32]) - 1;
                                float v = 0.f;
#pragma unroll
                                for (int j = 0; j < 32; ++j) v = j == j0 ? acc[q + j] : v;
                                if (large[q / 32] && n < kMaxLarge)
                                    a.large[(int64_t)row * kMaxLarge + n++] =
                                        make_int2(cb + q - a.n0 + j0, f2bf(v - bf2f(f2bf(v))));
                                large[q / 32] &= large[q / 32] - 1;
                            }
                        }
                    }
                } else if (EPI == HG_DX && !a.bf16_out) {
#pragma unroll
                    for (int q = 0; q < kUnit; q += 32) {
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
                    for (int q = 0; q < kUnit; q += 64) {
                        reuse();
                        stage16(q);
                        put(xc + q);
                    }
                }
            }
        }
        if (EPI != HG_FWD && lane == 0) store_wait_all();
    } else {
        if constexpr (kEpi == 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLo ? 72 : 40));
        if (warp == 0 || warp == 3) {
            // ---------------- producers (whole warps): A, and B
            const bool isA = warp == 0;
            uint32_t s = 0, ph = 1;   // stage, and the parity of its last release
            Item t;
            for (int i = first; ok && item_of(a, i, t); i += step) {
                const int k0 = t.k0, k1 = t.k1;
                const int2 ex = extra(t);
                const int ma = (t.m * CTAS + (int)rank) * 128;
                const int nb = a.n0 + t.n * BN + (int)rank * 128;
                // rows of A that each CTA of the cluster loads (what lies below them in
                // shared memory only reaches rows that are not stored)
                auto arows = [&](int r) {
                    const int left = a.M - (t.m * CTAS + r) * 128;
                    return kAMn || left >= 128 ? 128 : left > 0 ? a.tail : 0;
                };
                const uint32_t bytes = CTAS * kOpBytes + (arows(0) + (CTAS == 2 ? arows(1) : 0)) * 128u;
                const int mine = arows(rank);
                auto slot_free = [&]() {
                    return ok = __all_sync(0xffffffffu, mbar_wait(empty(s), ph, a.err, 1, a.wait_ns));
                };
                auto next = [&]() {
                    __syncwarp();
                    if (++s == stages) s = 0, ph ^= 1;
                };
                // an extra step's rows of B: lanes 0-15 gather four each, fetched a step ahead
                auto rows_of = [&](int e) {
                    return kLo && !isA && lane < 16 && e < ex.y
                               ? __ldcg((const int4 *)(a.lidx + (int64_t)(ex.x + e) * 64 + lane * 4))
                               : make_int4(0, 0, 0, 0);
                };
                for (int k = k0; k < k1; ++k) {
                    const uint32_t fb = CTAS == 2 ? map_leader(full(s)) : full(s);
                    const uint32_t sb = s0 + s * stage_bytes, sa = sb + kOpBytes;
                    if (!slot_free()) break;
                    const int second = kLo && a.terms == 2 && k >= a.kone;   // the remainders' turn
                    const int kk = second ? k - a.kone : k, xo = second ? a.aoff : 0;
                    if (isA) {
                        if (rank == 0) expect_tx_warp(full(s), bytes);
                        const int ka = kk * kBK;
                        if constexpr (kAMn) {
                            load_2d_warp<CTAS>(sa, &tmA, ma + xo, ka, fb);
                            load_2d_warp<CTAS>(sa + 8192, &tmA, ma + xo + 64, ka, fb);
                        } else if (mine) {
                            load_2d_warp<CTAS>(sa, mine == 128 ? &tmA : &tmAt, ka + xo, ma, fb);
                        }
                    } else {
                        const int kb = a.kb0 + kk * kBK;
                        if constexpr (kBMn) {
                            load_2d_warp<CTAS>(sb, &tmB, nb, kb, fb);
                            load_2d_warp<CTAS>(sb + 8192, &tmB, nb + 64, kb, fb);
                        } else {
                            load_2d_warp<CTAS>(sb, &tmB, kb, nb, fb);
                        }
                    }
                    next();
                }
                int4 r = rows_of(0);
                for (int e = 0; kLo && ok && e < ex.y; ++e) {
                    const uint32_t fb = CTAS == 2 ? map_leader(full(s)) : full(s);
                    const uint32_t sb = s0 + s * stage_bytes, sa = sb + kOpBytes;
                    const int st = ex.x + e;
                    const int4 rn = rows_of(e + 1);
                    if (!slot_free()) break;
                    if (isA) {
                        if (rank == 0) expect_tx_warp(full(s), CTAS * 2 * kOpBytes);
                        if constexpr (kAMn) {   // remainders [step][64][256 rows]
                            load_2d_warp<CTAS>(sa, &tmLoA, ma % kListRows, st * 64, fb);
                            load_2d_warp<CTAS>(sa + 8192, &tmLoA, ma % kListRows + 64, st * 64, fb);
                        } else {                // [step][256 rows][64]
                            load_2d_warp<CTAS>(sa, &tmLoA, 0, st * kListRows + ma % kListRows, fb);
                        }
                    } else if (lane < 16) {
                        r.x += a.lb0, r.y += a.lb0, r.z += a.lb0, r.w += a.lb0;
                        gather4<CTAS>(sb + lane * 512, &tmLoB, nb, r, fb);
                        gather4<CTAS>(sb + 8192 + lane * 512, &tmLoB, nb + 64, r, fb);
                    }
                    r = rn;
                    next();
                }
            }
        } else if (warp == 1) {
            // ---------------- MMA issuer
            if (rank == 0) {
                const uint32_t idesc = tc::idesc_bf16(CTAS * 128, BN, kAMn) | ((uint32_t)kBMn << 16);
                constexpr uint32_t kAStep = kAMn ? 2048 >> 4 : 32 >> 4;   // 16 k
                constexpr uint32_t kBStep = kBMn ? 2048 >> 4 : 32 >> 4;
                const uint64_t db0 = desc_of<kBMn>(s0), da0 = desc_of<kAMn>(s0 + kOpBytes);
                uint32_t s = 0, ph = 0, gc = 0;
                Item t;
                for (int i = first; ok && item_of(a, i, t); i += step) {
                    const int k0 = t.k0, k1 = t.k1;
                    const int2 ex = extra(t);
                    for (int c0 = k0; ok && c0 < k1; c0 += kChunk, ++gc) {
                        const uint32_t b = gc & 1;
                        // (every lane waits; the outcome is made uniform)
                        ok = __all_sync(0xffffffffu, mbar_wait(tempty(b), ((gc >> 1) & 1) ^ 1, a.err, 2, a.wait_ns));
                        if (!ok) break;
                        tc_fence_after();
                        int c1 = c0 + kChunk;
                        if (c1 >= k1) c1 = k1 + ex.y;   // (the extra steps join the last chunk)
                        for (int k = c0; k < c1; ++k) {
                            ok = __all_sync(0xffffffffu, mbar_wait(full(s), ph, a.err, 3, a.wait_ns));
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t da = da0 + s * (stage_bytes >> 4), db = db0 + s * (stage_bytes >> 4);
                            mma_step_warp<CTAS>(tmem + b * BN, da, db, kAStep, kBStep, idesc, k > c0, empty(s));
                            if (++s == stages) s = 0, ph ^= 1;
                        }
                        // (withheld by the test hook: the epilogue's bounded wait runs out)
                        if (ok && i != a.skip_item) commit_warp<CTAS>(tfull(b));
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
    if (EPI == HG_DW && a.beside) grid_wait();
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
