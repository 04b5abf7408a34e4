// head.cu -- losses of the vocabulary head: token log-probabilities and
// distillation from a teacher's top logits, forward and backward, without
// keeping the logits.  The products run on the tensor cores
// (head_gemm.cuh); this file holds the per-token kernels, the workspace
// layout, the choice of tiles and the entry points.
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "head_gemm.cuh"

namespace pmoe {
namespace tc {
// gemm_tc.cu: the bounded-wait limit and withheld item of the next products: the
// armed test hook (once), else the default limit and none
void take_wait_hook(uint64_t &wait_ns, int &skip_item);
}  // namespace tc
namespace hg {

constexpr int kMaxK = 256;                    // teacher entries per token
constexpr int kSms = 152;                     // SMs of a GB300
constexpr int64_t kPieceBytes = 512ll << 20;  // most bytes of G of a vocabulary piece

constexpr int kAnchors = 4;
constexpr float kAnchorQ = 0.25f;
// A token's anchors, [T][kAnchors]: vocabulary id (-1: none), place among the
// token's entries, entry of G
struct Anchors {
    int32_t *id;
    int *place;
    float *g;
};
// What k_head_teacher needs in the backward (coef NULL: forward)
struct TeacherGrad {
    const uint16_t *X, *W;
    int d;
    const float *lse, *g;
    float2 *coef;            // [T] factor of G, and least |G| of an entry that keeps its remainder
    uint16_t *xz;            // [T][d] X with zeros for the rows without gradient, or NULL
};

// x . w over d columns by a warp: exact products of BF16 rows, 8 columns a lane
// at a time, then a tree.  The order is fixed, so forward and backward agree.
// (Read past L1: the forward's call comes before its kernel's wait.)
__device__ __forceinline__ float row_dot(const uint16_t *x, const uint16_t *w, int d)
{
    float a = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x & 31; i < d / 8; i += 32) {
        const uint4 u = __ldcg((const uint4 *)x + i), v = __ldcg((const uint4 *)w + i);
        const uint32_t us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a = fmaf(bf2f((uint16_t)us[j]), bf2f((uint16_t)vs[j]), a);
            a = fmaf(bf2f((uint16_t)(us[j] >> 16)), bf2f((uint16_t)(vs[j] >> 16)), a);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
}
// dW = G^T X would take 0 * NaN from a row of X that has no gradient, whatever
// it holds: DW reads a copy in which such rows are zero, made by the warp that
// knows the row's factor.  (T = 4096, d = 2048, V = 32000, forward and both
// gradients: 1351 us with the copy, 1343 without.)
__device__ __forceinline__ void copy_row(uint16_t *__restrict__ out, const uint16_t *__restrict__ x, int d, float cf)
{
#pragma unroll 4
    for (int i = threadIdx.x & 31; i < d / 8; i += 32)
        ((uint4 *)out)[i] = cf != 0.f ? ((const uint4 *)x)[i] : make_uint4(0, 0, 0, 0);
}
// Least |G| of an entry that keeps its remainder: `share` of the factor's size,
// and not below the least normal number, as a threshold that underflows to
// zero would list every column, those past the vocabulary's end among them
__device__ __forceinline__ float least_large(float cf, float share)
{
    return fmaxf(kLarge * share * fabsf(cf), 1.17549435e-38f);
}
// p - q of an entry with logit z
__device__ __forceinline__ float p_minus_q(float z, float scale, float lse, float q)
{
    return expm1f(__fmul_rn(z, scale) - lse) + (1.f - q);
}

// ------------------------------------------------------------------ targets
// The backward's first kernel also clears the counters of its first piece.
__device__ __forceinline__ void clear(int *p, int n)
{
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) p[i] = 0;
}

// Distillation: the teacher's K entries of a token as probabilities, q =
// softmax(scale t) over the entries present.  Entries with one id become one:
// q is their sum and h their sum of q log q.  They are placed in vocabulary
// order, and for every unit of 128 vocabulary entries that has some, tab
// holds 256 + the place of its first and mask its columns, so that the GEMM's
// epilogue takes a unit's entries one after the other.
// A warp per token sorts 32 kN words (id << 8 | slot; kGone last) in its
// registers, word i of a lane being element 32 i + lane, by a bitonic network
// (comparing every entry with every other one takes K / 32 times as many steps
// as there are words).
constexpr uint32_t kGone = 0xFFFFFFFFu;   // (V < 2^24: no id reaches it)
template <int kN>
__global__ void __launch_bounds__(128) k_head_teacher(int T, int V, int K, float scale, const int32_t *__restrict__ t_idx,
                                                      const float *__restrict__ t_logits,
                                                      float *__restrict__ q, float *__restrict__ h,
                                                      int *__restrict__ nent, uint16_t *__restrict__ tab,
                                                      uint4 *__restrict__ mask, int NU, Anchors an, TeacherGrad b,
                                                      int *__restrict__ zero, int nzero, DevErr *err)
{
    constexpr int kAll = 32 * kN;
    __shared__ float2 sq[4][kAll];            // (q, q log q) by slot
    __shared__ uint32_t sk[4][kAll];          // the sorted words
    __shared__ __align__(16) uint32_t smask[4][kAll][4];   // by the place of a unit's first entry
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * 4 + warp;
    grid_wait();
    grid_go();
    clear(zero, nzero);
    if (t >= T) return;
    const float inf = __int_as_float(0x7f800000);
    uint32_t w[kN];
    float x[kN], m = -inf;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int k = i * 32 + lane;
        w[i] = kGone;
        x[i] = -inf;
        if (k < K) {
            const int id = t_idx[(int64_t)t * K + k];
            const float l = t_logits[(int64_t)t * K + k] * scale;
            if (id >= V) record_error(err, PMOE_ERR_BAD_INDEX, t, id);
            if (id >= 0 && id < V && l != -inf) {   // (a logit of -inf has probability zero)
                w[i] = (uint32_t)id << 8 | k;
                x[i] = l;
                m = fmaxf(m, l);
            }
        }
        *(uint4 *)smask[warp][k] = make_uint4(0, 0, 0, 0);
    }
    for (int u = lane; u < NU; u += 32) tab[(int64_t)t * NU + u] = 0;
    float s = 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
    for (int i = 0; i < kN; ++i) s += w[i] != kGone ? expf(x[i] - m) : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float ls = logf(s);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const float qk = w[i] != kGone ? expf(x[i] - m) / s : 0.f;
        sq[warp][i * 32 + lane] = make_float2(qk, qk > 0.f ? qk * (x[i] - m - ls) : 0.f);
    }
#pragma unroll
    for (int k = 2; k <= kAll; k *= 2)
#pragma unroll
        for (int j = k / 2; j; j /= 2) {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const bool up = ((i * 32 + lane) & k) == 0;
                if (j < 32) {
                    const uint32_t o = __shfl_xor_sync(0xffffffffu, w[i], j);
                    w[i] = ((lane & j) == 0) == up ? min(w[i], o) : max(w[i], o);
                } else if ((i & (j / 32)) == 0) {   // (the pair lies in this lane)
                    const int e = i | (j / 32);
                    const uint32_t lo = min(w[i], w[e]), hi = max(w[i], w[e]);
                    w[i] = up ? lo : hi;
                    w[e] = up ? hi : lo;
                }
            }
        }
#pragma unroll
    for (int i = 0; i < kN; ++i) sk[warp][i * 32 + lane] = w[i];
    __syncwarp();
    int n = 0, f0 = 0;   // ids so far; place of the first id of the current unit
    int na = 0;          // anchors so far
    int place[kN], first[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int e = i * 32 + lane;
        const uint32_t before = e ? sk[warp][e - 1] : kGone;
        const bool has = w[i] != kGone, lead = has && (e == 0 || before >> 8 != w[i] >> 8);
        const bool opens = lead && (e == 0 || (before >> 8) / kUnit != (w[i] >> 8) / kUnit);
        const unsigned bl = __ballot_sync(0xffffffffu, lead), bo = __ballot_sync(0xffffffffu, opens);
        const unsigned below = (1u << lane) - 1u, upto = below | 1u << lane;
        place[i] = lead ? n + __popc(bl & below) : -1;
        const int src = 31 - __clz(bo & upto);   // the lane that opens this entry's unit (-1: an earlier word)
        first[i] = src >= 0 ? n + __popc(bl & ((1u << src) - 1u)) : f0;
        const int last = 31 - __clz(bo);
        if (last >= 0) f0 = n + __popc(bl & ((1u << last) - 1u));
        n += __popc(bl);
        const uint32_t id = w[i] >> 8;
        float2 v = make_float2(0.f, 0.f);
        if (lead) {
            v = sq[warp][w[i] & 255];
            for (int j = e + 1; j < kAll && sk[warp][j] >> 8 == id && sk[warp][j] != kGone; ++j) {   // the same id, slots ascending
                const float2 o = sq[warp][sk[warp][j] & 255];
                v.x += o.x;
                v.y += o.y;
            }
            const int64_t at = (int64_t)t * K + place[i];
            q[at] = v.x;
            if (h) h[at] = v.y;
            atomicOr(&smask[warp][first[i]][id % kUnit / 32], 1u << (id & 31));
        }
        const unsigned ba = __ballot_sync(0xffffffffu, v.x >= kAnchorQ);
        const int slot = na + __popc(ba & below);
        if (v.x >= kAnchorQ && slot < kAnchors) {
            an.id[t * kAnchors + slot] = (int32_t)id;
            an.place[t * kAnchors + slot] = place[i];
        }
        for (unsigned m2 = b.coef ? ba : 0u; m2; m2 &= m2 - 1) {   // backward: the anchors' entries of G
            const int src = __ffs(m2) - 1, sl = na + __popc(ba & ((1u << src) - 1u));
            const int aid = __shfl_sync(0xffffffffu, (int)id, src);
            const float aq = __shfl_sync(0xffffffffu, v.x, src);
            const float z = row_dot(b.X + (int64_t)t * b.d, b.W + (int64_t)aid * b.d, b.d);
            if (lane == 0 && sl < kAnchors) an.g[t * kAnchors + sl] = b.g[t] * scale * p_minus_q(z, scale, b.lse[t], aq);
        }
        na += __popc(ba);
    }
    if (lane >= na && lane < kAnchors) an.id[t * kAnchors + lane] = -1;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (place[i] >= 0 && place[i] == first[i]) {
            const int64_t u = (int64_t)t * NU + (w[i] >> 8) / kUnit;
            tab[u] = (uint16_t)(256 + place[i]);
            mask[u] = *(const uint4 *)smask[warp][first[i]];
        }
    if (lane == 0) nent[t] = n;
    if (b.coef) {
        const float cf = n ? b.g[t] * scale : 0.f;
        if (lane == 0) b.coef[t] = make_float2(cf, least_large(cf, 1.f));
        if (b.xz) copy_row(b.xz + (int64_t)t * b.d, b.X + (int64_t)t * b.d, b.d, cf);
    }
}

// Log-probability, backward, a warp per token: G = coef (p - onehot) with coef =
// -g s (0: no target), its entry at the target, and the least entry that keeps
// its remainder.
__global__ void __launch_bounds__(128) k_head_target(int T, int V, int d, float scale, const uint16_t *__restrict__ X,
                                                     const uint16_t *__restrict__ W, const int32_t *__restrict__ target,
                                                     const float *__restrict__ lse, const float *__restrict__ g,
                                                     float2 *__restrict__ coef, uint16_t *__restrict__ xz, Anchors an,
                                                     int *__restrict__ zero, int nzero, DevErr *err)
{
    const int t = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    grid_wait();
    grid_go();
    clear(zero, nzero);
    if (t >= T) return;
    const int y = target[t];
    const bool has = y >= 0 && y < V;
    const float z = has ? row_dot(X + (int64_t)t * d, W + (int64_t)y * d, d) : 0.f;
    if (y >= V && lane == 0) record_error(err, PMOE_ERR_BAD_INDEX, t, y);
    const float cf = has ? -g[t] * scale : 0.f, e = has ? p_minus_q(z, scale, lse[t], 1.f) : 0.f;
    if (lane < kAnchors) {
        an.id[t * kAnchors + lane] = lane == 0 && has ? y : -1;
        an.g[t * kAnchors + lane] = lane == 0 ? cf * e : 0.f;
    }
    // (not below 1e-4, where 1 - p_y is no longer a bound for the other entries as computed)
    if (lane == 0) coef[t] = make_float2(cf, least_large(cf, fminf(fmaxf(fabsf(e), 1e-4f), 1.f)));
    if (xz) copy_row(xz + (int64_t)t * d, X + (int64_t)t * d, d, cf);
}

// ------------------------------------------------------------------ combine
// One CTA per token joins the NU softmax partials in one fixed order, adds the
// anchors, which the partials leave out, and forms the token's value.  A partial
// (m, s) stands for s 2^M with M = c m as rounded.  With `top` the largest
// logit and L = ln sum_v exp(scale (z_v - top)), lse = scale top + L (scale z as
// rounded in the backward too) and a log-probability is scale (z - top) - L:
// where an anchor is the largest, L = log1p(the others) however small they are.
__global__ void __launch_bounds__(128) k_head_combine(int V, int K, int NU, int d, float scale, float c,
                                                      const uint16_t *__restrict__ X, const uint16_t *__restrict__ W,
                                                      const float2 *__restrict__ part, const float *__restrict__ zt,
                                                      const int32_t *__restrict__ target, const int *__restrict__ nent,
                                                      const float *__restrict__ q, const float *__restrict__ h,
                                                      Anchors an, float *__restrict__ value, float *__restrict__ lse,
                                                      DevErr *err)
{
    __shared__ float2 sw[4];
    __shared__ float sz[kAnchors];
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float ninf = -__int_as_float(0x7f800000);
    // (before the wait: all of this was complete when the GEMM before started)
    int id[kAnchors] = {-1, -1, -1, -1}, place[kAnchors] = {0, 0, 0, 0};
    if (target) {
        const int y = __ldcg(target + t);
        if (y >= V && threadIdx.x == 0) record_error(err, PMOE_ERR_BAD_INDEX, (int)t, y);
        if (y >= 0 && y < V) id[0] = y;
    } else {
#pragma unroll
        for (int n = 0; n < kAnchors; ++n) {
            id[n] = __ldcg(an.id + t * kAnchors + n);
            if (id[n] >= 0) place[n] = __ldcg(an.place + t * kAnchors + n);
        }
    }
    static_assert(kAnchors == 4, "an anchor for each of the CTA's warps");
    const int mine = warp == 0 ? id[0] : warp == 1 ? id[1] : warp == 2 ? id[2] : id[3];
    if (mine >= 0) {
        const float z = row_dot(X + t * d, W + (int64_t)mine * d, d);
        if (lane == 0) sz[warp] = z;
    }
    grid_wait();
    grid_go();
    const float2 *p = part + t * NU;
    float m = ninf, s = 0.f;
    auto join = [&](float om, float os) {   // (no partials yet: m = -inf, s = 0; a NaN stays one)
        const float n = fmaxf(m, om), N = __fmul_rn(n, c);
        const float x = m == ninf ? s : s * exp2f(__fmul_rn(m, c) - N);
        const float y = om == ninf ? os : os * exp2f(__fmul_rn(om, c) - N);
        m = n;
        s = x + y;
    };
#pragma unroll 4
    for (int i = threadIdx.x; i < NU; i += 128) join(p[i].x, p[i].y);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s, o);
        join(om, os);
    }
    if (lane == 0) sw[warp] = make_float2(m, s);
    __syncthreads();
    if (warp) return;
    const float za[kAnchors] = {sz[0], sz[1], sz[2], sz[3]};   // (only where id >= 0)
    m = sw[0].x;
    s = sw[0].y;
    for (int i = 1; i < 4; ++i) join(sw[i].x, sw[i].y);
    float top = m;
    int lead = -1;   // the anchor that is the largest, if one is
#pragma unroll
    for (int n = 0; n < kAnchors; ++n)
        if (id[n] >= 0 && za[n] >= top) {
            if (lead < 0 || za[n] > top) lead = n;
            top = za[n];
        }
    // sums relative to c top, which the partials' M differs from by its rounding
    const float off = fmaf(top, c, -__fmul_rn(m, c));
    float rest = m == ninf ? s : s * exp2f(-off);
#pragma unroll
    for (int n = 0; n < kAnchors; ++n)
        if (id[n] >= 0 && n != lead) rest += exp2f((za[n] - top) * c);
    const float L = lead >= 0 ? log1pf(rest) : 0.6931471805599453f * log2f(rest);
    const float l = __fadd_rn(__fmul_rn(top, scale), L);
    auto logp = [&](float z) { return (z - top) * scale - L; };
    float v = 0.f;
    if (!target) {
        const int n = nent[t];
        for (int k = lane; k < n; k += 32) {
            const int64_t at = t * K + k;
            float z = zt[at];
#pragma unroll
            for (int e = 0; e < kAnchors; ++e)
                if (id[e] >= 0 && place[e] == k) z = za[e];
            v += h[at] - q[at] * logp(z);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    } else if (id[0] >= 0) {
        v = logp(za[0]);
    }
    if (lane == 0) {
        value[t] = v;
        lse[t] = l;
    }
}

// ------------------------------------------------------------------ large entries
// The extra K steps of one product, one CTA per 256 output rows.  The
// entries of the rows take consecutive columns of A, in (token, vocabulary
// id) order whatever order GRAD's threads listed them in.
//   DX (kDw 0): rows are tokens, a column's row of B is its vocabulary entry;
//   a block's entries have their own place (kMaxLarge steps of 64 each 256
//   tokens at most)
//   DW (kDw 1): rows are vocabulary entries, the row of B is the token; `fl`
//   names the blocks of 128 tokens to look at, four tokens a thread.  A
//   block's steps are taken from a counter, so blocks may come in any order,
//   but a block's own columns, and with them its sums, are fixed.
// The entries found are kept in shared memory while there is room, else the
// tokens are read again once the block's steps are known.
constexpr int kLargeThreads = 1024, kLargeKept = 1024;   // (threads: at most)
constexpr int kLargeSteps = kListRows * kMaxLarge / 64;   // of a block of tokens
struct LargeShared {
    int warp[kLargeThreads / 32], base;
    int3 kept[kLargeKept];   // (token - t0, vocabulary entry, remainder)
};

// Exclusive sum of n over the CTA's threads, and the total
__device__ __forceinline__ int large_scan(LargeShared &sh, int n, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sh.warp[warp] = x;
    __syncthreads();
    int s = lane < warps ? sh.warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    const int before = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
    total = __shfl_sync(0xffffffffu, s, 31);
    return (warp ? before : 0) + x - n;
}

template <int kDw>
__device__ void large_steps(LargeShared &sh, int blk, int T, const int *__restrict__ cnt, const int2 *__restrict__ large,
                            const uint8_t *__restrict__ fl, int fs, int *__restrict__ steps, int2 *__restrict__ lists,
                            int32_t *__restrict__ lidx, uint16_t *__restrict__ lo)
{
    constexpr int R = kDw ? 4 : 1;   // tokens a thread
    const int tid = threadIdx.x, t0 = kDw ? 0 : blk * kListRows, t1 = kDw ? T : min(T, t0 + kListRows);
    int64_t first = -1;              // the block's first step, once it is known
    auto put = [&](int at, int t, int v, int rem) {
        if (first < 0) {
            if (at < kLargeKept) sh.kept[at] = make_int3(t - t0, v, rem);
            return;
        }
        const int64_t st = first + at / 64;
        const int c = at % 64;
        lidx[st * 64 + c] = kDw ? t : v;
        lo[st * 64 * kListRows + (kDw ? c * kListRows + v % kListRows : (t - t0) * 64 + c)] = (uint16_t)rem;
    };
    auto ours = [&](int id) { return !kDw || id / kListRows == blk; };
    // all entries of the block, each with its column; returns their number.
    // (Most tokens have one or two; loops over a token's entries stay loops:
    // unrolled, the code's own fetches took longer than its work.)
    auto walk = [&]() {
        int total = 0;
        for (int b = t0; b < t1; b += blockDim.x * R) {
            const int t = b + tid * R;
            int c[R], n[R], sum = 0;
            int2 f[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {   // (all first loads at once)
                c[r] = t + r < t1 ? min(cnt[t + r], kMaxLarge) : 0;
                f[r] = t + r < t1 ? large[(int64_t)(t + r) * kMaxLarge] : make_int2(0, 0);
            }
            const bool look = t < t1 && (!kDw || fl[(int64_t)blk * fs + (t >> 7)] != 0);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                n[r] = look && c[r] > 0 && ours(f[r].x);
                if (look)
#pragma unroll 1
                    for (int j = 1; j < c[r]; ++j) n[r] += ours(large[(int64_t)(t + r) * kMaxLarge + j].x);
                sum += n[r];
            }
            int all, at = total + large_scan(sh, sum, all);
            total += all;
            if (sum) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int2 *x = large + (int64_t)(t + r) * kMaxLarge;
                    if (n[r]) {
#pragma unroll 1
                        for (int j = 0; j < c[r]; ++j) {
                            const int2 v = x[j];
                            if (!ours(v.x)) continue;
                            int place = 0;   // ascending by vocabulary id
#pragma unroll 1
                            for (int i = 0; i < c[r] && c[r] > 1; ++i) place += ours(x[i].x) && x[i].x < v.x;
                            put(at + place, t + r, v.x, v.y);
                        }
                    }
                    at += n[r];
                }
            }
        }
        return total;
    };
    const int total = walk(), ns = (total + 63) / 64;
    if (tid == 0) {
        sh.base = !kDw ? blk * kLargeSteps : ns ? atomicAdd(steps, ns) : 0;
        lists[blk] = make_int2(sh.base, ns);
    }
    __syncthreads();
    if (!ns) return;
    first = sh.base;
    uint4 *z = (uint4 *)(lo + first * 64 * kListRows);
    for (int i = tid; i < ns * 64 * kListRows / 8; i += blockDim.x) z[i] = make_uint4(0, 0, 0, 0);
    for (int i = total + tid; i < ns * 64; i += blockDim.x) lidx[first * 64 + i] = 0;   // (its column of A is zero)
    __syncthreads();
    if (total <= kLargeKept) {
        for (int i = tid; i < total; i += blockDim.x)
            put(i, t0 + sh.kept[i].x, sh.kept[i].y, sh.kept[i].z);
    } else {
        walk();
    }
}

// CTAs 0 .. nx-1: DX's blocks, the others DW's
__global__ void __launch_bounds__(kLargeThreads) k_head_large(int nx, int T, const int *cnt, const int2 *large,
                                                              const uint8_t *fl, int fs, int *steps, int2 *lists0,
                                                              int32_t *lidx0, uint16_t *lo0, int2 *lists1,
                                                              int32_t *lidx1, uint16_t *lo1)
{
    __shared__ LargeShared sh;
    grid_wait();
    grid_go();
    if ((int)blockIdx.x < nx) large_steps<0>(sh, blockIdx.x, T, cnt, large, fl, fs, steps, lists0, lidx0, lo0);
    else large_steps<1>(sh, blockIdx.x - nx, T, cnt, large, fl, fs, steps, lists1, lidx1, lo1);
}

struct Parts {
    int mt, nt, gm, whole, tile, splits;   // the tiling of DX (tile: rows and columns)
    int cut, rows, cols;                   // cut tiles, and what is kept of one
};
// dX = bf16(sum of the FP32 parts): `first` holds every tile's first part, `rest`
// [splits - 1][cut][rows][cols] the further ones of the tiles that were cut.
// T x d (d % 64 == 0), a thread 4 columns of a row; kS threads share the parts
// of the same columns, and their sums are added in order.
template <int kS>
__global__ void __launch_bounds__(256) k_head_sum(int T, int d, Parts p, const float *__restrict__ first,
                                                  const float *__restrict__ rest, uint16_t *__restrict__ out)
{
    __shared__ float4 sh[kS > 1 ? 256 : 1];
    constexpr int kCols = 256 / kS;
    const int64_t n = (int64_t)T * d, i = (blockIdx.x * (int64_t)kCols + threadIdx.x % kCols) * 4;
    const int strand = threadIdx.x / kCols;
    grid_wait();
    grid_go();
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n) {
        const int row = (int)(i / d), col = (int)(i % d), m = row / p.tile, c = col / p.tile, g = m / p.gm;
        const int item = g * p.gm * p.nt + c * min(p.gm, p.mt - g * p.gm) + m - g * p.gm;
        if (strand == 0) a = *(const float4 *)(first + i);
        if (item >= p.whole) {
            const int64_t step = (int64_t)p.cut * p.rows * p.cols;
            const int s0 = strand ? strand : kS;
            const float *x1 = rest + ((int64_t)(item - p.whole) * p.rows + row - m * p.tile) * p.cols + col - c * p.tile +
                              (s0 - 1) * step;
#pragma unroll 4
            for (int s = s0; s < p.splits; s += kS, x1 += kS * step) {
                const float4 x = *(const float4 *)x1;
                a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
            }
        }
    }
    if constexpr (kS > 1) {
        sh[threadIdx.x] = a;
        __syncthreads();
        if (strand) return;
#pragma unroll
        for (int s = 1; s < kS; ++s) {
            const float4 x = sh[s * kCols + threadIdx.x];
            a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
        }
    }
    if (i < n) *(uint2 *)(out + i) = make_uint2(pack_bf2(a.x, a.y), pack_bf2(a.z, a.w));
}

// ------------------------------------------------------------------ plan
static bool head_ok(const pmoe_head_dims &h)
{
    return h.T >= 0 && h.d > 0 && h.d % 64 == 0 && h.d <= 8192 && h.V > 0 && h.V < (1 << 24) && h.K >= 0 &&
           h.K <= kMaxK && h.T <= (1 << 24);
}

// Vocabulary entries per piece of the backward: G of one piece is at most
// kPieceBytes; pieces of equal size, multiples of 256.  Every further piece
// adds dX's FP32 sums to memory once more: T = 4096, d = 2048, V = 131072 runs
// its backward in 2826 us with pieces of 128 MB, 2701 with 256, 2675 with 512,
// 2645 with 1024.
static int piece_of(int T, int V)
{
    int64_t most = kPieceBytes / (2ll * std::max(T, 1)) / 256 * 256;
    most = std::max<int64_t>(most, 256);
    const int64_t np = cdiv(V, most);
    return (int)(cdiv(cdiv(V, np), 256) * 256);
}

// Whether G's remainders are kept in whole (2 terms) instead of in lists: for
// small vocabularies, where a block of 256 entries has long lists.  With about
// 2.5 large entries a token, the lists lengthen K by 640 / V and DW's take one
// CTA 0.33 us for every 64 entries of its block; two terms double K and write G
// twice.  (Forward and both gradients, two terms against lists: T = 4013, d = 192,
// V = 263 46 against 145 us; T = 8000, d = 128, V = 1500 84 against 129; at T = 4000,
// d = 512, V = 3000 both take 91.)
static int terms_of(const pmoe_head_dims &h)
{
    const int piece = piece_of(h.T, h.V);
    if (piece < h.V || 4ll * h.T * piece > kPieceBytes) return 1;
    const double tv = (double)h.T * h.V, mma = 4 * tv * h.d / 1.5e9;   // us
    const double lists = 0.33 * h.T * 2.5 * 256 / (64.0 * h.V) + mma * 640 / h.V, twice = mma + tv * 2 / 5e6;
    return twice < lists ? 2 : 1;
}

struct Tiling {
    int ctas, bn;
    int mt, nt, gm;      // gm: m tiles that run together
    int whole;           // tiles taken whole, the others cut into
    int splits, kper;    // `splits` items of kper K steps
};
// Tiles of an M x N product over ksteps K steps.  `split`: tiles of the last,
// partly filled round may be cut along K, their parts then being added up.
// (T = 4096, d = 2048, V = 131072: backward 2692 us without, 2675 with; T = 64,
// V = 32000: 127 us without, 57 with.)
// The number of parts is the one of least time by this estimate: a K step of
// a tile takes 0.28 us (the tensor cores' rate at 1.8 GHz), each round 2 us
// to fill and to drain, each part's FP32 tile goes to memory and back, and
// a launch to add them 4 us.
static Tiling tiling(int64_t M, int64_t N, int64_t ksteps, bool split)
{
    Tiling t;
    // A pair of CTAs on a 256 x 256 tile reads each operand half as often as
    // single CTAs on 128 x 128; single CTAs fill the GPU with smaller products.
    // Forward and backward at d = 2048, V = 4864, singles for all products against
    // pairs for all: 38 tiles of 256 (T = 512) 53.8 against 59.6 us, 76 tiles
    // (T = 1024) 74 against 76 (71 by this rule: dX has fewer), 152 tiles
    // (T = 2048) 123 against 104 (115 by this rule, dX's 64 tiles as singles).
    t.ctas = cdiv(M, 256) * cdiv(N, 256) >= kSms / 2 && M > 128 ? 2 : 1;
    t.bn = 128 * t.ctas;
    t.mt = (int)cdiv(M, 128 * t.ctas);
    t.nt = (int)cdiv(N, t.bn);
    // m tiles that run together: their rows of A stay in L2 while the n tiles
    // pass; groups of equal size.  T = 8192, d = 7168, V = 32768, forward and
    // backward: 6.78 ms by this rule, 6.82 with groups of 8 tiles, 6.99 with 48 MB
    // alone, 6.96 with 96 MB, 7.39 with all tiles in one group.
    const int64_t stripe = 2ll * 128 * t.ctas * ksteps * kBK;
    const int64_t most = std::max<int64_t>(8, (48ll << 20) / std::max<int64_t>(stripe, 1));
    t.gm = (int)cdiv(t.mt, cdiv(t.mt, most));
    const int64_t slots = kSms / t.ctas, tiles = (int64_t)t.mt * t.nt, cut = tiles % slots;
    int64_t best = 1;
    if (split && cut) {
        const double part = 2.0 * 128 * t.ctas * t.bn * 4 / 6e6;   // us
        double least = 0;
        for (int64_t s = 1; s <= std::min<int64_t>(ksteps, 2 * kSms); ++s) {
            const double us = cdiv(cut * s, slots) * (cdiv(ksteps, s) * 0.28 + 2) + (s > 1 ? cut * s * part + 4 : 0);
            if (s == 1 || us < least) {
                least = us;
                best = s;
            }
        }
    }
    t.whole = (int)(best > 1 ? tiles - cut : tiles);
    t.kper = (int)cdiv(std::max<int64_t>(ksteps, 1), best);
    t.splits = (int)cdiv(std::max<int64_t>(ksteps, 1), t.kper);
    return t;
}
static Tiling dx_tiling(const pmoe_head_dims &h)
{
    return tiling(h.T, h.d, cdiv(std::min(piece_of(h.T, h.V), h.V), kBK) * terms_of(h), true);
}

struct Ws {
    DevErr *err;
    float *q, *h;            // teacher entries [T][K]: q, q log q
    int *nent;               // [T] their number
    uint16_t *tab;           // [T][NU]
    uint4 *mask;             // [T][NU]
    float *zt;               // [T][K]
    float2 *part;            // [T][NU]
    Anchors an;
    float2 *coef;            // [T] factor and least large entry of G
    uint16_t *xz;            // [T][d] X, zero in the rows without gradient (for dW)
    int terms;
    uint16_t *G;             // [T][terms][piece]
    // G's large entries: per token, then as the extra K steps of DX and DW
    int *cnt;                // [T], then the step counter and the flags: zeroed per piece
    uint8_t *fl;             // [piece / 256][fs]
    int *steps;              // DW's steps taken so far
    size_t zero_bytes;
    int fs;
    int2 *large;             // [T][kMaxLarge]
    int2 *lists[2];          // per 256 rows: first step and number of steps
    int32_t *lidx[2];        // [steps][64]
    uint16_t *lo[2];         // [steps] remainders: DX [256 tokens][64], DW [64][256 entries]
    int max_steps[2];
    float *dx, *dxp;         // FP32 parts of dX: [T][d], and those of the cut tiles beyond the first
    Parts parts;
    size_t bytes;
};
static Ws carve(void *base, const pmoe_head_dims &h, int op)
{
    size_t off = 0;
    auto take = [&](size_t n) {
        uint8_t *p = base ? (uint8_t *)base + off : nullptr;
        off += (n + 255) & ~(size_t)255;
        return p;
    };
    Ws w{};
    const size_t T = h.T, K = h.K;
    w.err = (DevErr *)take(kHdrBytes);
    w.q = (float *)take(T * K * 4);
    w.tab = (uint16_t *)take(K ? T * cdiv(h.V, kUnit) * 2 : 0);
    w.mask = (uint4 *)take(K ? T * cdiv(h.V, kUnit) * 16 : 0);
    w.nent = (int *)take(K ? T * 4 : 0);
    w.an.id = (int32_t *)take(T * kAnchors * 4);
    w.an.place = (int *)take(T * kAnchors * 4);
    if (op == PMOE_HEAD_FORWARD) {
        w.h = (float *)take(T * K * 4);
        w.zt = (float *)take(T * K * 4);
        w.part = (float2 *)take(T * cdiv(h.V, kUnit) * 8);
    } else {
        const int piece = piece_of(h.T, h.V);
        const Tiling t = dx_tiling(h);
        w.coef = (float2 *)take(T * 8);
        w.xz = (uint16_t *)take(T * h.d * 2);
        w.an.g = (float *)take(T * kAnchors * 4);
        w.terms = terms_of(h);
        w.G = (uint16_t *)take(T * piece * w.terms * 2);
        const int blocks[2] = {(int)cdiv(h.T, kListRows), piece / kListRows};
        w.fs = (int)cdiv(h.T, 128);
        w.zero_bytes = (T * 4 + 4 + (size_t)blocks[1] * w.fs + 3) & ~(size_t)3;
        uint8_t *z = take(w.zero_bytes);
        w.cnt = (int *)z;
        w.steps = w.cnt + T;
        w.fl = (uint8_t *)(w.steps + 1);
        w.large = (int2 *)take(T * kMaxLarge * 8);
        for (int i = 0; i < 2; ++i) {
            w.max_steps[i] = i == 0 ? blocks[0] * kLargeSteps : (int)(cdiv((int64_t)h.T * kMaxLarge, 64) + blocks[1]);
            w.lists[i] = (int2 *)take((size_t)blocks[i] * 8);
            w.lidx[i] = (int32_t *)take((size_t)w.max_steps[i] * 64 * 4);
            w.lo[i] = (uint16_t *)take((size_t)w.max_steps[i] * 64 * kListRows * 2);
        }
        // (few tokens: only their rows of a tile are kept; T = 1 writes its row and no more)
        w.parts = {t.mt, t.nt, t.gm, t.whole, t.bn, t.splits, t.mt * t.nt - t.whole, std::min(t.bn, h.T), std::min(t.bn, h.d)};
        if (t.splits > 1 || piece < h.V) w.dx = (float *)take(T * h.d * 4);
        if (t.splits > 1)
            w.dxp = (float *)take((size_t)(t.splits - 1) * w.parts.cut * w.parts.rows * w.parts.cols * 4);
    }
    w.bytes = off;
    return w;
}

// ------------------------------------------------------------------ launch
// BF16 or FP32 row-major [planes][rows][cols] (planes 0: a 2-D map [rows][cols]),
// 128-byte swizzle, boxes of box_rows x box_cols (128 bytes), zeros past the end
static bool make_map(CUtensorMap *m, const void *base, bool f32, int64_t cols, int64_t rows, int64_t planes, int box_cols,
                     int box_rows)
{
    // (through the runtime's driver entry point: the library does not link libcuda)
    static const decltype(&cuTensorMapEncodeTiled) encode = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                            cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return (decltype(&cuTensorMapEncodeTiled))(ok ? p : nullptr);
    }();
    if (!encode) return false;
    const cuuint64_t e = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * e, (cuuint64_t)rows * cols * e};
    const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1}, estr[3] = {1, 1, 1};
    return encode(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, planes > 0 ? 3 : 2,
                  const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
struct Operand {
    const void *base;
    int64_t cols, rows;
    bool mn;                 // the contiguous axis is M (or N), not K
};
static bool map_operand(CUtensorMap *m, const Operand &o)
{
    return make_map(m, o.base, false, o.cols, o.rows, 0, kBK, o.mn ? 64 : 128);
}

template <int CTAS, int BN, int EPI>
static bool launch_as(const CUtensorMap &ma, const CUtensorMap &mt, const CUtensorMap &mb, const CUtensorMap (&mo)[2],
                      const CUtensorMap (&ml)[2], const Args &a, cudaStream_t st)
{
    constexpr auto kern = k_head_gemm<CTAS, BN, EPI>;
    if (!set_attribute<kern, cudaFuncAttributeMaxDynamicSharedMemorySize>(smem_of(BN))) return false;
    const int64_t items = a.whole + ((int64_t)a.mt * a.nt - a.whole) * a.splits;
    const int64_t clusters = std::min<int64_t>(items, gemm_num_sms() / CTAS);
    return launch_chained<kern>((unsigned)(clusters * CTAS), threads_of(BN),
                          smem_of(BN), CTAS, st, ma, mt, mb, mo[0], mo[1], ml[0], ml[1], a);
}

// One product: M x N outputs over ksteps K steps, with the tiles of `t`; `out`,
// `part`: the maps of the outputs and of the cut tiles' further parts (or NULL);
// `lo`: DX, DW: the remainders of G's large entries
template <int EPI>
static bool launch(const Tiling &t, const Operand &A, const Operand &B, const CUtensorMap *out, const CUtensorMap *part,
                   const Operand *lo, Args a, cudaStream_t st)
{
    CUtensorMap ma, mt, mb, mo[2], ml[2];
    a.tail = (int)(A.rows % 128);
    // (fewer than 128 rows: A's only boxes are the tail's)
    memset(&ma, 0, sizeof ma);
    if (((A.mn || A.rows >= 128) && !map_operand(&ma, A)) || !map_operand(&mb, B)) return false;
    a.abytes = kOpBytes;
    // (with extra K steps A's tiles are always whole)
    if ((EPI == HG_FWD || EPI == HG_GRAD) && A.rows < 128) a.abytes = (int)cdiv(a.tail, 8) * 1024;
    a.stages = std::min(kMaxStages, kRingBytes / (kOpBytes + a.abytes));
    memset(&mt, 0, sizeof mt);
    if (!A.mn && a.tail && !make_map(&mt, A.base, false, A.cols, A.rows, 0, kBK, a.tail)) return false;
    memset(mo, 0, sizeof mo);
    memset(ml, 0, sizeof ml);
    if (out) mo[0] = *out;
    if (part) mo[1] = *part;
    // (rows of B are gathered one by one: boxes of one row)
    if (lo && (!map_operand(&ml[0], *lo) || !make_map(&ml[1], B.base, false, B.cols, B.rows, 0, kBK, 1))) return false;
    a.mt = t.mt;
    a.nt = t.nt;
    a.splits = t.splits;
    a.kper = t.kper;
    a.whole = t.whole;
    a.gm = t.gm;
    return t.ctas == 2 ? launch_as<2, 256, EPI>(ma, mt, mb, mo, ml, a, st) : launch_as<1, 128, EPI>(ma, mt, mb, mo, ml, a, st);
}

// ------------------------------------------------------------------ passes
template <auto K>
using Kernel = std::integral_constant<decltype(K), K>;

static bool launch_teacher(const pmoe_head_dims &h, float scale, const int32_t *idx, const float *t_logits, const Ws &w,
                           const TeacherGrad &b, int *zero, int nzero, cudaStream_t st)
{
    auto launch = [&](auto kern) {
        return launch_chained<decltype(kern)::value>((unsigned)cdiv(h.T, 4), 128, 0, 1, st, h.T, h.V, h.K, scale, idx,
                                                     t_logits, w.q, w.h, w.nent, w.tab, w.mask, (int)cdiv(h.V, kUnit),
                                                     w.an, b, zero, nzero, w.err);
    };
    return h.K <= 32    ? launch(Kernel<k_head_teacher<1>>())
           : h.K <= 64  ? launch(Kernel<k_head_teacher<2>>())
           : h.K <= 128 ? launch(Kernel<k_head_teacher<4>>())
                        : launch(Kernel<k_head_teacher<8>>());
}

static pmoe_status forward(const pmoe_head_dims &h, const void *X, const void *W, float scale, const int32_t *idx,
                           const float *t_logits, bool distill, float *value, float *lse, const Ws &w, cudaStream_t st)
{
    const int K = distill ? h.K : 1;
    if (distill) {
        if (!launch_teacher(h, scale, idx, t_logits, w, TeacherGrad{}, nullptr, 0, st)) return PMOE_ERR_CUDA;
    }
    Args a{};
    a.M = h.T;
    a.N = h.V;
    a.V = h.V;
    a.ksteps = h.d / kBK;
    a.c = scale * 1.4426950408889634f;
    a.NU = (int)cdiv(h.V, kUnit);
    a.part = w.part;
    a.zt = w.zt;
    a.target = distill ? nullptr : idx;
    a.anchor = (const int4 *)w.an.id;
    a.tab = w.tab;
    a.mask = w.mask;
    a.K = K;
    a.err = w.err;
    tc::take_wait_hook(a.wait_ns, a.skip_item);
    if (!launch<HG_FWD>(tiling(h.T, h.V, a.ksteps, false), {X, h.d, h.T, false}, {W, h.d, h.V, false}, nullptr, nullptr,
                        nullptr, a, st))
        return PMOE_ERR_CUDA;
    return launch_chained<k_head_combine>((unsigned)h.T, 128, 0, 1, st, h.V, K, a.NU, h.d, scale, a.c, (const uint16_t *)X,
                          (const uint16_t *)W, w.part, w.zt, a.target, w.nent, w.q, w.h, w.an, value, lse, w.err)
               ? PMOE_OK
               : PMOE_ERR_CUDA;
}

static pmoe_status backward(const pmoe_head_dims &h, const void *X, const void *W, float scale, const int32_t *idx,
                            const float *t_logits, bool distill, const float *lse, const float *g, void *dX, void *dW,
                            const Ws &w, cudaStream_t st)
{
    const int K = distill ? h.K : 1;
    const int nzero = (int)(w.zero_bytes / 4);
    // (this kernel clears the counters of the first piece)
    const uint16_t *x = (const uint16_t *)X, *wt = (const uint16_t *)W;
    uint16_t *xz = dW ? w.xz : nullptr;
    const bool made =
        distill ? launch_teacher(h, scale, idx, t_logits, w, TeacherGrad{x, wt, h.d, lse, g, w.coef, xz}, w.cnt, nzero, st)
                : launch_chained<k_head_target>((unsigned)cdiv(h.T, 4), 128, 0, 1, st, h.T, h.V, h.d, scale, x, wt, idx, lse, g,
                                                w.coef, xz, w.an, w.cnt, nzero, w.err);
    if (!made) return PMOE_ERR_CUDA;
    const int piece = piece_of(h.T, h.V);
    const Tiling tx = dx_tiling(h);
    uint64_t wait_ns;
    int skip_item;
    tc::take_wait_hook(wait_ns, skip_item);
    for (int v0 = 0; v0 < h.V; v0 += piece) {
        const int vc = std::min(piece, h.V - v0);
        const int64_t ldg = (int64_t)piece * w.terms;
        CUtensorMap mo;
        Args b{};   // what the piece's products share
        b.terms = w.terms;
        b.aoff = piece;
        b.cnt = w.cnt;
        b.large = w.large;
        b.fl = dW ? w.fl : nullptr;
        b.fs = w.fs;
        b.wait_ns = wait_ns;
        b.skip_item = skip_item;
        b.err = w.err;
        if (v0 > 0 && cudaMemsetAsync(w.cnt, 0, w.zero_bytes, st) != cudaSuccess) return PMOE_ERR_CUDA;
        {   // G = coef (softmax(Z) - q) of this piece
            Args a = b;
            a.M = h.T;
            a.N = piece;
            a.n0 = v0;
            a.V = h.V;
            a.ksteps = h.d / kBK;
            a.scale = scale;
            a.target = distill ? nullptr : idx;
            a.tab = w.tab;
            a.mask = w.mask;
            a.q = w.q;
            a.NU = (int)cdiv(h.V, kUnit);
            a.K = K;
            a.lse = lse;
            a.coef = w.coef;
            a.anchor = (const int4 *)w.an.id;
            a.anchor_g = (const float4 *)w.an.g;
            if (!make_map(&mo, w.G, false, ldg, h.T, 1, 64, 32) ||
                !launch<HG_GRAD>(tiling(h.T, vc, a.ksteps, false), {X, h.d, h.T, false}, {W, h.d, h.V, false}, &mo,
                                 nullptr, nullptr, a, st))
                return PMOE_ERR_CUDA;
        }
        const int nx = dX ? (int)cdiv(h.T, kListRows) : 0, nw = dW ? (int)cdiv(vc, kListRows) : 0;
        // a block of tokens takes 256 threads; blocks of the vocabulary look at all tokens, four a thread
        const unsigned threads = nw == 0 || h.T <= 4 * kListRows ? kListRows : kLargeThreads;
        if (w.terms == 1 &&
            !launch_chained<k_head_large>((unsigned)(nx + nw), threads, 0, 1, st, nx, h.T, w.cnt, w.large, w.fl, w.fs, w.steps,
                            w.lists[0], w.lidx[0], w.lo[0], w.lists[1], w.lidx[1], w.lo[1]))
            return PMOE_ERR_CUDA;
        if (dX) {
            Args a = b;
            a.M = h.T;
            a.N = h.d;
            a.kone = (int)cdiv(vc, kBK);
            a.ksteps = a.kone * w.terms;
            a.kb0 = v0;
            a.bf16_out = w.dx == nullptr;
            a.accumulate = v0 > 0;
            Tiling t = tx;
            CUtensorMap mp;
            const Parts &p = w.parts;
            const bool made =
                (w.dx ? make_map(&mo, w.dx, true, h.d, h.T, 1, 32, 32) : make_map(&mo, dX, false, h.d, h.T, 1, 64, 32)) &&
                (!w.dxp || make_map(&mp, w.dxp, true, p.cols, p.rows, (int64_t)(p.splits - 1) * p.cut, 32, 32));
            // (a last, shorter piece: shorter parts, perhaps fewer; the other sums then stand)
            t.kper = (int)cdiv(a.ksteps, tx.splits);
            t.splits = (int)cdiv(a.ksteps, t.kper);
            a.lists = w.lists[0];
            a.lidx = w.lidx[0];
            a.lb0 = v0;
            const Operand lo{w.lo[0], 64, (int64_t)w.max_steps[0] * kListRows, false};
            if (!made ||
                !launch<HG_DX>(t, {w.G, ldg, h.T, false}, {W, h.d, h.V, true}, &mo, w.dxp ? &mp : nullptr, &lo, a, st))
                return PMOE_ERR_CUDA;
        }
        if (dW) {
            Args a = b;
            a.M = vc;
            a.N = h.d;
            a.kone = (int)cdiv(h.T, kBK);
            a.ksteps = a.kone * w.terms;
            a.beside = dX != nullptr;
            a.lists = w.lists[1];
            a.lidx = w.lidx[1];
            const Operand lo{w.lo[1], kListRows, (int64_t)w.max_steps[1] * 64, true};
            if (!make_map(&mo, (uint16_t *)dW + (int64_t)v0 * h.d, false, h.d, vc, 1, 64, 32) ||
                !launch<HG_DW>(tiling(vc, h.d, a.ksteps, false), {w.G, ldg, h.T, true}, {xz, h.d, h.T, true}, &mo, nullptr,
                               &lo, a, st))
                return PMOE_ERR_CUDA;
        }
    }
    if (dX && w.dx) {
        const int64_t n = (int64_t)h.T * h.d;
        // (T = 60, d = 64, V = 38592, a tile in 64 parts: the backward takes 29.4 us with 16 threads for
        // the parts of a column, 29.9 with one)
        const bool ok = tx.splits >= 16
                            ? launch_chained<k_head_sum<16>>((unsigned)cdiv(n, 64), 256, 0, 1, st, h.T, h.d, w.parts, w.dx,
                                                             w.dxp, (uint16_t *)dX)
                            : launch_chained<k_head_sum<1>>((unsigned)cdiv(n, 1024), 256, 0, 1, st, h.T, h.d, w.parts, w.dx,
                                                            w.dxp, (uint16_t *)dX);
        if (!ok) return PMOE_ERR_CUDA;
    }
    return PMOE_OK;
}

// Argument checks shared by the entry points; PMOE_OK to go on
static pmoe_status check(const pmoe_head_dims &h, float scale, std::initializer_list<const void *> needed,
                         std::initializer_list<const void *> optional, const void *ws, size_t ws_bytes, size_t need)
{
    if (!(scale > 0.f) || !std::isfinite(scale)) return PMOE_ERR_INVALID_ARG;
    for (const void *p : needed)
        if ((h.T > 0 && !p) || ((uintptr_t)p & 15)) return PMOE_ERR_INVALID_ARG;
    for (const void *p : optional)
        if ((uintptr_t)p & 15) return PMOE_ERR_INVALID_ARG;
    if (!ws || ws_bytes < need || ((uintptr_t)ws & 15)) return PMOE_ERR_WORKSPACE;
    return PMOE_OK;
}

}  // namespace hg
}  // namespace pmoe

using namespace pmoe;

extern "C" {

size_t head_workspace_bytes(pmoe_head_dims dims, int op)
{
    if (!hg::head_ok(dims) || (op != PMOE_HEAD_FORWARD && op != PMOE_HEAD_BACKWARD)) return 0;
    return hg::carve(nullptr, dims, op).bytes;
}

pmoe_status head_logprob_forward(pmoe_head_dims dims, const void *X, const void *W, float scale, const int32_t *target,
                                 float *logp, float *lse, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    if (!hg::head_ok(dims)) return PMOE_ERR_INVALID_ARG;
    const hg::Ws w = hg::carve(ws, dims, PMOE_HEAD_FORWARD);
    const pmoe_status s = hg::check(dims, scale, {X, W, target, logp, lse}, {}, ws, ws_bytes, w.bytes);
    if (s != PMOE_OK || dims.T == 0) return s;
    return hg::forward(dims, X, W, scale, target, nullptr, false, logp, lse, w, stream);
}

pmoe_status head_logprob_backward(pmoe_head_dims dims, const void *X, const void *W, float scale, const int32_t *target,
                                  const float *lse, const float *g, void *dX, void *dW, void *ws, size_t ws_bytes,
                                  cudaStream_t stream)
{
    if (!hg::head_ok(dims) || (!dX && !dW)) return PMOE_ERR_INVALID_ARG;
    const hg::Ws w = hg::carve(ws, dims, PMOE_HEAD_BACKWARD);
    const pmoe_status s = hg::check(dims, scale, {X, W, target, lse, g}, {dX, dW}, ws, ws_bytes, w.bytes);
    if (s != PMOE_OK) return s;
    if (dims.T == 0)
        return !dW || cudaMemsetAsync(dW, 0, (size_t)dims.V * dims.d * 2, stream) == cudaSuccess ? PMOE_OK : PMOE_ERR_CUDA;
    return hg::backward(dims, X, W, scale, target, nullptr, false, lse, g, dX, dW, w, stream);
}

pmoe_status head_distill_forward(pmoe_head_dims dims, const void *X, const void *W, float scale, const int32_t *t_idx,
                                 const float *t_logits, float *loss, float *lse, void *ws, size_t ws_bytes,
                                 cudaStream_t stream)
{
    if (!hg::head_ok(dims) || dims.K < 1) return PMOE_ERR_INVALID_ARG;
    const hg::Ws w = hg::carve(ws, dims, PMOE_HEAD_FORWARD);
    const pmoe_status s = hg::check(dims, scale, {X, W, t_idx, t_logits, loss, lse}, {}, ws, ws_bytes, w.bytes);
    if (s != PMOE_OK || dims.T == 0) return s;
    return hg::forward(dims, X, W, scale, t_idx, t_logits, true, loss, lse, w, stream);
}

pmoe_status head_distill_backward(pmoe_head_dims dims, const void *X, const void *W, float scale, const int32_t *t_idx,
                                  const float *t_logits, const float *lse, const float *g, void *dX, void *dW, void *ws,
                                  size_t ws_bytes, cudaStream_t stream)
{
    if (!hg::head_ok(dims) || dims.K < 1 || (!dX && !dW)) return PMOE_ERR_INVALID_ARG;
    const hg::Ws w = hg::carve(ws, dims, PMOE_HEAD_BACKWARD);
    const pmoe_status s = hg::check(dims, scale, {X, W, t_idx, t_logits, lse, g}, {dX, dW}, ws, ws_bytes, w.bytes);
    if (s != PMOE_OK) return s;
    if (dims.T == 0)
        return !dW || cudaMemsetAsync(dW, 0, (size_t)dims.V * dims.d * 2, stream) == cudaSuccess ? PMOE_OK : PMOE_ERR_CUDA;
    return hg::backward(dims, X, W, scale, t_idx, t_logits, true, lse, g, dX, dW, w, stream);
}

}  // extern "C"
