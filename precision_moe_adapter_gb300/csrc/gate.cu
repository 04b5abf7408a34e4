// gate.cu -- the gate of a layer that routes by scores: sigmoid or softmax of
// the logits, a balancing bias that takes part in the choice alone, groups of
// experts, the top k, weights renormalised; and its gradient.
//
// The choice is the one of the exact scores.  Without a bias the order of the
// experts is that of their logits, and keys of the logits decide.  With one, c =
// score + bias is formed in FP32 first; where two experts that the choice has to
// tell apart lie within the error of their c, the candidates' c are formed again in
// FP64, one candidate a lane.  They are neighbours down to the k-th place and on through
// those that are close to it, each to the next: among equal ones, whose order needs no
// closer look, the last may have a neighbour that stands before all of them.  The same
// holds for the last group in and the first one out, with the c of the experts that
// count for their groups.  Where that does not settle it, all of the token's c are
// formed in FP64.
#include <cmath>
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace pmoe {
namespace gate {

constexpr int kMaxGroups = 32;
constexpr uint32_t kAll = 0xffffffffu;

struct Args {
    int T, E, k, G, top, gsum, gsize;   // gsize: experts of a group
    int sublog, per;                    // 2^sublog lanes look at a group, per experts each
    uint32_t gmagic;                    // e / gsize is the high half of e gmagic (0: e)
    int softmax, renorm, has_bias, grouped;
    float factor;
    const float *logits, *bias;
    int32_t *idx;
    float *w;
};

// Keys in the order of the values, -0 as +0 (the sum with +0 is +0); 0 is an expert that
// is taken or out
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t u = __float_as_uint(v + 0.f);
    return max(u ^ ((uint32_t)((int)u >> 31) | 0x80000000u), 1u);
}
__device__ __forceinline__ float of_key(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t key_of(double v)
{
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.);
    const uint64_t k = (u >> 63) ? ~u : u | 0x8000000000000000ull;
    return k ? k : 1ull;
}
__device__ __forceinline__ double of_key(uint64_t k)
{
    return __longlong_as_double((long long)((k >> 63) ? k & 0x7fffffffffffffffull : ~k));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k)
{
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (uint64_t)hi << 32 | lo;
}
template <class F>
__device__ __forceinline__ F warp_sum(F v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float warp_fmax(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// exp(l - m) for l <= m, with the rounding of the difference taken back
__device__ __forceinline__ float exp_below(float l, float m)
{
    const float d = l - m;
    if (!(d > -200.f)) return d != d ? d : 0.f;          // (also l = -inf)
    const float t = d + m, err = (l - t) - (m - (t - d));   // l - m = d + err
    return expf(d) * (1.f + err);
}
// The same where 2^-22 and the difference's rounding (2^-24 of it) will do
__device__ __forceinline__ float exp_below_fast(float l, float m) { return ex2((l - m) * 1.4426950408889634f); }
__device__ __forceinline__ float sigmoid(float l) { return 1.f / (1.f + expf(-l)); }

// Where the row's softmax stands: its largest logit and 1 / sum
struct Norm {
    float m, inv;
};

// The factor of the lane's expert: s, or with renorm s / (sum of s + 1e-20).  The
// quotient is formed from scores relative to the largest chosen one, so that it
// keeps its accuracy where all of them are below FP32's range.
constexpr float kLnEps = -46.0517019f;   // ln(1e-20)
__device__ __forceinline__ float share(bool softmax, bool renorm, float l, bool live, Norm n)
{
    float s = 0.f, eps = 1e-20f;
    if (!renorm) return !live ? 0.f : softmax ? exp_below(l, n.m) * n.inv : sigmoid(l);
    const float base = of_key(warp_max(key_of(live ? l : -INFINITY)));
    if (base == -INFINITY) return 0.f;
    if (softmax) {
        if (live) s = exp_below(l, base);
        eps = expf(n.m - base + kLnEps) / n.inv;
    } else if (base > 0.f) {
        if (live) s = sigmoid(l);
    } else {
        if (live) s = exp_below(l, base) * sigmoid(-l);
        eps = expf(kLnEps - base);
    }
    return s / (warp_sum(s) + eps);
}

// The two largest values (keys, or FP32 numbers) seen so far
__device__ __forceinline__ void top2(uint64_t &a, uint64_t &b, uint64_t x)
{
    const uint64_t lo = x < a ? x : a;
    a = x < a ? a : x;
    b = lo > b ? lo : b;
}
__device__ __forceinline__ void top2(float &a, float &b, float x)
{
    const float lo = fminf(x, a);
    a = fmaxf(a, x);
    b = fmaxf(b, lo);
}

// Keeps the best `top` of G groups: lane g < G gives its group's score; the kept
// ones as a mask (ties to the lower group), and through `in`, `out` the least
// score kept and the largest not kept.
template <class Key>
__device__ __forceinline__ uint32_t keep_groups(Key score, int G, int top, Key &in, Key &out)
{
    const int lane = threadIdx.x & 31;
    int rank = 0;
    for (int g = 0; g < G; ++g) {
        const Key s = __shfl_sync(kAll, score, g);
        rank += s > score || (s == score && g < lane);
    }
    const bool kept = lane < G && rank < top;
    in = ~warp_max(kept ? ~score : (Key)0);
    out = warp_max(lane < G && !kept ? score : (Key)0);
    return __ballot_sync(kAll, kept);
}

// Each group's score in lane g < G, from the values of its experts in shared memory
// (expert e at e + e / 32): `val` makes it of the two best ones (`none`: not there).
template <class F, class V>
__device__ __forceinline__ auto group_score(const F *buf, const Args &a, F none, V val)
{
    const int lane = threadIdx.x & 31, sub = 1 << a.sublog;   // lanes of a group
    const int g = lane >> a.sublog, j = lane & (sub - 1);
    F x = none, y = none;
    if (g < a.G) {
        const int e0 = g * a.gsize;
        const int e1 = e0 + min((j + 1) * a.per, a.gsize);
#pragma unroll 4
        for (int e = e0 + j * a.per; e < e1; ++e) top2(x, y, buf[e + (e >> 5)]);
    }
    for (int o = 1; o < sub; o *= 2) {
        const F x2 = __shfl_xor_sync(kAll, x, o), y2 = __shfl_xor_sync(kAll, y, o);
        top2(x, y, x2);
        top2(x, y, y2);
    }
    return __shfl_sync(kAll, val(x, y), min(lane << a.sublog, 31));
}

__device__ __forceinline__ double exact_c(const Args &a, const float *row, int e, Norm n, double zinv)
{
    const double l = (double)row[e];
    const double s = a.softmax ? exp(l - (double)n.m) * zinv : 1. / (1. + exp(-l));
    return l == -INFINITY ? -INFINITY : s + (a.has_bias ? (double)a.bias[e] : 0.);
}
__device__ __forceinline__ double exact_zinv(const Args &a, const float *row, Norm n)
{
    if (!a.softmax) return 1.;
    double z = 0.;
    for (int e = threadIdx.x & 31; e < a.E; e += 32) z += exp((double)row[e] - (double)n.m);
    return 1. / warp_sum(z);
}

// Whether FP32 cannot tell x >= y apart: values off by up to err / 2 and their rounding
__device__ __forceinline__ bool near(float x, float y, float err)
{
    return y != -INFINITY && !(x - y > err + 2.3841858e-7f * (fabsf(x) + fabsf(y)));
}

// Whether two experts have the same logit and bias, and so the same c to the last bit: a
// tie, which goes to the lower id without a closer look
__device__ __forceinline__ bool same(const Args &a, const float *row, int e, int f)
{
    return row[e] == row[f] && (!a.has_bias || a.bias[e] == a.bias[f]);
}

// The groups' choice from FP64 scores: FP64 values are formed of the experts that count
// in each group by their FP32 ones; 0 where those (off by up to terr / 2) do not tell
// which ones count.
__device__ __noinline__ uint32_t keep_groups_exact(const Args &a, const float *row, Norm n, const float *buf, float terr)
{
    const int lane = threadIdx.x & 31, sub = 1 << a.sublog, g = lane >> a.sublog, j = lane & (sub - 1);
    const int e0 = g * a.gsize + j * a.per, e1 = g < a.G ? g * a.gsize + min((j + 1) * a.per, a.gsize) : 0;
    float x = -INFINITY, y = -INFINITY;   // the two largest, and their experts
    int xi = 0, yi = 0;
    auto put = [&](float k, int e) {
        if (k > x) y = x, yi = xi, x = k, xi = e;
        else if (k > y) y = k, yi = e;
    };
    for (int e = e0; e < e1; ++e) put(buf[e + (e >> 5)], e);
    for (int o = 1; o < sub; o *= 2) {
        const float x2 = __shfl_xor_sync(kAll, x, o), y2 = __shfl_xor_sync(kAll, y, o);
        const int xi2 = __shfl_xor_sync(kAll, xi, o), yi2 = __shfl_xor_sync(kAll, yi, o);
        put(x2, xi2);
        put(y2, yi2);
    }
    xi = __shfl_sync(kAll, xi, lane - j);   // (of equal ones each lane may have found others)
    yi = __shfl_sync(kAll, yi, lane - j);
    if (a.has_bias) {   // one that does not count and is close to the last that does, unless all of them are the same
        const float last = a.gsum == 2 ? y : x;
        const int li = a.gsum == 2 ? yi : xi;
        const bool other = a.gsum == 2 && near(x, y, terr) && !same(a, row, xi, yi);
        bool close = false;
        for (int e = e0; e < e1; ++e)
            if (e != xi && (a.gsum == 1 || e != yi) && near(last, buf[e + (e >> 5)], terr))
                close = close || other || !same(a, row, e, li);
        if (__any_sync(kAll, close)) return 0;
    }
    const double zinv = exact_zinv(a, row, n);
    double s = exact_c(a, row, xi, n, zinv);
    if (a.gsum == 2 && y != -INFINITY) s += exact_c(a, row, yi, n, zinv);
    if (x == -INFINITY) s = -INFINITY;
    uint64_t in, out;
    return keep_groups(__shfl_sync(kAll, key_of(s), min(lane << a.sublog, 31)), a.G, a.top, in, out);
}

// The largest keys in shared memory (expert e at e + e / 32), in order: lane j < rounds
// returns the j-th expert (and leaves the keys in `keys`)
template <class Key>
__device__ __noinline__ int choose(const Args &a, Key *buf, int rounds, Key *keys)
{
    const int lane = threadIdx.x & 31;
    int mine = 0;
    Key key = 0;
    for (int j = 0; j < rounds; ++j) {
        Key best = 0;
        int id = 0x7fffffff;
        for (int e = lane; e < a.E; e += 32) {
            const Key v = buf[e + (e >> 5)];
            if (v > best) best = v, id = e;
        }
        const Key m = warp_max(best);
        const int e = (int)__reduce_min_sync(kAll, best == m ? (uint32_t)id : 0x7fffffffu);
        if (e < a.E && e % 32 == lane) buf[e + (e >> 5)] = 0;
        __syncwarp();
        if (lane == j && e < a.E) mine = e, key = m;
    }
    if (keys) keys[lane] = key;
    __syncwarp();
    return mine;
}
// Whether an expert that `choose` has left is close to the one at place `at` (off by up to
// err / 2, lane j has the key and the expert of place j), the same ones only if `alike`
__device__ __noinline__ bool close_left(const Args &a, const float *row, const uint32_t *buf, uint32_t key, int id, int at,
                                        bool alike, float err)
{
    const float x = of_key(__shfl_sync(kAll, key, at));
    const int f = __shfl_sync(kAll, id, at);
    bool close = false;
    for (int e = threadIdx.x & 31; e < a.E; e += 32) {
        const uint32_t k = buf[e + (e >> 5)];
        if (k && near(x, of_key(k), err)) close = close || alike || !same(a, row, e, f);
    }
    return __any_sync(kAll, close);
}
// The first place from the k-th on that the next one is not close to (bit j: places j and
// j + 1 are close; bit 31 is clear)
__device__ __forceinline__ int run_end(uint32_t close, int k) { return k - 1 + __ffs((int)~(close >> (k - 1))) - 1; }
// The whole choice in FP64
__device__ __noinline__ int choose_exact(const Args &a, const float *row, Norm n, uint64_t *buf)
{
    const int lane = threadIdx.x & 31;
    const double zinv = exact_zinv(a, row, n);
    for (int e = lane; e < a.E; e += 32) buf[e + (e >> 5)] = key_of(exact_c(a, row, e, n, zinv));
    __syncwarp();
    if (a.grouped) {
        uint64_t in, out;
        const uint64_t s = group_score(buf, a, (uint64_t)0, [&](uint64_t x, uint64_t y) {
            return a.gsum == 1 || y <= 1 || of_key(y) == -INFINITY ? x : key_of(of_key(x) + of_key(y));
        });
        const uint32_t kept = keep_groups(s, a.G, a.top, in, out);
        __syncwarp();
        for (int e = lane; e < a.E; e += 32)
            if (!(kept >> (e / a.gsize) & 1u)) buf[e + (e >> 5)] = 0;
        __syncwarp();
    }
    return choose(a, buf, a.k, (uint64_t *)nullptr);
}
// The FP64 order of a few candidates (lane < cnt has one): lane j < k returns the j-th
__device__ __noinline__ int order_exact(const Args &a, const float *row, Norm n, int e, int cnt, int *slot)
{
    const int lane = threadIdx.x & 31;
    const double zinv = exact_zinv(a, row, n);
    const uint64_t c = lane < cnt ? key_of(exact_c(a, row, e, n, zinv)) : 0ull;
    int rank = 0;
    for (int j = 0; j < cnt; ++j) {
        const uint64_t o = __shfl_sync(kAll, c, j);
        const int oe = __shfl_sync(kAll, e, j);
        rank += o > c || (o == c && oe < e);
    }
    __syncwarp();
    if (lane < cnt) slot[rank] = e;
    __syncwarp();
    return slot[lane];
}

// One warp a token, experts 32 i + lane in a lane's registers
//
// The best k are found among few candidates: the (k + 2)-th largest of the lanes' own
// largest values bounds the (k + 2)-th largest of all from below, and the experts from
// there up (some 11 for k = 8, E = 384) are gathered, one a lane, and ranked.  (Taking the
// largest k times over, each time looking through all of them again, took 1280 instructions
// a token at k = 8, E = 384, against 870, and 18.6 us for 8192 tokens against 12.)  The values
// of that search are c by approximate exponentials (by tanh.approx it was no faster); the
// candidates' scores are computed in full.
//
// Bound by the issue of instructions, 60 to 70% of the slots at 32 warps an SM: 870 a token for
// E = 384 without groups, 1180 for E = 256 with 8 (23 us for 16384 tokens; their logits are 2.5
// us of HBM).  Fewer registers (12 CTAs of 4 warps an SM) or more (6) take the same or 10% longer.
// CTAs of 4 warps an SM: 8 (64 registers) up to 512 experts, 5 up to 1024.  With the registers
// that the compiler takes by itself 8192 tokens of 512 experts, biased, take 16.7 us instead of
// 12.7, of 1024 28 instead of 23 (with 4 CTAs 25).
constexpr int ctas_an_sm(int n) { return n <= 16 ? 8 : n <= 32 ? 5 : 1; }
enum Mode { kLogits = 0, kBias = 1, kGroups = 2 };   // neither a bias nor groups; a bias; groups
template <int kN, int kWarps, int kMode>
__global__ void __launch_bounds__(32 * kWarps, ctas_an_sm(kN)) k_gate(const Args a)
{
    const bool has_bias = kMode == kGroups ? a.has_bias : kMode == kBias, softmax = a.softmax;
    constexpr bool grouped = kMode == kGroups;
    extern __shared__ uint64_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // keys of a token: FP32 ones, of FP64 values for a close call
    uint64_t *buf = (uint64_t *)((uint8_t *)smem + (size_t)warp * (((a.E + a.E / 32 + 1) * (has_bias ? 8 : 4) + 7) & ~7));
    __shared__ int cand_id[kWarps][32];
    __shared__ float cand_c[kWarps][32], cand_s[kWarps][32];
    int *ci = cand_id[warp];
    float *cc = cand_c[warp], *cs = cand_s[warp];
    grid_wait();
    grid_go();
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T; t += (int64_t)gridDim.x * kWarps) {
        const float *row = a.logits + t * a.E;
        float v[kN];   // -inf: no expert, or one that cannot be chosen
        Norm n{0.f, 1.f};
        // (all loads on their way at once: the barrier keeps them from being put off to their uses)
        constexpr bool kBiasFirst = kN <= 16;
        float bias[kBiasFirst ? kN : 1];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int e = i * 32 + lane;
            v[i] = e < a.E ? row[e] : -INFINITY;
            if constexpr (kBiasFirst) bias[i] = has_bias && e < a.E ? a.bias[e] : 0.f;
        }
        if constexpr (kBiasFirst) __syncwarp();
        if (softmax) {
            float m = v[0];
#pragma unroll
            for (int i = 1; i < kN; ++i) m = fmaxf(m, v[i]);
            m = warp_fmax(m);
            n.m = m == -INFINITY ? 0.f : m;   // (no expert can be chosen: all scores are zero)
            if (has_bias || grouped || !a.renorm) {
                float z = 0.f;
                if (has_bias) {   // (v is the exponential from here on; -inf stays)
#pragma unroll
                    for (int i = 0; i < kN; ++i) {
                        const float x = exp_below_fast(v[i], n.m);
                        z += x;
                        v[i] = v[i] == -INFINITY ? v[i] : x;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kN; ++i) z += exp_below_fast(v[i], n.m);
                }
                z = warp_sum(z);
                n.inv = z > 0.f ? 1.f / z : z == 0.f ? 0.f : z;
            }
        }
        if (has_bias) {
            // (a loop for each form: a choice within one costs some 500 instructions a token)
            auto form = [&](auto score) {
                constexpr int kB = kN < 8 ? kN : 8;   // biases loaded at once where not all were
#pragma unroll
                for (int i0 = 0; i0 < kN; i0 += kB) {
                    float late[kB];
                    if constexpr (!kBiasFirst) {
#pragma unroll
                        for (int i = 0; i < kB; ++i) {
                            const int e = (i0 + i) * 32 + lane;
                            late[i] = e < a.E ? a.bias[e] : 0.f;
                        }
                        __syncwarp();
                    }
#pragma unroll
                    for (int i = i0; i < i0 + kB && i < kN; ++i) {
                        const float c = score(v[i], kBiasFirst ? bias[kBiasFirst ? i : 0] : late[i - i0]);
                        v[i] = v[i] == -INFINITY ? -INFINITY : c;
                    }
                }
            };
            if (softmax) form([&](float x, float b) { return fmaf(x, n.inv, b); });
            else form([](float l, float b) { return rcp(1.f + ex2(l * -1.4426950408889634f)) + b; });
        }
        // Bounds of the error of the difference of two c beside their own rounding.  Sigmoid:
        // a score by ex2 and rcp (v) is off by less than 2^-21 / 2, one by sigmoid() (the
        // candidates') by less than 2^-22 (the exponential's 2 units times s (1 - s), a sum
        // and a quotient).  Softmax: the row's sum adds a unit of 2^-24 a term.
        const float terr = softmax ? n.inv * (float)(kN + 16) * 1.1920929e-7f : 9.5367432e-7f;
        const float cerr = softmax ? terr : 4.7683716e-7f;
        int mine = 0, cnt = 0;
        bool whole = false;   // too close to call in FP32, for the groups or among many
        uint32_t kept = kAll;
        auto group_of = [&](uint32_t e) { return (a.gmagic ? __umulhi(e, a.gmagic) : e) & 31u; };
        if constexpr (grouped) {
            float *vb = (float *)buf;
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int e = i * 32 + lane;
                if (e < a.E) vb[e + (e >> 5)] = v[i];
            }
            __syncwarp();
            // (without a bias v is the logit: sums of two are of the scores)
            float size = 0.f;   // of what the lane's group is the sum of
            const float score = group_score(vb, a, -INFINITY, [&](float x, float y) {
                if (a.gsum == 1 || x == -INFINITY) return x;
                if (has_bias) {
                    if (y == -INFINITY) return x;
                    size = fabsf(x) + fabsf(y);
                    return x + y;
                }
                if (softmax) return exp_below(x, n.m) + exp_below(y, n.m);
                return sigmoid(x) + sigmoid(y);
            });
            uint32_t in, out;
            kept = keep_groups(key_of(score), a.G, a.top, in, out);
            const float x = of_key(in), y = of_key(out);   // the least score kept, the largest one not
            bool tie = false;
            if (has_bias && a.gsum == 1) tie = near(x, y, terr);
            else if (has_bias) {
                // (terms of opposite sign leave of their sum less than they are rounded by: the largest of
                // all groups bounds that)
                const float most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(size)));
                tie = near(0.5f * x, 0.5f * y, terr + 1.1920929e-7f * most) || most > 3.4e38f;
            }
            else if (a.gsum == 2) tie = y != -INFINITY && !(x - y > 1.9073486e-6f * x + 1e-36f);   // (each score to 2^-21)
            if (tie) {
                kept = keep_groups_exact(a, row, n, vb, terr);
                whole = kept == 0;
            }
#pragma unroll
            for (int i = 0; i < kN; ++i) v[i] = kept >> group_of(i * 32 + lane) & 1u ? v[i] : -INFINITY;
            __syncwarp();
        }
        float s = 0.f;
        bool scored = false;   // s is the lane's score
        int close = 0;         // the first so many lanes' experts are to be put in order by FP64 values
        if (!whole) {
            float best = v[0];
#pragma unroll
            for (int i = 1; i < kN; ++i) best = fmaxf(best, v[i]);
            // the lanes' largest values sorted, descending (a bitonic network)
#pragma unroll
            for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
                for (int o = size / 2; o; o /= 2) {
                    const float other = __shfl_xor_sync(kAll, best, o);
                    const bool up = ((lane & o) == 0) == ((lane & size) == 0);
                    best = up ? fmaxf(best, other) : fminf(best, other);
                }
            }
            // (-inf: fewer lanes have any that can be chosen, all are candidates)
            const float least = __shfl_sync(kAll, best, min(a.k + 2, 32) - 1);
            const bool all = least == -INFINITY;
            // (less by twice the error of the values)
            const float from = all        ? -3.402823466e38f
                               : has_bias ? least - (terr + 4.7683716e-7f * fabsf(least))
                                          : least;
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const bool in = v[i] >= from;
                const uint32_t b = __ballot_sync(kAll, in);
                if (b) {
                    const int at = cnt + __popc(b & ((1u << lane) - 1u));
                    if (in && at < 32) ci[at] = i * 32 + lane;
                    cnt += __popc(b);
                }
            }
            __syncwarp();
            if (cnt > 32 || cnt < a.k || (has_bias && cnt == a.k && !all)) {
                // many candidates (k near the number of lanes, many equal ones) or few that can be chosen
                whole = has_bias && a.k == 32;
                if (!whole) {   // by FP32 keys, the largest one at a time
                    uint32_t *kb = (uint32_t *)buf;
#pragma unroll
                    for (int i = 0; i < kN; ++i) {   // (0: of a group that is out)
                        const int e = i * 32 + lane;
                        if (e < a.E) kb[e + (e >> 5)] = kept >> group_of(e) & 1u ? key_of(v[i]) : 0u;
                    }
                    __syncwarp();
                    mine = choose(a, kb, has_bias ? min(a.k + 2, 32) : a.k, (uint32_t *)cc);
                    if (has_bias) {
                        // close ones are put in order by their FP64 values, unless they go on behind the
                        // places that were found.  (Where all are the same, the same ones behind them may.)
                        const uint32_t mk = ((uint32_t *)cc)[lane], nk = __shfl_down_sync(kAll, mk, 1);
                        const uint32_t nb = __ballot_sync(kAll, lane < 31 && mk && nk && near(of_key(mk), of_key(nk), terr));
                        if (nb << (32 - a.k)) {
                            const int nid = __shfl_down_sync(kAll, mine, 1), end = run_end(nb, a.k);
                            const uint32_t b = __ballot_sync(kAll, (nb >> lane & 1u) && !same(a, row, mine, nid));
                            if (b & ((1u << end) - 1u)) close = end + 1;
                            whole = end + 1 == min(a.k + 2, 32) && close_left(a, row, kb, mk, mine, end, close != 0, terr);
                        }
                    }
                }
            } else {
                const int e = lane < cnt ? ci[lane] : 0;
                const float l = lane < cnt ? row[e] : -INFINITY;
                float c = l;
                if (has_bias) {
                    s = softmax ? exp_below(l, n.m) * n.inv : sigmoid(l);
                    if (lane < cnt) c = s + a.bias[e];
                }
                int rank = 0;
#pragma unroll 4
                for (int j = 0; j < cnt; ++j) {
                    const float o = __shfl_sync(kAll, c, j);
                    rank += o > c || (o == c && j < lane);
                }
                __syncwarp();
                if (lane < cnt) ci[rank] = e, cc[rank] = c, cs[rank] = s;
                __syncwarp();
                mine = lane < cnt ? ci[lane] : 0;
                c = lane < cnt ? cc[lane] : -INFINITY;
                if (has_bias) {
                    s = cs[lane];
                    const float nc = __shfl_down_sync(kAll, c, 1);
                    const uint32_t nb = __ballot_sync(kAll, lane + 1 < cnt && near(c, nc, cerr));
                    scored = true;
                    if (nb << (32 - a.k)) {
                        const int nid = __shfl_down_sync(kAll, mine, 1);
                        const uint32_t b = __ballot_sync(kAll, (nb >> lane & 1u) && !same(a, row, mine, nid));
                        scored = !(b & ((1u << run_end(nb, a.k)) - 1u));
                    }
                    if (!scored) close = cnt;
                } else {
                    s = softmax ? exp_below(c, n.m) * n.inv : sigmoid(c);
                    scored = true;
                }
            }
            __syncwarp();
        }
        if (whole) mine = choose_exact(a, row, n, buf);
        else if (close) mine = order_exact(a, row, n, mine, close, ci);
        // the weights: the scores without the bias
        const bool live = lane < a.k;
        float w = 0.f;
        if (scored) {
            if (!live) s = 0.f;
            const float D = a.renorm ? warp_sum(s) : 1.f;
            w = a.renorm ? s / D : s;          // (1e-20 is below half a unit of D)
            scored = D > 0.25f;
        }
        if (!scored) w = share(softmax, a.renorm, live ? row[mine] : 0.f, live, n);
        if (live) {
            a.idx[t * a.k + lane] = mine;
            a.w[t * a.k + lane] = a.factor * w;
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------------ gradient
// With D = sum of the chosen scores + 1e-20 (or 1), the gradient of score j is
//   ds_j = factor / D (dw_j - [renorm] sum_i dw_i s_i / D)
// and that of the logits
//   sigmoid: dl_j = ds_j s_j (1 - s_j) of the chosen experts, else 0
//   softmax: dl_e = s_e ([chosen] ds_e - sum_j ds_j s_j)
// An expert that idx names twice takes both parts.
struct BwdArgs {
    int T, E, k;
    int softmax, renorm, accumulate;
    float factor;
    const float *logits;
    const int32_t *idx;
    const float *dw;
    float *dl;
};

// Sums over the kW lanes of a token
template <int kW>
__device__ __forceinline__ float token_sum(float v)
{
#pragma unroll
    for (int o = kW / 2; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
// The parts g of the same expert (e, and whose token: `same` has its lanes) summed in
// order for the first lane that has it; false in the other lanes
__device__ __forceinline__ bool first_of(uint32_t same, bool live, float &g)
{
    const int lane = threadIdx.x & 31;
    const bool first = live && (same & ((1u << lane) - 1u)) == 0;
    if (__any_sync(kAll, live && !first)) {
        float sum = 0.f;
        for (int j = 0; j < 32; ++j) {
            const float o = __shfl_sync(kAll, g, j);
            if (same >> j & 1u) sum += o;
        }
        g = sum;
    }
    return first;
}

// Sigmoid: kW lanes a token, the least power of two that holds k, as only the chosen logits
// are read.  (8192 tokens of 384 experts, k = 8: 7.1 us alone with 8 lanes, 10 with a warp a token.)
template <int kW, int kWarps>
__global__ void __launch_bounds__(32 * kWarps) k_gate_backward_sigmoid(const BwdArgs a)
{
    constexpr int kTok = 32 / kW;   // tokens of a warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % kW;
    grid_wait();
    grid_go();
    for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * kTok; t0 < a.T; t0 += (int64_t)gridDim.x * kWarps * kTok) {
        const int64_t t = t0 + lane / kW;
        int e = -1;
        float dw = 0.f;
        if (t < a.T && j < a.k) {
            e = a.idx[t * a.k + j];
            dw = a.dw[t * a.k + j];
        }
        const bool live = e >= 0 && e < a.E;
        const float l = live ? a.logits[t * a.E + e] : -INFINITY;
        if (!live) dw = 0.f;
        if (!a.accumulate) {   // zeros around the chosen experts
            float *out = a.dl + t0 * a.E;
            const int n = (int)(a.T - t0 < kTok ? a.T - t0 : kTok) * a.E;
            int i = 0;
            if (((t0 * a.E) & 3) == 0) {
                for (i = lane; i < n / 4; i += 32) ((float4 *)out)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                i = n & ~3;
            }
            for (i += lane; i < n; i += 32) out[i] = 0.f;
        }
        float p = sigmoid(l);
        if (a.renorm) {
            const float D = token_sum<kW>(p);
            p = p / (D + 1e-20f);
            if (__any_sync(kAll, !(D > 0.25f))) {   // (small scores: relative to the largest one, as in share)
                float base = l;
#pragma unroll
                for (int o = kW / 2; o; o >>= 1) base = fmaxf(base, __shfl_xor_sync(kAll, base, o));
                const float r = base == -INFINITY ? 0.f : exp_below(l, base) * sigmoid(-l);
                const float all = token_sum<kW>(r) + expf(kLnEps - base);
                if (!(base > 0.f)) p = base == -INFINITY ? 0.f : r / all;
            }
        }
        const float mean = a.renorm ? token_sum<kW>(dw * p) : 0.f;
        // ds_j s_j = factor (dw_j - mean) p_j with p_j the weight before its factor;
        // 1 - s as the score of the opposite logit: it keeps its accuracy near 0
        float g = live ? a.factor * (dw - mean) * p * sigmoid(-l) : 0.f;
        const bool first = first_of(__match_any_sync(kAll, live ? e << 5 | lane / kW : -1 - lane), live, g);
        __syncwarp();   // (orders the zeros before what takes their place)
        if (first) {
            float *q = a.dl + t * a.E + e;
            *q = a.accumulate ? *q + g : g;
        }
    }
}

// Softmax: a warp a token, experts 32 i + lane in a lane's registers
template <int kN, int kWarps>
__global__ void __launch_bounds__(32 * kWarps) k_gate_backward_softmax(const BwdArgs a)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_wait();
    grid_go();
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T; t += (int64_t)gridDim.x * kWarps) {
        const float *row = a.logits + t * a.E;
        float *out = a.dl + t * a.E;
        const int e = lane < a.k ? a.idx[t * a.k + lane] : -1;
        const bool live = e >= 0 && e < a.E;
        const float dw = live ? a.dw[t * a.k + lane] : 0.f;
        const float l = live ? row[e] : 0.f;
        float v[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = i * 32 + lane < a.E ? row[i * 32 + lane] : -INFINITY;
        float m = v[0];
#pragma unroll
        for (int i = 1; i < kN; ++i) m = fmaxf(m, v[i]);
        m = warp_fmax(m);
        if (m == -INFINITY) m = 0.f;
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < kN; ++i) z += v[i] = exp_below_fast(v[i], m);
        z = warp_sum(z);
        const float inv = z > 0.f ? 1.f / z : z == 0.f ? 0.f : z;
        const float p = share(true, a.renorm, l, live, Norm{m, inv});
        const float mean = a.renorm ? warp_sum(dw * p) : 0.f;
        float g = live ? a.factor * (dw - mean) * p : 0.f;
        const float c = -inv * warp_sum(g);
        const bool first = first_of(__match_any_sync(kAll, live ? e : -1 - lane), live, g);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int j = i * 32 + lane;
            if (j < a.E) out[j] = a.accumulate ? fmaf(v[i], c, out[j]) : v[i] * c;
        }
        __syncwarp();   // (orders the row's stores before what is added to them)
        if (first) out[e] += g;
        __syncwarp();
    }
}

static bool ok(const pmoe_gate &g)
{
    if (g.T < 0 || g.E < 1 || g.E > 4096 || g.k < 1 || g.k > 32 || g.k > g.E) return false;
    if (g.groups < 1 || g.groups > kMaxGroups || g.E % g.groups || g.topk_groups < 1 || g.topk_groups > g.groups) return false;
    if (g.k > g.topk_groups * (g.E / g.groups)) return false;
    if (g.group_sum != 1 && g.group_sum != 2) return false;
    if (g.score != PMOE_SCORE_SIGMOID && g.score != PMOE_SCORE_SOFTMAX) return false;
    if (!std::isfinite(g.factor)) return false;
    return (int64_t)g.T * g.k <= (int64_t)INT32_MAX / 2;
}
static bool aligned(std::initializer_list<const void *> ps)
{
    for (const void *p : ps)
        if ((uintptr_t)p & 15) return false;
    return true;
}

// f(the experts a lane holds)
template <class F>
static bool by_size(int E, F f)
{
    const int n = (int)cdiv(E, 32);
    return n <= 1    ? f(std::integral_constant<int, 1>())
           : n <= 2  ? f(std::integral_constant<int, 2>())
           : n <= 4  ? f(std::integral_constant<int, 4>())
           : n <= 8  ? f(std::integral_constant<int, 8>())
           : n <= 12 ? f(std::integral_constant<int, 12>())
           : n <= 16 ? f(std::integral_constant<int, 16>())
           : n <= 32 ? f(std::integral_constant<int, 32>())
                     : f(std::integral_constant<int, 128>());
}
static unsigned ctas_of(int T, int warps)
{
    return (unsigned)std::min<int64_t>(cdiv(T, warps), (int64_t)gemm_num_sms() * 128);
}

template <int kN>
static bool launch_as(const Args &a, cudaStream_t st)
{
    constexpr int kWarps = 4;
    const size_t smem = (size_t)kWarps * (((a.E + a.E / 32 + 1) * (a.has_bias ? 8 : 4) + 7) & ~7);
    auto launch = [&](auto mode) {
        constexpr auto kern = k_gate<kN, kWarps, decltype(mode)::value>;
        if (smem > 40 * 1024 &&
            !set_attribute<kern, cudaFuncAttributeMaxDynamicSharedMemorySize>((int)(kWarps * (32 * kN + kN + 1) * 8)))
            return false;
        return launch_chained<kern>(ctas_of(a.T, kWarps), 32 * kWarps, smem, 1, st, a);
    };
    // (the groups' and the bias's code costs the cases without them registers)
    return a.grouped    ? launch(std::integral_constant<int, kGroups>())
           : a.has_bias ? launch(std::integral_constant<int, kBias>())
                        : launch(std::integral_constant<int, kLogits>());
}
static bool launch_backward(const BwdArgs &a, cudaStream_t st)
{
    if (a.softmax)
        return by_size(a.E, [&](auto n) {
            constexpr int kN = decltype(n)::value, kWarps = kN > 32 ? 4 : 8;
            return launch_chained<k_gate_backward_softmax<kN, kWarps>>(ctas_of(a.T, kWarps), 32 * kWarps, 0, 1, st, a);
        });
    auto launch = [&](auto w) {
        constexpr int kW = decltype(w)::value;
        return launch_chained<k_gate_backward_sigmoid<kW, 4>>(ctas_of(a.T, 4 * (32 / kW)), 128, 0, 1, st, a);
    };
    return a.k <= 4    ? launch(std::integral_constant<int, 4>())
           : a.k <= 8  ? launch(std::integral_constant<int, 8>())
           : a.k <= 16 ? launch(std::integral_constant<int, 16>())
                       : launch(std::integral_constant<int, 32>());
}

}  // namespace gate
}  // namespace pmoe

using namespace pmoe;

extern "C" {

pmoe_status moe_gate_forward(pmoe_gate g, const float *logits, const float *bias, int32_t *idx, float *w,
                             cudaStream_t stream)
{
    if (!gate::ok(g) || (g.T > 0 && (!logits || !idx || !w)) || !gate::aligned({logits, bias, idx, w}))
        return PMOE_ERR_INVALID_ARG;
    if (g.T == 0) return PMOE_OK;
    gate::Args a{};
    a.T = g.T;
    a.E = g.E;
    a.k = g.k;
    a.G = g.groups;
    a.top = g.topk_groups;
    a.gsum = g.group_sum;
    a.gsize = g.E / g.groups;
    while ((2 << a.sublog) * a.G <= 32) ++a.sublog;
    a.per = (a.gsize + (1 << a.sublog) - 1) >> a.sublog;
    a.gmagic = a.gsize > 1 ? (uint32_t)(((1ull << 32) + a.gsize - 1) / a.gsize) : 0u;
    a.softmax = g.score == PMOE_SCORE_SOFTMAX;
    a.renorm = g.renorm != 0;
    a.has_bias = bias != nullptr;
    a.grouped = g.topk_groups < g.groups;
    a.factor = g.factor;
    a.logits = logits;
    a.bias = bias;
    a.idx = idx;
    a.w = w;
    const bool done = gate::by_size(g.E, [&](auto n) { return gate::launch_as<decltype(n)::value>(a, stream); });
    return done ? PMOE_OK : PMOE_ERR_CUDA;
}

pmoe_status moe_gate_backward(pmoe_gate g, const float *logits, const int32_t *idx, const float *d_topk_w,
                              int accumulate, float *dlogits, cudaStream_t stream)
{
    if (!gate::ok(g) || (g.T > 0 && (!logits || !idx || !d_topk_w || !dlogits)) ||
        !gate::aligned({logits, idx, d_topk_w, dlogits}))
        return PMOE_ERR_INVALID_ARG;
    if (g.T == 0) return PMOE_OK;
    gate::BwdArgs a{g.T, g.E, g.k, g.score == PMOE_SCORE_SOFTMAX, g.renorm != 0, accumulate != 0, g.factor,
                    logits, idx, d_topk_w, dlogits};
    return gate::launch_backward(a, stream) ? PMOE_OK : PMOE_ERR_CUDA;
}

}  // extern "C"
