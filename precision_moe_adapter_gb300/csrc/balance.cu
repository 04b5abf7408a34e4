// balance.cu -- the router's training side: the load-balance loss with the
// per-expert counts, and the gradient of the router logits from that loss and
// from the routing weights (moe_backward_data's d_topk_w).
//
// Both passes read the [T, E] logits once and hold a token's row in
// registers, NI values per thread of its group: a warp per token up to 1024
// experts, a CTA per token above (rows of up to 4096 do not fit a warp's
// registers).  The work per token is a chain of short steps (row, maximum,
// sum, dot), so what counts is that all of a token's loads are on their way
// at once and that enough tokens are in flight; three launches in a chain.
#include <cmath>

#include "common.cuh"
#include "pdl.cuh"

namespace pmoe {
namespace bal {

constexpr int kThreads = 256;      // backward
constexpr int kRedThreads = 1024;  // reduction, at most
constexpr float kNegInf = -INFINITY;

struct Ws {
    DevErr *err;
    float *psum;             // [slots][Ep] probability sums of a (slab, sequence) overlap
    int32_t *cnt;            // [slots][Ep] counts
    int32_t *ntok;           // [slots] tokens
    int L, slots, Ep;
    size_t bytes;
};
// Tokens are cut into slabs of L; a slab and a sequence that overlap own the
// partial sums in slot slab + sequence (overlaps form a staircase, so the
// slots are distinct).
static Ws carve(void *base, int T, int E, int nseq)
{
    size_t off = 0;
    auto take = [&](size_t n) {
        uint8_t *p = base ? (uint8_t *)base + off : nullptr;
        off += (n + 255) & ~(size_t)255;
        return p;
    };
    Ws w;
    // (16 warps share a slab; slabs of short sequences hold about two of them)
    const int64_t least = std::min<int64_t>(16, std::max<int64_t>(1, 2ll * T / nseq));
    w.L = (int)std::max<int64_t>(least, T > 16 * 2 * 152 ? cdiv(cdiv(T, 2 * 152), 16) * 16 : 0);
    w.slots = (int)cdiv(std::max(T, 1), w.L) + nseq;
    w.Ep = (E + 3) & ~3;
    w.err = (DevErr *)take(kHdrBytes);
    w.psum = (float *)take((size_t)w.slots * w.Ep * 4);
    w.cnt = (int32_t *)take((size_t)w.slots * w.Ep * 4);
    w.ntok = (int32_t *)take((size_t)w.slots * 4);
    w.bytes = off;
    return w;
}

// Sequence bounds, held inside [0, T] whatever the caller's array says
__device__ __forceinline__ int seq_at(const int32_t *seq, int s, int nseq, int T)
{
    if (!seq) return s == 0 ? 0 : T;
    return min(max(seq[s], 0), T);
}
// The sequence that holds token t: the last s with seq[s] <= t (nseq if t is
// past the last sequence's end, -1 before the first).  By a whole warp, 32
// bounds at a time: a search in halves would wait for a load at every step.
__device__ __forceinline__ int seq_of(const int32_t *seq, int nseq, int T, int t)
{
    if (!seq) return t < T ? 0 : 1;
    const int lane = threadIdx.x & 31;
    int lo = 0, len = nseq + 1;   // the first bound > t is in [lo, lo + len], known > t at lo + len
    while (len > 0) {
        const int stride = (len + 31) >> 5, i = lo + (lane + 1) * stride - 1;
        const unsigned b = __ballot_sync(0xffffffffu, i >= lo + len || seq_at(seq, i, nseq, T) > t);
        const int f = b ? __ffs(b) - 1 : 32;   // the first stride whose last bound is > t
        const int end = lo + len;
        lo = min(lo + f * stride, end);
        len = stride > 1 ? min(stride - 1, end - lo) : 0;
    }
    return lo - 1;
}

// Threads of the forward's CTAs: 16 warps share a slab, or one group of TPT
// threads is the CTA (its reductions are CTA barriers)
constexpr int fwd_threads(int tpt) { return tpt > 32 ? tpt : 512; }

// Reductions over a group of TPT threads (a warp, or the whole CTA)
template <int TPT, class Op>
__device__ __forceinline__ float group_reduce(float v, Op op, float *sh)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if constexpr (TPT > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
        __syncthreads();
        v = sh[0];
        for (int i = 1; i < TPT / 32; ++i) v = op(v, sh[i]);
    }
    return v;
}
struct Max {
    __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Add {
    __device__ float operator()(float a, float b) const { return a + b; }
};

// Thread `tid` of a group holds NI columns of a row, in runs of V (V = 4:
// 16-byte loads, where E is a multiple of 4; else 1): value i is column
template <int TPT, int V>
__device__ __forceinline__ int col_of(int tid, int i) { return (i / V * TPT + tid) * V + i % V; }

template <int TPT, int V, int NI>
__device__ __forceinline__ void row_load(const float *__restrict__ l, int E, int tid, float (&p)[NI])
{
#pragma unroll
    for (int i = 0; i < NI; i += V) {
        const int e = col_of<TPT, V>(tid, i);
        if constexpr (V == 4) {
            const float4 x = e < E ? *(const float4 *)(l + e) : make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
            p[i] = x.x, p[i + 1] = x.y, p[i + 2] = x.z, p[i + 3] = x.w;
        } else {
            p[i] = e < E ? l[e] : kNegInf;
        }
    }
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// softmax of such a row; a row of -inf only has p = 0.  In base 2: the
// rounding of m log2(e) is common to the row and cancels, the rest is one
// rounding of each exponent and exp2's own error.
template <int TPT, int NI>
__device__ __forceinline__ void row_softmax(float (&p)[NI], float *sh)
{
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < NI; ++i) m = fmaxf(m, p[i]);
    m = group_reduce<TPT>(m, Max(), sh);
    constexpr float kLog2e = 1.4426950408889634f;
    const float m2 = m == kNegInf ? 0.f : m * kLog2e;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        p[i] = ex2(fmaf(p[i], kLog2e, -m2));
        s += p[i];
    }
    s = group_reduce<TPT>(s, Add(), sh);
    const float inv = m == kNegInf ? 0.f : 1.f / s;
#pragma unroll
    for (int i = 0; i < NI; ++i) p[i] *= inv;
}

// ------------------------------------------------------------------ forward
// Partial sums of one slab: per overlapping sequence, the token groups' sums
// of p (added in group order), the counts (integer atomics: order-free) and
// the number of tokens.  A group loads its next row while it works on one.
template <int TPT, int V, int NI>
__global__ void __launch_bounds__(fwd_threads(TPT)) k_balance_partial(int T, int E, int k, int L, int Ep,
                                                                 const float *__restrict__ logits,
                                                                 const int32_t *__restrict__ idx,
                                                                 const uint8_t *__restrict__ valid,
                                                                 const int32_t *__restrict__ seq, int nseq,
                                                                 float *__restrict__ psum, int32_t *__restrict__ cnt,
                                                                 int32_t *__restrict__ ntok, DevErr *err)
{
    constexpr int kFwdThreads = fwd_threads(TPT);
    extern __shared__ float sm[];   // [groups][Ep] sums, then [Ep] counts
    __shared__ float sh[kFwdThreads / 32];
    __shared__ int sn;
    constexpr int kGroups = kFwdThreads / TPT;
    int *sc = (int *)(sm + kGroups * Ep);
    const int grp = threadIdx.x / TPT, tid = threadIdx.x % TPT;
    const int t0 = blockIdx.x * L, t1 = min(T, t0 + L);
    grid_wait();
    grid_go();
    for (int s = max(0, seq_of(seq, nseq, T, t0)); s < nseq; ++s) {
        const int a0 = seq_at(seq, s, nseq, T), b0 = seq_at(seq, s + 1, nseq, T);
        if (a0 >= t1) break;
        const int a = max(a0, t0), b = min(b0, t1);
        if (a >= b) continue;
        __syncthreads();   // the previous sequence's sums have been written out
        for (int e = threadIdx.x; e < E; e += kFwdThreads) sc[e] = 0;
        if (threadIdx.x == 0) sn = 0;
        __syncthreads();
        float acc[NI], next[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[i] = 0.f;
        int n = 0, t = a + grp;
        if (t < b) row_load<TPT, V>(logits + (int64_t)t * E, E, tid, next);
        for (; t < b; t += kGroups) {
            float p[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) p[i] = next[i];
            const bool use = !valid || valid[t];
            const int e = tid < k ? idx[(int64_t)t * k + tid] : 0;
            if (t + kGroups < b) row_load<TPT, V>(logits + (int64_t)(t + kGroups) * E, E, tid, next);
            if (!use) continue;
            row_softmax<TPT, NI>(p, sh);
#pragma unroll
            for (int i = 0; i < NI; ++i) acc[i] += p[i];
            if (tid < k) {
                if (e >= 0 && e < E) atomicAdd(&sc[e], 1);
                else record_error(err, PMOE_ERR_BAD_INDEX, t, e);
            }
            ++n;
        }
#pragma unroll
        for (int i = 0; i < NI; i += V) {
            const int e = col_of<TPT, V>(tid, i);
            if (e >= E) continue;
            if constexpr (V == 4) *(float4 *)(sm + grp * Ep + e) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
            else sm[grp * Ep + e] = acc[i];
        }
        if (tid == 0) atomicAdd(&sn, n);
        __syncthreads();
        const int64_t slot = (int64_t)blockIdx.x + s;
        for (int e = threadIdx.x; e < Ep; e += kFwdThreads) {
            float v = 0.f;
            if (e < E) {
#pragma unroll
                for (int g = 0; g < kGroups; ++g) v += sm[g * Ep + e];
            }
            psum[slot * Ep + e] = v;
            cnt[slot * Ep + e] = e < E ? sc[e] : 0;
        }
        if (threadIdx.x == 0) ntok[slot] = sn;
    }
}

// One cluster of C CTAs per sequence, each with `cols` (a multiple of 32) of
// the experts: the slots are added in blockDim / cols interleaved strands,
// then the strands, then the CTAs' shares of the loss, always in order.
// loss = E / (k n) sum_e c_e pmean_e.
__global__ void __launch_bounds__(kRedThreads) k_balance_reduce(int T, int E, int k, int L, int Ep, int cols, int C,
                                                                const int32_t *__restrict__ seq, int nseq,
                                                                const float *__restrict__ psum,
                                                                const int32_t *__restrict__ cnt,
                                                                const int32_t *__restrict__ ntok,
                                                                int32_t *__restrict__ counts,
                                                                int32_t *__restrict__ n_out,
                                                                float *__restrict__ pmean, float *__restrict__ loss,
                                                                DevErr *err)
{
    __shared__ float sp[kRedThreads];
    __shared__ int sq[kRedThreads];
    __shared__ float sw[kRedThreads / 32], sl[8];   // sl: the CTAs' shares (CTA 0)
    __shared__ int sn;
    const int s = blockIdx.x / C, r = blockIdx.x % C;
    // CTA 0's shared memory may be written once CTA 0 has started: every CTA
    // arrives here and waits just before its store
    if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    grid_wait();
    grid_go();
    const int a = seq_at(seq, s, nseq, T), b = seq_at(seq, s + 1, nseq, T);
    if (seq && threadIdx.x == 0 && r == 0 && (seq[s] < 0 || seq[s + 1] < seq[s] || seq[s + 1] > T))
        record_error(err, PMOE_ERR_BAD_INDEX, s, seq[s]);
    const int first = a / L, last = b > a ? (b - 1) / L : first - 1;
    if (threadIdx.x == 0) sn = 0;
    __syncthreads();
    int n = 0;
    for (int i = first + threadIdx.x; i <= last; i += blockDim.x) n += ntok[i + s];
    if (n) atomicAdd(&sn, n);
    const int strands = blockDim.x / cols, strand = threadIdx.x / cols, col = threadIdx.x % cols;
    const int e = r * cols + col;
    float v = 0.f;
    int c = 0;
    if (strand < strands && e < E) {
#pragma unroll 8
        for (int i = first + strand; i <= last; i += strands) {
            v += psum[(int64_t)(i + s) * Ep + e];
            c += cnt[(int64_t)(i + s) * Ep + e];
        }
    }
    sp[threadIdx.x] = v;
    sq[threadIdx.x] = c;
    __syncthreads();
    n = sn;
    const float inv = n > 0 ? 1.f / (float)n : 0.f;
    float part = 0.f;
    if (threadIdx.x < cols && e < E) {
        for (int g = 1; g < strands; ++g) {
            v += sp[g * cols + col];
            c += sq[g * cols + col];
        }
        counts[(int64_t)s * E + e] = c;
        pmean[(int64_t)s * E + e] = v * inv;
        part = (float)c * (v * inv);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if ((threadIdx.x & 31) == 0) sw[threadIdx.x >> 5] = part;
    __syncthreads();
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (threadIdx.x == 0) {
        float t = 0.f;
        for (int i = 0; i < (int)blockDim.x / 32; ++i) t += sw[i];
        if (C == 1) {
            sl[0] = t;
        } else {   // into CTA 0's sl[r]
            uint32_t ad = (uint32_t)__cvta_generic_to_shared(&sl[r]), remote;
            asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(ad));
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote), "f"(t) : "memory");
        }
    }
    __syncwarp();
    if (C > 1)
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (threadIdx.x == 0 && r == 0) {
        float t = 0.f;
        for (int i = 0; i < C; ++i) t += sl[i];
        loss[s] = t * ((float)E / (float)k) * inv;
        n_out[s] = n;
    }
}

// ------------------------------------------------------------------ backward
// dlogit_e = p_e (a_e - sum_e' p_e' a_e') with a_e = g E c_e / (k n^2) of the
// token's sequence, plus w_j (dw_j - sum_i w_i dw_i) at the selected experts.
template <int TPT, int V, int NI>
__global__ void __launch_bounds__(kThreads) k_route_backward(int T, int E, int k, const float *__restrict__ logits,
                                                             const int32_t *__restrict__ idx,
                                                             const float *__restrict__ w, const float *__restrict__ dw,
                                                             const uint8_t *__restrict__ valid,
                                                             const int32_t *__restrict__ seq, int nseq,
                                                             const int32_t *__restrict__ counts,
                                                             const int32_t *__restrict__ ntok,
                                                             const float *__restrict__ gl, float *__restrict__ dlogits,
                                                             DevErr *err)
{
    __shared__ float sh[kThreads / 32];
    extern __shared__ float rows[];   // a row of gradients per group
    const int tid = threadIdx.x % TPT, Ep = (E + 3) & ~3;
    const int t = blockIdx.x * (kThreads / TPT) + threadIdx.x / TPT;
    grid_wait();
    grid_go();
    if (t >= T) return;
    // all loads first: the row, the selection, the sequence's counts
    float d[NI];
    if (gl) row_load<TPT, V>(logits + (int64_t)t * E, E, tid, d);
    const int lane = threadIdx.x & 31;
    int e = -1;
    float wj = 0.f, gj = 0.f;
    if (dw && lane < k) {   // every warp forms the k terms, lane j slot j
        e = idx[(int64_t)t * k + lane];
        wj = w[(int64_t)t * k + lane];
        gj = dw[(int64_t)t * k + lane];
    }
    const bool counted = gl && (!valid || valid[t]);
    int n = 0;
    float c[NI], f = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) c[i] = 0.f;
    if (counted) {
        const int s = seq_of(seq, nseq, T, t);
        n = s >= 0 && s < nseq ? ntok[s] : 0;
        if (n > 0) {
            f = gl[s] * ((float)E / (float)k) / ((float)n * (float)n);
#pragma unroll
            for (int i = 0; i < NI; i += V) {
                const int col = col_of<TPT, V>(tid, i);
                if (col >= E) continue;
                if constexpr (V == 4) {
                    const int4 x = *(const int4 *)(counts + (int64_t)s * E + col);
                    c[i] = (float)x.x, c[i + 1] = (float)x.y, c[i + 2] = (float)x.z, c[i + 3] = (float)x.w;
                } else {
                    c[i] = (float)counts[(int64_t)s * E + col];
                }
            }
        }
    }
    if (n > 0) {
        row_softmax<TPT, NI>(d, sh);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) dot += d[i] * c[i];
        dot = group_reduce<TPT>(dot, Add(), sh);
#pragma unroll
        for (int i = 0; i < NI; ++i) d[i] *= f * (c[i] - dot);
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) d[i] = 0.f;
    }
    if (dw) {
        // the selected experts' terms are added in shared memory, by the lane of
        // each slot; where slots share an expert, the first one's lane adds all
        float *row = rows + threadIdx.x / TPT * Ep;
#pragma unroll
        for (int i = 0; i < NI; i += V) {
            const int col = col_of<TPT, V>(tid, i);
            if (col >= E) continue;
            if constexpr (V == 4) *(float4 *)(row + col) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
            else row[col] = d[i];
        }
        if constexpr (TPT > 32) __syncthreads();
        else __syncwarp();
        if (tid < 32) {
            if (lane < k && (e < 0 || e >= E)) {
                record_error(err, PMOE_ERR_BAD_INDEX, t, e);
                e = -1;
                wj = 0.f;
            }
            float dot = wj * gj;
#pragma unroll
            for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            float x = wj * (gj - dot);
            const unsigned same = __match_any_sync(0xffffffffu, e);
            if (__any_sync(0xffffffffu, e >= 0 && __popc(same) > 1)) {
                float sum = 0.f;
                for (int j = 0; j < k; ++j) {
                    const float y = __shfl_sync(0xffffffffu, x, j);
                    if (same >> j & 1u) sum += y;
                }
                x = sum;
            }
            if (e >= 0 && lane == __ffs(same) - 1) row[e] += x;
        }
        if constexpr (TPT > 32) __syncthreads();
        else __syncwarp();
#pragma unroll
        for (int i = 0; i < NI; i += V) {
            const int col = col_of<TPT, V>(tid, i);
            if (col >= E) continue;
            if constexpr (V == 4) *(float4 *)(dlogits + (int64_t)t * E + col) = *(const float4 *)(row + col);
            else dlogits[(int64_t)t * E + col] = row[col];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (col_of<TPT, V>(tid, i) < E) dlogits[(int64_t)t * E + col_of<TPT, V>(tid, i)] = d[i];
    }
}

// The variant by the number of experts: f(threads per token, values per load,
// values per thread).  Rows of a multiple of 4 floats are 16-byte aligned.
template <int N>
using Int = std::integral_constant<int, N>;
template <int V, class F>
static void by_width(int E, F f)
{
    if (E <= 32 * V) f(Int<32>(), Int<V>(), Int<V>());
    else if (E <= 128) f(Int<32>(), Int<V>(), Int<4>());
    else if (E <= 256) f(Int<32>(), Int<V>(), Int<8>());
    else if (E <= 384) f(Int<32>(), Int<V>(), Int<12>());
    else if (E <= 512) f(Int<32>(), Int<V>(), Int<16>());
    else if (E <= 1024) f(Int<32>(), Int<V>(), Int<32>());
    else f(Int<256>(), Int<V>(), Int<16>());   // E <= 4096
}
template <class F>
static void by_experts(int E, F f)
{
    if (E % 4 == 0) by_width<4>(E, f);
    else by_width<1>(E, f);
}

// T, E and k alone: a router needs no layer behind it
static bool sizes_ok(const pmoe_dims &d, int nseq)
{
    return d.T >= 0 && d.E > 0 && d.E <= 4096 && d.k > 0 && d.k <= 32 && d.k <= d.E &&
           (int64_t)d.T * d.k <= INT32_MAX / 2 && nseq >= 1 && nseq <= (1 << 20);
}

static bool aligned(std::initializer_list<const void *> ps)
{
    for (const void *p : ps)
        if ((uintptr_t)p & 15) return false;
    return true;
}

}  // namespace bal
}  // namespace pmoe

using namespace pmoe;

extern "C" {

size_t moe_balance_ws_bytes(pmoe_dims dims, int32_t nseq)
{
    if (!bal::sizes_ok(dims, nseq)) return 0;
    return bal::carve(nullptr, dims.T, dims.E, nseq).bytes;
}

pmoe_status moe_balance_forward(pmoe_dims dims, const float *logits, const int32_t *idx, const uint8_t *valid,
                                const int32_t *seq, int32_t nseq, int32_t *counts, int32_t *ntok, float *pmean,
                                float *loss, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    if (!bal::sizes_ok(dims, nseq) || (!seq && nseq != 1)) return PMOE_ERR_INVALID_ARG;
    if ((dims.T > 0 && (!logits || !idx)) || !counts || !ntok || !pmean || !loss) return PMOE_ERR_INVALID_ARG;
    if (!bal::aligned({logits, idx, valid, seq, counts, ntok, pmean, loss})) return PMOE_ERR_INVALID_ARG;
    const bal::Ws w = bal::carve(ws, dims.T, dims.E, nseq);
    if (!ws || ws_bytes < w.bytes || !bal::aligned({ws})) return PMOE_ERR_WORKSPACE;
    bool ok = true;
    if (dims.T > 0)
        bal::by_experts(dims.E, [&](auto tpt, auto v, auto ni) {
            constexpr auto kern = bal::k_balance_partial<tpt.value, v.value, ni.value>;
            const size_t sm = (size_t)(bal::fwd_threads(tpt.value) / tpt.value + 1) * w.Ep * 4;
            // (up to 17 rows of 1024 floats: 69 KB)
            ok = set_attribute<kern, cudaFuncAttributeMaxDynamicSharedMemorySize>(17 * 4096) &&
                 launch_chained<kern>((unsigned)cdiv(dims.T, w.L), bal::fwd_threads(tpt.value), sm, 1, stream, dims.T, dims.E,
                                dims.k, w.L, w.Ep, logits, idx, valid, seq, nseq, w.psum, w.cnt, w.ntok, w.err);
        });
    // CTAs per sequence: 32 experts each up to 8 CTAs, then more experts each
    const int cols = (int)(cdiv(dims.E, 256) * 32), C = (int)cdiv(dims.E, cols);
    // few slots a sequence: smaller CTAs start sooner (forward of 37 sequences of 16384 tokens, E = 256:
    // 12.6 us with 256 threads, 15.0 with 1024); one long sequence: more strands (8192 tokens, E = 384:
    // 8.9 us with 1024, 11.8 with 256)
    const unsigned threads = w.slots / nseq >= 64 ? bal::kRedThreads : std::max(256, cols);
    ok = ok && launch_chained<bal::k_balance_reduce>((unsigned)(nseq * C), threads, 0, C, stream, dims.T, dims.E,
                              dims.k, w.L, w.Ep, cols, C, seq, nseq, w.psum, w.cnt, w.ntok, counts, ntok, pmean, loss,
                              w.err);
    return ok ? PMOE_OK : PMOE_ERR_CUDA;
}

pmoe_status moe_route_backward(pmoe_dims dims, const float *logits, const int32_t *idx, const float *w,
                               const float *d_topk_w, const uint8_t *valid, const int32_t *seq, int32_t nseq,
                               const int32_t *counts, const int32_t *ntok, const float *g_loss, float *dlogits, void *ws,
                               size_t ws_bytes, cudaStream_t stream)
{
    if (!bal::sizes_ok(dims, nseq) || (!seq && nseq != 1)) return PMOE_ERR_INVALID_ARG;
    if (!d_topk_w && !g_loss) return PMOE_ERR_INVALID_ARG;
    if (dims.T > 0 && (!dlogits || (d_topk_w && (!idx || !w)) || (g_loss && (!logits || !counts || !ntok))))
        return PMOE_ERR_INVALID_ARG;
    if (!bal::aligned({logits, idx, w, d_topk_w, valid, seq, counts, ntok, g_loss, dlogits})) return PMOE_ERR_INVALID_ARG;
    const bal::Ws b = bal::carve(ws, dims.T, dims.E, nseq);
    if (!ws || ws_bytes < b.bytes || !bal::aligned({ws})) return PMOE_ERR_WORKSPACE;
    if (dims.T == 0) return PMOE_OK;
    bool ok = true;
    bal::by_experts(dims.E, [&](auto tpt, auto v, auto ni) {
        const unsigned groups = bal::kThreads / tpt.value;   // (rows of at most 32 KB in all)
        ok = launch_chained<bal::k_route_backward<tpt.value, v.value, ni.value>>((unsigned)cdiv(dims.T, groups),
                            bal::kThreads, (size_t)groups * b.Ep * 4, 1, stream, dims.T, dims.E, dims.k, logits, idx, w, d_topk_w, valid, seq,
                            nseq, counts, ntok, g_loss, dlogits, b.err);
    });
    return ok ? PMOE_OK : PMOE_ERR_CUDA;
}

}  // extern "C"
