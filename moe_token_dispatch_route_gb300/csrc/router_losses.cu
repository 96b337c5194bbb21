// The router's losses and the gradient of its logits.
// Tokens are cut into groups (sequences) of seq_len; masked tokens count nowhere.  With p the token's scores in sum 1
// (softmax, or logistic scores over their sum), n the group's counted tokens and load[e] its picks of expert e:
//   balance loss  b / G  sum_g E / (k n^2) sum_e load[e] sum_t p[t][e]
//   z loss        z / N  sum_t lse_t^2,   lse = log sum_e exp(logit),  N all counted tokens
// and, with w_e = b E load[e] / (G k n^2), the gradient of a counted token's logits
//   softmax:  p_e (w_e - sum_j p_j w_j),   logistic: the same times 1 - s_e,   + 2 z lse / N softmax_e
// plus the gates': topk_w as the routing computes it from the picks' logits, times dtopk_w.
// With logistic scores p and the gradient are taken of logits relative to the token's largest one where that is far below 0, and
// the w_e less their mean: neither changes the formulas.
// Bound by instruction issue when large (the exponentials and sums: 60 to 67% of the slots, DRAM a quarter) and by launch
// latency when small.  32768 tokens of 256 experts: 38 us in all; the logits twice and dlogits once
// would be 15 at a plain copy's rate.  65536 tokens of 8 and of 64 experts: 21 to 22 and 46 to 51 us, 0.9 and 7.4 at that rate: a
// token's shuffles, picks and loop are paid for one or two experts a lane.
//
// A token is held by 8 to 32 lanes, VPL experts each; its sums are shuffles.  A CTA stays within one group, so
// the forward pass keeps its experts' score sums in registers over all its tokens and the backward pass its w_e.  The
// CTAs' sums are joined in a fixed order by a second kernel, whose last CTA adds the groups'.
#include <algorithm>
#include <type_traits>

#include "moe_internal.cuh"
#include "serve.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kRouterThreads = 256, kRouterWarps = kRouterThreads / 32;

// How a call's tokens are shared out: `chunks` CTAs a group, `chunk` tokens each.
struct Split {
    int chunk, chunks;
    long long blocks;
};
Split split_of(int T, int E, int seq_len, int groups, int sm_count) {
    const int per_pass = kRouterWarps * (E <= 8 ? 4 : E <= 16 ? 2 : 1);  // tokens that a CTA takes at a time
    const long long want = std::max<long long>(2 * per_pass, ((long long)T + 4 * sm_count - 1) / (4 * sm_count));
    Split s;
    s.chunks = (int)std::max<long long>(1, (seq_len + want - 1) / want);
    s.chunk = (seq_len + s.chunks - 1) / s.chunks;
    s.blocks = (long long)groups * s.chunks;
    return s;
}

// Experts of a joining CTA, and how many CTAs a group's experts are shared out to (one where a group has one CTA's sums).
constexpr int kJoinExperts = 32;
__host__ __device__ inline int expert_parts(int E, const Split& s) { return s.chunks > 1 ? (E + kJoinExperts - 1) / kJoinExperts : 1; }

// Scratch: a count of the CTAs that have joined; sum_e load[e] sum_t p[t][e] of each group and part of its experts; the groups' z
// sums; then (chunks > 1) each CTA's score sums, load, z sum and tokens.
struct Partials {
    unsigned* joined;  // the first kernel sets it to 0
    float* dot;        // [groups][expert_parts]
    float* z;          // [groups]
    float* part;       // [blocks][2 E + 2]
    __host__ __device__ Partials(const RouterLossArgs& a, const Split& s)
        : joined(static_cast<unsigned*>(a.scratch)), dot(static_cast<float*>(a.scratch) + 4),
          z(dot + (size_t)a.groups * expert_parts(a.E, s)), part(z + a.groups) {}
};

template <int GL>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = GL / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
template <int GL>
__device__ __forceinline__ float lanes_max(float v) {
    if constexpr (GL == 32) {
        asm("redux.sync.max.f32 %0, %0, 0xFFFFFFFF;" : "+f"(v));
    } else {
#pragma unroll
        for (int o = GL / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    }
    return v;
}

// Whether `v` holds in all GL lanes of this one's token.
template <int GL>
__device__ __forceinline__ bool all_lanes(bool v) {
    if constexpr (GL == 32) return __all_sync(kFull, v);
    const unsigned lanes = ((1u << (GL & 31)) - 1u) << (threadIdx.x & 31 & ~(GL - 1));
    return (__ballot_sync(kFull, v) & lanes) == lanes;
}

// e^x for x <= 0, within 2 + 1.2 |x| units in the last place: the far terms that are off by more are the small ones.
__device__ __forceinline__ float exp_of(float x) {
    float p;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(__fmul_rn(x, 1.4426950408889634f)));
    return p;
}

// s = 1 / (1 + e^-l) and 1 - s from e^-|l|, which does not overflow: neither is the other's difference from 1, which
// would lose a far logit's small one.
struct Logistic {
    float s, rest;
    __device__ Logistic() {}
    __device__ explicit Logistic(float l) {
        const float e = exp_of(-fabsf(l)), big = __fdividef(1.f, 1.f + e), small = e * big;
        s = l >= 0.f ? big : small;
        rest = l >= 0.f ? small : big;
    }
};

// How a token's experts lie in its lanes: GL lanes, VPL experts each, VEC of them side by side.  With VEC 4 all exist
// (E = 32 VPL) and are loaded and stored four at a time.  Forward and backward in us, logistic scores, with four and with one
// side by side: 65536 tokens of 128 experts 24.4 + 30.2 and 25.1 + 31.3, 32768 of 256 20.4 + 19.4 and 21.1 + 30.6, 16384 of 512
// 18.9 + 23.1 and 21.4 + 24.3.  Other numbers of experts have not been tried with four.
template <int GL, int VPL, int VEC>
struct Lanes {
    static constexpr int kCols = GL * VPL;
    static __device__ __forceinline__ int expert(int sub, int i) { return i / VEC * GL * VEC + sub * VEC + i % VEC; }
    static __device__ __forceinline__ void load(const float* row, int sub, int E, bool there, float (&l)[VPL]) {
#pragma unroll
        for (int i = 0; i < VPL; i += VEC) {
            const int e = expert(sub, i);
            if constexpr (VEC == 4) {
                const float4 v = there ? __ldg(reinterpret_cast<const float4*>(row + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
                l[i] = v.x;
                l[i + 1] = v.y;
                l[i + 2] = v.z;
                l[i + 3] = v.w;
            } else {
                l[i] = e < E ? (there ? __ldg(row + e) : 0.f) : __uint_as_float(0xFF800000u);
            }
        }
    }
    static __device__ __forceinline__ void store(float* row, int sub, int E, const float (&d)[VPL]) {
#pragma unroll
        for (int i = 0; i < VPL; i += VEC) {
            const int e = expert(sub, i);
            if constexpr (VEC == 4) __stcs(reinterpret_cast<float4*>(row + e), make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]));
            else if (e < E) __stcs(row + e, d[i]);
        }
    }
};

// What is read of a token; in the forward pass while the one before it is worked on.  A masked token may hold anything, and 0
// times a NaN is one: its logits are read only where `masked_too` (gates that are entries of the softmax over them all).
template <int GL, int VPL, int VEC>
struct Token {
    float l[VPL], dw;
    int pick;  // lane j's: pick j, or -1
    bool there, counted;
    __device__ __forceinline__ void fetch(const RouterLossArgs& a, long long t, long long t1, int sub, bool gates, bool masked_too) {
        there = t < t1;
        counted = there && (!a.mask || __ldg(a.mask + t));
        pick = -1;
        dw = 0.f;
        if (there && sub < a.k && a.topk_idx) {
            pick = __ldg(a.topk_idx + (size_t)t * a.k + sub);
            if (gates) dw = __ldg(a.dtopk_w + (size_t)t * a.k + sub);
        }
        const bool read = counted || (there && masked_too);
        Lanes<GL, VPL, VEC>::load(a.logits + (read ? (size_t)t * a.E : 0), sub, a.E, read, l);
    }
};

// A token's softmax numerators x (e^(logit - top)) with their sum and lse where they are wanted, and its logistic scores, up to a
// common factor where all of them are far below 1.
template <int GL, int VPL, bool SIG>
struct Scores {
    float x[VPL], top, xsum, lse;
    Logistic g[SIG ? VPL : 1];
    float total;  // of the scores
    // Called by whole warps; l is used up.
    __device__ __forceinline__ void compute(float (&l)[VPL], bool want_lse) {
        top = xsum = lse = 0.f;
        float high = l[0];  // of this lane's
#pragma unroll
        for (int i = 1; i < VPL; ++i) high = fmaxf(high, l[i]);
        if (!SIG || want_lse) {
            top = lanes_max<GL>(high);
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                x[i] = exp_of(l[i] - top);
                xsum += x[i];
            }
            xsum = lanes_sum<GL>(xsum);
            if (want_lse) lse = top + logf(xsum);
        }
        if constexpr (SIG) {
            // Below kFar 1 + e^l is 1 and a score e^l: what its token's shares are made of does not change by a common factor, and
            // with the largest logit at kFar no share that matters is flushed to 0 (from -87 on all of them would be).
            constexpr float kFar = -18.f;
            if (__any_sync(kFull, all_lanes<GL>(high < kFar))) {
                const float highest = lanes_max<GL>(high);
                if (highest < kFar) {
#pragma unroll
                    for (int i = 0; i < VPL; ++i) l[i] = (l[i] - highest) + kFar;
                }
            }
            total = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                g[i] = Logistic(l[i]);
                total += g[i].s;
            }
            total = lanes_sum<GL>(total);
        } else {
            total = xsum;
        }
    }
    __device__ __forceinline__ float score(int i) const { return SIG ? g[SIG ? i : 0].s : x[i]; }
};

// A group's E / (k n^2) sum_e load[e] sum_t p[t][e].
__device__ __forceinline__ float group_balance(const RouterLossArgs& a, float dot, int n) {
    return n > 0 ? dot * ((float)a.E / ((float)a.k * (float)n * (float)n)) : 0.f;
}

// Sum over a CTA, in every thread.
template <int WARPS>
__device__ __forceinline__ float cta_sum(float v, float (&red)[WARPS]) {
    v = lanes_sum<32>(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < WARPS ? red[threadIdx.x & 31] : 0.f;
    return lanes_sum<32>(v);
}

// (512 experts: four CTAs an SM, 16384 tokens of logistic scores in 19.2 us; with the 73 registers that it would take otherwise 20.4)
template <int GL, int VPL, int VEC, bool SIG>
__global__ void __launch_bounds__(kRouterThreads, VEC == 4 && VPL == 16 ? 4 : 0) balance_kernel(const RouterLossArgs a, Split sp) {
    using L = Lanes<GL, VPL, VEC>;
    constexpr int kCols = L::kCols;
    __shared__ float sums[kRouterWarps][kCols];
    __shared__ int hist[kCols];
    __shared__ float red[kRouterWarps];
    wait_for_kernel_before();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane % GL;
    const long long g = blockIdx.x / sp.chunks;
    const int chunk = blockIdx.x % sp.chunks;
    const long long t0 = g * a.seq_len + (long long)chunk * sp.chunk;
    const long long t1 = min(min(t0 + sp.chunk, (g + 1) * (long long)a.seq_len), (long long)a.T);
    const Partials pt(a, sp);
    if (blockIdx.x == 0 && tid == 0) *pt.joined = 0u;
    for (int e = tid; e < kCols; e += kRouterThreads) hist[e] = 0;
    __syncthreads();
    float acc[VPL], z = 0.f;
    int n = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = 0.f;
    constexpr int kPass = kRouterWarps * (32 / GL);
    const bool want = a.z != 0.f;
    Token<GL, VPL, VEC> next;
    next.fetch(a, t0 + warp * (32 / GL) + lane / GL, t1, sub, false, false);
    for (long long tw = t0 + warp * (32 / GL); tw < t1; tw += kPass) {
        Token<GL, VPL, VEC> now = next;
        if (tw + kPass < t1) next.fetch(a, tw + kPass + lane / GL, t1, sub, false, false);
        const bool live = now.counted;
        if (!__any_sync(kFull, live)) continue;
        if (live && (unsigned)now.pick < (unsigned)a.E) atomicAdd(&hist[now.pick], 1);
        Scores<GL, VPL, SIG> sc;
        sc.compute(now.l, want);
        if (live) {
            const float inv = __fdividef(1.f, sc.total);
#pragma unroll
            for (int i = 0; i < VPL; ++i) acc[i] = fmaf(sc.score(i), inv, acc[i]);
            if (sub == 0) {
                z = fmaf(sc.lse, sc.lse, z);
                ++n;
            }
        }
    }
    // the lane groups' sums, then the warps'
#pragma unroll
    for (int o = 16; o >= GL; o >>= 1)
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] += __shfl_xor_sync(kFull, acc[i], o);
    if (lane < GL)
#pragma unroll
        for (int i = 0; i < VPL; ++i) sums[warp][L::expert(sub, i)] = acc[i];
    z = cta_sum(z, red);
    const int tokens = (int)cta_sum((float)n, red);  // (below 2^24: a chunk)
    float dot = 0.f;
    float* part = pt.part + (size_t)blockIdx.x * (2 * a.E + 2);
    for (int e = tid; e < a.E; e += kRouterThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kRouterWarps; ++w) v += sums[w][e];
        if (sp.chunks > 1) {
            part[e] = v;
            part[a.E + e] = __int_as_float(hist[e]);
        } else {
            a.load[g * a.E + e] = hist[e];
            dot = fmaf(v, (float)hist[e], dot);
        }
    }
    if (sp.chunks > 1) {
        if (tid == 0) {
            part[2 * a.E] = z;
            part[2 * a.E + 1] = __int_as_float(tokens);
        }
        return;
    }
    dot = cta_sum(dot, red);
    if (tid == 0) {
        pt.dot[g] = dot;
        pt.z[g] = z;
        a.tokens[g] = tokens;
        if (a.groups == 1) {
            a.tokens[1] = tokens;
            a.loss[0] = a.balance != 0.f ? a.balance * group_balance(a, dot, tokens) : 0.f;  // (0 times what may be no number)
            a.loss[1] = tokens > 0 ? a.z * (z / (float)tokens) : 0.f;
        }
    }
}

// The groups' losses, added in their order by one CTA.
template <int WARPS>
__device__ __forceinline__ void total_of_groups(const RouterLossArgs& a, const Split& sp, float (&red)[WARPS], int* count) {
    const Partials pt(a, sp);
    const int parts = expert_parts(a.E, sp);
    float bal = 0.f, z = 0.f;
    int n = 0;
#pragma unroll 4
    for (int g = threadIdx.x; g < a.groups; g += 32 * WARPS) {
        float dot = 0.f;
        for (int i = 0; i < parts; ++i) dot += __ldcg(pt.dot + (size_t)g * parts + i);
        const int tokens = __ldcg(a.tokens + g);
        bal += group_balance(a, dot, tokens);
        z += __ldcg(pt.z + g);
        n += tokens;
    }
    if (threadIdx.x == 0) *count = 0;
    bal = cta_sum(bal, red);
    z = cta_sum(z, red);
    if (n) atomicAdd(count, n);
    __syncthreads();
    if (threadIdx.x == 0) {
        a.tokens[a.groups] = *count;
        a.loss[0] = a.balance != 0.f ? a.balance * (bal / (float)a.groups) : 0.f;
        a.loss[1] = *count > 0 ? a.z * (z / (float)*count) : 0.f;
    }
}

// Adds the CTAs' sums of a group: a CTA takes 32 experts, a warp every 32nd CTA's, joined in their order.  (One CTA a group
// took 190 us for 16384 tokens of 1000 experts in one group.)  The last one to end adds the groups'.
constexpr int kJoinThreads = 1024;
__global__ void __launch_bounds__(kJoinThreads) balance_groups_kernel(const RouterLossArgs a, Split sp) {
    __shared__ float sums[32][kJoinExperts + 1];
    __shared__ int loads[32][kJoinExperts + 1];
    __shared__ float red[kJoinThreads / 32];
    __shared__ int count;
    __shared__ bool last;
    wait_for_kernel_before();
    const int parts = expert_parts(a.E, sp), g = (int)(blockIdx.x / parts), piece = (int)(blockIdx.x % parts);
    const size_t pitch = 2 * a.E + 2;
    const Partials pt(a, sp);
    const float* part = pt.part + (size_t)g * sp.chunks * pitch;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = piece * kJoinExperts + lane;
    float v = 0.f;
    int load = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int c = warp; c < sp.chunks; c += 32) {
            v += __ldcg(part + c * pitch + e);
            load += __float_as_int(__ldcg(part + c * pitch + a.E + e));
        }
    }
    float z = 0.f;
    int n = 0;
    if (piece == 0)
        for (int c = threadIdx.x; c < sp.chunks; c += kJoinThreads) {
            z += __ldcg(part + c * pitch + 2 * a.E);
            n += __float_as_int(__ldcg(part + c * pitch + 2 * a.E + 1));
        }
    sums[warp][lane] = v;
    loads[warp][lane] = load;
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    if (warp == 0) {
        v = 0.f;
        load = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            v += sums[i][lane];
            load += loads[i][lane];
        }
        if (e < a.E) a.load[(size_t)g * a.E + e] = load;
        const float dot = lanes_sum<32>(e < a.E ? v * (float)load : 0.f);
        if (lane == 0) pt.dot[(size_t)g * parts + piece] = dot;
    }
    if (piece == 0) {
        z = cta_sum(z, red);
        if (n) atomicAdd(&count, n);
        __syncthreads();
        if (threadIdx.x == 0) {
            pt.z[g] = z;
            a.tokens[g] = count;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(pt.joined, 1u) == gridDim.x - 1u;
        __threadfence();
    }
    __syncthreads();
    if (last) total_of_groups(a, sp, red, &count);
}

// Groups that a CTA of the first kernel each has done: their total.
__global__ void __launch_bounds__(kJoinThreads) balance_total_kernel(const RouterLossArgs a, Split sp) {
    __shared__ float red[kJoinThreads / 32];
    __shared__ int count;
    wait_for_kernel_before();
    total_of_groups(a, sp, red, &count);
}

template <int GL, int VPL, int VEC, bool SIG>
__global__ void __launch_bounds__(kRouterThreads) router_backward_kernel(const RouterLossArgs a, Split sp) {
    using L = Lanes<GL, VPL, VEC>;
    constexpr int kCols = L::kCols, kPer = 32 / GL;  // tokens of a warp
    __shared__ __align__(16) float delta[kRouterWarps * kPer][kCols];    // the gates' gradient of a token's picks
    wait_for_kernel_before();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane % GL;
    const long long g = blockIdx.x / sp.chunks;
    const int chunk = blockIdx.x % sp.chunks;
    const long long t0 = g * a.seq_len + (long long)chunk * sp.chunk;
    const long long t1 = min(min(t0 + sp.chunk, (g + 1) * (long long)a.seq_len), (long long)a.T);
    float* mine = delta[warp * kPer + lane / GL];
    float w[VPL];
    {
        const int n = a.balance != 0.f ? __ldg(a.tokens + g) : 0;
        const float coef = n > 0 ? a.balance * ((float)a.E / ((float)a.groups * (float)a.k * (float)n * (float)n)) : 0.f;
        float picks = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = L::expert(sub, i);
            w[i] = coef != 0.f && e < a.E ? (float)__ldg(a.load + g * a.E + e) : 0.f;
            picks += w[i];
            mine[e] = 0.f;
        }
        // Less their mean: p_e (w_e - sum_j p_j w_j) is the same for it, and an even load's common part does not cancel in fp32.
        const float mean = lanes_sum<GL>(picks) / (float)a.E;
#pragma unroll
        for (int i = 0; i < VPL; ++i) w[i] = L::expert(sub, i) < a.E ? coef * (w[i] - mean) : 0.f;
    }
    const int all = a.z != 0.f ? __ldg(a.tokens + a.groups) : 0;
    const float zc = all > 0 ? 2.f * a.z / (float)all : 0.f;
    const bool losses = a.balance != 0.f || a.z != 0.f;
    const bool full = losses || (!SIG && !a.renorm);  // the gradient is not of the picks alone
    __syncwarp();
    for (long long tw = t0 + warp * kPer; tw < t1; tw += kRouterWarps * kPer) {
        Token<GL, VPL, VEC> now;
        now.fetch(a, tw + lane / GL, t1, sub, a.dtopk_w != nullptr, a.dtopk_w && !SIG && !a.renorm);
        const long long t = tw + lane / GL;
        const bool there = now.there, counted = now.counted;
        float d[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) d[i] = 0.f;
        // the picks: lane j holds pick j
        const int pick = a.dtopk_w && (unsigned)now.pick < (unsigned)a.E ? now.pick : -1;
        const float pl = pick >= 0 ? __ldg(a.logits + (size_t)t * a.E + pick) : __uint_as_float(0xFF800000u), dw = pick >= 0 ? now.dw : 0.f;
        float gate_dot = 0.f, pick_p = 0.f;
        if (full) {
            Scores<GL, VPL, SIG> sc;
            sc.compute(now.l, zc != 0.f);
            const float inv = __fdividef(1.f, sc.total);
            if (!SIG && !a.renorm) {  // gates that are entries of the softmax over all experts
                pick_p = pick >= 0 ? exp_of(pl - sc.top) * inv : 0.f;
                gate_dot = lanes_sum<GL>(pick_p * dw);
            }
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) dot = fmaf(sc.score(i) * inv, w[i], dot);
            dot = lanes_sum<GL>(dot);
            const float zt = counted ? zc * sc.lse * (SIG && zc != 0.f ? __fdividef(1.f, sc.xsum) : inv) : 0.f;
            const float pinv = counted ? inv : 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const float v = sc.score(i) * pinv * (w[i] - dot);
                if constexpr (SIG) d[i] = v * sc.g[i].rest;
                else d[i] = fmaf(-gate_dot * inv, sc.x[i], v);
            }
            if (zc != 0.f)
#pragma unroll
                for (int i = 0; i < VPL; ++i) d[i] = fmaf(zt, sc.x[i], d[i]);
        }
        if (a.dtopk_w) {
            float v;
            if (!SIG && !a.renorm) {
                v = pick_p * dw;
            } else if (!a.renorm) {
                const Logistic g(pl);
                v = dw * g.s * g.rest;
            } else {
                float s = 0.f;
                if (SIG) {
                    s = pick >= 0 ? Logistic(pl).s : 0.f;
                } else {
                    const float top = lanes_max<GL>(pl);
                    s = pick >= 0 ? exp_of(pl - top) : 0.f;
                }
                const float gate = s * __fdividef(1.f, lanes_sum<GL>(s));
                v = gate * (dw - lanes_sum<GL>(gate * dw));
                if (SIG) v *= Logistic(pl).rest;
            }
            if (pick >= 0) atomicAdd(mine + pick, v);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < VPL; i += VEC) {
                if constexpr (VEC == 4) {
                    const float4 v4 = *reinterpret_cast<const float4*>(mine + L::expert(sub, i));
                    d[i] += v4.x;
                    d[i + 1] += v4.y;
                    d[i + 2] += v4.z;
                    d[i + 3] += v4.w;
                } else {
                    d[i] += mine[L::expert(sub, i)];
                }
            }
            __syncwarp();
            if (pick >= 0) mine[pick] = 0.f;
            __syncwarp();
        }
        if (there) L::store(a.dlogits + (size_t)t * a.E, sub, a.E, d);
    }
}

// go(lanes a token, experts a lane, experts side by side, logistic scores)
template <class Go>
cudaError_t by_experts(const RouterLossArgs& a, bool vec, Go go) {
    using std::integral_constant;
    auto lanes = [&](auto gl, auto vpl, auto v) {
        return a.sigmoid ? go(gl, vpl, v, std::true_type()) : go(gl, vpl, v, std::false_type());
    };
    constexpr integral_constant<int, 1> one;
    constexpr integral_constant<int, 4> four;
    constexpr integral_constant<int, 32> warp;
    const int E = a.E;
    if (E <= 8) return lanes(integral_constant<int, 8>(), one, one);
    if (E <= 16) return lanes(integral_constant<int, 16>(), one, one);
    if (E <= 32) return lanes(warp, one, one);
    if (E <= 64) return lanes(warp, integral_constant<int, 2>(), one);
    if (vec && E == 128) return lanes(warp, four, four);
    if (vec && E == 256) return lanes(warp, integral_constant<int, 8>(), four);
    if (vec && E == 512) return lanes(warp, integral_constant<int, 16>(), four);
    if (E <= 128) return lanes(warp, four, one);
    if (E <= 256) return lanes(warp, integral_constant<int, 8>(), one);
    if (E <= 512) return lanes(warp, integral_constant<int, 16>(), one);
    return lanes(warp, integral_constant<int, 32>(), one);
}

}  // namespace

size_t balance_scratch_bytes(int T, int E, int seq_len, int sm_count) {
    const int groups = (int)(((long long)T + seq_len - 1) / seq_len);
    const Split s = split_of(T, E, seq_len, groups, sm_count);
    return sizeof(float) * (4 + (size_t)groups * (expert_parts(E, s) + 1) + (s.chunks > 1 ? (size_t)s.blocks * (2 * (size_t)E + 2) : 0));
}

cudaError_t launch_balance_loss(const RouterLossArgs& a, int sm_count, cudaStream_t stream) {
    const Split sp = split_of(a.T, a.E, a.seq_len, a.groups, sm_count);
    if (sp.blocks >= (1LL << 31)) return cudaErrorInvalidValue;
    const bool vec = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
    cudaError_t e = by_experts(a, vec, [&](auto gl, auto vpl, auto v, auto sig) {
        return launch_after(balance_kernel<decltype(gl)::value, decltype(vpl)::value, decltype(v)::value, decltype(sig)::value>,
                            (unsigned)sp.blocks, kRouterThreads, 0, stream, a, sp);
    });
    if (e == cudaSuccess && sp.chunks > 1)
        e = launch_after(balance_groups_kernel, (unsigned)(a.groups * expert_parts(a.E, sp)), kJoinThreads, 0, stream, a, sp);
    if (e == cudaSuccess && sp.chunks == 1 && a.groups > 1) e = launch_after(balance_total_kernel, 1u, kJoinThreads, 0, stream, a, sp);
    return e;
}

cudaError_t launch_router_backward(const RouterLossArgs& a, int sm_count, cudaStream_t stream) {
    const Split sp = split_of(a.T, a.E, a.seq_len, a.groups, sm_count);
    if (sp.blocks >= (1LL << 31)) return cudaErrorInvalidValue;
    const bool vec = (reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits)) % 16 == 0;
    return by_experts(a, vec, [&](auto gl, auto vpl, auto v, auto sig) {
        return launch_after(router_backward_kernel<decltype(gl)::value, decltype(vpl)::value, decltype(v)::value, decltype(sig)::value>,
                            (unsigned)sp.blocks, kRouterThreads, 0, stream, a, sp);
    });
}

}  // namespace moe
