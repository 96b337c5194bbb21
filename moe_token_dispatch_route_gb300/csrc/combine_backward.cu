// Gradient of the gate-weighted combine out[t] = sum_j w[t][j] Y[dest[t k + j]]:
//   dY[dest[t k + j]] = w[t][j] dout[t]      (bf16)
//   dw[t][j] = <dout[t], Y[dest[t k + j]]>   (fp32 sums)
//
// Bound by HBM: reads T rows of dout and S = T k rows of Y, writes S rows of dY.  A group of
// threads, a CTA or for narrow rows a warp, takes one token: each of its threads reads 8 columns of
// dout once and the same columns of up to KMAX of the token's rows of Y, all in flight at once.
// T = 8192, k = 8, N = 4096, Y bf16 and dout fp32: 181 us, 6.7 TB/s (0.98 of a plain copy's rate).
#include <algorithm>

#include "train.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256;

// Eight columns of Y as they are in memory.
template <bool BF16>
struct Row8;
template <>
struct Row8<true> {
    uint4 a;
    __device__ void load(const void* Y, size_t i) { a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(Y) + i)); }
    __device__ float dot(const float (&g)[8], float s) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fmaf(g[2 * j + 1], bf16_hi(w[j]), fmaf(g[2 * j], bf16_lo(w[j]), s));
        return s;
    }
};
template <>
struct Row8<false> {
    float4 a, b;
    __device__ void load(const void* Y, size_t i) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(Y) + i);
        a = __ldcs(p);
        b = __ldcs(p + 1);
    }
    __device__ float dot(const float (&g)[8], float s) const {
        s = fmaf(g[3], a.w, fmaf(g[2], a.z, fmaf(g[1], a.y, fmaf(g[0], a.x, s))));
        return fmaf(g[7], b.w, fmaf(g[6], b.z, fmaf(g[5], b.y, fmaf(g[4], b.x, s))));
    }
};

// GROUP threads (32 or 256) a token; KMAX slots at a time: the smallest of 2, 4 and 8 that holds k, whose
// registers are what limits the CTAs of an SM.
template <bool DB, bool YB, int GROUP, int KMAX>
__global__ void __launch_bounds__(kThreads, KMAX == 8 ? (YB ? 3 : 2) : 4) combine_backward_kernel(const CombineBackwardArgs a) {
    wait_for_kernel_before();
    __shared__ float red[2][KMAX][kThreads / 32];
    const int sub = threadIdx.x % GROUP, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kTokens = kThreads / GROUP;
    int turn = 0;
    for (long long t0 = (long long)blockIdx.x * kTokens; t0 < a.T; t0 += (long long)gridDim.x * kTokens) {
        const long long t = t0 + threadIdx.x / GROUP;
        if (t >= a.T) continue;  // GROUP 32: the whole warp
        for (int j0 = 0; j0 < a.k; j0 += KMAX, turn ^= 1) {
            int row[KMAX];
            float w[KMAX], acc[KMAX];
#pragma unroll
            for (int j = 0; j < KMAX; ++j) {
                const bool slot = j0 + j < a.k;
                const int r = slot ? __ldg(a.dest + t * a.k + j0 + j) : -1;
                row[j] = r >= 0 && r < a.S ? r : -1;
                w[j] = slot ? __ldg(a.w + t * a.k + j0 + j) : 0.f;
                acc[j] = 0.f;
            }
            for (int n = sub * 8; n < a.N; n += GROUP * 8) {
                float g[8];
                Row8<YB> y[KMAX];
                load8<DB>(a.dout, (size_t)t * a.N + n, g);
#pragma unroll
                for (int j = 0; j < KMAX; ++j)
                    if (row[j] >= 0) y[j].load(a.Y, (size_t)row[j] * a.N + n);
#pragma unroll
                for (int j = 0; j < KMAX; ++j) {
                    if (row[j] < 0) continue;
                    acc[j] = y[j].dot(g, acc[j]);
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = g[i] * w[j];
                    store8<true>(a.dY, (size_t)row[j] * a.N + n, o);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int j = 0; j < KMAX; ++j) acc[j] += __shfl_xor_sync(kFull, acc[j], o);
            if constexpr (GROUP == 32) {
#pragma unroll
                for (int j = 0; j < KMAX; ++j)
                    if (lane == j && j0 + j < a.k) a.dw[t * a.k + j0 + j] = acc[j];
            } else {
                if (lane == 0)
#pragma unroll
                    for (int j = 0; j < KMAX; ++j) red[turn][j][warp] = acc[j];
                __syncthreads();  // the two arrays of `red` alternate: one barrier is enough
                if (threadIdx.x < KMAX && j0 + threadIdx.x < a.k) {
                    float s = 0.f;
#pragma unroll
                    for (int i = 0; i < kThreads / 32; ++i) s += red[turn][threadIdx.x][i];
                    a.dw[t * a.k + j0 + threadIdx.x] = s;
                }
            }
        }
    }
}

template <bool DB, bool YB, int GROUP, int KMAX>
cudaError_t go(const CombineBackwardArgs& a, int sm_count, cudaStream_t stream) {
    constexpr int kTokens = kThreads / GROUP;
    // 32 CTAs an SM, of few tokens each, rather than as many as are resident: 8192 tokens, k = 8, N = 4096, fp32
    // 251 us, 268 with those
    const long long ctas = ((long long)a.T + kTokens - 1) / kTokens;
    return launch_after(combine_backward_kernel<DB, YB, GROUP, KMAX>, (unsigned)std::min<long long>(ctas, (long long)sm_count * 32), kThreads, 0,
                        stream, a);
}

template <bool DB, bool YB>
cudaError_t launch(const CombineBackwardArgs& a, int sm_count, cudaStream_t stream) {
    // A CTA has 8 columns a thread for rows of 2048.  Narrower ones leave threads idle: a warp a token is faster
    // once there are tokens for all the warps (us, CTA and warp; 16384 tokens, k = 4: N = 512 50 and 25,
    // 1024 66 and 57, 1408 82 and 78; 2048 with 8192 tokens 56 and 57), and slower by its passes over the row before
    // (333 tokens, k = 8, N = 1024: 6.7 and 9.2; N = 512, k = 4: 7.1 and 6.9).
    if (a.N <= 512 || (a.N < 2048 && a.T > 8 * sm_count)) {
        if (a.k <= 2) return go<DB, YB, 32, 2>(a, sm_count, stream);
        if (a.k <= 4) return go<DB, YB, 32, 4>(a, sm_count, stream);
        return go<DB, YB, 32, 8>(a, sm_count, stream);
    }
    if (a.k <= 2) return go<DB, YB, 256, 2>(a, sm_count, stream);
    if (a.k <= 4) return go<DB, YB, 256, 4>(a, sm_count, stream);
    return go<DB, YB, 256, 8>(a, sm_count, stream);
}

}  // namespace

cudaError_t launch_combine_backward(const CombineBackwardArgs& a, int sm_count, cudaStream_t stream) {
    if (a.dout_bf16) return a.y_bf16 ? launch<true, true>(a, sm_count, stream) : launch<true, false>(a, sm_count, stream);
    return a.y_bf16 ? launch<false, true>(a, sm_count, stream) : launch<false, false>(a, sm_count, stream);
}

}  // namespace moe
