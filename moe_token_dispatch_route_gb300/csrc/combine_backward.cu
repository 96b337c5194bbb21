// Gradient of the gate-weighted combine out[t] = sum_j w[t][j] Y[dest[t k + j]]:
//   dY[dest[t k + j]] = w[t][j] dout[t]      (bf16)
//   dw[t][j] = <dout[t], Y[dest[t k + j]]>   (fp32 sums)
#include <algorithm>

#include "train.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256;

// one CTA per routed slot
template <bool DB, bool YB>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const CombineBackwardArgs a) {
    __shared__ float red[kThreads / 32];
    for (long long s = blockIdx.x; s < a.S; s += gridDim.x) {
        const int row = __ldg(a.dest + s);
        const float w = __ldg(a.w + s);
        const size_t t = (size_t)(s / a.k);
        float acc = 0.f;
        if (row >= 0 && row < a.S) {
            for (int n = threadIdx.x * 8; n < a.N; n += kThreads * 8) {
                float g[8], y[8];
                load8<DB>(a.dout, t * a.N + n, g);
                load8<YB>(a.Y, (size_t)row * a.N + n, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc = fmaf(g[j], y[j], acc);
                    g[j] *= w;
                }
                store8<true>(a.dY, (size_t)row * a.N + n, g);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kThreads / 32; ++i) acc += red[i];
            a.dw[s] = acc;
        }
    }
}

}  // namespace

cudaError_t launch_combine_backward(const CombineBackwardArgs& a, int sm_count, cudaStream_t stream) {
    const int grid = (int)std::min<long long>(a.S, (long long)sm_count * 8);
    if (a.dout_bf16) {
        if (a.y_bf16) combine_backward_kernel<true, true><<<grid, kThreads, 0, stream>>>(a);
        else combine_backward_kernel<true, false><<<grid, kThreads, 0, stream>>>(a);
    } else {
        if (a.y_bf16) combine_backward_kernel<false, true><<<grid, kThreads, 0, stream>>>(a);
        else combine_backward_kernel<false, false><<<grid, kThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace moe
