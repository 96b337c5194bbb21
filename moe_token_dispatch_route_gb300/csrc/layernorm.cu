// Layer norm of token rows and its gradient.
//   mean = sum x / d,  rstd = 1 / sqrt(sum (x - mean)^2 / d + eps),
//   y = (x - mean) rstd gamma + beta
// and, with xh = (x - mean) rstd and v = dy gamma,
//   dx = rstd (v - sum v / d - xh (sum v xh) / d) + dres,
//   dgamma = sum_t dy xh,  dbeta = sum_t dy.
// All sums are fp32.
#include <algorithm>

#include "train.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256;

// Sums of N values over the CTA, the same bits in every thread.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(kFull, v[i], o);
    __syncthreads();
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[i * 32 + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = 0.f;
        for (int w = 0; w < kThreads / 32; ++w) s += red[i * 32 + w];
        v[i] = s;
    }
}

template <bool XB>
__global__ void __launch_bounds__(kThreads) layernorm_kernel(const LayernormArgs a) {
    __shared__ float red[64];
    const float inv_d = 1.f / (float)a.d;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t row = (size_t)t * a.d;
        float s[1] = {0.f};
        for (int c = threadIdx.x * 8; c < a.d; c += kThreads * 8) {
            float v[8];
            load8<XB>(a.x, row + c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += v[j];
        }
        block_sum(s, red);
        const float mean = s[0] * inv_d;
        float q[1] = {0.f};
        for (int c = threadIdx.x * 8; c < a.d; c += kThreads * 8) {
            float v[8];
            load8<XB>(a.x, row + c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) q[0] = fmaf(v[j] - mean, v[j] - mean, q[0]);
        }
        block_sum(q, red);
        const float rstd = 1.f / sqrtf(q[0] * inv_d + a.eps);
        for (int c = threadIdx.x * 8; c < a.d; c += kThreads * 8) {
            float v[8];
            load8<XB>(a.x, row + c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float g = a.gamma ? __ldg(a.gamma + c + j) : 1.f;
                const float b = a.beta ? __ldg(a.beta + c + j) : 0.f;
                v[j] = fmaf((v[j] - mean) * rstd, g, b);
            }
            store8<true>(a.y, row + c, v);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[t] = mean;
            if (a.rstd) a.rstd[t] = rstd;
        }
    }
}

template <bool DYB, bool XB>
__global__ void __launch_bounds__(kThreads) layernorm_dx_kernel(const LayernormBackwardArgs a) {
    __shared__ float red[64];
    const float inv_d = 1.f / (float)a.d;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t row = (size_t)t * a.d;
        const float mean = __ldg(a.mean + t), rstd = __ldg(a.rstd + t);
        float s[2] = {0.f, 0.f};
        for (int c = threadIdx.x * 8; c < a.d; c += kThreads * 8) {
            float v[8], x[8];
            load8<DYB>(a.dy, row + c, v);
            load8<XB>(a.x, row + c, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float vg = v[j] * (a.gamma ? __ldg(a.gamma + c + j) : 1.f);
                s[0] += vg;
                s[1] = fmaf(vg, (x[j] - mean) * rstd, s[1]);
            }
        }
        block_sum(s, red);
        const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
        for (int c = threadIdx.x * 8; c < a.d; c += kThreads * 8) {
            float v[8], x[8], r[8] = {};
            load8<DYB>(a.dy, row + c, v);
            load8<XB>(a.x, row + c, x);
            if (a.dres) load8<XB>(a.dres, row + c, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float vg = v[j] * (a.gamma ? __ldg(a.gamma + c + j) : 1.f);
                const float xh = (x[j] - mean) * rstd;
                v[j] = fmaf(rstd, vg - m1 - xh * m2, r[j]);
            }
            store8<XB>(a.dx, row + c, v);
        }
    }
}

// one CTA per 32 columns: 8 warps take every 8th row, then a sum over the warps
template <bool DYB, bool XB>
__global__ void __launch_bounds__(kThreads) layernorm_dweight_kernel(const LayernormBackwardArgs a) {
    __shared__ float sg[kThreads / 32][32], sb[kThreads / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float g = 0.f, b = 0.f;
    if (c < a.d) {
        for (int t = warp; t < a.T; t += kThreads / 32) {
            const size_t i = (size_t)t * a.d + c;
            const float dy = DYB ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.dy)[i] << 16)
                                 : static_cast<const float*>(a.dy)[i];
            const float x = XB ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.x)[i] << 16)
                               : static_cast<const float*>(a.x)[i];
            g = fmaf(dy, (x - __ldg(a.mean + t)) * __ldg(a.rstd + t), g);
            b += dy;
        }
    }
    sg[warp][lane] = g;
    sb[warp][lane] = b;
    __syncthreads();
    if (warp == 0 && c < a.d) {
        for (int w = 1; w < kThreads / 32; ++w) {
            g += sg[w][lane];
            b += sb[w][lane];
        }
        if (a.dgamma) a.dgamma[c] = g;
        if (a.dbeta) a.dbeta[c] = b;
    }
}

template <bool DYB, bool XB>
cudaError_t backward(const LayernormBackwardArgs& a, int sm_count, cudaStream_t stream) {
    layernorm_dx_kernel<DYB, XB><<<std::min(a.T, sm_count * 8), kThreads, 0, stream>>>(a);
    if (a.dgamma || a.dbeta)
        layernorm_dweight_kernel<DYB, XB><<<(a.d + 31) / 32, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layernorm(const LayernormArgs& a, int sm_count, cudaStream_t stream) {
    const int grid = std::min(a.T, sm_count * 8);
    if (a.x_bf16) layernorm_kernel<true><<<grid, kThreads, 0, stream>>>(a);
    else layernorm_kernel<false><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

size_t layernorm_backward_scratch_bytes(int, int, int) { return 256; }

cudaError_t launch_layernorm_backward(const LayernormBackwardArgs& a, int sm_count, cudaStream_t stream) {
    if (a.dy_bf16) return a.x_bf16 ? backward<true, true>(a, sm_count, stream) : backward<true, false>(a, sm_count, stream);
    return a.x_bf16 ? backward<false, true>(a, sm_count, stream) : backward<false, false>(a, sm_count, stream);
}

}  // namespace moe
