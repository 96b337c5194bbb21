// The two gradients of the per-expert grouped product Y_i = A_i W_e(i):
//   input gradient   dA_i = dY_i W_e(i)^T            (i over expert e's rows)
//   weight gradient  dW_e = A_e^T dY_e               (summed over expert e's rows)
// bf16 operands, fp32 sums, output fp32 or bf16 (rounded once).
#include <algorithm>

#include "moe_internal.cuh"
#include "train.cuh"

namespace moe {
namespace {

constexpr int kTile = 64, kStep = 16, kChunk = 512, kCtaThreads = 256;

__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

__device__ __forceinline__ void put(const GroupedGradArgs& a, size_t i, float v) {
    if (a.out_bf16) static_cast<uint16_t*>(a.out)[i] = (uint16_t)bf16x2(v, 0.f);
    else if (a.accumulate) static_cast<float*>(a.out)[i] += v;
    else static_cast<float*>(a.out)[i] = v;
}

// Offsets have to ascend from 0 to S: they bound every access.
__device__ __forceinline__ bool offsets_ok(const GroupedGradArgs& a) {
    int bad = __ldg(a.offsets) != 0 || __ldg(a.offsets + a.E) != a.S;
    for (int e = threadIdx.x; e < a.E; e += kCtaThreads) bad |= __ldg(a.offsets + e + 1) < __ldg(a.offsets + e);
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) report_error(a.status, kStDevice, -2, __ldg(a.offsets + a.E), 0);
    return !bad;
}

// A 64 x 64 tile of P Q with P [m][k] and Q [k][n] read through the given strides; 4 x 4
// values a thread.  Sums of kChunk products are added up one by one: a single running sum
// over 16384 products was 1.5e-6 (norm) from the 64-bit result.
__device__ __forceinline__ void tile_product(const uint16_t* P, size_t pm, size_t pk, int m, const uint16_t* Q,
                                             size_t qk, size_t qn, int n, int K, float (&sum)[4][4]) {
    float acc[4][4] = {};
    __shared__ float sp[kStep][kTile + 1], sq[kStep][kTile + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int k0 = 0; k0 < K; k0 += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += kCtaThreads) {
            const int kp = pk == 1 ? i % kStep : i / kTile, r = pk == 1 ? i / kStep : i % kTile;
            sp[kp][r] = (r < m && k0 + kp < K) ? widen(__ldg(P + r * pm + (k0 + kp) * pk)) : 0.f;
            const int kq = qk == 1 ? i % kStep : i / kTile, c = qk == 1 ? i / kStep : i % kTile;
            sq[kq][c] = (c < n && k0 + kq < K) ? widen(__ldg(Q + (k0 + kq) * qk + c * qn)) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kStep; ++kk) {
            float p[4], q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = sp[kk][ty * 4 + i];
                q[i] = sq[kk][tx * 4 + i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(p[i], q[j], acc[i][j]);
        }
        __syncthreads();
        if ((k0 + kStep) % kChunk == 0 || k0 + kStep >= K) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum[i][j] += acc[i][j];
                    acc[i][j] = 0.f;
                }
        }
    }
}

// grid: (d / 64, row tiles strided over the CTAs of y, expert)
__global__ void __launch_bounds__(kCtaThreads) dgrad_kernel(const GroupedGradArgs a) {
    if (!offsets_ok(a)) return;
    const int e = blockIdx.z, seg0 = __ldg(a.offsets + e), cnt = __ldg(a.offsets + e + 1) - seg0;
    const int c0 = blockIdx.x * kTile, cols = min(kTile, a.d - c0);
    for (int r0 = blockIdx.y * kTile; r0 < cnt; r0 += gridDim.y * kTile) {
        const int rows = min(kTile, cnt - r0);
        float acc[4][4] = {};
        tile_product(a.dY + (size_t)(seg0 + r0) * a.N, a.N, 1, rows, a.W + ((size_t)e * a.d + c0) * a.N, 1, a.N, cols,
                     a.N, acc);
        const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j)
                if (ty * 4 + i < rows && tx * 4 + j < cols)
                    put(a, (size_t)(seg0 + r0 + ty * 4 + i) * a.d + c0 + tx * 4 + j, acc[i][j]);
    }
}

// grid: (N / 64, d / 64 strided over the CTAs of y, expert)
__global__ void __launch_bounds__(kCtaThreads) wgrad_kernel(const GroupedGradArgs a) {
    if (!offsets_ok(a)) return;
    const int e = blockIdx.z, seg0 = __ldg(a.offsets + e), cnt = __ldg(a.offsets + e + 1) - seg0;
    const int c0 = blockIdx.x * kTile, cols = min(kTile, a.N - c0);
    for (int r0 = blockIdx.y * kTile; r0 < a.d; r0 += gridDim.y * kTile) {
        const int rows = min(kTile, a.d - r0);
        float acc[4][4] = {};
        tile_product(a.A + (size_t)seg0 * a.d + r0, 1, a.d, rows, a.dY + (size_t)seg0 * a.N + c0, a.N, 1, cols, cnt, acc);
        const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j)
                if (ty * 4 + i < rows && tx * 4 + j < cols)
                    put(a, ((size_t)e * a.d + r0 + ty * 4 + i) * a.N + c0 + tx * 4 + j, acc[i][j]);
    }
}

}  // namespace

cudaError_t launch_grouped_dgrad(const GroupedGradArgs& a, int, cudaStream_t stream) {
    dgrad_kernel<<<dim3((a.d + kTile - 1) / kTile, std::min(64, (a.S + kTile - 1) / kTile), a.E), kCtaThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_grouped_wgrad(const GroupedGradArgs& a, int, cudaStream_t stream) {
    wgrad_kernel<<<dim3((a.N + kTile - 1) / kTile, std::min(64, (a.d + kTile - 1) / kTile), a.E), kCtaThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
