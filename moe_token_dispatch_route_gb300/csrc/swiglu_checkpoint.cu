// The SwiGLU activation with its pre-activations kept in 8 bits, and the backward pass that
// uses them.
//
// GU row = [gate g (F columns) | up u (F columns)].  Each half of a row is cut into blocks of
// 128 columns; with amax the block's largest magnitude,
//   scale = fp32(amax / 127),  inv = fp32(127 / amax),  code = nearest even of fp32(x inv),
// so code is in [-127, 127] and the stored value is code * scale.  A block whose amax is
// zero, or so small that inv is not finite (amax < 2^-121), has scale 0 and codes 0.  A block that holds an
// infinity or a NaN has scale NaN: all of it is restored as NaN, so an overflow of the
// forward pass shows in the gradients.
//   forward:  H = silu(g) u from the values themselves;
//   backward: with g, u the stored values and s = 1 / (1 + e^-g),
//             dU = dH g s,  dG = dH u s (1 + g (1 - s)),  H = g s u again.
#include <algorithm>

#include "train.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256;
constexpr int kLanes = kCkptBlock / 8;   // 16 lanes of 8 columns share a block
constexpr float kMinAmax = 3.7615819e-37f;  // 2^-121: the smallest amax that is stored

// 1 / (1 + e^-g) from e^-|g|, which does not overflow: far negative g keeps its small result
__device__ __forceinline__ float sigmoid(float g) {
    const float e = expf(-fabsf(g));
    return (g >= 0.f ? 1.f : e) / (1.f + e);
}

// Scale of the block of 16 lanes and this lane's 8 codes (two words); every lane of the
// warp takes part.
__device__ __forceinline__ uint2 quantize8(const float (&v)[8], float& scale) {
    uint32_t m = 0;  // magnitudes compare as integers: NaN > infinity > finite
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
    const float amax = __uint_as_float(m);
    if (m >= 0x7F800000u) {
        scale = __uint_as_float(0x7FC00000u);
        return make_uint2(0u, 0u);
    }
    if (amax < kMinAmax) {
        scale = 0.f;
        return make_uint2(0u, 0u);
    }
    scale = __fdiv_rn(amax, 127.f);
    const float inv = __fdiv_rn(127.f, amax);
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = (uint32_t)__float2int_rn(__fmul_rn(v[j], inv)) & 0xFFu;
    return make_uint2(q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24, q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24);
}

__device__ __forceinline__ void restore8(uint2 q, float scale, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = (float)(int8_t)(q.x >> (8 * j)) * scale;
        v[4 + j] = (float)(int8_t)(q.y >> (8 * j)) * scale;
    }
}

// A half-warp takes one block of one row (its gate and its up columns).
template <bool GUB>
__global__ void __launch_bounds__(kThreads) swiglu_checkpoint_kernel(const SwigluCkptArgs a) {
    const int nb = ckpt_blocks(a.F);
    const long long units = a.S * nb;
    const int sub = threadIdx.x & (kLanes - 1);
    const long long step = (long long)gridDim.x * (kThreads / kLanes);
    const long long first = (long long)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    // whole warps stay in the loop (the shuffles need every lane)
    for (long long u = first; u - (threadIdx.x & 31) / kLanes < units; u += step) {
        const bool live_unit = u < units;
        const long long row = live_unit ? u / nb : 0;
        const int b = live_unit ? (int)(u % nb) : 0;
        const int c = b * kCkptBlock + sub * 8;
        const bool live = live_unit && c < a.F;  // F % 8 == 0
        float g[8] = {}, up[8] = {};
        const size_t i = (size_t)row * 2 * a.F + c;
        if (live) {
            load8<GUB>(a.GU, i, g);
            load8<GUB>(a.GU, i + a.F, up);
        }
        float sg, su;
        const uint2 qg = quantize8(g, sg), qu = quantize8(up, su);
        if (!live) continue;
        *reinterpret_cast<uint2*>(a.codes + i) = qg;
        *reinterpret_cast<uint2*>(a.codes + i + a.F) = qu;
        if (sub == 0) {
            a.scales[row * 2 * nb + b] = sg;
            a.scales[row * 2 * nb + nb + b] = su;
        }
        if (a.H) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = g[j] * sigmoid(g[j]) * up[j];
            store8<true>(a.H, (size_t)row * a.F + c, g);
        }
    }
}

template <bool DHB>
__global__ void __launch_bounds__(kThreads) swiglu_backward_kernel(const SwigluCkptBackwardArgs a) {
    const int nb = ckpt_blocks(a.F), nv = a.F / 8;
    const long long units = a.S * nv;
    for (long long u = (long long)blockIdx.x * kThreads + threadIdx.x; u < units; u += (long long)gridDim.x * kThreads) {
        const long long row = u / nv;
        const int c = (int)(u % nv) * 8;
        const size_t i = (size_t)row * 2 * a.F + c, h = (size_t)row * a.F + c;
        float g[8], up[8], dh[8];
        restore8(__ldcs(reinterpret_cast<const uint2*>(a.codes + i)), __ldg(a.scales + row * 2 * nb + c / kCkptBlock), g);
        restore8(__ldcs(reinterpret_cast<const uint2*>(a.codes + i + a.F)),
                 __ldg(a.scales + row * 2 * nb + nb + c / kCkptBlock), up);
        load8<DHB>(a.dH, h, dh);
        float dg[8], du[8], hh[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = sigmoid(g[j]), act = g[j] * s;
            hh[j] = act * up[j];
            du[j] = dh[j] * act;
            dg[j] = dh[j] * up[j] * (s * (1.f + g[j] * (1.f - s)));
        }
        store8<true>(a.dGU, i, dg);
        store8<true>(a.dGU, i + a.F, du);
        if (a.H) store8<true>(a.H, h, hh);
    }
}

}  // namespace

cudaError_t launch_swiglu_checkpoint(const SwigluCkptArgs& a, int sm_count, cudaStream_t stream) {
    const long long blocks = (a.S * ckpt_blocks(a.F) + kThreads / kLanes - 1) / (kThreads / kLanes);
    const int grid = (int)std::min<long long>(blocks, (long long)sm_count * 8);
    if (a.gu_bf16) swiglu_checkpoint_kernel<true><<<grid, kThreads, 0, stream>>>(a);
    else swiglu_checkpoint_kernel<false><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_checkpoint_backward(const SwigluCkptBackwardArgs& a, int sm_count, cudaStream_t stream) {
    const long long blocks = (a.S * (a.F / 8) + kThreads - 1) / kThreads;
    const int grid = (int)std::min<long long>(blocks, (long long)sm_count * 8);
    if (a.dh_bf16) swiglu_backward_kernel<true><<<grid, kThreads, 0, stream>>>(a);
    else swiglu_backward_kernel<false><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
