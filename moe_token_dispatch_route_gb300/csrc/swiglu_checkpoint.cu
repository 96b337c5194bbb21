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
//
// Both kernels are bound by HBM.  A thread takes 8 columns of the gate and the same 8 of the up
// half; the 16 threads of a block find its amax by shuffles.  The row and block of a thread's next unit are stepped,
// not divided out.
#include <algorithm>

#include "train.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256;
constexpr int kLanes = kCkptBlock / 8;      // 16 threads of 8 columns share a block
constexpr float kMinAmax = 3.7615819e-37f;  // 2^-121: the smallest amax that is stored

// 1 / (1 + e^-g) from e^-|g|, which does not overflow: far negative g keeps its small result.
// The approximations are within a few units of 2^-24, far below the rounding to bf16 that follows.
__device__ __forceinline__ float sigmoid(float g) {
    const float e = __expf(-fabsf(g));
    return __fdividef(g >= 0.f ? 1.f : e, 1.f + e);
}

// Scale of the 16 threads' block and this thread's 8 codes (two words); every lane of the warp
// takes part.
__device__ __forceinline__ uint2 quantize8(const float (&v)[8], float& scale) {
    uint32_t m = 0;  // magnitudes compare as integers: NaN > infinity > finite
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
    const float amax = __uint_as_float(m);
    if (m >= 0x7F800000u || amax < kMinAmax) {
        scale = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : 0.f;
        return make_uint2(0u, 0u);
    }
    scale = __fdiv_rn(amax, 127.f);
    const float inv = __fdiv_rn(127.f, amax);
    // fp32(x inv) is at most 127 and a bit in magnitude: adding 1.5 * 2^23 rounds it to the
    // nearest even integer, whose two's complement is the sum's low byte
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __float_as_uint(__fadd_rn(__fmul_rn(v[j], inv), 12582912.f));
    auto pack = [&](int i) {
        return __byte_perm(__byte_perm(q[i], q[i + 1], 0x0040), __byte_perm(q[i + 2], q[i + 3], 0x0040), 0x5410);
    };
    return make_uint2(pack(0), pack(4));
}

// The stored values of 8 codes.  A code plus 128 is put in the low byte of 2^23's bits.
__device__ __forceinline__ void restore8(uint2 q, float scale, float (&v)[8]) {
    const uint32_t w[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = (__uint_as_float(__byte_perm(w[j / 4], 0x4B000000u, 0x7540 | (j & 3))) - 8388736.f) * scale;
}

// (row, part) of unit u of `parts` per row, and the step to unit u + stride.
struct Walk {
    long long row, row_step;
    int part, part_step, parts;
    __device__ Walk(long long u, long long stride, int parts_) : parts(parts_) {
        row = u / parts;
        part = (int)(u - row * parts);
        row_step = stride / parts;
        part_step = (int)(stride - row_step * parts);
    }
    __device__ void next() {
        row += row_step;
        part += part_step;
        if (part >= parts) {
            part -= parts;
            ++row;
        }
    }
};

// Sixteen threads take one block of one row (its gate and its up columns).
template <bool GUB>
__global__ void __launch_bounds__(kThreads) swiglu_checkpoint_kernel(const SwigluCkptArgs a) {
    const int nb = ckpt_blocks(a.F);
    const int sub = threadIdx.x & (kLanes - 1), part = threadIdx.x / kLanes;
    Walk at((long long)blockIdx.x * (kThreads / kLanes) + part, (long long)gridDim.x * (kThreads / kLanes), nb);
    // every lane of a warp stays as long as the warp's first unit is a unit (the shuffles need all)
    for (;; at.next()) {
        const bool unit = at.row < a.S;
        if (!__any_sync(kFull, unit)) return;
        const int c = at.part * kCkptBlock + sub * 8;
        const bool live = unit && c < a.F;  // F % 8 == 0
        float g[8] = {}, up[8] = {};
        const size_t i = (size_t)at.row * 2 * a.F + c;
        if (live) {
            load8<GUB>(a.GU, i, g);
            load8<GUB>(a.GU, i + a.F, up);
        }
        float sg, su;
        const uint2 qg = quantize8(g, sg), qu = quantize8(up, su);
        if (!live) continue;
        __stcs(reinterpret_cast<uint2*>(a.codes + i), qg);
        __stcs(reinterpret_cast<uint2*>(a.codes + i + a.F), qu);
        if (sub == 0) {
            a.scales[at.row * 2 * nb + at.part] = sg;
            a.scales[at.row * 2 * nb + nb + at.part] = su;
        }
        if (a.H) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = g[j] * sigmoid(g[j]) * up[j];
            store8<true>(a.H, (size_t)at.row * a.F + c, g);
        }
    }
}

template <bool DHB>
__global__ void __launch_bounds__(kThreads) swiglu_backward_kernel(const SwigluCkptBackwardArgs a) {
    const int nb = ckpt_blocks(a.F);
    Walk at((long long)blockIdx.x * kThreads + threadIdx.x, (long long)gridDim.x * kThreads, a.F / 8);
    for (; at.row < a.S; at.next()) {
        const int c = at.part * 8;
        const size_t i = (size_t)at.row * 2 * a.F + c, h = (size_t)at.row * a.F + c;
        const float* scale = a.scales + at.row * 2 * nb + c / kCkptBlock;
        float g[8], up[8], dh[8], dg[8], du[8];
        restore8(__ldcs(reinterpret_cast<const uint2*>(a.codes + i)), __ldg(scale), g);
        restore8(__ldcs(reinterpret_cast<const uint2*>(a.codes + i + a.F)), __ldg(scale + nb), up);
        load8<DHB>(a.dH, h, dh);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = sigmoid(g[j]), act = g[j] * s, du_dh = up[j] * dh[j];
            dg[j] = du_dh * fmaf(act, 1.f - s, s);  // s (1 + g (1 - s))
            du[j] = dh[j] * act;
            g[j] = act * up[j];
        }
        store8<true>(a.dGU, i, dg);
        store8<true>(a.dGU, i + a.F, du);
        if (a.H) store8<true>(a.H, h, g);
    }
}

// threads of a launch: `per_sm` CTAs on every SM, fewer where there is less to do
template <class Kernel, class Args>
cudaError_t go(Kernel kernel, const Args& a, long long threads, int sm_count, cudaStream_t stream) {
    const long long ctas = (threads + kThreads - 1) / kThreads;
    kernel<<<(int)std::min<long long>(ctas, (long long)sm_count * 8), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_swiglu_checkpoint(const SwigluCkptArgs& a, int sm_count, cudaStream_t stream) {
    const long long threads = a.S * ckpt_blocks(a.F) * kLanes;
    return a.gu_bf16 ? go(swiglu_checkpoint_kernel<true>, a, threads, sm_count, stream)
                     : go(swiglu_checkpoint_kernel<false>, a, threads, sm_count, stream);
}

cudaError_t launch_swiglu_checkpoint_backward(const SwigluCkptBackwardArgs& a, int sm_count, cudaStream_t stream) {
    const long long threads = a.S * (a.F / 8);
    return a.dh_bf16 ? go(swiglu_backward_kernel<true>, a, threads, sm_count, stream)
                     : go(swiglu_backward_kernel<false>, a, threads, sm_count, stream);
}

}  // namespace moe
