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
// Both kernels are bound by HBM, and close to it by their instructions.  A thread takes 8 columns of the gate and the
// same 8 of the up half; the 16 threads of a block find its amax by shuffles.  The row and block of a
// thread's next unit are stepped, not divided out.
// bf16, S = 16384, F = 14336: forward 305 us, 6.2 TB/s (0.92 of a plain copy's rate); backward 365 us, 6.5 TB/s (0.95).
// S = 65536, F = 1408: forward 123 us, both 265 us.
#include <algorithm>

#include "train.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256;
constexpr int kLanes = kCkptBlock / 8;      // 16 threads of 8 columns share a block
constexpr float kMinAmax = 3.7615819e-37f;  // 2^-121: the smallest amax that is stored

// 1 / (1 + e^-g) from e^-|g|, which does not overflow: far negative g keeps its small result.
// The exponential is within 2 + 1.173 |g| units in its last place and the quotient within 2: 2e-6 of the result at
// |g| = 10, 1.2e-5 at 80, below the 2^-9 of the rounding to bf16 that follows.
__device__ __forceinline__ float sigmoid(float g) {
    const float e = __expf(-fabsf(g));
    return __fdividef(g >= 0.f ? 1.f : e, 1.f + e);
}

// Eight columns as they are in memory, so that the next unit's can be on their way in few registers.
// amax(): their largest magnitude's fp32 bits.  Magnitudes compare as integers: NaN > infinity > finite.
template <bool BF16>
struct Raw;
template <>
struct Raw<true> {
    uint4 a = {0, 0, 0, 0};
    __device__ void load(const void* p, size_t i) { a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i)); }
    __device__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16_lo(w[j]);
            v[2 * j + 1] = bf16_hi(w[j]);
        }
    }
    __device__ uint32_t amax() const {  // two at a time
        constexpr uint32_t kAbs = 0x7FFF7FFFu;
        const uint32_t m = __vmaxu2(__vmaxu2(a.x & kAbs, a.y & kAbs), __vmaxu2(a.z & kAbs, a.w & kAbs));
        return max(m & 0xFFFF0000u, m << 16);
    }
};
template <>
struct Raw<false> {
    float4 a = {0.f, 0.f, 0.f, 0.f}, b = {0.f, 0.f, 0.f, 0.f};
    __device__ void load(const void* p, size_t i) {
        a = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
        b = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i) + 1);
    }
    __device__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    __device__ uint32_t amax() const {
        float v[8];
        get(v);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        return m;
    }
};

// One of the four quotients of a block pair: a block's scale or its inverse.
// amax / 127 (or NaN, or 0 below the smallest amax) and 127 / amax (0 where the codes are 0).
__device__ __forceinline__ float quotient(uint32_t amax_bits, bool inverse) {
    const float amax = __uint_as_float(amax_bits);
    if (amax_bits >= 0x7F800000u) return inverse ? 0.f : __uint_as_float(0x7FC00000u);
    if (amax < kMinAmax) return 0.f;
    return __fdiv_rn(inverse ? 127.f : amax, inverse ? amax : 127.f);
}

// Eight codes.  fp32(x inv) is at most 127 and a bit in magnitude: adding 1.5 * 2^23 rounds it to
// the nearest even integer, whose two's complement is the sum's low byte.  inv = 0 is a block of
// codes 0 (x may be infinite or NaN there).
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
    if (inv == 0.f) return make_uint2(0u, 0u);
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

// Sixteen threads take one block of one row (its gate and its up columns); the next unit's loads
// are issued before this one's arithmetic.
template <bool GUB>
__global__ void __launch_bounds__(kThreads) swiglu_checkpoint_kernel(const SwigluCkptArgs a) {
    wait_for_kernel_before();
    const int nb = ckpt_blocks(a.F);
    const int sub = threadIdx.x & (kLanes - 1), part = threadIdx.x / kLanes;
    Walk at((long long)blockIdx.x * (kThreads / kLanes) + part, (long long)gridDim.x * (kThreads / kLanes), nb);
    auto live = [&] { return at.row < a.S && at.part * kCkptBlock + sub * 8 < a.F; };  // F % 8 == 0
    Raw<GUB> rg, ru;
    auto fetch = [&] {
        if (live()) {
            const size_t i = (size_t)at.row * 2 * a.F + at.part * kCkptBlock + sub * 8;
            rg.load(a.GU, i);
            ru.load(a.GU, i + a.F);
        } else {
            rg = ru = Raw<GUB>();
        }
    };
    fetch();
    // every lane of a warp stays while one of its lanes has a unit (the shuffles need all)
    while (__any_sync(kFull, at.row < a.S)) {
        float g[8], up[8];
        rg.get(g);
        ru.get(up);
        uint32_t mg = rg.amax(), mu = ru.amax();
        const bool mine = live(), stored = at.row < a.S;
        const long long row = at.row;
        const int b = at.part, c = b * kCkptBlock + sub * 8;
        at.next();
        fetch();
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) {
            mg = max(mg, __shfl_xor_sync(kFull, mg, o));
            mu = max(mu, __shfl_xor_sync(kFull, mu, o));
        }
        // one division a thread: threads 0-3 of each four take the gate's inverse, the up's
        // inverse, the gate's scale and the up's scale
        const float quot = quotient(sub & 1 ? mu : mg, (sub & 2) == 0);
        const float ig = __shfl_sync(kFull, quot, threadIdx.x & 28), iu = __shfl_sync(kFull, quot, (threadIdx.x & 28) + 1);
        if ((sub == 2 || sub == 3) && stored) a.scales[row * 2 * nb + (sub & 1 ? nb : 0) + b] = quot;
        if (!mine) continue;
        const uint2 qg = codes8(g, ig), qu = codes8(up, iu);
        const size_t i = (size_t)row * 2 * a.F + c;
        __stcs(reinterpret_cast<uint2*>(a.codes + i), qg);
        __stcs(reinterpret_cast<uint2*>(a.codes + i + a.F), qu);
        if (a.H) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = g[j] * sigmoid(g[j]) * up[j];
            store8<true>(a.H, (size_t)row * a.F + c, g);
        }
    }
}

template <bool DHB>
__global__ void __launch_bounds__(kThreads) swiglu_backward_kernel(const SwigluCkptBackwardArgs a) {
    wait_for_kernel_before();
    const int nb = ckpt_blocks(a.F);
    Walk at((long long)blockIdx.x * kThreads + threadIdx.x, (long long)gridDim.x * kThreads, a.F / 8);
    uint2 qg, qu;
    float sg, su;
    Raw<DHB> rh;
    auto fetch = [&] {
        if (at.row >= a.S) return;
        const int c = at.part * 8;
        const size_t i = (size_t)at.row * 2 * a.F + c;
        const float* scale = a.scales + at.row * 2 * nb + c / kCkptBlock;
        qg = __ldcs(reinterpret_cast<const uint2*>(a.codes + i));
        qu = __ldcs(reinterpret_cast<const uint2*>(a.codes + i + a.F));
        sg = __ldg(scale);
        su = __ldg(scale + nb);
        rh.load(a.dH, (size_t)at.row * a.F + c);
    };
    fetch();
    while (at.row < a.S) {
        const int c = at.part * 8;
        const size_t i = (size_t)at.row * 2 * a.F + c, h = (size_t)at.row * a.F + c;
        float g[8], up[8], dh[8], dg[8], du[8];
        restore8(qg, sg, g);
        restore8(qu, su, up);
        rh.get(dh);
        at.next();
        fetch();
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

// threads of a launch: four CTAs on every SM of bf16 inputs, three of fp32, fewer where there is less to do.  More loads
// in flight are slower, not faster (forward, S = 16384, F = 14336, us: bf16 333 with three, 305 with four, 330 with five
// resident; fp32 468 with two, 428 with three, 451 with four, 511 with five).
template <class Kernel, class Args>
cudaError_t go(Kernel kernel, const Args& a, long long threads, bool bf16, int sm_count, cudaStream_t stream) {
    const long long ctas = (threads + kThreads - 1) / kThreads;
    return launch_after(kernel, (unsigned)std::min<long long>(ctas, (long long)sm_count * (bf16 ? 4 : 3)), kThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_swiglu_checkpoint(const SwigluCkptArgs& a, int sm_count, cudaStream_t stream) {
    const long long threads = a.S * ckpt_blocks(a.F) * kLanes;
    return a.gu_bf16 ? go(swiglu_checkpoint_kernel<true>, a, threads, true, sm_count, stream)
                     : go(swiglu_checkpoint_kernel<false>, a, threads, false, sm_count, stream);
}

cudaError_t launch_swiglu_checkpoint_backward(const SwigluCkptBackwardArgs& a, int sm_count, cudaStream_t stream) {
    const long long threads = a.S * (a.F / 8);
    return a.dh_bf16 ? go(swiglu_backward_kernel<true>, a, threads, true, sm_count, stream)
                     : go(swiglu_backward_kernel<false>, a, threads, false, sm_count, stream);
}

}  // namespace moe
