// RMS norm of token rows with the residual's addition before it and an 8-bit output beside or in place of the bf16 one.
//   h = x + res (rounded to the residual's type, stored),  rstd = 1 / sqrt(sum h^2 / d + eps),  y = h rstd gamma,
// the sum in fp32 over the stored values (where their squares pass its range, of scaled ones).  The 8-bit output is y before
// it is rounded to bf16: e4m3 codes and a scale for each 128 columns of a row.  Bound by HBM: x and the residual are read once
// and h stays in registers between the sum and the results (rows above 32768 columns are read back from L2).
//
// A row is held by TPR threads (a power of two from 16 to 1024), vectors of 8 columns, so 16 neighbouring threads hold a
// block of 128 and find its amax by shuffles.  8192 x 4096, fp32 x, bf16 residual, both outputs: 60.1 us, 0.91 of a plain
// copy's rate.
#include <algorithm>
#include <type_traits>

#include "serve.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kVpt = 4;       // vectors of a thread
constexpr int kMaxRow = 1024 * 8 * kVpt;
constexpr int kWide = 1024;
constexpr float kLargest = 3.402823466e38f;
__host__ __device__ constexpr int cta_threads(int tpr) { return tpr > 128 ? tpr : 128; }

template <bool BF16>
__device__ __forceinline__ float rounded(float v) {
    return BF16 ? __uint_as_float((uint32_t)(bf16x2(v, 0.f) & 0xFFFFu) << 16) : v;
}

// Sum over the TPR threads of a row, the same bits in each of them; `red` alternates from call to call.
template <int TPR, int CTA>
__device__ __forceinline__ float row_sum(float v, float (&red)[CTA / 32]) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if constexpr (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) red[warp] = v;
        __syncthreads();
        v = red[warp / kWarps * kWarps + lane % kWarps];
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    }
    return v;
}

// The results of 8 columns: called by all lanes of a warp (`mine`: the columns exist).
__device__ __forceinline__ void results8(const RmsnormArgs& a, const float (&h)[8], float rstd, size_t row, int c, bool mine) {
    float y[8];
    if (mine) {
        float g[8];
        if (a.gamma) {
            const float4 u = __ldg(reinterpret_cast<const float4*>(a.gamma + c)), v = __ldg(reinterpret_cast<const float4*>(a.gamma + c) + 1);
            g[0] = u.x; g[1] = u.y; g[2] = u.z; g[3] = u.w;
            g[4] = v.x; g[5] = v.y; g[6] = v.z; g[7] = v.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = 1.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = h[j] * rstd * g[j];
        if (a.y) store8<true>(a.y, row * a.d + c, y);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.f;
    }
    if (a.codes) {
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(y[j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(kFull, amax, o));
        // the block's first thread divides for the scale, the others for its inverse
        const int in_block = threadIdx.x & 15;
        const float quotient = block_quotient(amax, in_block != 0);
        const float inv = __shfl_sync(kFull, quotient, (threadIdx.x & 31 & ~15) + 1);
        if (mine) {
            if (in_block == 0) a.scales[row * scale_blocks(a.d) + c / kScaleBlock] = quotient;
            __stcs(reinterpret_cast<uint2*>(a.codes + row * a.d + c),
                   make_uint2(e4m3x4(y[0], y[1], y[2], y[3], inv), e4m3x4(y[4], y[5], y[6], y[7], inv)));
        }
    }
}

// Rows that are finite but whose mean square and eps are not (values from some 1e18 up): a CTA that has met one (`met`, by thread) goes
// over its rows again, sums the squares of 2^-96 h and writes the results of such rows once more.  h is what each thread
// has stored, or x; its plain sum is the same bits as before.  (Done where it is met, the second sum cost the other rows up to 6%.)
template <bool XB, bool HB, int TPR, int CTA>
__device__ __forceinline__ void far_rows(const RmsnormArgs& a, bool met, float inv_d, float (&red)[2][CTA / 32]) {
    if (!__syncthreads_or(met)) return;
    constexpr int kRows = CTA / TPR;
    constexpr float kDown = 0x1p-96f;
    const int c0 = (int)(threadIdx.x % TPR) * 8;
    for (long long t0 = (long long)blockIdx.x * kRows; t0 < a.T; t0 += (long long)gridDim.x * kRows) {
        const long long t = t0 + threadIdx.x / TPR;
        const bool row = t < a.T;
        const size_t at = row ? (size_t)t * a.d : 0;
        auto load = [&](int c, float(&h)[8]) {
            if (a.h) load8<HB>(a.h, at + c, h);
            else load8<XB>(a.x, at + c, h);
        };
        float s = 0.f, v = 0.f;
#pragma unroll 1
        for (int c = c0; row && c < a.d; c += TPR * 8) {
            float h[8];
            load(c, h);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s = fmaf(h[j], h[j], s);
                v = fmaf(h[j] * kDown, h[j] * kDown, v);
            }
        }
        s = row_sum<TPR, CTA>(s, red[0]);
        v = row_sum<TPR, CTA>(v, red[1]);
        const bool far = fmaf(s, inv_d, a.eps) > kLargest;
        if (!__syncthreads_or(far)) continue;  // (and all have read the sums)
        const float rstd = kDown / sqrtf(v * inv_d + a.eps * kDown * kDown);
        if (row && far && c0 == 0 && a.rstd) a.rstd[t] = rstd;
#pragma unroll 1
        for (int base = 0; base < a.d; base += TPR * 8) {  // (whole warps: the blocks' amax is found by shuffles)
            const int c = base + c0;
            const bool mine = row && far && c < a.d;
            float h[8] = {};
            if (mine) load(c, h);
            results8(a, h, rstd, row ? (size_t)t : 0, c, mine);
        }
    }
}

template <bool XB, bool HB, int TPR>
__global__ void __launch_bounds__(cta_threads(TPR), 1024 / cta_threads(TPR)) rmsnorm_kernel(const RmsnormArgs a) {
    constexpr int kCta = cta_threads(TPR), kRows = kCta / TPR;
    __shared__ float red[2][kCta / 32];
    wait_for_kernel_before();
    const int sub = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const float inv_d = 1.f / (float)a.d;
    int turn = 0;
    bool met = false;
    for (long long t0 = (long long)blockIdx.x * kRows; t0 < a.T; t0 += (long long)gridDim.x * kRows, turn ^= 1) {
        const long long t = t0 + group;
        const bool row = t < a.T;
        const size_t at = row ? (size_t)t * a.d : 0;
        float h[kVpt][8];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int c = (sub + i * TPR) * 8;
            if (row && c < a.d) {
                load8<XB>(a.x, at + c, h[i]);
                if (a.res) {
                    float r[8];
                    load8<HB>(a.res, at + c, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[i][j] = rounded<HB>(h[i][j] + r[j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int c = (sub + i * TPR) * 8;
            if (a.h && row && c < a.d) store8<HB>(a.h, at + c, h[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(h[i][j], h[i][j], s);
        }
        s = row_sum<TPR, kCta>(s, red[turn]);
        const float mean = fmaf(s, inv_d, a.eps), rstd = 1.f / sqrtf(mean);
        met |= mean > kLargest;
        if (row && sub == 0 && a.rstd) a.rstd[t] = rstd;
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int c = (sub + i * TPR) * 8;
            results8(a, h[i], rstd, row ? (size_t)t : 0, c, row && c < a.d);
        }
    }
    far_rows<XB, HB, TPR, kCta>(a, met, inv_d, red);
}

// d > 32768: h is read back
template <bool XB, bool HB>
__global__ void __launch_bounds__(kWide) rmsnorm_wide_kernel(const RmsnormArgs a) {
    __shared__ float red[2][kWide / 32];
    wait_for_kernel_before();
    const float inv_d = 1.f / (float)a.d;
    int turn = 0;
    bool met = false;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        const size_t at = (size_t)t * a.d;
        float s = 0.f;
        for (int c = threadIdx.x * 8; c < a.d; c += kWide * 8) {
            float h[8];
            load8<XB>(a.x, at + c, h);
            if (a.res) {
                float r[8];
                load8<HB>(a.res, at + c, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[j] = rounded<HB>(h[j] + r[j]);
            }
            if (a.h) store8<HB>(a.h, at + c, h);
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(h[j], h[j], s);
        }
        s = row_sum<kWide, kWide>(s, red[turn]);
        const float mean = fmaf(s, inv_d, a.eps), rstd = 1.f / sqrtf(mean);
        met |= mean > kLargest;
        if (threadIdx.x == 0 && a.rstd) a.rstd[t] = rstd;
        for (int c0 = 0; c0 < a.d; c0 += kWide * 8) {  // (whole warps: the blocks' amax is found by shuffles)
            const int c = c0 + threadIdx.x * 8;
            float h[8] = {};
            if (c < a.d) {  // what this thread has stored, or x
                if (a.h) load8<HB>(a.h, at + c, h);
                else load8<XB>(a.x, at + c, h);
            }
            results8(a, h, rstd, (size_t)t, c, c < a.d);
        }
    }
    far_rows<XB, HB, kWide, kWide>(a, met, inv_d, red);
}

template <bool XB, bool HB>
cudaError_t rows(const RmsnormArgs& a, int sm_count, cudaStream_t s) {
    if (a.d > kMaxRow) return launch_after(rmsnorm_wide_kernel<XB, HB>, (unsigned)std::min(a.T, 2 * sm_count), kWide, 0, s, a);
    auto go = [&](auto tpr) {
        constexpr int kTpr = decltype(tpr)::value, kCta = cta_threads(kTpr), kRows = kCta / kTpr;
        const unsigned grid = (unsigned)std::min(((long long)a.T + kRows - 1) / kRows, (long long)sm_count * (1024 / kCta));
        return launch_after(rmsnorm_kernel<XB, HB, kTpr>, grid, kCta, 0, s, a);
    };
    int tpr = 16;
    while (tpr * 8 * kVpt < a.d) tpr *= 2;
    switch (tpr) {
        case 16: return go(std::integral_constant<int, 16>());
        case 32: return go(std::integral_constant<int, 32>());
        case 64: return go(std::integral_constant<int, 64>());
        case 128: return go(std::integral_constant<int, 128>());
        case 256: return go(std::integral_constant<int, 256>());
        case 512: return go(std::integral_constant<int, 512>());
        default: return go(std::integral_constant<int, 1024>());
    }
}

}  // namespace

cudaError_t launch_rmsnorm(const RmsnormArgs& a, int sm_count, cudaStream_t stream) {
    if (a.x_bf16) return a.h_bf16 ? rows<true, true>(a, sm_count, stream) : rows<true, false>(a, sm_count, stream);
    return a.h_bf16 ? rows<false, true>(a, sm_count, stream) : rows<false, false>(a, sm_count, stream);
}

}  // namespace moe
