// The experts' weights in 8 bits: W bf16 [E][d][N] -> e4m3 codes [E][N][d] and a scale for each block of 128 x 128, the
// layout of the block-scaled per-expert product (the reduction d is the contiguous axis of both its operands).
// Bound by HBM: 2 bytes in and 1 out a weight (64 experts of 2048 x 2816: 175 us, 0.93 of a plain copy's rate).
//
// A CTA takes a block at a time.  A thread holds 4 consecutive rows of d by 8 columns, twice; it packs the codes of four
// rows into a word a column, and the words cross shared memory to leave as rows of 128 bytes.
#include <algorithm>

#include "serve.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256;
constexpr int kCtasPerSm = 5;  // (64 experts of 2048 x 2816: 184 us with four, 177 with five)

__global__ void __launch_bounds__(kThreads, kCtasPerSm) quantize_weights_kernel(const QuantizeWeightsArgs a) {
    __shared__ uint32_t words[128 * 32];  // [column of W][words of 4 rows]; word w of column n is at w ^ 2 (n / 8)
    __shared__ uint32_t red[2][kThreads / 32];
    wait_for_kernel_before();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int v = tid & 15, g = tid >> 4;  // columns 8v .. 8v + 7; rows 4g .. 4g + 3, and 64 more
    const int n_half = a.N / a.halves, nb = scale_blocks(n_half), db = scale_blocks(a.d);
    const long long blocks = (long long)a.E * a.halves * nb * db;
    int turn = 0;
    for (long long b = blockIdx.x; b < blocks; b += gridDim.x, turn ^= 1) {
        // neighbours in N run together: their rows of W are neighbours in memory
        const int i = (int)(b % nb);
        const long long r = b / nb;
        const int half = (int)(r % a.halves);
        const long long q = r / a.halves;
        const int j = (int)(q % db), e = (int)(q / db);
        const int cols = min(128, n_half - 128 * i), rows = min(128, a.d - 128 * j);
        const int n0 = half * n_half + 128 * i, d0 = 128 * j;
        uint4 x[2][4];
        uint32_t amax = 0;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int row = 64 * s + 4 * g + k;
                x[s][k] = make_uint4(0, 0, 0, 0);
                if (row < rows && 8 * v < cols)
                    x[s][k] = __ldcs(reinterpret_cast<const uint4*>(a.W + ((size_t)e * a.d + d0 + row) * a.N + n0 + 8 * v));
            }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                constexpr uint32_t kAbs = 0x7FFF7FFFu;
                const uint4 u = x[s][k];
                const uint32_t m = __vmaxu2(__vmaxu2(u.x & kAbs, u.y & kAbs), __vmaxu2(u.z & kAbs, u.w & kAbs));
                amax = max(amax, max(m & 0xFFFF0000u, m << 16));
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(kFull, amax, o));
        if (lane == 0) red[turn][warp] = amax;
        __syncthreads();  // (and all have read the words of the block before)
        amax = red[turn][lane & 7];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(kFull, amax, o));
        const float inv = block_quotient(amax, true);
        if (tid == 0) a.scales[((size_t)e * a.halves * nb + (size_t)half * nb + i) * db + j] = block_quotient(amax, false);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t* u[4] = {&x[s][0].x, &x[s][1].x, &x[s][2].x, &x[s][3].x};
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                float f[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] = c & 1 ? bf16_hi(u[k][c / 2]) : bf16_lo(u[k][c / 2]);
                words[(8 * v + c) * 32 + ((16 * s + g) ^ (2 * v))] = e4m3x4(f[0], f[1], f[2], f[3], inv);
            }
        }
        __syncthreads();
        // 16 lanes a column of W: 8 bytes each
        const int pair = tid & 15;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int n = 16 * k + (tid >> 4);
            const uint2 w = *reinterpret_cast<const uint2*>(words + n * 32 + 2 * (pair ^ (n >> 3)));
            if (n < cols && 8 * pair < rows)
                __stcs(reinterpret_cast<uint2*>(a.codes + ((size_t)e * a.N + n0 + n) * a.d + d0 + 8 * pair), w);
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_quantize_weights(const QuantizeWeightsArgs& a, int sm_count, cudaStream_t stream) {
    const long long blocks = (long long)a.E * a.halves * scale_blocks(a.N / a.halves) * scale_blocks(a.d);
    return launch_after(quantize_weights_kernel, (unsigned)std::min<long long>(blocks, (long long)sm_count * kCtasPerSm), kThreads, 0,
                        stream, a);
}

}  // namespace moe
