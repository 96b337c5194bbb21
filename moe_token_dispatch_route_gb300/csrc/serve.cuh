// Declarations of the 8-bit forward operators (RMS norm with an 8-bit output, the experts' weights in 8
// bits, the block-scaled per-expert product) and of the router's losses: launch parameter blocks.
#pragma once

#include "train.cuh"

namespace moe {

constexpr int kScaleBlock = 128;  // columns (and, of weights, rows) that share one scale
__host__ __device__ constexpr int scale_blocks(int n) { return n / kScaleBlock + (n % kScaleBlock != 0); }

struct RmsnormArgs {
    const void* x;       // [T][d], fp32 or bf16
    int x_bf16;
    const void* res;     // [T][d] of h's type, or null
    void* h;             // [T][d] or null (no residual)
    int h_bf16;
    const float* gamma;  // [d] or null (1)
    float eps;
    uint16_t* y;         // bf16 [T][d] or null
    uint8_t* codes;      // e4m3 [T][d] or null
    float* scales;       // [T][scale_blocks(d)], with codes
    float* rstd;         // [T] or null
    int T, d;
};
cudaError_t launch_rmsnorm(const RmsnormArgs& a, int sm_count, cudaStream_t stream);

struct QuantizeWeightsArgs {
    const uint16_t* W;  // bf16 [E][d][N]
    uint8_t* codes;     // e4m3 [E][N][d]
    float* scales;      // [E][halves * scale_blocks(N / halves)][scale_blocks(d)]
    int E, d, N, halves;
};
cudaError_t launch_quantize_weights(const QuantizeWeightsArgs& a, int sm_count, cudaStream_t stream);

struct GroupedFp8Args {
    const uint8_t* A;        // e4m3 [S][d], or [T][d] with perm
    const float* A_scales;   // [rows of A][scale_blocks(d)]
    const int32_t* perm;     // [S] or null: row i is A's row perm[i] / k
    const int32_t* offsets;  // [E+1]
    const uint8_t* W;        // e4m3 [E][N][d]
    const float* W_scales;   // [E][halves * scale_blocks(N / halves)][scale_blocks(d)]
    int glu;                 // 1: N = 2F, gate then up; out H, not Y
    void* Y;                 // [S][N], fp32 or bf16
    int out_bf16;
    uint8_t* H;              // e4m3 [S][F]
    float* H_scales;         // [S][scale_blocks(F)]
    int32_t* status;
    long long timeout_ns;
    int T, S, d, E, k, N;
};
cudaError_t launch_grouped_fp8(const GroupedFp8Args& a, int device, int sm_count, cudaStream_t stream);

struct RouterLossArgs {
    const float* logits;      // [T][E]
    const int32_t* topk_idx;  // [T][k]
    const float* dtopk_w;     // [T][k] or null (backward)
    const uint8_t* mask;      // [T] or null: nonzero counts
    int seq_len;              // tokens of a group; the last one may be shorter
    int groups;
    float balance, z;
    int renorm, sigmoid;
    float* loss;              // [2]
    int32_t* load;            // [groups][E]
    int32_t* tokens;          // [groups + 1]
    float* dlogits;           // [T][E]
    void* scratch;
    int T, E, k;
};
size_t balance_scratch_bytes(int T, int E, int seq_len, int sm_count);
cudaError_t launch_balance_loss(const RouterLossArgs& a, int sm_count, cudaStream_t stream);
cudaError_t launch_router_backward(const RouterLossArgs& a, int sm_count, cudaStream_t stream);

// e4m3 bytes [..][cols] as 128-byte swizzled boxes of 128 columns
bool map_e4m3_2d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows);
// weights [E][halves][n][cols]: boxes of 128 columns by 128 rows of one half of one expert
bool map_e4m3_weights(CUtensorMap* map, const void* base, uint64_t E, uint64_t halves, uint64_t n, uint64_t cols);

#if defined(__CUDACC__)

// 8-bit storage of a block: with amax its largest magnitude,
//   scale = fp32(amax / 448),  inv = fp32(448 / amax),  code = nearest even e4m3 of fp32(x inv).
// fp32(x inv) is at most 448 and a bit, which rounds to 448, the largest e4m3 value.  A block below 2^-117 (whose
// scale would be subnormal) has scale 0 and codes 0, one with an infinity or a NaN scale NaN and codes 0.
constexpr float kE4m3Max = 448.f;
constexpr float kMinAmax8 = 6.0185310762101144e-36f;  // 2^-117

// The block's scale, or (inverse) what its values are multiplied by; amax as its fp32 bits: magnitudes compare as
// integers, NaN > infinity > finite.
__device__ __forceinline__ float block_quotient(uint32_t amax_bits, bool inverse) {
    const float amax = __uint_as_float(amax_bits);
    if (amax_bits >= 0x7F800000u) return inverse ? 0.f : __uint_as_float(0x7FC00000u);
    if (amax < kMinAmax8) return 0.f;
    return __fdiv_rn(inverse ? kE4m3Max : amax, inverse ? amax : kE4m3Max);
}

// four codes; inv = 0 is a block of codes 0 (its values may be infinite or NaN)
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float inv) {
    const float2 scale = make_float2(inv, inv), x = __fmul2_rn(make_float2(a, b), scale), y = __fmul2_rn(make_float2(c, d), scale);
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x.y), "f"(x.x));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y.y), "f"(y.x));
    return inv == 0.f ? 0u : (uint32_t)lo | (uint32_t)hi << 16;
}

#endif  // __CUDACC__

}  // namespace moe
