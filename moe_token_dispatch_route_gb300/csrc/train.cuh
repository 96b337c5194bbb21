// Declarations of the training operators (layer norm, the SwiGLU activation with its 8-bit
// checkpoint, the gradients of the grouped product and of the combine): launch parameter
// blocks and the plan fields their entry points need.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

// What the entry points in train_api.cu need of a plan.
struct PlanView {
    int T, d, E, k, N;
    long long S;
    int out_bf16;     // element type of the plan's Y
    int device, sm_count;
    long long timeout_ns;
    size_t split_off;  // offset in the workspace of the area for split reductions; 0: none
};
bool plan_view(moe_plan_t plan, PlanView* v);

struct LayernormArgs {
    const void* x;       // [T][d], fp32 or bf16
    int x_bf16;
    const float* gamma;  // [d] or null (1)
    const float* beta;   // [d] or null (0)
    float eps;
    uint16_t* y;         // bf16 [T][d]
    float* mean;         // [T] or null
    float* rstd;         // [T] or null
    int T, d;
};
cudaError_t launch_layernorm(const LayernormArgs& a, int sm_count, cudaStream_t stream);

struct LayernormBackwardArgs {
    const void* dy;      // [T][d], fp32 or bf16
    int dy_bf16;
    const void* x;       // [T][d], fp32 or bf16
    int x_bf16;          // also the type of dres and dx
    const float* gamma;  // [d] or null (1)
    const float* mean;   // [T]
    const float* rstd;   // [T]
    const void* dres;    // [T][d] or null
    void* dx;            // [T][d]
    float* dgamma;       // [d] or null
    float* dbeta;        // [d] or null
    float* partial;      // scratch: partial sums of dgamma and dbeta
    int T, d;
    int device;
};
size_t layernorm_backward_scratch_bytes(int T, int d, int sm_count);
cudaError_t launch_layernorm_backward(const LayernormBackwardArgs& a, int sm_count, cudaStream_t stream);

constexpr int kCkptBlock = 128;  // columns that share one scale
__host__ __device__ constexpr int ckpt_blocks(int F) { return (F + kCkptBlock - 1) / kCkptBlock; }

struct SwigluCkptArgs {
    const void* GU;   // [S][2F], fp32 or bf16: gate columns, then up columns
    int gu_bf16;
    uint16_t* H;      // bf16 [S][F] or null
    int8_t* codes;    // [S][2F]
    float* scales;    // [S][2 * ckpt_blocks(F)]
    long long S;
    int F;
};
cudaError_t launch_swiglu_checkpoint(const SwigluCkptArgs& a, int sm_count, cudaStream_t stream);

struct SwigluCkptBackwardArgs {
    const void* dH;   // [S][F], fp32 or bf16
    int dh_bf16;
    const int8_t* codes;
    const float* scales;
    uint16_t* H;      // bf16 [S][F] or null: the activation again, from the checkpoint
    uint16_t* dGU;    // bf16 [S][2F]
    long long S;
    int F;
};
cudaError_t launch_swiglu_checkpoint_backward(const SwigluCkptBackwardArgs& a, int sm_count, cudaStream_t stream);

struct CombineBackwardArgs {
    const void* dout;     // [T][N], fp32 or bf16
    int dout_bf16;
    const void* Y;        // [S][N], fp32 or bf16
    int y_bf16;
    const float* w;       // [T][k]
    const int32_t* dest;  // [T*k]
    uint16_t* dY;         // bf16 [S][N]
    float* dw;            // [T][k]
    int T, k, N;
    long long S;
};
cudaError_t launch_combine_backward(const CombineBackwardArgs& a, int sm_count, cudaStream_t stream);

struct GroupedGradArgs {
    const uint16_t* A;       // bf16 [S][d]   (weight gradient)
    const uint16_t* dY;      // bf16 [S][N]
    const uint16_t* W;       // bf16 [E][d][N] (input gradient)
    const int32_t* offsets;  // [E+1]
    void* out;               // dA [S][d] or dW [E][d][N]
    int out_bf16;
    int accumulate;          // weight gradient, fp32: out += instead of out =
    int32_t* status;
    uint32_t* hdr;           // workspace header
    void* split;             // workspace of split reductions, or null
    long long timeout_ns;
    int S, d, E, N;
};
cudaError_t launch_grouped_dgrad(const GroupedGradArgs& a, int device, int sm_count, cudaStream_t stream);
cudaError_t launch_grouped_wgrad(const GroupedGradArgs& a, int device, int sm_count, cudaStream_t stream);
size_t grouped_grad_split_bytes(long long S, int d, int E, int N, int sm_count);

// bf16 [rows][cols], 128-byte swizzle, and the same as 64-column chunks loaded two at a time
// (false where cols % 64 != 0)
bool map_bf16_2d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint32_t box_cols,
                 uint32_t box_rows);
bool map_bf16_chunks(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows);

#if defined(__CUDACC__)

// Launches a kernel that may start while the one before it in the stream is ending: it calls
// wait_for_kernel_before() itself, before it reads or writes memory.  2 us less from kernel to kernel
// (layer norm gradient, 8192 x 4096 bf16: 53.8 -> 51.6 us).
template <class Kernel, class... Args>
cudaError_t launch_after(Kernel kernel, unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// fp32 -> bf16, nearest even, two values packed
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// eight consecutive elements [i, i+8) of an fp32 or bf16 array, widened to fp32
// (i a multiple of 8 elements from a 16-byte aligned base)
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, size_t i, float (&v)[8]) {
    if constexpr (BF16) {
        const uint4 h = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i));
        const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16_lo(w[j]);
            v[2 * j + 1] = bf16_hi(w[j]);
        }
    } else {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
        const float4 a = __ldcs(p), b = __ldcs(p + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* base, size_t i, const float (&v)[8]) {
    if constexpr (BF16) {
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i),
               make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])));
    } else {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
        __stcs(p, make_float4(v[0], v[1], v[2], v[3]));
        __stcs(p + 1, make_float4(v[4], v[5], v[6], v[7]));
    }
}

#endif  // __CUDACC__

}  // namespace moe
