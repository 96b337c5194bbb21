// C ABI of the training operators (declared in include/moe.h): argument checks and launches.
#include <cmath>

#include "moe_internal.cuh"
#include "train.cuh"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// a device array that has to be there
bool need(const void* p, size_t a) { return p && aligned(p, a); }
// one that may be left out
bool may(const void* p, size_t a) { return aligned(p, a); }

bool dtype_ok(int32_t t) { return t == MOE_OUT_F32 || t == MOE_OUT_BF16; }

// Makes the plan's device current for the duration of a call.
struct DeviceScope {
    int prev = -1, dev;
    bool ok;
    explicit DeviceScope(int d) : dev(d) {
        ok = cudaGetDevice(&prev) == cudaSuccess && (prev == dev || cudaSetDevice(dev) == cudaSuccess);
    }
    ~DeviceScope() {
        if (prev >= 0 && prev != dev) cudaSetDevice(prev);
    }
};

moe_status_t launched(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    cudaGetLastError();
    return MOE_ERR_CUDA;
}

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

void* split_area(const PlanView& v, void* workspace) {
    return v.split_off ? static_cast<uint8_t*>(workspace) + v.split_off : nullptr;
}

}  // namespace

extern "C" {

moe_status_t moe_backward_scratch(moe_plan_t plan, size_t* bytes) {
    PlanView v;
    if (!bytes || !plan_view(plan, &v)) return MOE_ERR_INVALID_ARG;
    *bytes = layernorm_backward_scratch_bytes(v.T, v.d, v.sm_count);
    return MOE_OK;
}

moe_status_t moe_layernorm(moe_plan_t plan, const void* x, int32_t x_dtype, const float* gamma, const float* beta,
                           float eps, uint16_t* y, float* mean, float* rstd, void* stream) {
    PlanView v;
    if (!plan_view(plan, &v) || !dtype_ok(x_dtype) || !(eps > 0.f) || std::isinf(eps)) return MOE_ERR_INVALID_ARG;
    if (v.T == 0) return MOE_OK;
    if (!need(x, 16) || !need(y, 16) || !may(gamma, 16) || !may(beta, 16) || !may(mean, 4) || !may(rstd, 4))
        return MOE_ERR_INVALID_ARG;
    DeviceScope scope(v.device);
    if (!scope.ok) return MOE_ERR_CUDA;
    LayernormArgs a{x, x_dtype == MOE_OUT_BF16, gamma, beta, eps, y, mean, rstd, v.T, v.d};
    return launched(launch_layernorm(a, v.sm_count, as_stream(stream)));
}

moe_status_t moe_layernorm_backward(moe_plan_t plan, const void* dy, int32_t dy_dtype, const void* x, int32_t x_dtype,
                                    const float* gamma, const float* mean, const float* rstd, const void* dres,
                                    void* dx, float* dgamma, float* dbeta, void* scratch, void* stream) {
    PlanView v;
    if (!plan_view(plan, &v) || !dtype_ok(dy_dtype) || !dtype_ok(x_dtype)) return MOE_ERR_INVALID_ARG;
    if (!may(dgamma, 16) || !may(dbeta, 16)) return MOE_ERR_INVALID_ARG;
    if ((dgamma || dbeta) && !need(scratch, 256)) return MOE_ERR_WORKSPACE;
    cudaStream_t s = as_stream(stream);
    if (v.T == 0) {
        DeviceScope scope(v.device);
        if (!scope.ok) return MOE_ERR_CUDA;
        cudaError_t e = cudaSuccess;
        if (dgamma) e = cudaMemsetAsync(dgamma, 0, sizeof(float) * v.d, s);
        if (e == cudaSuccess && dbeta) e = cudaMemsetAsync(dbeta, 0, sizeof(float) * v.d, s);
        return launched(e);
    }
    if (!need(dy, 16) || !need(x, 16) || !may(gamma, 16) || !need(mean, 4) || !need(rstd, 4) || !may(dres, 16) ||
        !need(dx, 16))
        return MOE_ERR_INVALID_ARG;
    DeviceScope scope(v.device);
    if (!scope.ok) return MOE_ERR_CUDA;
    LayernormBackwardArgs a{dy, dy_dtype == MOE_OUT_BF16, x, x_dtype == MOE_OUT_BF16, gamma, mean, rstd, dres, dx,
                            dgamma, dbeta, static_cast<float*>(scratch), v.T, v.d, v.device};
    return launched(launch_layernorm_backward(a, v.sm_count, s));
}

moe_status_t moe_swiglu_checkpoint(moe_plan_t plan, const void* GU, uint16_t* H, int8_t* codes, float* scales,
                                   void* stream) {
    PlanView v;
    if (!plan_view(plan, &v)) return MOE_ERR_INVALID_ARG;
    if (v.S == 0) return MOE_OK;
    if (!need(GU, 16) || !may(H, 16) || !need(codes, 16) || !need(scales, 4)) return MOE_ERR_INVALID_ARG;
    DeviceScope scope(v.device);
    if (!scope.ok) return MOE_ERR_CUDA;
    SwigluCkptArgs a{GU, v.out_bf16, H, codes, scales, v.S, v.N / 2};
    return launched(launch_swiglu_checkpoint(a, v.sm_count, as_stream(stream)));
}

moe_status_t moe_swiglu_checkpoint_backward(moe_plan_t plan, const void* dH, int32_t dh_dtype, const int8_t* codes,
                                            const float* scales, uint16_t* H, uint16_t* dGU, void* stream) {
    PlanView v;
    if (!plan_view(plan, &v) || !dtype_ok(dh_dtype)) return MOE_ERR_INVALID_ARG;
    if (v.S == 0) return MOE_OK;
    if (!need(dH, 16) || !need(codes, 16) || !need(scales, 4) || !may(H, 16) || !need(dGU, 16))
        return MOE_ERR_INVALID_ARG;
    DeviceScope scope(v.device);
    if (!scope.ok) return MOE_ERR_CUDA;
    SwigluCkptBackwardArgs a{dH, dh_dtype == MOE_OUT_BF16, codes, scales, H, dGU, v.S, v.N / 2};
    return launched(launch_swiglu_checkpoint_backward(a, v.sm_count, as_stream(stream)));
}

moe_status_t moe_combine_backward(moe_plan_t plan, const void* dout, int32_t dout_dtype, const void* Y,
                                  const float* topk_w, const int32_t* dest, uint16_t* dY, float* dtopk_w,
                                  void* stream) {
    PlanView v;
    if (!plan_view(plan, &v) || !dtype_ok(dout_dtype)) return MOE_ERR_INVALID_ARG;
    if (v.S == 0) return MOE_OK;
    if (!need(dout, 16) || !need(Y, 16) || !need(topk_w, 4) || !need(dest, 4) || !need(dY, 16) || !need(dtopk_w, 4))
        return MOE_ERR_INVALID_ARG;
    DeviceScope scope(v.device);
    if (!scope.ok) return MOE_ERR_CUDA;
    CombineBackwardArgs a{dout, dout_dtype == MOE_OUT_BF16, Y, v.out_bf16, topk_w, dest, dY, dtopk_w,
                          v.T, v.k, v.N, v.S};
    return launched(launch_combine_backward(a, v.sm_count, as_stream(stream)));
}

moe_status_t moe_grouped_gemm_dgrad(moe_plan_t plan, const uint16_t* dY, const int32_t* offsets, const uint16_t* W,
                                    void* dA, int32_t da_dtype, void* workspace, int32_t* dev_status, void* stream) {
    PlanView v;
    if (!plan_view(plan, &v) || !dtype_ok(da_dtype) || !need(dev_status, 4)) return MOE_ERR_INVALID_ARG;
    if (!need(workspace, 256)) return MOE_ERR_WORKSPACE;
    if (v.S == 0) return MOE_OK;
    if (!need(dY, 16) || !need(offsets, 4) || !need(W, 16) || !need(dA, 16)) return MOE_ERR_INVALID_ARG;
    DeviceScope scope(v.device);
    if (!scope.ok) return MOE_ERR_CUDA;
    GroupedGradArgs a{nullptr, dY, W, offsets, dA, da_dtype == MOE_OUT_BF16, 0, dev_status,
                      static_cast<uint32_t*>(workspace), split_area(v, workspace), v.timeout_ns, (int)v.S, v.d, v.E, v.N};
    return launched(launch_grouped_dgrad(a, v.device, v.sm_count, as_stream(stream)));
}

moe_status_t moe_grouped_gemm_wgrad(moe_plan_t plan, const uint16_t* A, const uint16_t* dY, const int32_t* offsets,
                                    void* dW, int32_t dw_dtype, int32_t accumulate, void* workspace,
                                    int32_t* dev_status, void* stream) {
    PlanView v;
    if (!plan_view(plan, &v) || !dtype_ok(dw_dtype) || !need(dev_status, 4) || (accumulate != 0 && accumulate != 1))
        return MOE_ERR_INVALID_ARG;
    if (accumulate && dw_dtype != MOE_OUT_F32) return MOE_ERR_UNSUPPORTED;  // gradients are summed in fp32
    if (!need(workspace, 256)) return MOE_ERR_WORKSPACE;
    if (!need(dW, 16)) return MOE_ERR_INVALID_ARG;
    DeviceScope scope(v.device);
    if (!scope.ok) return MOE_ERR_CUDA;
    cudaStream_t s = as_stream(stream);
    if (v.S == 0) {  // no rows: the sums are zero
        const size_t bytes = (size_t)v.E * v.d * v.N * (dw_dtype == MOE_OUT_BF16 ? 2 : 4);
        return accumulate ? MOE_OK : launched(cudaMemsetAsync(dW, 0, bytes, s));
    }
    if (!need(A, 16) || !need(dY, 16) || !need(offsets, 4)) return MOE_ERR_INVALID_ARG;
    GroupedGradArgs a{A, dY, nullptr, offsets, dW, dw_dtype == MOE_OUT_BF16, accumulate, dev_status,
                      static_cast<uint32_t*>(workspace), split_area(v, workspace), v.timeout_ns, (int)v.S, v.d, v.E, v.N};
    return launched(launch_grouped_wgrad(a, v.device, v.sm_count, s));
}

}  // extern "C"
