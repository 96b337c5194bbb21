// C ABI of the 8-bit forward operators and of the router's losses (declared in include/moe.h): argument checks and launches.
#include <cmath>

#include "moe_internal.cuh"
#include "serve.cuh"

using namespace moe;

namespace moe {
bool plan_route_shape(moe_plan_t plan, int* T, int* E, int* k, int* route_blocks, int* device, int* route_flags);
}

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool need(const void* p, size_t a) { return p && aligned(p, a); }  // a device array that has to be there
bool may(const void* p, size_t a) { return aligned(p, a); }        // one that may be left out
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

moe_status_t grouped_fp8(moe_plan_t plan, const uint8_t* A, const float* A_scales, const int32_t* perm, const int32_t* offsets,
                         const uint8_t* W, const float* W_scales, bool glu, void* out, float* H_scales, void* workspace,
                         int32_t* dev_status, void* stream) {
    PlanView v;
    if (!plan_view(plan, &v) || !need(dev_status, 4)) return MOE_ERR_INVALID_ARG;
    if (glu && v.N % 32 != 0) return MOE_ERR_UNSUPPORTED;  // H's rows are read back as operands: whole 16 bytes
    if (!need(workspace, 256)) return MOE_ERR_WORKSPACE;
    if (v.S == 0) return MOE_OK;
    if (!need(A, 16) || !need(A_scales, 4) || !may(perm, 4) || !need(offsets, 4) || !need(W, 16) || !need(W_scales, 4) ||
        !need(out, 16) || (glu && !need(H_scales, 4)))
        return MOE_ERR_INVALID_ARG;
    DeviceScope scope(v.device);
    if (!scope.ok) return MOE_ERR_CUDA;
    GroupedFp8Args a{};
    a.A = A;
    a.A_scales = A_scales;
    a.perm = perm;
    a.offsets = offsets;
    a.W = W;
    a.W_scales = W_scales;
    a.glu = glu;
    a.Y = glu ? nullptr : out;
    a.out_bf16 = v.out_bf16;
    a.H = glu ? static_cast<uint8_t*>(out) : nullptr;
    a.H_scales = H_scales;
    a.status = dev_status;
    a.timeout_ns = v.timeout_ns;
    a.T = v.T;
    a.S = (int)v.S;
    a.d = v.d;
    a.E = v.E;
    a.k = v.k;
    a.N = v.N;
    return launched(launch_grouped_fp8(a, v.device, v.sm_count, as_stream(stream)));
}

// The fields that both router calls share; false: an argument is invalid.
bool router_args(moe_plan_t plan, const PlanView& v, int32_t seq_len, float balance, float z, RouterLossArgs* a) {
    int T, E, k, blocks, device, flags;
    if (seq_len < 0 || !std::isfinite(balance) || !std::isfinite(z) || !plan_route_shape(plan, &T, &E, &k, &blocks, &device, &flags))
        return false;
    a->seq_len = seq_len == 0 || seq_len > v.T ? v.T : seq_len;
    a->groups = v.T == 0 ? 1 : (int)(((long long)v.T + a->seq_len - 1) / a->seq_len);
    a->balance = balance;
    a->z = z;
    a->renorm = (flags & MOE_ROUTE_RENORM) ? 1 : 0;
    a->sigmoid = (flags & MOE_ROUTE_SIGMOID) ? 1 : 0;
    a->T = v.T;
    a->E = v.E;
    a->k = v.k;
    return true;
}

}  // namespace

extern "C" {

moe_status_t moe_rmsnorm(moe_plan_t plan, const void* x, int32_t x_dtype, const void* res, int32_t h_dtype, const float* gamma,
                         float eps, void* h, uint16_t* y, uint8_t* codes, float* scales, float* rstd, void* stream) {
    PlanView v;
    if (!plan_view(plan, &v) || !dtype_ok(x_dtype) || !dtype_ok(h_dtype) || !(eps > 0.f) || std::isinf(eps))
        return MOE_ERR_INVALID_ARG;
    if (v.T == 0) return MOE_OK;  // (arrays of no rows may have no address)
    if (!res && h_dtype != x_dtype) return MOE_ERR_INVALID_ARG;  // without a residual h is x
    if (!need(x, 16) || !may(res, 16) || !may(h, 16) || (res && !h) || !may(gamma, 16) || !may(y, 16) || !may(codes, 16) ||
        !may(scales, 4) || !may(rstd, 4) || (codes != nullptr) != (scales != nullptr) || (!y && !codes))
        return MOE_ERR_INVALID_ARG;
    DeviceScope scope(v.device);
    if (!scope.ok) return MOE_ERR_CUDA;
    RmsnormArgs a{x, x_dtype == MOE_OUT_BF16, res, h, h_dtype == MOE_OUT_BF16, gamma, eps, y, codes, scales, rstd, v.T, v.d};
    return launched(launch_rmsnorm(a, v.sm_count, as_stream(stream)));
}

moe_status_t moe_rmsnorm_backward(moe_plan_t plan, const void* dy, int32_t dy_dtype, const void* h, int32_t h_dtype,
                                  const float* gamma, const float* rstd, const void* dres, void* dx, float* dgamma, void* scratch,
                                  void* stream) {
    PlanView v;
    if (!plan_view(plan, &v) || !dtype_ok(dy_dtype) || !dtype_ok(h_dtype) || !may(dgamma, 16)) return MOE_ERR_INVALID_ARG;
    if (dgamma && !need(scratch, 256)) return MOE_ERR_WORKSPACE;
    cudaStream_t s = as_stream(stream);
    if (v.T == 0) {
        DeviceScope scope(v.device);
        if (!scope.ok) return MOE_ERR_CUDA;
        return dgamma ? launched(cudaMemsetAsync(dgamma, 0, sizeof(float) * v.d, s)) : MOE_OK;
    }
    if (!need(dy, 16) || !need(h, 16) || !may(gamma, 16) || !need(rstd, 4) || !may(dres, 16) || !need(dx, 16))
        return MOE_ERR_INVALID_ARG;
    DeviceScope scope(v.device);
    if (!scope.ok) return MOE_ERR_CUDA;
    // the layer norm's gradient of rows whose mean is taken as 0
    LayernormBackwardArgs a{dy, dy_dtype == MOE_OUT_BF16, h, h_dtype == MOE_OUT_BF16, gamma, nullptr, rstd, dres, dx, dgamma,
                            nullptr, static_cast<float*>(scratch), v.T, v.d, v.device};
    return launched(launch_layernorm_backward(a, v.sm_count, s));
}

moe_status_t moe_quantize_weights(moe_plan_t plan, const uint16_t* W, int32_t halves, uint8_t* codes, float* scales, void* stream) {
    PlanView v;
    if (!plan_view(plan, &v) || (halves != 1 && halves != 2)) return MOE_ERR_INVALID_ARG;
    if (halves == 2 && v.N % 32 != 0) return MOE_ERR_UNSUPPORTED;
    if (!need(W, 16) || !need(codes, 16) || !need(scales, 4)) return MOE_ERR_INVALID_ARG;
    DeviceScope scope(v.device);
    if (!scope.ok) return MOE_ERR_CUDA;
    QuantizeWeightsArgs a{W, codes, scales, v.E, v.d, v.N, halves};
    return launched(launch_quantize_weights(a, v.sm_count, as_stream(stream)));
}

moe_status_t moe_grouped_gemm_fp8(moe_plan_t plan, const uint8_t* A, const float* A_scales, const int32_t* perm,
                                  const int32_t* offsets, const uint8_t* W, const float* W_scales, void* Y, void* workspace,
                                  int32_t* dev_status, void* stream) {
    return grouped_fp8(plan, A, A_scales, perm, offsets, W, W_scales, false, Y, nullptr, workspace, dev_status, stream);
}

moe_status_t moe_grouped_gemm_fp8_swiglu(moe_plan_t plan, const uint8_t* A, const float* A_scales, const int32_t* perm,
                                         const int32_t* offsets, const uint8_t* W1, const float* W1_scales, uint8_t* H,
                                         float* H_scales, void* workspace, int32_t* dev_status, void* stream) {
    return grouped_fp8(plan, A, A_scales, perm, offsets, W1, W1_scales, true, H, H_scales, workspace, dev_status, stream);
}

moe_status_t moe_balance_scratch(moe_plan_t plan, int32_t seq_len, size_t* bytes) {
    PlanView v;
    RouterLossArgs a{};
    if (!bytes || !plan_view(plan, &v) || !router_args(plan, v, seq_len, 0.f, 0.f, &a)) return MOE_ERR_INVALID_ARG;
    const size_t n = v.T == 0 ? 0 : balance_scratch_bytes(v.T, v.E, a.seq_len, v.sm_count);
    *bytes = n < 256 ? 256 : n;
    return MOE_OK;
}

moe_status_t moe_balance_loss(moe_plan_t plan, const float* logits, const int32_t* topk_idx, const uint8_t* mask, int32_t seq_len,
                              float balance, float z, float* loss, int32_t* load, int32_t* tokens, void* scratch, void* stream) {
    PlanView v;
    RouterLossArgs a{};
    if (!plan_view(plan, &v) || !router_args(plan, v, seq_len, balance, z, &a)) return MOE_ERR_INVALID_ARG;
    if (!need(scratch, 256)) return MOE_ERR_WORKSPACE;
    if (!need(loss, 4) || !need(load, 4) || !need(tokens, 4)) return MOE_ERR_INVALID_ARG;
    if (v.T > 0 && (!need(logits, 4) || !need(topk_idx, 4))) return MOE_ERR_INVALID_ARG;
    DeviceScope scope(v.device);
    if (!scope.ok) return MOE_ERR_CUDA;
    cudaStream_t s = as_stream(stream);
    if (v.T == 0) {
        cudaError_t e = cudaMemsetAsync(loss, 0, 2 * sizeof(float), s);
        if (e == cudaSuccess) e = cudaMemsetAsync(load, 0, sizeof(int32_t) * v.E, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(tokens, 0, 2 * sizeof(int32_t), s);
        return launched(e);
    }
    a.logits = logits;
    a.topk_idx = topk_idx;
    a.mask = mask;
    a.loss = loss;
    a.load = load;
    a.tokens = tokens;
    a.scratch = scratch;
    return launched(launch_balance_loss(a, v.sm_count, s));
}

moe_status_t moe_router_backward(moe_plan_t plan, const float* logits, const int32_t* topk_idx, const float* dtopk_w,
                                 const uint8_t* mask, int32_t seq_len, float balance, float z, const int32_t* load,
                                 const int32_t* tokens, float* dlogits, void* stream) {
    PlanView v;
    RouterLossArgs a{};
    if (!plan_view(plan, &v) || !router_args(plan, v, seq_len, balance, z, &a)) return MOE_ERR_INVALID_ARG;
    if (v.T == 0) return MOE_OK;
    if (!need(logits, 4) || !may(dtopk_w, 4) || (dtopk_w && !need(topk_idx, 4)) || !need(dlogits, 4) ||
        (balance != 0.f && !need(load, 4)) || ((balance != 0.f || z != 0.f) && !need(tokens, 4)))
        return MOE_ERR_INVALID_ARG;
    DeviceScope scope(v.device);
    if (!scope.ok) return MOE_ERR_CUDA;
    a.logits = logits;
    a.topk_idx = topk_idx;
    a.dtopk_w = dtopk_w;
    a.mask = mask;
    a.load = const_cast<int32_t*>(load);
    a.tokens = const_cast<int32_t*>(tokens);
    a.dlogits = dlogits;
    return launched(launch_router_backward(a, v.sm_count, as_stream(stream)));
}

}  // extern "C"
