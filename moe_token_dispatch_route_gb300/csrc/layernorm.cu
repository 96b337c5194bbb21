// Layer norm of token rows and its gradient.
//   mean = sum x / d,  rstd = 1 / sqrt(sum (x - mean)^2 / d + eps),
//   y = (x - mean) rstd gamma + beta
// and, with xh = (x - mean) rstd and v = dy gamma,
//   dx = rstd (v - sum v / d - xh (sum v xh) / d) + dres,
//   dgamma = sum_t dy xh,  dbeta = sum_t dy.
// All sums are fp32.  Both directions are bound by HBM: each input is read once and stays in
// registers between the sums over a row and the row's result.  Wider rows do not fit: above 32768 columns the forward
// kernel reads a row three times, and above 16384 the backward pass reads x and dy twice for dx and once more
// for dgamma and dbeta (the repeats within a row come from L2).
//
// A row is held by TPR threads (a power of two from 8 to 1024), VPT vectors of 8 columns each, so
// that the sums are one shuffle tree and, above a warp, one exchange through shared memory.  The
// backward kernel also keeps dgamma and dbeta of its columns, over all the rows of
// its CTA, in registers (shared memory for d > 8192); the CTAs' partial sums are added by a second
// kernel in a fixed order.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "train.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

// Eight columns as they are in memory.
template <bool BF16>
struct Raw {
    uint4 a;
    __device__ void load(const void* base, size_t i) { a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i)); }
    __device__ void take(const uint8_t* row, int c) { a = *reinterpret_cast<const uint4*>(row + c * 2); }  // from shared memory
    __device__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ uint32_t bits() const { return a.x | a.y | a.z | a.w; }
    __device__ float get(int j) const {
        const uint32_t w = j < 2 ? a.x : j < 4 ? a.y : j < 6 ? a.z : a.w;
        return j & 1 ? bf16_hi(w) : bf16_lo(w);
    }
};
template <>
struct Raw<false> {
    float4 a, b;
    __device__ void load(const void* base, size_t i) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
        a = __ldcs(p);
        b = __ldcs(p + 1);
    }
    __device__ void take(const uint8_t* row, int c) {
        a = *reinterpret_cast<const float4*>(row + c * 4);
        b = *reinterpret_cast<const float4*>(row + c * 4 + 16);
    }
    __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ uint32_t bits() const {
        return __float_as_uint(a.x) | __float_as_uint(a.y) | __float_as_uint(a.z) | __float_as_uint(a.w) |
               __float_as_uint(b.x) | __float_as_uint(b.y) | __float_as_uint(b.z) | __float_as_uint(b.w);
    }
    __device__ float get(int j) const {
        return j == 0 ? a.x : j == 1 ? a.y : j == 2 ? a.z : j == 3 ? a.w : j == 4 ? b.x : j == 5 ? b.y : j == 6 ? b.z : b.w;
    }
};

__device__ __forceinline__ void weights8(const float* w, int c, float none, float (&v)[8]) {
    if (w) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(w + c)), b = __ldg(reinterpret_cast<const float4*>(w + c) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = none;
    }
}

// CTA of a row group: at least `least` threads, whole rows.
__host__ __device__ constexpr int cta_threads(int tpr, int least) { return tpr > least ? tpr : least; }

// Sums of N values over the TPR threads of a row, the same bits in each of them.  `red` is used
// by one call at a time: two calls in a row need a CTA barrier or another array between them.
template <int TPR, int N, int CTA, class Barrier>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[CTA / 32], Barrier barrier) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], o);
    if constexpr (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        const int warp = threadIdx.x >> 5, first = warp / kWarps * kWarps;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[i][warp] = v[i];
        barrier();
        // a lane a warp, not every lane all warps: those loads alone were 15% of a row of 1024 threads (8192 x 8192
        // bf16, backward: 127 us, 109 so)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = red[i][first + (threadIdx.x & 31) % kWarps];
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], o);
    }
}

struct CtaBarrier {
    __device__ void operator()() const { __syncthreads(); }
};

// The same, passed once the words that `bits` is made of are in registers: a load of shared memory queues behind
// global stores, and a barrier alone does not wait for it to be done.
struct ReadBarrier {
    uint32_t bits;
    __device__ void operator()() const { __syncthreads_or(bits == 1u); }
};

// ------------------------------------------------------------------ forward

// Resident CTAs that the registers are cut for: 640 (bf16) or 512 threads an SM with two rows each,
// 1024 with one.
__host__ __device__ constexpr int forward_ctas(int cta, bool xb, int rows) {
    const int threads = rows == 1 ? 1024 : xb ? 640 : 512;
    return threads > cta ? threads / cta : 1;
}

// R rows at a time: the weights, 8 bytes a column from L1 where a row has 2 or 4, are read once for R
// rows, and R rows share each barrier (8192 x 4096: bf16 30 us with one row, 27 with two; fp32 36 and 33; launched while
// the kernel before ends 24.5, 5.5 TB/s, and 31).
template <bool XB, int TPR, int VPT, int R>
__global__ void __launch_bounds__(cta_threads(TPR, 128), forward_ctas(cta_threads(TPR, 128), XB, R)) layernorm_kernel(const LayernormArgs a) {
    wait_for_kernel_before();
    constexpr int kCta = cta_threads(TPR, 128), kRows = kCta / TPR * R;
    __shared__ float red_m[R][kCta / 32], red_v[R][kCta / 32];
    const int sub = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const float inv_d = 1.f / (float)a.d;
    for (long long t0 = (long long)blockIdx.x * kRows; t0 < a.T; t0 += (long long)gridDim.x * kRows) {
        const long long t = t0 + group * R;
        Raw<XB> x[R][VPT];
        float mean[R], rstd[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (sub + i * TPR) * 8;
                if (c < a.d && t + r < a.T) x[r][i].load(a.x, (size_t)(t + r) * a.d + c);
                else x[r][i].zero();
            }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) mean[r] += x[r][i].get(j);
        }
        row_sum<TPR, R, kCta>(mean, red_m, CtaBarrier());
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] *= inv_d;
            rstd[r] = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if ((sub + i * TPR) * 8 < a.d) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        rstd[r] = fmaf(x[r][i].get(j) - mean[r], x[r][i].get(j) - mean[r], rstd[r]);
                }
            }
        }
        row_sum<TPR, R, kCta>(rstd, red_v, CtaBarrier());
#pragma unroll
        for (int r = 0; r < R; ++r) rstd[r] = 1.f / sqrtf(rstd[r] * inv_d + a.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (sub + i * TPR) * 8;
            if (c >= a.d) continue;
            float g[8], b[8], y[8];
            weights8(a.gamma, c, 1.f, g);
            weights8(a.beta, c, 0.f, b);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (t + r >= a.T) continue;
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = fmaf((x[r][i].get(j) - mean[r]) * rstd[r], g[j], b[j]);
                store8<true>(a.y, (size_t)(t + r) * a.d + c, y);
            }
        }
        if (sub == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (t + r >= a.T) continue;
                if (a.mean) a.mean[t + r] = mean[r];
                if (a.rstd) a.rstd[t + r] = rstd[r];
            }
    }
}

// d > 32768: the row is read three times (from L2 after the first)
constexpr int kWide = 1024;
template <bool XB>
__global__ void __launch_bounds__(kWide) layernorm_wide_kernel(const LayernormArgs a) {
    __shared__ float red_m[1][kWide / 32], red_v[1][kWide / 32];
    const float inv_d = 1.f / (float)a.d;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t row = (size_t)t * a.d;
        float s[1] = {0.f}, q[1] = {0.f};
        for (int c = threadIdx.x * 8; c < a.d; c += kWide * 8) {
            float v[8];
            load8<XB>(a.x, row + c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += v[j];
        }
        row_sum<kWide, 1, kWide>(s, red_m, CtaBarrier());
        const float mean = s[0] * inv_d;
        for (int c = threadIdx.x * 8; c < a.d; c += kWide * 8) {
            float v[8];
            load8<XB>(a.x, row + c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) q[0] = fmaf(v[j] - mean, v[j] - mean, q[0]);
        }
        row_sum<kWide, 1, kWide>(q, red_v, CtaBarrier());
        const float rstd = 1.f / sqrtf(q[0] * inv_d + a.eps);
        for (int c = threadIdx.x * 8; c < a.d; c += kWide * 8) {
            float v[8], g[8], b[8];
            load8<XB>(a.x, row + c, v);
            weights8(a.gamma, c, 1.f, g);
            weights8(a.beta, c, 0.f, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = fmaf((v[j] - mean) * rstd, g[j], b[j]);
            store8<true>(a.y, row + c, v);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[t] = mean;
            if (a.rstd) a.rstd[t] = rstd;
        }
    }
}

// ------------------------------------------------------------------ backward

// Rows of at most 128 threads (d <= 1024).  A thread has one vector of 8 columns, so its sums and the
// row's xh and v are 40 registers and 1024 threads an SM fit: it is their number that hides the
// round trips of a row.
__host__ __device__ constexpr int back_cta(int tpr) { return tpr == 64 ? 512 : 1024; }

template <int TPR>
struct Back {
    // one CTA an SM, whose rows' sums are joined in shared memory before they are written (two CTAs for
    // 64 threads: there are 16 named barriers, one the CTA's); 32768 x 512, bf16 x and fp32 dy: 34 us
    // with CTAs of 256 threads, 31 with 1024
    static constexpr int kCta = back_cta(TPR);
    static constexpr int kRows = kCta / TPR;
    static constexpr int kCtasPerSm = 1024 / kCta;
    static constexpr int kCols = TPR * 8;
    static constexpr size_t kSmem = kRows > 1 ? (size_t)kRows * 2 * kCols * 4 : 0;  // at most 64 KB
};

// Barrier of the TPR threads of row group `group`.
template <int TPR, int CTA>
__device__ __forceinline__ void group_barrier(int group) {
    if constexpr (TPR == CTA) __syncthreads();
    else if constexpr (TPR > 32) asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
}

// Where a CTA's sums go: its partial sums [2][d], or the results themselves where it is the only one.
struct SumsOut {
    float *dgamma, *dbeta;
    __device__ explicit SumsOut(const LayernormBackwardArgs& a) {
        float* part = a.partial + (size_t)blockIdx.x * 2 * a.d;
        dgamma = gridDim.x == 1 ? a.dgamma : part;
        dbeta = gridDim.x == 1 ? a.dbeta : part + a.d;
    }
};

// A thread's sums of columns c .. c + 7.
__device__ __forceinline__ void write_sums(const float (&dg)[8], const float (&db)[8], int c, const SumsOut& out) {
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
        if (out.dgamma) *reinterpret_cast<float4*>(out.dgamma + c + j) = make_float4(dg[j], dg[j + 1], dg[j + 2], dg[j + 3]);
        if (out.dbeta) *reinterpret_cast<float4*>(out.dbeta + c + j) = make_float4(db[j], db[j + 1], db[j + 2], db[j + 3]);
    }
}

// The sums of a CTA's row groups, added in shared memory ([group][2][COLS]) in the groups' order.
template <int ROWS, int COLS, int CTA>
__device__ __forceinline__ void join_rows(float* joined, const float (&dg)[8], const float (&db)[8], int group, int c, int d, const SumsOut& out) {
    float* own = joined + group * 2 * COLS + c;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        own[j] = dg[j];
        own[COLS + j] = db[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * COLS; i += CTA) {
        const int col = i % COLS, half = i / COLS;
        float* to = half ? out.dbeta : out.dgamma;
        if (col >= d || !to) continue;
        float v = 0.f;
#pragma unroll
        for (int g = 0; g < ROWS; ++g) v += joined[g * 2 * COLS + i];
        to[col] = v;
    }
}

template <bool DYB, bool XB, int TPR>
__global__ void __launch_bounds__(Back<TPR>::kCta, Back<TPR>::kCtasPerSm) layernorm_backward_kernel(const LayernormBackwardArgs a) {
    using B = Back<TPR>;
    __shared__ float red[2][2][B::kCta / 32];
    extern __shared__ float joined[];  // [group][2][kCols]
    const int tid = threadIdx.x, sub = tid % TPR, group = tid / TPR, c = sub * 8;
    const float inv_d = 1.f / (float)a.d;
    const bool mine = c < a.d;  // this thread's columns exist
    wait_for_kernel_before();
    float dg[8], db[8], gamma[8];
    weights8(mine ? a.gamma : nullptr, c, 1.f, gamma);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[j] = db[j] = 0.f;
    const long long step = (long long)gridDim.x * B::kRows;
    long long t = (long long)blockIdx.x * B::kRows + group;
    int turn = 0;
    for (long long t0 = (long long)blockIdx.x * B::kRows; t0 < a.T; t0 += step, t += step, turn ^= 1) {
        const bool live = t < a.T && mine;
        const size_t at = live ? (size_t)t * a.d + c : 0;
        Raw<XB> x, res;
        Raw<DYB> dy;
        float mean = 0.f, rstd = 0.f;
        if (live) {
            x.load(a.x, at);
            dy.load(a.dy, at);
            mean = __ldg(a.mean + t);
            rstd = __ldg(a.rstd + t);
        } else {
            x.zero();
            dy.zero();
        }
        if (live && a.dres) res.load(a.dres, at);
        else res.zero();
        // xh and v = dy gamma stay in registers between the two halves
        float xh[8], v[8], s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float w = dy.get(j);
            xh[j] = (x.get(j) - mean) * rstd;
            v[j] = w * gamma[j];
            s[0] += v[j];
            s[1] = fmaf(v[j], xh[j], s[1]);
            dg[j] = fmaf(w, xh[j], dg[j]);
            db[j] += w;
        }
        // the two arrays of `red` alternate, so one barrier a row is enough
        row_sum<TPR, 2, B::kCta>(s, red[turn], [&] { group_barrier<TPR, B::kCta>(group); });
        if (!live) continue;
        const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = fmaf(rstd, fmaf(-xh[j], m2, v[j] - m1), res.get(j));
        store8<XB>(a.dx, at, v);
    }
    if (!a.dgamma && !a.dbeta) return;
    asm volatile("griddepcontrol.launch_dependents;");  // the joining kernel may start; it waits for this one's end
    join_rows<B::kRows, B::kCols, B::kCta>(joined, dg, db, group, c, a.d, SumsOut(a));
}

// 1024 < d <= 8192: a CTA holds one row, the same way, and its next rows are on their way in shared
// memory: one thread copies whole rows of x, dy and dres (cp.async.bulk, two rows ahead), so a row's
// round trip is behind the arithmetic of the rows before it.
// Measured, with the joining kernel, against the rows loaded into registers when they are needed: 8192 x 4096 bf16
// x and fp32 dy 66 -> 62 us, fp32 both 93 -> 86; 20000 x 992 the other way, 33 -> 43.  More rows ahead are slower: 8192 x
// 4096 bf16 54 us with two, 54.5 with three, 56 with four (fp32 dy 59 with two, 60 with three; launched while the kernel
// before ends 51.7 and 56.6, 5.9 TB/s).
template <bool DYB, bool XB, int TPR>
struct Ahead {
    static constexpr int kCta = TPR;
    static constexpr int kCtasPerSm = 1024 / kCta;
    static constexpr int kCols = TPR * 8;
    static constexpr int kXBytes = kCols * (XB ? 2 : 4), kDBytes = kCols * (DYB ? 2 : 4);
    static constexpr int kSlot = 2 * kXBytes + kDBytes;  // x, dy, dres of one row
    static constexpr int kStages = 2;
    static constexpr size_t kSmem = (size_t)kStages * kSlot;
};

__device__ __forceinline__ void copy_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// Bounded wait; a copy of memory that is there completes, so running out means a broken context.
__device__ __forceinline__ bool row_landed(uint32_t bar, uint32_t parity) {
    for (int i = 0; i < (1 << 22); ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        if (ok) return true;
    }
    return false;
}

template <bool DYB, bool XB, int TPR>
__global__ void __launch_bounds__(Ahead<DYB, XB, TPR>::kCta, Ahead<DYB, XB, TPR>::kCtasPerSm)
    layernorm_ahead_kernel(const LayernormBackwardArgs a) {
    using B = Ahead<DYB, XB, TPR>;
    __shared__ float red[2][2][B::kCta / 32];
    __shared__ uint64_t full[B::kStages];
    extern __shared__ __align__(128) uint8_t slots[];  // [stage]{x, dy, dres}
    const int c = threadIdx.x * 8;
    const float inv_d = 1.f / (float)a.d;
    const bool mine = c < a.d;  // this thread's columns exist
    const long long step = gridDim.x, first = blockIdx.x;
    const uint32_t slots_at = static_cast<uint32_t>(__cvta_generic_to_shared(slots));
    const uint32_t bars = static_cast<uint32_t>(__cvta_generic_to_shared(full));
    auto fetch = [&](long long t, int stage) {  // one thread
        if (t >= a.T) return;
        const uint32_t xb = (uint32_t)a.d * (XB ? 2 : 4), db = (uint32_t)a.d * (DYB ? 2 : 4);
        const uint32_t dst = slots_at + stage * B::kSlot, bar = bars + 8 * stage;
        const size_t row = (size_t)t * a.d;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"((a.dres ? 2 : 1) * xb + db) : "memory");
        copy_row(dst, static_cast<const uint8_t*>(a.x) + row * (XB ? 2 : 4), xb, bar);
        copy_row(dst + B::kXBytes, static_cast<const uint8_t*>(a.dy) + row * (DYB ? 2 : 4), db, bar);
        if (a.dres) copy_row(dst + B::kXBytes + B::kDBytes, static_cast<const uint8_t*>(a.dres) + row * (XB ? 2 : 4), xb, bar);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < B::kStages; ++s)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bars + 8 * s) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    wait_for_kernel_before();
    if (threadIdx.x == 0) {
        for (int s = 0; s < B::kStages; ++s) fetch(first + s * step, s);
    }
    float dg[8], db[8], gamma[8];
    weights8(mine ? a.gamma : nullptr, c, 1.f, gamma);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[j] = db[j] = 0.f;
    auto stats = [&](long long t) { return t < a.T ? make_float2(__ldg(a.mean + t), __ldg(a.rstd + t)) : make_float2(0.f, 0.f); };
    float2 next = stats(first);
    __syncthreads();
    int turn = 0, stage = 0;
    uint32_t phase = 0;
    bool landed = true;
    for (long long t = first; t < a.T; t += step, turn ^= 1) {
        float mean = next.x;
        const float rstd = next.y;
        next = stats(t + step);
        if (!row_landed(bars + 8 * stage, phase)) {
            landed = false;
            mean = __uint_as_float(0x7FC00000u);  // the row's result is NaN, not what was there before
        }
        // xh and v = dy gamma stay in registers between the two halves
        const uint8_t* slot = slots + stage * B::kSlot;
        float xh[8], v[8], s[2] = {0.f, 0.f};
        Raw<XB> res;
        res.zero();
        if (mine) {
            Raw<XB> x;
            Raw<DYB> dy;
            x.take(slot, c);
            dy.take(slot + B::kXBytes, c);
            if (a.dres) res.take(slot + B::kXBytes + B::kDBytes, c);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float w = dy.get(j);
                xh[j] = (x.get(j) - mean) * rstd;
                v[j] = w * gamma[j];
                s[0] += v[j];
                s[1] = fmaf(v[j], xh[j], s[1]);
                dg[j] = fmaf(w, xh[j], dg[j]);
                db[j] += w;
            }
        }
        // the two arrays of `red` alternate, so one barrier a row is enough; after it the CTA has
        // read the slot (the sums need all of x and dy)
        row_sum<TPR, 2, B::kCta>(s, red[turn], ReadBarrier{res.bits()});
        if (threadIdx.x == 0) fetch(t + B::kStages * step, stage);
        if (mine) {
            const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = fmaf(rstd, fmaf(-xh[j], m2, v[j] - m1), res.get(j));
            store8<XB>(a.dx, (size_t)t * a.d + c, v);
        }
        if (++stage == B::kStages) {
            stage = 0;
            phase ^= 1u;
        }
    }
    if (!landed)  // give copies that are late another chance to end before the CTA does
        for (int s = 0; s < B::kStages; ++s) row_landed(bars + 8 * s, phase);
    if (!a.dgamma && !a.dbeta) return;
    asm volatile("griddepcontrol.launch_dependents;");  // the joining kernel may start; it waits for this one's end
    if (mine) write_sums(dg, db, c, SumsOut(a));
}

// 8192 < d <= 16384: 1024 threads leave 64 registers each, so dgamma and dbeta are summed in shared
// memory (128 KB, which leaves no room for rows on their way) and the rows pass through registers.
constexpr int kTall = 1024;
constexpr size_t kTallSmem = (size_t)kTall * 2 * 8 * 2 * 4;

template <bool DYB, bool XB>
__global__ void __launch_bounds__(kTall, 1) layernorm_tall_kernel(const LayernormBackwardArgs a) {
    wait_for_kernel_before();
    constexpr int VPT = 2;
    __shared__ float red[2][2][kTall / 32];
    extern __shared__ float4 sums4[];
    const int tid = threadIdx.x;
    const float inv_d = 1.f / (float)a.d;
    // four columns of vector i are float4 (4 i + 2 half + j / 4) kTall + tid: no two lanes share a bank,
    // and every thread uses its own alone
#pragma unroll
    for (int i = 0; i < 4 * VPT; ++i) sums4[i * kTall + tid] = make_float4(0.f, 0.f, 0.f, 0.f);
    int turn = 0;
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        const size_t row = (size_t)t * a.d;
        const float mean = __ldg(a.mean + t), rstd = __ldg(a.rstd + t);
        Raw<XB> x[VPT];
        Raw<DYB> dy[VPT];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * kTall) * 8;
            if (c < a.d) {
                x[i].load(a.x, row + c);
                dy[i].load(a.dy, row + c);
            } else {
                x[i].zero();
                dy[i].zero();
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * kTall) * 8;
            if (c >= a.d) continue;
            float g[8];
            weights8(a.gamma, c, 1.f, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = dy[i].get(j) * g[j];
                s[0] += v;
                s[1] = fmaf(v, (x[i].get(j) - mean) * rstd, s[1]);
            }
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                float4& g4 = sums4[(4 * i + j / 4) * kTall + tid];
                float4& b4 = sums4[(4 * i + 2 + j / 4) * kTall + tid];
                float4 u = g4, v = b4;
                u.x = fmaf(dy[i].get(j), (x[i].get(j) - mean) * rstd, u.x);
                u.y = fmaf(dy[i].get(j + 1), (x[i].get(j + 1) - mean) * rstd, u.y);
                u.z = fmaf(dy[i].get(j + 2), (x[i].get(j + 2) - mean) * rstd, u.z);
                u.w = fmaf(dy[i].get(j + 3), (x[i].get(j + 3) - mean) * rstd, u.w);
                v.x += dy[i].get(j);
                v.y += dy[i].get(j + 1);
                v.z += dy[i].get(j + 2);
                v.w += dy[i].get(j + 3);
                g4 = u;
                b4 = v;
            }
        }
        row_sum<kTall, 2, kTall>(s, red[turn], CtaBarrier());
        const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (tid + i * kTall) * 8;
            if (c >= a.d) continue;
            float g[8], r[8] = {}, o[8];
            weights8(a.gamma, c, 1.f, g);
            if (a.dres) load8<XB>(a.dres, row + c, r);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[j] = fmaf(rstd, dy[i].get(j) * g[j] - m1 - (x[i].get(j) - mean) * rstd * m2, r[j]);
            store8<XB>(a.dx, row + c, o);
        }
    }
    if (!a.dgamma && !a.dbeta) return;
    asm volatile("griddepcontrol.launch_dependents;");
    const SumsOut out(a);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (tid + i * kTall) * 8;
        if (c >= a.d) continue;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            float* to = v >> 1 ? out.dbeta : out.dgamma;
            if (to) *reinterpret_cast<float4*>(to + c + (v & 1) * 4) = sums4[(4 * i + v) * kTall + tid];
        }
    }
}

// Adds the CTAs' partial sums, [parts][2 d] -> dgamma, dbeta.  A CTA takes 32 columns: 8 lanes read
// 128 bytes of a part, a warp four parts, the CTA 64; a lane's sums are added over the warp's
// four parts by shuffles and over the warps in order.
constexpr int kJoin = 512;
__global__ void __launch_bounds__(kJoin) layernorm_join_kernel(const float* partial, int parts, int d, float* dgamma, float* dbeta) {
    __shared__ float4 sums[kJoin / 32][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q = lane & 7;
    const int c = blockIdx.x * 32 + q * 4;  // 2 d is a multiple of 32
    wait_for_kernel_before();
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 5
    for (int p = warp * 4 + (lane >> 3); p < parts; p += kJoin / 8) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(partial + (size_t)p * 2 * d + c));
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
    }
#pragma unroll
    for (int o = 8; o < 32; o *= 2) {
        v.x += __shfl_xor_sync(kFull, v.x, o);
        v.y += __shfl_xor_sync(kFull, v.y, o);
        v.z += __shfl_xor_sync(kFull, v.z, o);
        v.w += __shfl_xor_sync(kFull, v.w, o);
    }
    if (lane < 8) sums[warp][q] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        const float* col = reinterpret_cast<const float*>(sums) + threadIdx.x;
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kJoin / 32; ++w) t += col[w * 32];
        const int at = blockIdx.x * 32 + threadIdx.x;
        if (at < d) {
            if (dgamma) dgamma[at] = t;
        } else if (dbeta) {
            dbeta[at - d] = t;
        }
    }
}

// d > 16384: dx with the row read twice (from L2 the second time); dgamma and dbeta by columns
template <bool DYB, bool XB>
__global__ void __launch_bounds__(kWide) layernorm_wide_dx_kernel(const LayernormBackwardArgs a) {
    __shared__ float red[2][2][kWide / 32];
    const float inv_d = 1.f / (float)a.d;
    int turn = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        const size_t row = (size_t)t * a.d;
        const float mean = __ldg(a.mean + t), rstd = __ldg(a.rstd + t);
        float s[2] = {0.f, 0.f};
        for (int c = threadIdx.x * 8; c < a.d; c += kWide * 8) {
            float v[8], x[8], g[8];
            load8<DYB>(a.dy, row + c, v);
            load8<XB>(a.x, row + c, x);
            weights8(a.gamma, c, 1.f, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[0] = fmaf(v[j], g[j], s[0]);
                s[1] = fmaf(v[j] * g[j], (x[j] - mean) * rstd, s[1]);
            }
        }
        row_sum<kWide, 2, kWide>(s, red[turn], CtaBarrier());
        const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
        for (int c = threadIdx.x * 8; c < a.d; c += kWide * 8) {
            float v[8], x[8], g[8], r[8] = {};
            load8<DYB>(a.dy, row + c, v);
            load8<XB>(a.x, row + c, x);
            weights8(a.gamma, c, 1.f, g);
            if (a.dres) load8<XB>(a.dres, row + c, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = fmaf(rstd, v[j] * g[j] - m1 - (x[j] - mean) * rstd * m2, r[j]);
            store8<XB>(a.dx, row + c, v);
        }
    }
}

template <bool DYB, bool XB>
__global__ void __launch_bounds__(256) layernorm_wide_dweight_kernel(const LayernormBackwardArgs a) {
    __shared__ float sg[8][32], sb[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float g = 0.f, b = 0.f;
    if (c < a.d) {
        for (int t = warp; t < a.T; t += 8) {
            const size_t i = (size_t)t * a.d + c;
            const float dy = DYB ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.dy)[i] << 16)
                                 : static_cast<const float*>(a.dy)[i];
            const float x = XB ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.x)[i] << 16)
                               : static_cast<const float*>(a.x)[i];
            g = fmaf(dy, (x - __ldg(a.mean + t)) * __ldg(a.rstd + t), g);
            b += dy;
        }
    }
    sg[warp][lane] = g;
    sb[warp][lane] = b;
    __syncthreads();
    if (warp == 0 && c < a.d) {
        for (int w = 1; w < 8; ++w) {
            g += sg[w][lane];
            b += sb[w][lane];
        }
        if (a.dgamma) a.dgamma[c] = g;
        if (a.dbeta) a.dbeta[c] = b;
    }
}

// ------------------------------------------------------------------ launches

int pow2_at_least(int v) {
    int p = 8;
    while (p < v) p *= 2;
    return p;
}

// threads of a row: vectors of 8 columns, `vpt` a thread
int row_threads(int d, int vpt) { return pow2_at_least((d / 8 + vpt - 1) / vpt); }

constexpr int kForwardMax = 1024 * 8 * 4;
constexpr int kBackwardMax = 1024 * 8, kTallMax = 1024 * 8 * 2;
constexpr int kAheadMin = 256;  // threads of a row from which the next rows are copied ahead

template <bool XB, int R>
void forward_rows(const LayernormArgs& a, int sm_count, cudaStream_t s) {
    auto go = [&](auto tpr) {
        constexpr int kTpr = decltype(tpr)::value, kCta = cta_threads(kTpr, 128), kRows = kCta / kTpr * R;
        const int grid = (int)std::min(((long long)a.T + kRows - 1) / kRows, (long long)sm_count * (2048 / kCta));
        launch_after(layernorm_kernel<XB, kTpr, 4, R>, grid, kCta, 0, s, a);  // (an error is seen below)
    };
    switch (row_threads(a.d, 4)) {
        case 8: go(std::integral_constant<int, 8>()); break;
        case 16: go(std::integral_constant<int, 16>()); break;
        case 32: go(std::integral_constant<int, 32>()); break;
        case 64: go(std::integral_constant<int, 64>()); break;
        case 128: go(std::integral_constant<int, 128>()); break;
        case 256: go(std::integral_constant<int, 256>()); break;
        default:
            if constexpr (R == 1) {
                if (a.d <= kForwardMax / 2) go(std::integral_constant<int, 512>());
                else go(std::integral_constant<int, 1024>());
            }
    }
}

template <bool XB>
cudaError_t forward(const LayernormArgs& a, int sm_count, cudaStream_t s) {
    const int tpr = row_threads(a.d, 4);
    if (a.d > kForwardMax) {
        layernorm_wide_kernel<XB><<<std::min(a.T, sm_count), kWide, 0, s>>>(a);
    } else if (tpr <= 256 && a.T > sm_count * (1024 / tpr)) {
        forward_rows<XB, 2>(a, sm_count, s);
    } else {
        // few rows: one at a time, on as many SMs as there are; and rows of 512 threads and more, of
        // which two at a time leave too few on an SM (8192 x 12000 bf16: 98 us with one, 113 with two)
        forward_rows<XB, 1>(a, sm_count, s);
    }
    return cudaGetLastError();
}

// CTAs of the backward kernels, all resident at once, and their partial sums
int backward_parts(int T, int d, int sm_count) {
    if (d > kBackwardMax) return std::min(T, sm_count);
    const int tpr = row_threads(d, 1), cta = tpr >= kAheadMin ? tpr : back_cta(tpr), rows = cta / tpr;
    return (int)std::min(((long long)T + rows - 1) / rows, (long long)sm_count * (1024 / cta));
}

cudaError_t join(const LayernormBackwardArgs& a, int parts, cudaStream_t s) {
    return launch_after(layernorm_join_kernel, 2 * a.d / 32, kJoin, 0, s, (const float*)a.partial, parts, a.d, a.dgamma, a.dbeta);
}

// Launches a kernel whose shared memory may be over the default limit of 48 KB, the static part included;
// `ready`: the devices (by bit) where its limit is raised.
template <class Kernel>
cudaError_t launch_big(Kernel kernel, const LayernormBackwardArgs& a, int grid, int cta, size_t smem,
                       std::atomic<unsigned long long>& ready, cudaStream_t s) {
    const unsigned long long bit = a.device < 64 ? 1ull << a.device : 0;
    if (smem > 32 * 1024 && !(ready.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    return launch_after(kernel, grid, cta, smem, s, a);
}

template <bool DYB, bool XB>
cudaError_t backward(const LayernormBackwardArgs& a, int sm_count, cudaStream_t s) {
    if (a.d > kTallMax) {
        layernorm_wide_dx_kernel<DYB, XB><<<std::min(a.T, sm_count), kWide, 0, s>>>(a);
        if (a.dgamma || a.dbeta) layernorm_wide_dweight_kernel<DYB, XB><<<(a.d + 31) / 32, 256, 0, s>>>(a);
        return cudaGetLastError();
    }
    const int parts = backward_parts(a.T, a.d, sm_count);
    cudaError_t e = cudaSuccess;
    auto go = [&](auto tpr) {
        constexpr int kTpr = decltype(tpr)::value;
        static std::atomic<unsigned long long> ready{0};
        if constexpr (kTpr >= kAheadMin) {
            using B = Ahead<DYB, XB, kTpr>;
            e = launch_big(layernorm_ahead_kernel<DYB, XB, kTpr>, a, parts, B::kCta, B::kSmem, ready, s);
        } else {
            using B = Back<kTpr>;
            e = launch_big(layernorm_backward_kernel<DYB, XB, kTpr>, a, parts, B::kCta, B::kSmem, ready, s);
        }
    };
    static std::atomic<unsigned long long> tall_ready{0};
    if (a.d > kBackwardMax) e = launch_big(layernorm_tall_kernel<DYB, XB>, a, parts, kTall, kTallSmem, tall_ready, s);
    else switch (row_threads(a.d, 1)) {
        case 8: go(std::integral_constant<int, 8>()); break;
        case 16: go(std::integral_constant<int, 16>()); break;
        case 32: go(std::integral_constant<int, 32>()); break;
        case 64: go(std::integral_constant<int, 64>()); break;
        case 128: go(std::integral_constant<int, 128>()); break;
        case 256: go(std::integral_constant<int, 256>()); break;
        case 512: go(std::integral_constant<int, 512>()); break;
        default: go(std::integral_constant<int, 1024>()); break;
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess && (a.dgamma || a.dbeta) && parts > 1) e = join(a, parts, s);
    return e;
}

}  // namespace

cudaError_t launch_layernorm(const LayernormArgs& a, int sm_count, cudaStream_t stream) {
    return a.x_bf16 ? forward<true>(a, sm_count, stream) : forward<false>(a, sm_count, stream);
}

size_t layernorm_backward_scratch_bytes(int T, int d, int sm_count) {
    if (d > kTallMax || T == 0) return 256;
    return (size_t)backward_parts(T, d, sm_count) * 2 * d * sizeof(float);
}

cudaError_t launch_layernorm_backward(const LayernormBackwardArgs& a, int sm_count, cudaStream_t stream) {
    if (a.dy_bf16) return a.x_bf16 ? backward<true, true>(a, sm_count, stream) : backward<true, false>(a, sm_count, stream);
    return a.x_bf16 ? backward<false, true>(a, sm_count, stream) : backward<false, false>(a, sm_count, stream);
}

}  // namespace moe
