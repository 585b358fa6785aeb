// moe_topk_backward: the gradient of the routing weights with respect to the
// router's logits, the choice of experts held fixed.  With g_j = rsf * grad_j,
// z = x or softcap * tanh(x / softcap):
//
//   softmax            dz_e = p_e (g_e - sum_l g_l p_l)   (g_e = 0 if not chosen)
//   softmax, renorm    v_j = p_j / sum_l p_l is the softmax of the chosen z
//                      alone: dz_j = v_j (g_j - sum_l g_l v_l), others 0
//   sigmoid            dz_j = g_j p_j (1 - p_j)
//   sigmoid, renorm    v_j = p_j / sum_l p_l: dz_j = v_j (g_j - sum_l g_l v_l) (1 - p_j)
//   softcap            dx = dz / cosh(x / softcap)^2
//
// Shares v_j come from scores scaled by exp(-m), m the largest chosen logit (of the
// sigmoid's: where it is negative): sums of scores that fp32 cannot hold, as
// sigmoids from about -87 on, never appear.  A scaled sum is 0 only where all its
// logits are -inf; such a row gets zeros.
//
// Lane j of a group of L lanes (8, 16 or 32, as k needs) holds slot j of a row.
// The row of the gradient is filled first, with zeros or, for the softmax
// without renormalisation, with -p_e sum_l g_l p_l from registers; then each
// slot's lane stores its own element over it (the warp's barrier between
// orders the two).  Reads k logits a row (the whole row only for the softmax
// without renormalisation) and writes M * E values: HBM writes bound large
// batches, launch latency the small ones.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>
#include <cstdio>

#include "moe_routing.h"
#include "sm100_ptx.cuh"

namespace moe {

int set_error(int status, const char* msg);
int set_cuda_error(cudaError_t err, const char* what);

namespace {

constexpr int kGradWarps = 4;

struct GradArgs {
    const float* grad;
    const void* logits;
    const int32_t* ids;
    void* out;
    int64_t M;
    int E, k, scoring, renorm;
    float rsf, softcap;
};

__device__ __forceinline__ float load_f32(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float cap(float x, float c) { return c != 0.0f ? c * tanhf(x / c) : x; }
// d cap / d x = 1 / cosh(x / c)^2, with e = exp(-2 |x / c|).  (1 - tanh^2 has 6% of
// error left at 8 caps and is 0 from 9 on.)
__device__ __forceinline__ float cap_slope(float x, float c) {
    if (c == 0.0f) return 1.0f;
    const float e = expf(-2.0f * fabsf(x / c));
    return 4.0f * e / ((1.0f + e) * (1.0f + e));
}

// p / sum, 0 where nothing was summed (a NaN stays one).
__device__ __forceinline__ float share(float p, float sum) { return sum != 0.0f ? p / sum : 0.0f; }

// Sum over the slots of this group that share this lane's expert, and whether
// this lane is the first of them.
template <int L>
__device__ __forceinline__ float joint(float v, int id, bool mine, int k, bool* first) {
    const int lane = threadIdx.x & 31, g0 = lane & ~(L - 1);
    float sum = 0.0f;
    *first = mine;
    for (int j = 0; j < k; ++j) {
        const float t = __shfl_sync(0xffffffffu, v, g0 + j);
        const int i = __shfl_sync(0xffffffffu, mine ? id : -1, g0 + j);
        if (mine && i == id) {
            sum += t;
            if (g0 + j < lane) *first = false;
        }
    }
    return sum;
}

// Everything but the dense softmax: nothing outside the chosen experts.
template <typename T, int L>
__global__ void __launch_bounds__(kGradWarps * 32) chosen_kernel(GradArgs a, int wide) {
    const int lane = threadIdx.x & 31, slot = lane % L;
    const int64_t row = ((int64_t)blockIdx.x * kGradWarps + (threadIdx.x >> 5)) * (32 / L) + lane / L;
    ptx::griddep_wait();
    const bool live = row < a.M;
    const T* x = static_cast<const T*>(a.logits) + row * a.E;
    T* out = static_cast<T*>(a.out) + row * a.E;

    const int id = live && slot < a.k ? __ldg(a.ids + row * a.k + slot) : -1;
    const bool mine = (uint32_t)id < (uint32_t)a.E;
    const float g = mine ? a.rsf * __ldg(a.grad + row * a.k + slot) : 0.0f;
    const float raw = mine ? load_f32(x + id) : 0.0f;
    if (live) {
        if (wide) {  // rows of whole 16-byte pieces
            const int n = a.E * (int)sizeof(T) / 16;
            for (int c = slot; c < n; c += L) reinterpret_cast<uint4*>(out)[c] = make_uint4(0, 0, 0, 0);
        } else {
            for (int e = slot; e < a.E; e += L) put(out + e, 0.0f);
        }
    }
    float v;
    if (a.scoring == MOE_SCORE_SOFTMAX) {
        const float z = cap(raw, a.softcap);
        const float m = group_max<L>(mine ? z : -INFINITY);
        float p = mine ? expf(z - (m == -INFINITY ? 0.0f : m)) : 0.0f;
        p = share(p, group_sum<L>(p));
        const float mean = group_sum<L>(g * p);
        v = p * (g - mean) * cap_slope(raw, a.softcap);
    } else {
        const float q = mine ? 1.0f / (1.0f + expf(raw)) : 0.0f;  // 1 - p without cancellation
        float p = mine ? 1.0f / (1.0f + expf(-raw)) : 0.0f, mean = 0.0f;
        if (a.renorm) {
            const float m = fminf(group_max<L>(mine ? raw : -INFINITY), 0.0f);
            // all of them negative: p exp(-m) = exp(raw - m) q
            if (mine && !(raw > 0.0f)) p = expf(raw - (m == -INFINITY ? 0.0f : m)) * q;
            p = share(p, group_sum<L>(p));
            mean = group_sum<L>(g * p);
        }
        v = p * (g - mean) * q;
    }
    bool first;
    const float sum = joint<L>(v, id, mine, a.k, &first);
    __syncwarp();
    if (first) put(out + id, sum);
}

// The softmax without renormalisation: every expert of the row takes part.
// One warp per row, the row's values in registers (up to 1024 experts).
template <typename T>
__global__ void __launch_bounds__(kGradWarps * 32) dense_kernel(GradArgs a, int wide) {
    constexpr int N = 16 / (int)sizeof(T);  // values of a 16-byte piece
    constexpr int PIECES = 1024 / 32 / N;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kGradWarps + (threadIdx.x >> 5);
    ptx::griddep_wait();
    if (row >= a.M) return;
    const T* x = static_cast<const T*>(a.logits) + row * a.E;
    T* out = static_cast<T*>(a.out) + row * a.E;

    const int id = lane < a.k ? __ldg(a.ids + row * a.k + lane) : -1;
    const bool mine = (uint32_t)id < (uint32_t)a.E;
    const float g = mine ? a.rsf * __ldg(a.grad + row * a.k + lane) : 0.0f;
    const float raw = mine ? load_f32(x + id) : 0.0f;

    // values e = (lane + 32 i) * N + u, -inf past the row
    float z[PIECES][N];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        if (i * 32 * N >= a.E) break;
        const int e0 = (lane + 32 * i) * N;
        union {
            uint4 v;
            T t[N];
        } c;
        if (wide && e0 < a.E) c.v = *reinterpret_cast<const uint4*>(x + e0);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            float t = -INFINITY;
            if (e0 + u < a.E) t = cap(wide ? (float)c.t[u] : load_f32(x + e0 + u), a.softcap);
            z[i][u] = t;
            top = fmaxf(top, t);
        }
    }
    top = group_max<32>(top);
    if (top == -INFINITY) top = 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        if (i * 32 * N >= a.E) break;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            z[i][u] = expf(z[i][u] - top);
            s += z[i][u];
        }
    }
    const float total = group_sum<32>(s);
    const float p = mine ? share(expf(cap(raw, a.softcap) - top), total) : 0.0f;
    const float rest = group_sum<32>(g * p), rest_total = share(rest, total);
    bool first;
    const float sum = joint<32>(g * p, id, mine, a.k, &first);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int e0 = (lane + 32 * i) * N;
        if (e0 >= a.E) break;
        union {
            uint4 v;
            T t[N];
        } c;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            float t = -rest_total * z[i][u];
            if (a.softcap != 0.0f && e0 + u < a.E) t *= cap_slope(load_f32(x + e0 + u), a.softcap);
            put(&c.t[u], t);
        }
        if (wide) {
            *reinterpret_cast<uint4*>(out + e0) = c.v;
        } else {
#pragma unroll
            for (int u = 0; u < N; ++u)
                if (e0 + u < a.E) out[e0 + u] = c.t[u];
        }
    }
    __syncwarp();
    if (first) put(out + id, (sum - rest * p) * cap_slope(raw, a.softcap));
}

template <typename T>
void (*pick(const GradArgs& a, int* rows_per_warp))(GradArgs, int) {
    *rows_per_warp = 1;
    if (a.scoring == MOE_SCORE_SOFTMAX && !a.renorm) return dense_kernel<T>;
    if (a.k > 16) return chosen_kernel<T, 32>;
    *rows_per_warp = a.k > 8 ? 2 : 4;
    return a.k > 8 ? chosen_kernel<T, 16> : chosen_kernel<T, 8>;
}

}  // namespace
}  // namespace moe

extern "C" int moe_topk_backward(const float* grad_weights, const void* gating_output, int dtype,
                                 const int32_t* topk_ids, int64_t M, int32_t E, int32_t k, int scoring,
                                 int32_t renormalize, float routed_scaling_factor, float softcap,
                                 void* grad_logits, void* stream) {
    using namespace moe;
    char msg[256];
    const char* who = "moe_topk_backward";
    auto invalid = [&](const char* what) {
        snprintf(msg, sizeof msg, "%s: %s", who, what);
        return set_error(MOE_ERR_INVALID_ARG, msg);
    };
    if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16)
        return invalid("dtype is neither MOE_DTYPE_F32 nor MOE_DTYPE_BF16");
    if (M < 0 || E < 1 || k < 1) return invalid("M must not be negative, E and k must be positive");
    if (scoring != MOE_SCORE_SOFTMAX && scoring != MOE_SCORE_SIGMOID)
        return invalid("scoring is neither MOE_SCORE_SOFTMAX nor MOE_SCORE_SIGMOID");
    if (!std::isfinite(routed_scaling_factor)) return invalid("routed_scaling_factor is not finite");
    if (!std::isfinite(softcap)) return invalid("softcap is not finite");
    if (softcap != 0.0f && scoring != MOE_SCORE_SOFTMAX) return invalid("softcap goes with softmax scoring only");
    if (E > 1024 || k > 32 || M > ((1ll << 31) - 1) / k) {
        snprintf(msg, sizeof msg, "%s: E=%d > 1024, k=%d > 32 or M*k >= 2^31", who, E, k);
        return set_error(MOE_ERR_UNSUPPORTED, msg);
    }
    if (M == 0) return MOE_OK;
    const size_t esz = dtype == MOE_DTYPE_F32 ? 4 : 2;
    auto bad = [](const void* p, size_t n) { return !p || reinterpret_cast<uintptr_t>(p) % n != 0; };
    if (bad(grad_weights, 4) || bad(gating_output, esz) || bad(topk_ids, 4) || bad(grad_logits, esz))
        return invalid("a pointer is null or not aligned to its element size");

    GradArgs a{grad_weights, gating_output, topk_ids, grad_logits, M, E, k, scoring, renormalize ? 1 : 0,
               routed_scaling_factor, softcap};
    int rows = 1;
    auto kern = dtype == MOE_DTYPE_F32 ? pick<float>(a, &rows) : pick<__nv_bfloat16>(a, &rows);
    const int wide = (size_t)E * esz % 16 == 0 && !bad(gating_output, 16) && !bad(grad_logits, 16);
    rows *= kGradWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((M + rows - 1) / rows), 1, 1);
    cfg.blockDim = dim3(kGradWarps * 32, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t err = cudaLaunchKernelEx(&cfg, kern, a, wide);
    return err == cudaSuccess ? MOE_OK : set_cuda_error(err, "moe_topk_backward launch");
}
