// moe_topk_backward: the gradient of the routing weights with respect to the
// router's logits, the choice of experts held fixed.  With g_j = rsf * grad_j,
// z = x or softcap * tanh(x / softcap):
//
//   softmax            dz_e = p_e (g_e - sum_l g_l p_l)   (g_e = 0 if not chosen)
//   softmax, renorm    v_j = p_j / sum_l p_l is the softmax of the chosen z
//                      alone: dz_j = v_j (g_j - sum_l g_l v_l), others 0
//   sigmoid            dz_j = g_j p_j (1 - p_j)
//   sigmoid, renorm    S = sum_l p_l: dz_j = (g_j - sum_l g_l p_l / S) / S * p_j (1 - p_j)
//   softcap            dx = dz (1 - tanh(x / softcap)^2)
//
// One warp per row, lane j holds slot j (k <= 32); the row of the gradient is
// put together in shared memory and stored whole.  Reads k logits a row (the
// whole row only for the softmax without renormalisation) and writes M * E
// values: bound by HBM writes for large batches, by launch latency below.
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kGradWarps * 32) topk_backward_kernel(GradArgs a) {
    extern __shared__ float s_rows[];
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kGradWarps + (threadIdx.x >> 5);
    ptx::griddep_wait();
    if (row >= a.M) return;
    const T* x = static_cast<const T*>(a.logits) + row * a.E;
    float* dz = s_rows + (threadIdx.x >> 5) * a.E;
    const bool capped = a.softcap != 0.0f;

    int id = lane < a.k ? __ldg(a.ids + row * a.k + lane) : -1;
    const bool mine = (uint32_t)id < (uint32_t)a.E;
    const float g = mine ? a.rsf * __ldg(a.grad + row * a.k + lane) : 0.0f;
    float z = mine ? load_f32(x + id) : 0.0f;
    if (capped) z = a.softcap * tanhf(z / a.softcap);

    float v;            // this slot's dz
    float rest = 0.0f;  // softmax without renormalisation: sum_l g_l p_l
    float top = 0.0f, total = 1.0f;
    const bool dense = a.scoring == MOE_SCORE_SOFTMAX && !a.renorm;
    if (dense) {
        top = -INFINITY;
        for (int e = lane; e < a.E; e += 32) {
            float t = load_f32(x + e);
            if (capped) t = a.softcap * tanhf(t / a.softcap);
            dz[e] = t;
            top = fmaxf(top, t);
        }
        top = warp_max(top);
        float s = 0.0f;
        for (int e = lane; e < a.E; e += 32) s += expf(dz[e] - top);
        total = warp_sum(s);
        const float p = mine ? expf(z - top) / total : 0.0f;
        rest = warp_sum(g * p);
        v = g * p;
    } else if (a.scoring == MOE_SCORE_SOFTMAX) {
        const float m = warp_max(mine ? z : -INFINITY);
        float p = mine ? expf(z - m) : 0.0f;
        const float s = warp_sum(p);
        p = mine ? p / s : 0.0f;
        v = p * (g - warp_sum(g * p));
    } else {
        const float p = mine ? 1.0f / (1.0f + expf(-z)) : 0.0f;
        const float q = mine ? 1.0f / (1.0f + expf(z)) : 0.0f;  // 1 - p without cancellation
        if (a.renorm) {
            const float s = warp_sum(p);
            const float mean = warp_sum(g * p);
            v = mine ? (g - mean / s) / s * p * q : 0.0f;
        } else {
            v = g * p * q;
        }
    }
    // an expert chosen twice gets both slots' share, from the first of them
    const unsigned same = __match_any_sync(0xffffffffu, mine ? id : -1 - lane);
    float sum = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        const float t = __shfl_sync(0xffffffffu, v, j);
        if (same >> j & 1) sum += t;
    }
    const bool first = mine && (__ffs(same) - 1 == lane);

    __syncwarp();
    for (int e = lane; e < a.E; e += 32) dz[e] = dense ? -rest * (expf(dz[e] - top) / total) : 0.0f;
    __syncwarp();
    if (first) dz[id] += sum;
    __syncwarp();
    T* out = static_cast<T*>(a.out) + row * a.E;
    for (int e = lane; e < a.E; e += 32) {
        float t = dz[e];
        if (capped) {
            const float h = tanhf(load_f32(x + e) / a.softcap);
            t *= 1.0f - h * h;
        }
        put(out + e, t);
    }
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((M + kGradWarps - 1) / kGradWarps), 1, 1);
    cfg.blockDim = dim3(kGradWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = (size_t)kGradWarps * E * 4;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t err = dtype == MOE_DTYPE_F32 ? cudaLaunchKernelEx(&cfg, topk_backward_kernel<float>, a)
                                             : cudaLaunchKernelEx(&cfg, topk_backward_kernel<__nv_bfloat16>, a);
    return err == cudaSuccess ? MOE_OK : set_cuda_error(err, "moe_topk_backward launch");
}
