// The experts' products over the segments of expert-sorted rows:
//
//   moe_expert_matmul              out[p] = f(W_e x[p] + b_e) (gated: f(g) * u) + residual[p]
//   moe_expert_matmul_grad_input   grad_x[p] = (W_e^T grad_out[p]) through f' at preact[p]
//   moe_expert_matmul_grad_weight  grad_W_e = sum_p grad_out[p] x[p]^T, grad_b_e = sum_p grad_out[p]
//
// Simple form: 64 x 64 tiles on the CUDA cores, fp32 sums.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstdio>

#include "moe_routing.h"

namespace moe {

int set_error(int status, const char* msg);
int set_cuda_error(cudaError_t err, const char* what);

namespace {

using bf16 = __nv_bfloat16;

constexpr int kT = 64;
constexpr int kKB = 16;

struct MatArgs {
    const bf16* x;       // forward: x; grad_input: grad_out; grad_weight: grad_out
    const bf16* w;       // forward, grad_input: weight; grad_weight: x
    const int32_t* off;
    int64_t P;
    int K, N, E;         // of the weight (N without the gate's doubling)
    const float* bias;
    int act, gated;
    const bf16* extra;   // forward: residual; grad_input: preact
    void* out;
    bf16* preact;
    float* grad_bias;
};

__device__ __forceinline__ float act_f(float z, int act) {
    if (act == MOE_ACT_SILU) return z / (1.0f + expf(-z));
    if (act == MOE_ACT_GELU) return z * normcdff(z);
    return z;
}

__device__ __forceinline__ float act_df(float z, int act) {
    if (act == MOE_ACT_SILU) {
        const float p = 1.0f / (1.0f + expf(-z));
        return p * (1.0f + z * (1.0f - p));
    }
    if (act == MOE_ACT_GELU) return normcdff(z) + z * 0.3989422804014327f * expf(-0.5f * z * z);
    return 1.0f;
}

__device__ __forceinline__ void segment(const MatArgs& a, int e, int64_t* begin, int64_t* end) {
    const int64_t b = a.off[e], t = a.off[e + 1];
    *begin = b < 0 ? 0 : b > a.P ? a.P : b;
    *end = t < *begin ? *begin : t > a.P ? a.P : t;
}

// blockIdx: x = column tile, y = row tiles of the expert in strides, z = expert.
// GRAD false: D[p, n] = sum_k x[p, k] w[e, n, k]; true: D[p, k] = sum_n x[p, n] w[e, n, k].
template <bool GRAD>
__global__ void __launch_bounds__(256) simple_rows_kernel(MatArgs a) {
    __shared__ float sa[kKB][kT + 1], sb[2][kKB][kT + 1];
    int64_t begin, end;
    segment(a, blockIdx.z, &begin, &end);
    const int R = GRAD ? a.N : a.K;  // reduction length
    const int C = GRAD ? a.K : a.N;  // output columns
    const int nz = !GRAD && a.gated ? 2 : 1;
    const int Nz = a.N * nz;
    const bf16* w = a.w + (int64_t)blockIdx.z * Nz * a.K;
    const int c0 = blockIdx.x * kT, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (int64_t r0 = begin + (int64_t)blockIdx.y * kT; r0 < end; r0 += (int64_t)gridDim.y * kT) {
        float acc[2][4][4] = {};
        for (int k0 = 0; k0 < R; k0 += kKB) {
            for (int i = threadIdx.x; i < kT * kKB; i += 256) {
                const int r = i / kKB, kk = i % kKB;
                sa[kk][r] = r0 + r < end && k0 + kk < R ? __bfloat162float(a.x[(r0 + r) * R + k0 + kk]) : 0.0f;
                for (int h = 0; h < nz; ++h) {
                    const int c = c0 + r;
                    const bool in = c < C && k0 + kk < R;
                    sb[h][kk][r] = !in ? 0.0f
                                   : GRAD ? __bfloat162float(w[(int64_t)(k0 + kk) * a.K + c])
                                          : __bfloat162float(w[((int64_t)h * a.N + c) * a.K + k0 + kk]);
                }
            }
            __syncthreads();
            for (int kk = 0; kk < kKB; ++kk)
                for (int h = 0; h < nz; ++h)
                    for (int i = 0; i < 4; ++i)
                        for (int j = 0; j < 4; ++j)
                            acc[h][i][j] = fmaf(sa[kk][ty * 4 + i], sb[h][kk][tx * 4 + j], acc[h][i][j]);
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int64_t r = r0 + ty * 4 + i;
                const int c = c0 + tx * 4 + j;
                if (r >= end || c >= C) continue;
                if (GRAD) {
                    const float q = acc[0][i][j];
                    bf16* out = (bf16*)a.out;
                    if (!a.extra) {
                        out[r * C + c] = __float2bfloat16_rn(q);
                    } else if (a.gated) {
                        const float g = __bfloat162float(a.extra[r * 2 * C + c]);
                        const float u = __bfloat162float(a.extra[r * 2 * C + C + c]);
                        out[r * 2 * C + c] = __float2bfloat16_rn(q * u * act_df(g, a.act));
                        out[r * 2 * C + C + c] = __float2bfloat16_rn(q * act_f(g, a.act));
                    } else {
                        out[r * C + c] = __float2bfloat16_rn(q * act_df(__bfloat162float(a.extra[r * C + c]), a.act));
                    }
                } else {
                    float z[2] = {acc[0][i][j], acc[1][i][j]};
                    for (int h = 0; h < nz; ++h) {
                        if (a.bias) z[h] += a.bias[(int64_t)blockIdx.z * Nz + h * a.N + c];
                        if (a.preact) a.preact[r * Nz + h * a.N + c] = __float2bfloat16_rn(z[h]);
                    }
                    float v = act_f(z[0], a.act);
                    if (a.gated) v *= z[1];
                    if (a.extra) v += __bfloat162float(a.extra[r * C + c]);
                    ((bf16*)a.out)[r * C + c] = __float2bfloat16_rn(v);
                }
            }
    }
}

// blockIdx: x = K tile, y = N tile, z = expert.
template <typename T>
__global__ void __launch_bounds__(256) simple_weight_kernel(MatArgs a) {
    __shared__ float sa[kKB][kT + 1], sb[kKB][kT + 1];
    int64_t begin, end;
    segment(a, blockIdx.z, &begin, &end);
    const int n0 = blockIdx.y * kT, k0 = blockIdx.x * kT, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {}, sum = 0.0f;
    for (int64_t p0 = begin; p0 < end; p0 += kKB) {
        for (int i = threadIdx.x; i < kT * kKB; i += 256) {
            const int pp = i / kT, c = i % kT;
            const bool in = p0 + pp < end;
            sa[pp][c] = in && n0 + c < a.N ? __bfloat162float(a.x[(p0 + pp) * a.N + n0 + c]) : 0.0f;
            sb[pp][c] = in && k0 + c < a.K ? __bfloat162float(a.w[(p0 + pp) * a.K + k0 + c]) : 0.0f;
        }
        __syncthreads();
        for (int pp = 0; pp < kKB; ++pp) {
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[pp][ty * 4 + i], sb[pp][tx * 4 + j], acc[i][j]);
            if (threadIdx.x < kT) sum += sa[pp][threadIdx.x];
        }
        __syncthreads();
    }
    T* out = static_cast<T*>(a.out) + (int64_t)blockIdx.z * a.N * a.K;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + ty * 4 + i, k = k0 + tx * 4 + j;
            if (n < a.N && k < a.K) out[(int64_t)n * a.K + k] = T(acc[i][j]);
        }
    if (a.grad_bias && blockIdx.x == 0 && threadIdx.x < kT && n0 + (int)threadIdx.x < a.N)
        a.grad_bias[(int64_t)blockIdx.z * a.N + n0 + threadIdx.x] = sum;
}

bool bad(const void* p, size_t n) { return !p || reinterpret_cast<uintptr_t>(p) % n != 0; }
bool bad_opt(const void* p, size_t n) { return p && bad(p, n); }

// Checks shared by the three calls (pointers apart).
int check_sizes(const char* who, int64_t P, int K, int N, int E, int activation, int gated) {
    char msg[256];
    if (P < 0 || K < 1 || N < 1 || E < 1) {
        snprintf(msg, sizeof msg, "%s: P=%lld must not be negative, K=%d, N=%d and E=%d must be positive", who,
                 (long long)P, K, N, E);
        return set_error(MOE_ERR_INVALID_ARG, msg);
    }
    if (activation < MOE_ACT_NONE || activation > MOE_ACT_GELU || gated < 0 || gated > 1) {
        snprintf(msg, sizeof msg, "%s: activation %d or gated %d is not one of the documented values", who,
                 activation, gated);
        return set_error(MOE_ERR_INVALID_ARG, msg);
    }
    if (K % 8 != 0 || N % 8 != 0) {
        snprintf(msg, sizeof msg, "%s: K=%d and N=%d must be multiples of 8", who, K, N);
        return set_error(MOE_ERR_UNSUPPORTED, msg);
    }
    if (E > 1024 || P >= (1ll << 31) || K > (1 << 24) || N > (1 << 24)) {
        snprintf(msg, sizeof msg, "%s: E=%d > 1024, P=%lld >= 2^31, or K=%d or N=%d > 2^24", who, E, (long long)P, K, N);
        return set_error(MOE_ERR_UNSUPPORTED, msg);
    }
    return MOE_OK;
}

int bad_pointer(const char* who) {
    char msg[256];
    snprintf(msg, sizeof msg, "%s: a pointer is null or not aligned (rows 16 bytes, offsets and bias 4)", who);
    return set_error(MOE_ERR_INVALID_ARG, msg);
}

int row_tiles(int64_t P) {
    const int64_t t = (P + kT - 1) / kT;
    return (int)(t < 64 ? t : 64);
}

int launched(const char* who) {
    cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? MOE_OK : set_cuda_error(err, who);
}

}  // namespace
}  // namespace moe

extern "C" {

int moe_expert_matmul(const void* x, const void* weight, const int32_t* expert_offsets, int64_t P, int32_t K,
                      int32_t N, int32_t E, const float* bias, int activation, int32_t gated, const void* residual,
                      void* out, void* preact_out, void* stream) {
    using namespace moe;
    const char* who = "moe_expert_matmul";
    const int rc = check_sizes(who, P, K, N, E, activation, gated);
    if (rc != MOE_OK) return rc;
    if (P == 0) return MOE_OK;
    if (bad(x, 16) || bad(weight, 16) || bad(expert_offsets, 4) || bad_opt(bias, 4) || bad_opt(residual, 16) ||
        bad(out, 16) || bad_opt(preact_out, 16))
        return bad_pointer(who);
    MatArgs a{(const bf16*)x, (const bf16*)weight, expert_offsets, P, K, N, E, bias, activation, gated,
              (const bf16*)residual, out, (bf16*)preact_out, nullptr};
    simple_rows_kernel<false><<<dim3((N + kT - 1) / kT, row_tiles(P), E), 256, 0, (cudaStream_t)stream>>>(a);
    return launched(who);
}

int moe_expert_matmul_grad_input(const void* grad_out, const void* weight, const int32_t* expert_offsets, int64_t P,
                                 int32_t K, int32_t N, int32_t E, const void* preact, int activation, int32_t gated,
                                 void* grad_x, void* stream) {
    using namespace moe;
    const char* who = "moe_expert_matmul_grad_input";
    const int rc = check_sizes(who, P, K, N, E, activation, gated);
    if (rc != MOE_OK) return rc;
    if (!preact && P > 0 && (activation != MOE_ACT_NONE || gated))
        return set_error(MOE_ERR_INVALID_ARG, "moe_expert_matmul_grad_input: an activation needs its preact");
    if (P == 0) return MOE_OK;
    if (bad(grad_out, 16) || bad(weight, 16) || bad(expert_offsets, 4) || bad_opt(preact, 16) || bad(grad_x, 16))
        return bad_pointer(who);
    MatArgs a{(const bf16*)grad_out, (const bf16*)weight, expert_offsets, P, K, N, E, nullptr, activation, gated,
              (const bf16*)preact, grad_x, nullptr, nullptr};
    simple_rows_kernel<true><<<dim3((K + kT - 1) / kT, row_tiles(P), E), 256, 0, (cudaStream_t)stream>>>(a);
    return launched(who);
}

int moe_expert_matmul_grad_weight(const void* grad_out, const void* x, const int32_t* expert_offsets, int64_t P,
                                  int32_t K, int32_t N, int32_t E, int dtype, void* grad_weight, float* grad_bias,
                                  void* stream) {
    using namespace moe;
    const char* who = "moe_expert_matmul_grad_weight";
    if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16)
        return set_error(MOE_ERR_INVALID_ARG,
                         "moe_expert_matmul_grad_weight: dtype is neither MOE_DTYPE_F32 nor MOE_DTYPE_BF16");
    const int rc = check_sizes(who, P, K, N, E, MOE_ACT_NONE, 0);
    if (rc != MOE_OK) return rc;
    if ((P > 0 && (bad(grad_out, 16) || bad(x, 16))) || bad(expert_offsets, 4) || bad(grad_weight, 16) ||
        bad_opt(grad_bias, 4))
        return bad_pointer(who);
    MatArgs a{(const bf16*)grad_out, (const bf16*)x, expert_offsets, P, K, N, E, nullptr, 0, 0, nullptr,
              grad_weight, nullptr, grad_bias};
    const dim3 grid((K + kT - 1) / kT, (N + kT - 1) / kT, E);
    if (dtype == MOE_DTYPE_F32)
        simple_weight_kernel<float><<<grid, 256, 0, (cudaStream_t)stream>>>(a);
    else
        simple_weight_kernel<bf16><<<grid, 256, 0, (cudaStream_t)stream>>>(a);
    return launched(who);
}

}  // extern "C"
