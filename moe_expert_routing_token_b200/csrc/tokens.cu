// Token rows to their places in expert order and back, with gradients:
//
//   moe_gather_tokens            sorted[s(t, j)] = x[t]
//   moe_gather_tokens_backward   grad_x[t] = sum_j grad_sorted[s(t, j)]
//   moe_combine_tokens           out[t] = residual[t] + sum_j w[t, j] y[s(t, j)]
//   moe_combine_tokens_backward  grad_y[s(t, j)] = w[t, j] grad_out[t],
//                                grad_w[t, j] = <grad_out[t], y[s(t, j)]>
//
// s is the expert permutation's scatter index (token-major), so every kernel
// walks tokens: a token's own row is read or written once and its k places
// are visited from registers.  No arithmetic to speak of; HBM traffic bounds
// all four.  Sums run over j ascending in fp32, so results do not depend on
// scheduling.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstdio>

#include "moe_routing.h"
#include "sm100_ptx.cuh"

namespace moe {

int set_error(int status, const char* msg);
int set_cuda_error(cudaError_t err, const char* what);

namespace {

constexpr int kTokThreads = 128;
constexpr int kTokWarps = kTokThreads / 32;

// VB bytes of a row as one access; N values of T in it.
template <int VB> struct Vec;
template <> struct Vec<16> { using type = uint4; };
template <> struct Vec<8> { using type = uint2; };
template <> struct Vec<4> { using type = uint32_t; };
template <> struct Vec<2> { using type = uint16_t; };

template <typename T, int VB>
struct Chunk {
    static constexpr int N = VB / (int)sizeof(T);
    using V = typename Vec<VB>::type;
    union {
        V v;
        T t[N];
    };
    __device__ __forceinline__ Chunk() {}
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Places of up to 32 slots from j0 on: lane j holds slot j0 + j's, 0xffffffff
// if it has none; the return value has a bit for each slot that has.
__device__ __forceinline__ uint32_t places(const int32_t* scatter, int64_t t, int k, int j0, uint32_t P, int lane,
                                           uint32_t* place) {
    *place = j0 + lane < k ? (uint32_t)__ldg(scatter + t * k + j0 + lane) : 0xffffffffu;
    return __ballot_sync(0xffffffffu, *place < P);
}

// Accesses a lane has in flight per row: 64 bytes, at most 12 accesses; for sums
// half of that, at most 9: an odd width a little past a power of two takes no
// more segments than the power (sums of 6 x 4096 fp32 rows of 515 / 1031 / 2051:
// 12.6 / 22.0 / 39.8 us; with eight 13.8 / 22.4 / 40.0, with ten 12.7 / 22.4 / 39.7).
template <int VB> constexpr int unroll() { return VB >= 16 ? 4 : VB >= 8 ? 8 : 12; }
template <int VB> constexpr int sum_unroll() { return VB >= 16 ? 2 : VB >= 8 ? 4 : 9; }

// A row's n accesses in `segs` even segments of up to 32 * U (a multiple of 32):
// a short last one costs as much latency as a whole one.  The warps of a block
// have the same segment of consecutive tokens.
struct Split {
    uint32_t segs, span;
    Split(int64_t n, int U) {
        segs = (uint32_t)((n + 32 * U - 1) / (32 * U));
        span = (uint32_t)((n + 32 * (int64_t)segs - 1) / (32 * (int64_t)segs)) * 32;
    }
};

// One warp per (token, segment).
template <typename T, int VB>
__global__ void __launch_bounds__(kTokThreads)
    gather_kernel(const T* x, int64_t M, int64_t H, const int32_t* __restrict__ scatter, int k, uint32_t P,
                  T* sorted, uint32_t segs, uint32_t span) {
    using C = Chunk<T, VB>;
    constexpr int U = unroll<VB>();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)(blockIdx.x / segs) * kTokWarps + (threadIdx.x >> 5);
    const uint32_t at = blockIdx.x % segs * span + lane;  // this lane's first access in the row
    const int left = (int)min((int64_t)span - lane, H / C::N - at);  // the segment's end from there
    ptx::griddep_wait();
    if (t >= M) return;
    typename C::V v[U];
    bool loaded = false;
    const auto* src = reinterpret_cast<const typename C::V*>(x + t * H) + at;
    for (int j0 = 0; j0 < k; j0 += 32) {
        uint32_t place;
        uint32_t todo = places(scatter, t, k, j0, P, lane, &place);
        if (todo && !loaded) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (32 * u < left) v[u] = src[32 * u];
            loaded = true;
        }
        for (; todo; todo &= todo - 1) {
            const uint32_t p = __shfl_sync(0xffffffffu, place, __ffs(todo) - 1);
            auto* dst = reinterpret_cast<typename C::V*>(sorted + (int64_t)p * H) + at;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (32 * u < left) dst[32 * u] = v[u];
        }
    }
}

// One warp per (token, segment): the weighted sum of the token's rows, R of
// them in flight at a time (without weights there is no residual either).
// Bound by the latency of a warp's two dependent reads, places and rows, where
// accesses are narrow: as many blocks an SM as the sums leave registers for.
// (From warm caches, 6 x 8191 fp32 rows of 1031, an eighth of the experts here:
// 10.3 us with nine, 10.5 with eight; with ten, whose registers spill, 11.9.
// 6 x 4096 bf16 rows of 1028, all experts: 10.4 with eight, 19.6 with ten.  From
// HBM the first takes 14.9, the second 17.6.)
constexpr int sum_blocks(int VB, bool weighted) {
    return VB >= 16 ? 6 : VB >= 8 ? (weighted ? 5 : 8) : weighted ? 8 : 9;
}

template <typename T, int VB, bool WEIGHTED>
__global__ void __launch_bounds__(kTokThreads, sum_blocks(VB, WEIGHTED))
    combine_kernel(const T* y, int64_t M, int64_t H, const int32_t* __restrict__ scatter, int k, uint32_t P,
                   const float* __restrict__ weights, const T* residual, T* out, uint32_t segs, uint32_t span) {
    using C = Chunk<T, VB>;
    constexpr int U = sum_unroll<VB>(), R = VB >= 16 ? 4 : 2;
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)(blockIdx.x / segs) * kTokWarps + (threadIdx.x >> 5);
    const uint32_t at = blockIdx.x % segs * span + lane;  // this lane's first access in the row
    const int left = (int)min((int64_t)span - lane, H / C::N - at);  // the segment's end from there
    ptx::griddep_wait();
    if (t >= M) return;
    float acc[U][C::N];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < C::N; ++i) acc[u][i] = 0.0f;
    C r[U];
    if (WEIGHTED && residual != nullptr) {
        const auto* res = reinterpret_cast<const typename C::V*>(residual + t * H) + at;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (32 * u < left) r[u].v = res[32 * u];
    }
    for (int j0 = 0; j0 < k; j0 += 32) {
        uint32_t place;
        uint32_t todo = places(scatter, t, k, j0, P, lane, &place);
        const float weight = WEIGHTED && j0 + lane < k ? __ldg(weights + t * k + j0 + lane) : 1.0f;
        while (todo) {
            C c[R][U];
            float w[R];
            const int rows = min(__popc(todo), R);
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (q >= rows) break;
                const int j = __ffs(todo) - 1;
                todo &= todo - 1;
                const uint32_t p = __shfl_sync(0xffffffffu, place, j);
                w[q] = WEIGHTED ? __shfl_sync(0xffffffffu, weight, j) : 1.0f;
                const auto* src = reinterpret_cast<const typename C::V*>(y + (int64_t)p * H) + at;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (32 * u < left) c[q][u].v = src[32 * u];
            }
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (q >= rows) break;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (32 * u < left)
#pragma unroll
                        for (int i = 0; i < C::N; ++i)
                            acc[u][i] = WEIGHTED ? fmaf(w[q], to_f32(c[q][u].t[i]), acc[u][i])
                                                 : acc[u][i] + to_f32(c[q][u].t[i]);
            }
        }
    }
    auto* dst = reinterpret_cast<typename C::V*>(out + t * H) + at;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (32 * u >= left) continue;
        C c;
#pragma unroll
        for (int i = 0; i < C::N; ++i)
            c.t[i] = from_f32<T>(WEIGHTED && residual != nullptr ? acc[u][i] + to_f32(r[u].t[i]) : acc[u][i]);
        dst[32 * u] = c.v;
    }
}

// W warps per (token, slot): a row of grad_y and one dot product.  The token's
// row of grad_out comes from cache for all but its first slot.  The dot product
// is summed in blocks, the U accesses of a round in two chains: 1.1e-7 off in the
// mean for fp32 rows of 7168, where one chain over a lane's whole share was
// 2.75e-7 (304 us for 4096 x 8 of them, both).  U accesses of either row in
// flight, as many as four blocks an SM have registers for (4096 x 6 bf16 rows of
// 1028: 25.8 us; 33.8 with eight in 100 registers).
template <typename T, int VB, int W>
__global__ void __launch_bounds__(256, 4)
    combine_backward_kernel(const T* grad_out, const T* y, int64_t pairs, int64_t H,
                            const int32_t* __restrict__ scatter, int k, const float* __restrict__ weights, T* grad_y,
                            float* grad_weights) {
    using C = Chunk<T, VB>;
    constexpr int U = VB >= 16 ? 4 : VB >= 8 ? (sizeof(T) == 4 ? 8 : 5) : 9;
    __shared__ float s_dot[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * (8 / W) + warp / W;
    ptx::griddep_wait();
    float dot = 0.0f;
    if (i < pairs) {
        const uint32_t p = (uint32_t)__ldg(scatter + i);
        if (p < pairs) {
            const float w = __ldg(weights + i);
            const int64_t n = H / C::N;
            const auto* g_row = reinterpret_cast<const typename C::V*>(grad_out + i / k * H);
            const auto* y_row = reinterpret_cast<const typename C::V*>(y + (int64_t)p * H);
            auto* d_row = reinterpret_cast<typename C::V*>(grad_y + (int64_t)p * H);
            for (int64_t c0 = (warp % W) * 32 + lane; c0 < n; c0 += 32 * W * U) {
                const int left = (int)(n - c0);
                const auto *gs = g_row + c0, *ys = y_row + c0;
                auto* ds = d_row + c0;
                C g[U], v[U];
                float part[2] = {0.0f, 0.0f};
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (32 * W * u < left) {
                        g[u].v = gs[32 * W * u];
                        v[u].v = ys[32 * W * u];
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (32 * W * u < left) {
                        C d;
#pragma unroll
                        for (int e = 0; e < C::N; ++e) {
                            part[u % 2] = fmaf(to_f32(g[u].t[e]), to_f32(v[u].t[e]), part[u % 2]);
                            d.t[e] = from_f32<T>(w * to_f32(g[u].t[e]));
                        }
                        ds[32 * W * u] = d.v;
                    }
                dot += part[0] + part[1];
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (W == 1 && lane == 0) grad_weights[i] = dot;
    }
    if constexpr (W > 1) {  // W = 8: the block's one pair
        if (lane == 0) s_dot[warp] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) s += s_dot[w];
            grad_weights[i] = s;
        }
    }
}

bool al(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Widest access that keeps every row of these arrays aligned.
template <typename T>
int access_bytes(int64_t H, const void* a, const void* b, const void* c = nullptr) {
    const size_t row = (size_t)H * sizeof(T);
    for (int vb = 16; vb > (int)sizeof(T); vb /= 2)
        if (row % vb == 0 && al(a, vb) && al(b, vb) && (!c || al(c, vb))) return vb;
    return sizeof(T);
}

template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), int64_t blocks, int threads, const char* who, void* stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t err = cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
    return err == cudaSuccess ? MOE_OK : set_cuda_error(err, who);
}

struct TokArgs {
    const char* who;
    int64_t M, H;
    const int32_t* scatter;
    int k;
    void* stream;
};

// Shared checks.  Returns MOE_OK to go on, -1 for an empty batch.
int check(const TokArgs& a, int dtype, std::initializer_list<const void*> rows,
          std::initializer_list<const void*> words) {
    char msg[256];
    if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) {
        snprintf(msg, sizeof msg, "%s: dtype %d is neither MOE_DTYPE_F32 nor MOE_DTYPE_BF16", a.who, dtype);
        return set_error(MOE_ERR_INVALID_ARG, msg);
    }
    if (a.M < 0 || a.H < 1 || a.k < 1) {
        snprintf(msg, sizeof msg, "%s: M=%lld must not be negative, H=%lld and k=%d must be positive", a.who,
                 (long long)a.M, (long long)a.H, a.k);
        return set_error(MOE_ERR_INVALID_ARG, msg);
    }
    if (a.M > ((1ll << 31) - 1) / a.k) {
        snprintf(msg, sizeof msg, "%s: M*k >= 2^31", a.who);
        return set_error(MOE_ERR_UNSUPPORTED, msg);
    }
    if (a.M == 0) return -1;
    const size_t esz = dtype == MOE_DTYPE_F32 ? 4 : 2;
    for (const void* p : rows)
        if (!p || !al(p, esz)) {
            snprintf(msg, sizeof msg, "%s: a row array is null or not aligned to its element size", a.who);
            return set_error(MOE_ERR_INVALID_ARG, msg);
        }
    for (const void* p : words)
        if (!p || !al(p, 4)) {
            snprintf(msg, sizeof msg, "%s: an index or weight array is null or not 4-byte aligned", a.who);
            return set_error(MOE_ERR_INVALID_ARG, msg);
        }
    return MOE_OK;
}

template <typename T, int VB>
int run_gather(const TokArgs& a, const void* x, void* sorted) {
    const Split s(a.H / (VB / (int)sizeof(T)), unroll<VB>());
    const int64_t blocks = (a.M + kTokWarps - 1) / kTokWarps * s.segs;
    if (blocks >= (1ll << 31)) return set_error(MOE_ERR_UNSUPPORTED, "moe_gather_tokens: M*H needs too many blocks");
    return launch(gather_kernel<T, VB>, blocks, kTokThreads, a.who, a.stream, (const T*)x, a.M, a.H, a.scatter, a.k,
                  (uint32_t)(a.M * a.k), (T*)sorted, s.segs, s.span);
}

template <typename T, int VB, bool WEIGHTED>
int run_combine(const TokArgs& a, const void* y, const float* w, const void* residual, void* out) {
    const Split s(a.H / (VB / (int)sizeof(T)), sum_unroll<VB>());
    const int64_t blocks = (a.M + kTokWarps - 1) / kTokWarps * s.segs;
    if (blocks >= (1ll << 31)) return set_error(MOE_ERR_UNSUPPORTED, "moe_combine_tokens: M*H needs too many blocks");
    return launch(combine_kernel<T, VB, WEIGHTED>, blocks, kTokThreads, a.who, a.stream, (const T*)y, a.M, a.H,
                  a.scatter, a.k, (uint32_t)(a.M * a.k), w, (const T*)residual, (T*)out, s.segs, s.span);
}

// A warp per pair from this many pairs on, a block per pair below.  Rows of 7168
// bf16, in us with a warp / a block: 10.5 / 8.5 for 1024 pairs, 13.9 / 14.7 for
// 2048, 22.3 / 26.7 for 4096; of 512 bf16: 4.6 / 3.6, 4.4 / 8.2, 4.6 / 14.3.
constexpr int64_t kWarpPairs = 4096;

template <typename T, int VB>
int run_combine_backward(const TokArgs& a, const void* g, const void* y, const float* w, void* gy, float* gw) {
    const int64_t pairs = a.M * a.k;
    const bool warps = pairs >= kWarpPairs;
    return launch(warps ? combine_backward_kernel<T, VB, 1> : combine_backward_kernel<T, VB, 8>,
                  warps ? (pairs + 7) / 8 : pairs, 256, a.who, a.stream, (const T*)g, (const T*)y, pairs, a.H,
                  a.scatter, a.k, w, (T*)gy, gw);
}

// F<T, VB>(args...) for the row type and access width.
#define MOE_TOK_DISPATCH(F, dtype, vb32, vb16, ...)                        \
    do {                                                                   \
        if ((dtype) == MOE_DTYPE_F32) {                                    \
            switch (vb32) {                                                \
                case 16: return F(float, 16)(__VA_ARGS__);                 \
                case 8: return F(float, 8)(__VA_ARGS__);                   \
                default: return F(float, 4)(__VA_ARGS__);                  \
            }                                                              \
        }                                                                  \
        switch (vb16) {                                                    \
            case 16: return F(__nv_bfloat16, 16)(__VA_ARGS__);             \
            case 8: return F(__nv_bfloat16, 8)(__VA_ARGS__);               \
            case 4: return F(__nv_bfloat16, 4)(__VA_ARGS__);               \
            default: return F(__nv_bfloat16, 2)(__VA_ARGS__);              \
        }                                                                  \
    } while (0)
#define MOE_GATHER(T, VB) run_gather<T, VB>
#define MOE_COMBINE(T, VB) run_combine<T, VB, true>
#define MOE_SUM(T, VB) run_combine<T, VB, false>
#define MOE_COMBINE_BWD(T, VB) run_combine_backward<T, VB>

}  // namespace
}  // namespace moe

extern "C" {

int moe_gather_tokens(const void* x, int dtype, int64_t M, int32_t H, const int32_t* scatter_indx, int32_t k,
                      void* sorted, void* stream) {
    using namespace moe;
    const TokArgs a{"moe_gather_tokens", M, H, scatter_indx, k, stream};
    const int rc = check(a, dtype, {x, sorted}, {scatter_indx});
    if (rc != MOE_OK) return rc < 0 ? MOE_OK : rc;
    MOE_TOK_DISPATCH(MOE_GATHER, dtype, access_bytes<float>(H, x, sorted), access_bytes<__nv_bfloat16>(H, x, sorted),
                     a, x, sorted);
}

int moe_gather_tokens_backward(const void* grad_sorted, int dtype, int64_t M, int32_t H,
                               const int32_t* scatter_indx, int32_t k, void* grad_x, void* stream) {
    using namespace moe;
    const TokArgs a{"moe_gather_tokens_backward", M, H, scatter_indx, k, stream};
    const int rc = check(a, dtype, {grad_sorted, grad_x}, {scatter_indx});
    if (rc != MOE_OK) return rc < 0 ? MOE_OK : rc;
    MOE_TOK_DISPATCH(MOE_SUM, dtype, access_bytes<float>(H, grad_sorted, grad_x),
                     access_bytes<__nv_bfloat16>(H, grad_sorted, grad_x), a, grad_sorted, nullptr, nullptr, grad_x);
}

int moe_combine_tokens(const void* y, int dtype, int64_t M, int32_t H, const int32_t* scatter_indx, int32_t k,
                       const float* topk_weights, const void* residual, void* out, void* stream) {
    using namespace moe;
    const TokArgs a{"moe_combine_tokens", M, H, scatter_indx, k, stream};
    const int rc = check(a, dtype, {y, residual ? residual : y, out}, {scatter_indx, topk_weights});
    if (rc != MOE_OK) return rc < 0 ? MOE_OK : rc;
    MOE_TOK_DISPATCH(MOE_COMBINE, dtype, access_bytes<float>(H, y, out, residual),
                     access_bytes<__nv_bfloat16>(H, y, out, residual), a, y, topk_weights, residual, out);
}

int moe_combine_tokens_backward(const void* grad_out, const void* y, int dtype, int64_t M, int32_t H,
                                const int32_t* scatter_indx, int32_t k, const float* topk_weights, void* grad_y,
                                float* grad_weights, void* stream) {
    using namespace moe;
    const TokArgs a{"moe_combine_tokens_backward", M, H, scatter_indx, k, stream};
    const int rc = check(a, dtype, {grad_out, y, grad_y}, {scatter_indx, topk_weights, grad_weights});
    if (rc != MOE_OK) return rc < 0 ? MOE_OK : rc;
    MOE_TOK_DISPATCH(MOE_COMBINE_BWD, dtype, access_bytes<float>(H, grad_out, y, grad_y),
                     access_bytes<__nv_bfloat16>(H, grad_out, y, grad_y), a, grad_out, y, topk_weights, grad_y,
                     grad_weights);
}

}  // extern "C"
