// The experts' products over the segments of expert-sorted rows, on the
// tcgen05 tensor cores:
//
//   moe_expert_matmul              out[p] = f(W_e x[p] + b_e) (gated: f(g) * u) + residual[p]
//   moe_expert_matmul_grad_input   grad_x[p] = (W_e^T grad_out[p]) through f' at preact[p]
//   moe_expert_matmul_grad_weight  grad_W_e = sum_p grad_out[p] x[p]^T, grad_b_e = sum_p grad_out[p]
//
// Two persistent kernels on CTA pairs, one CTA per SM, warp-specialised: two
// copying lanes, an issuing lane in the even CTA and eight epilogue warps
// around a ring of shared-memory stages and two TMEM accumulators, so that a
// tile's epilogue overlaps the next tile's products.  tcgen05.mma works on the
// pair (cta_group::2, M = 256): each CTA copies its own half of both operands
// and holds its own 128 rows of the result.
//
// expert_rows_kernel (the first two calls).  A tile is 256 rows of the WEIGHT
// times up to 256 tokens of one expert: the accumulator's lanes are output
// features and its columns tokens.  Segments have any length, and the column
// count of a pair's product goes in steps of 32, so a segment is cut into equal
// parts of at most 256 tokens in units of 32 instead of being padded to 128 or
// 256 rows; and a handful of tokens costs one narrow product over weights that
// stream past once.  grad_input differs only in the weight's orientation (its
// tile is MN-major: reduction along the weight's rows).  A gated tile holds
// gate and up rows interleaved by 8, so that both factors of an output meet in
// one thread's TMEM fragment.  The epilogue reads 16x256b fragments, works in
// fp32, and turns them token-major with transposing matrix moves through
// 80-byte shared-memory rows (a pitch without bank conflicts).
//
// expert_weight_kernel (grad_weight).  A tile is 256 x 256 of one expert's
// gradient, both operands MN-major with the reduction along tokens.  Where a
// segment's last 64-row stage runs over its end, the next segment's rows are
// zeroed in shared memory before the product.  Long segments are summed in
// parts, the later ones in the second accumulator and from there added onto the
// first.  The result leaves by tile stores, which clip at the matrix's ends.
//
// What bounds them (B200): long reductions over many rows, a pair's two SMs
// taking 64 bytes a cycle each from L2 (256 x 256 x 64 takes 516 cycles and
// brings 32 KB to either), 83% of the tensor pipe at 8 experts of 1024 rows,
// 7168 by 2 x 2048; under a lasting load the board's 1000 W, which lowers the
// clock to 1.05 - 1.3 GHz (1.70 ms for 32 such experts, 1130 TFLOP/s).  Few
// rows per expert: the weights' bytes from HBM (6.9 TB/s at 2 rows each).  Few
// tiles: one tile's latency.
//
// Every wait is bounded; a wait that runs out is counted
// (moe_watchdog_trips) and ends the block's work.  An accumulator whose
// products are not all in is never handed to an epilogue, of either CTA (the
// other one's flag is not set, only its own wait runs out): such a tile is not
// stored and, of a split reduction, not sent on.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstdio>
#include <mutex>
#include <unordered_map>

#include "expert_ptx.cuh"
#include "moe_routing.h"
#include "tma_host.cuh"

namespace moe {

int set_error(int status, const char* msg);
int set_cuda_error(cudaError_t err, const char* what);
int sm_count(int* dev, int* sms);

namespace {

using bf16 = __nv_bfloat16;

constexpr int kMaxE = 1024;
constexpr int kM = 128;                 // accumulator lanes: weight rows
constexpr int kBK = 64;                 // reduction per stage (one 128-byte swizzle row)
constexpr int kABytes = kM * kBK * 2;
constexpr int kAccCols = 256;           // TMEM columns of one accumulator
constexpr int kUnit = 32;               // token step of a pair's product
constexpr int kMaxStages = 12;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kPitch = 80;              // bytes of a staged token: 32 features and a bank shift
constexpr int kEpiBytes = 32 * kPitch;  // per epilogue warp: 32 tokens
constexpr int kSumBytes = kM * 32 * 4;  // a CTA's fp32 sums of a 32-token tile
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kStageNs = 2000;     // and per stage of a reduction that is waited for as a whole

static __device__ unsigned int g_watchdog_trips_experts;

enum Mode { kFwd, kFwdGated, kGrad, kGradGated };

struct RowArgs {
    const int32_t* off;
    int64_t P;
    int E;
    int red;             // reduction length
    unsigned tiles_f;    // pairs of feature tiles
    int tn_max;          // tokens per tile at most
    int stages, stage_bytes;
    int split;           // pairs of a cluster that share a tile's reduction
    int N;               // columns of one output part
    const float* bias;   // (E, N) or (E, 2 N)
    int act;
    const bf16* extra;   // forward: residual; gradient: preact
    bf16* out;
    bf16* preact;
};

struct WeightArgs {
    const int32_t* off;
    int64_t P;
    int E, N, K;
    unsigned tiles_n, tiles_k;  // of 256 x 256
    int stages;
    bool bias_next;
};

// The normal distribution's tail over its density at t >= 0 (Mills' ratio),
// sqrt(pi / 2) erfcx(t / sqrt 2): a rational function fitted here by weighted
// least squares to a relative error of 7e-7 (in fp32) up to t = 14, where the
// density leaves fp32.  With it Phi(-t) keeps its relative precision far out,
// in 7 multiply-adds and a reciprocal; normcdff's several branches made the
// epilogue of 32 x 32 values last longer than its tile's products.
__device__ __forceinline__ float2 mills(float2 t) {
    using namespace ptx;
    float2 p = fma2(t, both(0.04273192584514618f), 0.2996203303337097f);
    p = fma2(p, t, 0.9073256254196167f);
    p = fma2(p, t, 1.253313660621643f);
    float2 q = fma2(t, both(0.042736925184726715f), 0.2994176745414734f);
    q = fma2(q, t, 0.9534378051757812f);
    q = fma2(q, t, 1.5218068361282349f);
    q = fma2(q, t, 1.0f);
    return mul2(p, rcp_2(q));
}

// f(z) and, where asked for, f'(z) of two values.  Where the reduction is short the
// epilogue's time is the call's (6335 rows, 176 by 4664: 41 us with GELU, 24
// without an activation): two warps a scheduler, each a chain of dependent steps
// (issue slots 42% busy, fixed latencies the most frequent stall), hence two
// values an instruction wherever there is one for it; the approximate exponential's and reciprocal's few units in the 24th
// bit vanish in the rounding to bf16.  A NaN stays one.
template <int ACT, bool GRAD>
__device__ __forceinline__ float2 activate(float2 z, float2* slope) {
    using namespace ptx;
    constexpr float kLog2e = 1.4426950408889634f;
    if constexpr (ACT == MOE_ACT_SILU) {
        const float2 p = rcp_2(add2(exp2_2(mul2(z, -kLog2e)), both(1.0f)));
        const float2 f = mul2(z, p);
        if (GRAD) *slope = fma2(f, fma2(p, both(-1.0f), 1.0f), p);  // p + z p (1 - p)
        return f;
    }
    if constexpr (ACT == MOE_ACT_GELU) {
        const float2 u = make_float2(fabsf(z.x), fabsf(z.y));
        const float2 t = make_float2(min_nan(u.x, 14.0f), min_nan(u.y, 14.0f));
        const float2 density = mul2(exp2_2(mul2(mul2(t, t), -0.5f * kLog2e)), 0.3989422804014327f);
        const float2 tail = mul2(density, mills(t));  // Phi(-|z|)
        if (GRAD)
            *slope = fma2(make_float2(copysignf(t.x, z.x), copysignf(t.y, z.y)), density,
                          make_float2(z.x < 0.0f ? tail.x : 1.0f - tail.x, z.y < 0.0f ? tail.y : 1.0f - tail.y));
        // max(z, 0) - |z| Phi(-|z|)
        return fma2(mul2(t, -1.0f), tail, fma2(u, both(0.5f), mul2(z, 0.5f)));
    }
    if (GRAD) *slope = both(1.0f);
    return z;
}

__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

// Position in a ring of two accumulators.
struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int n) {
        if (++s == n) {
            s = 0;
            phase ^= 1;
        }
    }
};

// Position in the ring of stages: byte offset of the stage, of its barrier in
// each row of barriers, and the phase parity.  An issuing lane is one thread,
// whose dependent instructions take 4 cycles and more each: divisions by the
// stage count cost it more than a stage's products, and so do descriptors put
// together anew for each product.
struct Stages {
    uint32_t at = 0, bar = 0, phase = 0;
    __device__ __forceinline__ void step(uint32_t bytes, uint32_t all) {
        at += bytes;
        bar += 8;
        if (at == all) {
            at = bar = 0;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.b32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void give_up(volatile int* abort_flag) {
    *abort_flag = 1;
    atomicAdd(&g_watchdog_trips_experts, 1u);
}

// Gives the copies that a lane has issued time to land before it leaves after
// a wait that ran out (a millisecond; a copy takes a few microseconds).  Where
// all goes well they have landed when the last accumulator is complete.
__device__ __forceinline__ void settle() {
    const uint64_t until = ptx::globaltimer_ns() + 1000000;
    while (ptx::globaltimer_ns() < until) __nanosleep(1000);
}

// ---------------------------------------------------------------- segments
// begin[e] to begin[e + 1] are the rows of expert e; cum[e] counts the token
// tiles of the experts before it.  Offsets are clamped to [0, P] and made
// nondecreasing: whatever they hold, segments lie apart and inside the rows.
struct Segments {
    int* begin;     // E + 1
    unsigned* cum;  // E + 1
    __device__ __forceinline__ int count(int e) const { return begin[e + 1] - begin[e]; }
};
constexpr size_t segment_bytes(int E) { return (size_t)(E + 1) * 8; }

__device__ __forceinline__ unsigned tiles_of(int count, int tn_max) {
    return ((unsigned)count + tn_max - 1) / (unsigned)tn_max;
}

// This thread's offsets.
struct Offsets {
    static constexpr int N = (kMaxE + 1 + kThreads - 1) / kThreads;
    int32_t at[N];
    __device__ __forceinline__ void load(const int32_t* off, int E) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = threadIdx.x + i * kThreads;
            at[i] = e <= E ? __ldg(off + e) : 0;
        }
    }
};

// All threads of the block; ends with a barrier.
__device__ void load_segments(const Segments& s, const Offsets& off, int E, int64_t P, int tn_max) {
#pragma unroll
    for (int i = 0; i < Offsets::N; ++i) {
        const int e = threadIdx.x + i * kThreads;
        if (e > E) break;
        const int64_t v = off.at[i];
        s.begin[e] = (int)(v < 0 ? 0 : v > P ? P : v);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int per = (E + 32) / 32, e0 = threadIdx.x * per, e1 = min(e0 + per, E + 1);
        int top = 0;
        for (int e = e0; e < e1; ++e) top = max(top, s.begin[e]);
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, top, o);
            if ((int)threadIdx.x >= o) top = max(top, v);
        }
        top = __shfl_up_sync(0xffffffffu, top, 1);
        if (threadIdx.x == 0) top = 0;
        for (int e = e0; e < e1; ++e) s.begin[e] = top = max(top, s.begin[e]);
        __syncwarp();
        unsigned mine = 0;
        for (int e = e0; e < e1 && e < E; ++e) mine += tiles_of(s.count(e), tn_max);
        unsigned incl = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
            if ((int)threadIdx.x >= o) incl += v;
        }
        unsigned at = incl - mine;
        for (int e = e0; e < e1 && e < E; ++e) {
            s.cum[e] = at;
            at += tiles_of(s.count(e), tn_max);
        }
        if (threadIdx.x == 31) s.cum[E] = incl;
    }
    __syncthreads();
}

struct Tile {
    int e;      // expert
    int f;      // feature tile of this CTA of the pair
    int row0;   // first token row
    int valid;  // tokens of the tile
    int tn;     // valid rounded up to kUnit
};

// Tiles run over experts, then feature tiles, then the token tiles of the
// expert, so that neighbouring blocks share the weight's rows.
__device__ __forceinline__ Tile tile_at(const Segments& s, const RowArgs& a, unsigned tile, int rank) {
    int lo = 0, hi = a.E;  // cum[lo] * tiles_f <= tile < cum[hi] * tiles_f
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.cum[mid] * a.tiles_f <= tile) lo = mid;
        else hi = mid;
    }
    Tile t;
    t.e = lo;
    const unsigned parts = tiles_of(s.count(lo), a.tn_max);
    const unsigned in = tile - s.cum[lo] * a.tiles_f;
    const int f_pair = in / parts;
    t.f = 2 * f_pair + rank;
    const int part = in - f_pair * parts;
    // equal parts to within one unit of 32 tokens
    const int units = tiles_of(s.count(lo), kUnit), q = (unsigned)units / parts, more = units - q * (int)parts;
    const int first = part * q + (part < more ? part : more);
    t.row0 = s.begin[lo] + first * kUnit;
    t.tn = (q + (part < more ? 1 : 0)) * kUnit;
    const int left = s.count(lo) - first * kUnit;
    t.valid = left < t.tn ? left : t.tn;
    return t;
}

// ---------------------------------------------------------------- epilogue pieces
// A warp's 32 tokens of `width` bytes each (features ascending), staged at
// kPitch: 16-byte pieces between shared memory and rows of `ld` elements.
// Pieces past `valid` tokens or past `cols` columns are skipped (or zero).
template <int WIDTH>
__device__ __forceinline__ void stage_to_global(const uint8_t* stage, bf16* dst, int64_t ld, int valid, int cols,
                                                int lane) {
    constexpr int PER = WIDTH / 16;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int idx = lane + 32 * i, tok = idx / PER, piece = idx % PER;
        if (tok < valid && piece * 8 < cols)
            *reinterpret_cast<uint4*>(dst + tok * ld + piece * 8) =
                *reinterpret_cast<const uint4*>(stage + tok * kPitch + piece * 16);
    }
}

template <int WIDTH>
struct Rows {
    uint4 v[WIDTH / 16];
    __device__ __forceinline__ void load(const bf16* src, int64_t ld, int valid, int cols, int lane) {
        constexpr int PER = WIDTH / 16;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int idx = lane + 32 * i, tok = idx / PER, piece = idx % PER;
            v[i] = tok < valid && piece * 8 < cols ? *reinterpret_cast<const uint4*>(src + tok * ld + piece * 8)
                                                   : make_uint4(0, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void stage(uint8_t* stage, int lane) const {
        constexpr int PER = WIDTH / 16;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int idx = lane + 32 * i;
            *reinterpret_cast<uint4*>(stage + (idx / PER) * kPitch + (idx % PER) * 16) = v[i];
        }
    }
};

// Fragments of 32 features x 32 tokens: w[i][m] holds tokens 8 i + 2 (l % 4) +
// {0, 1} of feature 8 m + l / 4.
__device__ __forceinline__ void put32(uint32_t stage, const uint32_t (&w)[4][4], int lane) {
    const uint32_t at = stage + (lane % 8) * kPitch + (lane / 8) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) ptx::stmatrix_x4_trans(at + 8 * i * kPitch, w[i][0], w[i][1], w[i][2], w[i][3]);
}
__device__ __forceinline__ void get32(uint32_t stage, uint32_t (&w)[4][4], int lane) {
    const uint32_t at = stage + (lane % 8) * kPitch + (lane / 8) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) ptx::ldmatrix_x4_trans(at + 8 * i * kPitch, w[i][0], w[i][1], w[i][2], w[i][3]);
}
// The same for 16 features (two 8-feature groups, two token groups a move).
__device__ __forceinline__ void put16(uint32_t stage, const uint32_t (&w)[4][2], int lane) {
    const uint32_t at = stage + ((lane / 16) * 8 + lane % 8) * kPitch + (lane / 8 % 2) * 16;
#pragma unroll
    for (int i = 0; i < 4; i += 2)
        ptx::stmatrix_x4_trans(at + 8 * i * kPitch, w[i][0], w[i][1], w[i + 1][0], w[i + 1][1]);
}
__device__ __forceinline__ void get16(uint32_t stage, uint32_t (&w)[4][2], int lane) {
    const uint32_t at = stage + ((lane / 16) * 8 + lane % 8) * kPitch + (lane / 8 % 2) * 16;
#pragma unroll
    for (int i = 0; i < 4; i += 2)
        ptx::ldmatrix_x4_trans(at + 8 * i * kPitch, w[i][0], w[i][1], w[i + 1][0], w[i + 1][1]);
}

// First output column of a quarter's 32 lanes.
template <int MODE>
__device__ __forceinline__ int first_column(const Tile& t, int quarter) {
    return MODE == kFwdGated ? t.f * 64 + quarter * 16 : t.f * kM + quarter * 32;
}

// The bias of this thread's fragment rows: features l / 4 + 8 m, when gated of
// the gate (m 0, 1) and of the other factor (m 2, 3).
template <int MODE>
struct Bias {
    float b[4];
    __device__ __forceinline__ void load(const RowArgs& a, const Tile& t, int quarter, int lane) {
        if (MODE != kFwd && MODE != kFwdGated) return;
        if (a.bias == nullptr) return;
        const int col0 = first_column<MODE>(t, quarter) + lane / 4;
        const float* row = a.bias + (int64_t)t.e * (MODE == kFwdGated ? 2 : 1) * a.N;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int c = col0 + 8 * (MODE == kFwdGated ? m % 2 : m);
            b[m] = c < a.N ? __ldg(row + (MODE == kFwdGated ? m / 2 * a.N : 0) + c) : 0.0f;
        }
    }
};

// f of a fragment's values in place (of the gate's half only unless ALL), in
// the first `groups` groups of 8 tokens.
template <int ACT, bool ALL>
__device__ __forceinline__ void activate_all(float (&acc)[2][4][4], int groups) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= groups) break;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int p = 0; p < (ALL ? 4 : 2); p += 2) {
                const float2 v = activate<ACT, false>(make_float2(acc[h][i][p], acc[h][i][p + 1]), nullptr);
                acc[h][i][p] = v.x;
                acc[h][i][p + 1] = v.y;
            }
    }
}

// The fragment q taken on through f at the preactivations g (and, gated, the
// other factor u): w = q f'(g) [u], u = q f(g).
template <int ACT, bool GATED>
__device__ __forceinline__ void through_all(const float (&acc)[2][4][4], const uint32_t (&g)[4][4],
                                            uint32_t (&u)[4][4], uint32_t (&w)[4][4], int groups) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= groups) break;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            float2 q = make_float2(acc[m / 2][i][2 * (m % 2)], acc[m / 2][i][2 * (m % 2) + 1]), slope;
            const float2 f = activate<ACT, true>(unpack(g[i][m]), &slope);
            if constexpr (GATED) {
                const float2 v = unpack(u[i][m]), other = ptx::mul2(q, f);
                u[i][m] = pack(other.x, other.y);
                q = ptx::mul2(q, v);
            }
            q = ptx::mul2(q, slope);
            w[i][m] = pack(q.x, q.y);
        }
    }
}

// Split reductions: a warp's fragment to the first pair's CTA of the same rank
// (piece i of thread l at 16 (32 i + l)), and there on top of its own.
__device__ __forceinline__ void send_sums(uint32_t taddr, uint32_t sums, uint32_t joined, int rank, int quarter,
                                          int lane) {
    float acc[2][4][4];
    ptx::tmem_ld_frag32(taddr, acc);
    const uint32_t to = ptx::map_to_rank(sums + quarter * (kSumBytes / 4) + lane * 16, rank);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float* v = acc[i / 4][i % 4];
        ptx::st_cluster_f32x4(to + i * 512, v[0], v[1], v[2], v[3]);
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_to_rank(joined, rank));
}
__device__ __forceinline__ void add_sums(uint32_t taddr, const uint8_t* sums, int parts, int quarter, int lane) {
    float acc[2][4][4];
    ptx::tmem_ld_frag32(taddr, acc);
    for (int part = 0; part < parts; ++part) {
        const float4* from =
            reinterpret_cast<const float4*>(sums + part * kSumBytes + quarter * (kSumBytes / 4)) + lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 v = from[i * 32];
            float* to = acc[i / 4][i % 4];
            to[0] += v.x;
            to[1] += v.y;
            to[2] += v.z;
            to[3] += v.w;
        }
    }
    ptx::tmem_st_frag32(taddr, acc);
}

// A warp's part of the residual or the preactivations, 32 tokens of 32 lanes
// from tok0 on: on its way while the tile's products run, or the chunk before is
// worked on.  (Input gradient through GELU, 2886 rows, 4288 by 208: 28.3 us; 30.6
// with loads at the chunk's start from rows prefetched into L2.)
template <int MODE>
struct Extra {
    static constexpr int WIDTH = MODE == kFwdGated ? 32 : 64;  // bytes of one part per token
    Rows<WIDTH> in0, in1;
    __device__ __forceinline__ void load(const RowArgs& a, const Tile& t, int tok0, int quarter, int lane) {
        if (a.extra == nullptr) return;
        const int col0 = first_column<MODE>(t, quarter), valid = t.valid - tok0;
        const int64_t ld = MODE == kGradGated ? 2 * (int64_t)a.N : a.N;
        const bf16* p = a.extra + ((int64_t)t.row0 + tok0) * ld + col0;
        in0.load(p, ld, valid, a.N - col0, lane);
        if constexpr (MODE == kGradGated) in1.load(p + a.N, ld, valid, a.N - col0, lane);
    }
};

// One warp's 32 lanes x 32 tokens of the accumulator at taddr.
template <int MODE>
__device__ __forceinline__ void epilogue_chunk(const RowArgs& a, const Tile& t, const Bias<MODE>& bias,
                                               Extra<MODE>& extra, uint32_t taddr, int tok0, int quarter,
                                               uint8_t* stage, int lane) {
    const int valid = t.valid - tok0;                        // tokens of this chunk (may exceed 32)
    const int col0 = first_column<MODE>(t, quarter);
    const int cols = a.N - col0;                             // columns left (may be <= 0)
    const int64_t row0 = (int64_t)t.row0 + tok0;
    const uint32_t sst = ptx::smem_u32(stage);

    const int64_t ld_in = MODE == kGradGated ? 2 * (int64_t)a.N : a.N;
    float acc[2][4][4];
    ptx::tmem_ld_frag32(taddr, acc);
    const int groups = valid >= 32 ? 4 : (valid + 7) / 8;    // token groups of 8 in use

    if constexpr (MODE == kFwd) {
        uint32_t w[4][4] = {};
        if (a.bias != nullptr) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[m / 2][i][2 * (m % 2)] += bias.b[m];
                    acc[m / 2][i][2 * (m % 2) + 1] += bias.b[m];
                }
        }
        if (a.preact != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int m = 0; m < 4; ++m) w[i][m] = pack(acc[m / 2][i][2 * (m % 2)], acc[m / 2][i][2 * (m % 2) + 1]);
            put32(sst, w, lane);
            __syncwarp();
            stage_to_global<64>(stage, a.preact + row0 * a.N + col0, a.N, valid, cols, lane);
            __syncwarp();
        }
        uint32_t r[4][4];
        if (a.extra != nullptr) {
            extra.in0.stage(stage, lane);
            extra.load(a, t, tok0 + 64, quarter, lane);
            __syncwarp();
            get32(sst, r, lane);
            __syncwarp();
        }
        if (a.act == MOE_ACT_SILU) activate_all<MOE_ACT_SILU, true>(acc, groups);
        else if (a.act == MOE_ACT_GELU) activate_all<MOE_ACT_GELU, true>(acc, groups);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                float2 v = make_float2(acc[m / 2][i][2 * (m % 2)], acc[m / 2][i][2 * (m % 2) + 1]);
                if (a.extra != nullptr) v = ptx::add2(v, unpack(r[i][m]));
                w[i][m] = pack(v.x, v.y);
            }
        put32(sst, w, lane);
        __syncwarp();
        stage_to_global<64>(stage, a.out + row0 * a.N + col0, a.N, valid, cols, lane);
    } else if constexpr (MODE == kFwdGated) {
        const int64_t ld_z = 2 * (int64_t)a.N;
        if (a.bias != nullptr) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[h][i][0] += bias.b[h];
                    acc[h][i][1] += bias.b[h];
                    acc[h][i][2] += bias.b[2 + h];
                    acc[h][i][3] += bias.b[2 + h];
                }
        }
        uint32_t w[4][2] = {};
        if (a.preact != nullptr) {
#pragma unroll
            for (int part = 0; part < 2; ++part) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) w[i][h] = pack(acc[h][i][2 * part], acc[h][i][2 * part + 1]);
                put16(sst, w, lane);
                __syncwarp();
                stage_to_global<32>(stage, a.preact + row0 * ld_z + part * a.N + col0, ld_z, valid, cols, lane);
                __syncwarp();
            }
        }
        uint32_t r[4][2];
        if (a.extra != nullptr) {
            extra.in0.stage(stage, lane);
            extra.load(a, t, tok0 + 64, quarter, lane);
            __syncwarp();
            get16(sst, r, lane);
            __syncwarp();
        }
        if (a.act == MOE_ACT_SILU) activate_all<MOE_ACT_SILU, false>(acc, groups);
        else if (a.act == MOE_ACT_GELU) activate_all<MOE_ACT_GELU, false>(acc, groups);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float2 v = ptx::mul2(make_float2(acc[h][i][0], acc[h][i][1]), make_float2(acc[h][i][2], acc[h][i][3]));
                if (a.extra != nullptr) v = ptx::add2(v, unpack(r[i][h]));
                w[i][h] = pack(v.x, v.y);
            }
        put16(sst, w, lane);
        __syncwarp();
        stage_to_global<32>(stage, a.out + row0 * a.N + col0, a.N, valid, cols, lane);
    } else {
        uint32_t w[4][4] = {}, g[4][4], u[4][4] = {};
        if (a.extra != nullptr) {
            extra.in0.stage(stage, lane);
            __syncwarp();
            get32(sst, g, lane);
            __syncwarp();
            if constexpr (MODE == kGradGated) {
                extra.in1.stage(stage, lane);
                __syncwarp();
                get32(sst, u, lane);
                __syncwarp();
            }
            extra.load(a, t, tok0 + 64, quarter, lane);
        }
        if (a.extra == nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    w[i][m] = pack(acc[m / 2][i][2 * (m % 2)], acc[m / 2][i][2 * (m % 2) + 1]);
        } else if (a.act == MOE_ACT_SILU) {
            through_all<MOE_ACT_SILU, MODE == kGradGated>(acc, g, u, w, groups);
        } else if (a.act == MOE_ACT_GELU) {
            through_all<MOE_ACT_GELU, MODE == kGradGated>(acc, g, u, w, groups);
        } else {
            through_all<MOE_ACT_NONE, MODE == kGradGated>(acc, g, u, w, groups);
        }
        put32(sst, w, lane);
        __syncwarp();
        stage_to_global<64>(stage, a.out + row0 * ld_in + col0, ld_in, valid, cols, lane);
        if constexpr (MODE == kGradGated) {
            __syncwarp();
            put32(sst, u, lane);
            __syncwarp();
            stage_to_global<64>(stage, a.out + row0 * ld_in + a.N + col0, ld_in, valid, cols, lane);
        }
    }
    __syncwarp();
}

// Shared-memory layout behind the stage ring.  full (the even CTA's, for
// both): the copies of a stage have landed; tail: this CTA's copies of a stage
// that ends a segment have, and cut (the even CTA's, for both): what they
// brought of the next segment is zeroed; empty: a stage has been multiplied;
// acc_full, acc_empty (the even CTA's, for both): an accumulator is complete,
// has been read.
struct Control {
    uint64_t full[kMaxStages], tail[kMaxStages], cut[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
    uint64_t joined;     // split reductions: the other pairs' sums are here
    uint32_t tmem;
    int abort_flag;
};

// Barriers, TMEM and the meeting of the pair's two CTAs.
__device__ __forceinline__ uint32_t start_block(Control* c, int stages, int split, int warp) {
    if (warp == 0) {
        const int lane = threadIdx.x;
        if (lane < stages) {
            ptx::mbar_init(&c->full[lane], 1);
            ptx::mbar_init(&c->tail[lane], 1);
            ptx::mbar_init(&c->cut[lane], 2);
            ptx::mbar_init(&c->empty[lane], 1);
        } else if (lane >= 30) {
            ptx::mbar_init(&c->acc_full[lane - 30], 1);
            ptx::mbar_init(&c->acc_empty[lane - 30], 2 * kEpiWarps);
            if (lane == 30) ptx::mbar_init(&c->joined, 4 * (split > 1 ? split - 1 : 1));
            c->abort_flag = 0;
        }
        ptx::fence_mbar_init();
        __syncwarp();
    }
    if (warp == 2) {
        ptx::tmem_alloc_pair(&c->tmem, 2 * kAccCols);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    return c->tmem;
}

// Neither CTA of a pair leaves before the other: each reads the other's shared
// memory and arrives on its barriers.
__device__ __forceinline__ void end_block(uint32_t tmem, int warp) {
    ptx::tc_fence_before();
    ptx::cluster_sync();
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, 2 * kAccCols);
    }
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    expert_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmX16, RowArgs a) {
    constexpr bool GRAD = MODE == kGrad || MODE == kGradGated;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = ptx::smem_align<1024>(smem_raw);
    uint8_t* epi = ring + a.stages * a.stage_bytes;
    uint8_t* sums = epi + kEpiWarps * kEpiBytes;  // split reductions: the other pairs' parts
    Control* c = reinterpret_cast<Control*>(sums + (a.split - 1) * kSumBytes);
    int* seg_at = reinterpret_cast<int*>(c + 1);
    const Segments seg{seg_at, reinterpret_cast<unsigned*>(seg_at) + a.E + 1};
    volatile int* abort_flag = &c->abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // A cluster of `split` pairs has a tile at a time; `slice` is this pair's
    // part of the reduction, `lead` its even CTA.
    const int cta = (int)ptx::cluster_ctarank(), rank = cta & 1, lead = cta & ~1, slice = cta >> 1;
    const unsigned pair = blockIdx.x / (2 * a.split), pairs = gridDim.x / (2 * a.split);
    if (threadIdx.x == 0) {
        ptx::tma_prefetch_desc(&tmW);
        ptx::tma_prefetch_desc(&tmX);
        ptx::tma_prefetch_desc(&tmX16);
    }
    // The next kernel of the stream may set up as soon as SMs are free: another
    // such call with few tiles does so beside this one.
    ptx::griddep_launch_dependents();
    const uint32_t tmem = start_block(c, a.stages, a.split, warp);
    ptx::griddep_wait();
    Offsets offsets;
    offsets.load(a.off, a.E);
    load_segments(seg, offsets, a.E, a.P, a.tn_max);
    const unsigned tiles = seg.cum[a.E] * a.tiles_f;

    const uint32_t ring_at = ptx::smem_u32(ring), all = a.stages * a.stage_bytes;
    const uint32_t full = ptx::smem_u32(c->full), empty = ptx::smem_u32(c->empty);
    const int blocks_k = (a.red + kBK - 1) / kBK;  // this pair's: [k_lo, k_hi)
    const int k_lo = blocks_k * slice / a.split * kBK, k_hi = blocks_k * (slice + 1) / a.split * kBK;
    if (warp == 0 || warp == 3) {
        // Producers: warp 0 copies the weight's tile, warp 3 the tokens', both
        // to the even CTA's barrier.  One lane for both is late: a copy takes
        // it some 80 cycles to issue.
        if (elect_one()) {
            Stages r;
            bool ok = true, ready = true;  // ready: the stage at r is known to be empty
            const uint32_t full_pair = ptx::map_to_rank(full, lead);
            for (unsigned tile = pair; tile < tiles && ok; tile += pairs) {
                const Tile t = tile_at(seg, a, tile, rank);
                const int row0 = t.row0 + rank * (t.tn / 2);  // this CTA's half of the tokens
                const uint32_t bytes = 2 * kABytes + t.tn * (kBK * 2);
                for (int k = k_lo; k < k_hi; k += kBK) {
                    if (!ready && !ptx::bar_wait<false>(empty + r.bar, r.phase ^ 1, kWaitNs)) {
                        give_up(abort_flag);
                        ok = false;
                        break;
                    }
                    Stages next = r;
                    next.step(a.stage_bytes, all);
                    ready = ptx::bar_try(empty + next.bar, next.phase ^ 1);
                    const uint32_t at = ring_at + r.at, bar = full_pair + r.bar;
                    if (warp == 0) {
                        // Only the even CTA arrives: its barrier cannot complete
                        // before, however early the other's copies land.  (An
                        // arrival of the other one, a release at cluster scope,
                        // takes longer than a stage's products: 2.90 against
                        // 1.72 ms for the first product of 4096 x 8 rows.)
                        if (rank == 0) ptx::bar_expect(full + r.bar, bytes);
                        if constexpr (GRAD) {
                            ptx::tma_load(at, &tmW, t.f * kM, k, t.e, bar);
                            ptx::tma_load(at + kABytes / 2, &tmW, t.f * kM + 64, k, t.e, bar);
                        } else if constexpr (MODE == kFwdGated) {
                            ptx::tma_load(at, &tmW, k, 0, 0, t.f * 8, t.e, bar);
                        } else {
                            ptx::tma_load(at, &tmW, k, t.f * kM, t.e, bar);
                        }
                    } else {
                        uint32_t to = at + kABytes;
                        int row = row0;
                        for (int i = t.tn / 64; i > 0; --i, row += 32, to += 32 * kBK * 2)
                            ptx::tma_load(to, &tmX, k, row, bar);
                        if (t.tn & 32) ptx::tma_load(to, &tmX16, k, row, bar);
                    }
                    r = next;
                }
            }
            if (!ok) settle();
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            Stages r;
            Ring acc;
            bool ok = true, ready = false;  // ready: the stage at r is known to be full
            // descriptors of the first stage's operands; steps of 16 in the reduction
            const uint64_t ad0 = ptx::sdesc_sw128(ring_at, GRAD ? kABytes / 2 : 16, 1024);
            const uint64_t bd0 = ptx::sdesc_sw128(ring_at + kABytes, 16, 1024);
            const uint16_t ctas = (uint16_t)(3u << lead);
            constexpr uint64_t A_STEP = GRAD ? 2048 >> 4 : 32 >> 4, B_STEP = 32 >> 4;
            for (unsigned tile = pair; tile < tiles && ok; tile += pairs, acc.step(2)) {
                const Tile t = tile_at(seg, a, tile, rank);
                const uint32_t idesc = ptx::idesc_bf16_m256(t.tn, GRAD, false);
                if (!ptx::mbar_wait_cluster(&c->acc_empty[acc.s], acc.phase ^ 1, kWaitNs)) {
                    give_up(abort_flag);
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t d = tmem + acc.s * kAccCols;
                for (int k = k_lo; k < k_hi; k += kBK) {
                    if (!ready && !ptx::bar_wait<true>(full + r.bar, r.phase, kWaitNs)) {
                        give_up(abort_flag);
                        ok = false;
                        break;
                    }
                    // a look at the next stage's barrier takes as long as two
                    // narrow products to come back
                    Stages next = r;
                    next.step(a.stage_bytes, all);
                    ready = ptx::bar_try_cluster(full + next.bar, next.phase);
                    ptx::tc_fence_after();
                    const uint64_t ad = ad0 + (r.at >> 4), bd = bd0 + (r.at >> 4);
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        ptx::umma_bf16_pair(d, ad + kk * A_STEP, bd + kk * B_STEP, idesc, k != k_lo || kk != 0);
                    ptx::umma_commit_pair(empty + r.bar, ctas);
                    r = next;
                }
                if (ok) ptx::umma_commit_pair(ptx::smem_u32(&c->acc_full[acc.s]), ctas);
            }
        }
    } else if (warp >= 4) {
        const int ew = warp - 4, quarter = warp & 3, half = ew >> 2;
        uint8_t* stage = epi + ew * kEpiBytes;
        Ring acc;
        for (unsigned tile = pair; tile < tiles; tile += pairs, acc.step(2)) {
            const Tile t = tile_at(seg, a, tile, rank);
            Bias<MODE> bias;
            bias.load(a, t, quarter, lane);
            Extra<MODE> extra;
            if (slice == 0) extra.load(a, t, half * 32, quarter, lane);
            if (!ptx::mbar_wait(&c->acc_full[acc.s], acc.phase, kWaitNs + blocks_k * kStageNs)) {
                if (lane == 0) give_up(abort_flag);
                *abort_flag = 1;
            }
            __syncwarp();
            if (__any_sync(0xffffffffu, *abort_flag)) break;
            ptx::tc_fence_after();
            const uint32_t base = tmem + acc.s * kAccCols + (static_cast<uint32_t>(quarter * 32) << 16);
            if (a.split > 1 && half == 0) {
                // one chunk of 32 tokens; its sums meet in the first pair
                if (slice > 0) {
                    send_sums(base, ptx::smem_u32(sums) + (slice - 1) * kSumBytes, ptx::smem_u32(&c->joined), rank,
                              quarter, lane);
                } else if (__all_sync(0xffffffffu, ptx::mbar_wait_cluster(&c->joined, 0,
                                                                          kWaitNs + blocks_k * kStageNs))) {
                    add_sums(base, sums, a.split - 1, quarter, lane);
                } else {
                    if (lane == 0) give_up(abort_flag);
                    *abort_flag = 1;
                }
                __syncwarp();
                if (__any_sync(0xffffffffu, *abort_flag)) break;
            }
            for (int tok0 = half * 32; tok0 < t.valid && slice == 0; tok0 += 64)
                epilogue_chunk<MODE>(a, t, bias, extra, base + tok0, tok0, quarter, stage, lane);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::bar_arrive_remote(ptx::map_to_rank(ptx::smem_u32(&c->acc_empty[acc.s]), lead));
        }
    }
    __syncwarp();
    end_block(tmem, warp);
}

// ---------------------------------------------------------------- weight gradient
constexpr int kWN = 256;                          // columns of a tile (K side), half in each CTA
constexpr int kWEpiBytes = 32 * 128;               // staged by an epilogue warp for a tile store
constexpr int kWStageBytes = kABytes + kWN / 2 * kBK * 2;

// Products of 16 tokens for the last `left` (or 64) of a segment, and whether
// they take rows of the next segment, which have to be zeroed first.
__device__ __forceinline__ int steps_of(int left) { return left >= kBK ? kBK / 16 : (left + 15) / 16; }
__device__ __forceinline__ bool runs_over(int left) { return left < kBK && left % 16 != 0; }

// A segment's rows are summed in parts, whose sums are joined by rounded additions
// (the epilogue adds a part onto the first one's accumulator): the tensor core cuts
// its running sum to 24 bits at each step of 16 rows instead of rounding it, which
// grows with the steps: relative, for terms of random signs, 2.1e-6 after 2048 rows,
// 9.1e-6 after 8192, 1.5e-4 after 131072 (5.6e-6, 3.5e-5 and 8e-4 where all are
// positive).  Parts as the result's type needs them: an addition holds the products
// up for 0.85 us, 1600 cycles for 768 of TMEM traffic (fp32, 4 experts of 8192 rows,
// 4096 by 4096: 898 us, 774 - 802 in one sum; bf16 has one addition to 16384 rows).
template <typename T>
__device__ __forceinline__ int part_end(int p0, int count) {
    constexpr int kPart = sizeof(T) == 4 ? 2048 : 16384;
    return count - p0 > kPart ? p0 + kPart : count;
}

// A warp's 32 rows x 128 bytes, staged in the 128-byte swizzle of its tile
// store: lane r holds row r, whose 16-byte piece c lies at c ^ (r % 8).
template <typename T>
__device__ __forceinline__ void stage_row(uint8_t* stage, const float* v, int lane) {
    uint8_t* row = stage + lane * 128;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        uint4 w;
        if constexpr (sizeof(T) == 4)
            w = make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]),
                           __float_as_uint(v[4 * c + 3]));
        else
            w = make_uint4(pack(v[8 * c], v[8 * c + 1]), pack(v[8 * c + 2], v[8 * c + 3]),
                           pack(v[8 * c + 4], v[8 * c + 5]), pack(v[8 * c + 6], v[8 * c + 7]));
        *reinterpret_cast<uint4*>(row + ((c ^ (lane & 7)) * 16)) = w;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    expert_weight_kernel(const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmX,
                         const __grid_constant__ CUtensorMap tmOut, WeightArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = ptx::smem_align<1024>(smem_raw);
    uint8_t* epi = ring + a.stages * kWStageBytes;
    Control* c = reinterpret_cast<Control*>(epi + kEpiWarps * kWEpiBytes);
    int* seg_at = reinterpret_cast<int*>(c + 1);
    const Segments seg{seg_at, reinterpret_cast<unsigned*>(seg_at) + a.E + 1};
    volatile int* abort_flag = &c->abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)ptx::cluster_ctarank();
    const unsigned pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        ptx::tma_prefetch_desc(&tmY);
        ptx::tma_prefetch_desc(&tmX);
    }
    // (not to expert_bias_kernel, whose blocks would lie beside these: 13.5
    // against 11.4 us for 69 rows, 1080 by 1000)
    if (!a.bias_next) ptx::griddep_launch_dependents();
    const uint32_t tmem = start_block(c, a.stages, 1, warp);
    ptx::griddep_wait();
    Offsets offsets;
    offsets.load(a.off, a.E);
    load_segments(seg, offsets, a.E, a.P, kBK);
    const unsigned per_e = a.tiles_n * a.tiles_k, tiles = a.E * per_e;

    const uint32_t ring_at = ptx::smem_u32(ring);
    const uint32_t full = ptx::smem_u32(c->full), tail = ptx::smem_u32(c->tail), cut = ptx::smem_u32(c->cut),
                   empty = ptx::smem_u32(c->empty);
    const uint32_t all = a.stages * kWStageBytes;
    if (warp == 0 || warp == 2) {
        // Producers: warp 0 copies grad_out's tile, warp 2 x's.
        if (elect_one()) {
            Stages r;
            bool ok = true, ready = true;  // ready: the stage at r is known to be empty
            const uint32_t full_pair = ptx::map_to_rank(full, 0);
            const CUtensorMap* tm = warp == 0 ? &tmY : &tmX;
            const uint32_t part = ring_at + (warp == 0 ? 0 : kABytes);
            for (unsigned tile = pair; tile < tiles && ok; tile += pairs) {
                const int e = tile / per_e;
                const unsigned in = tile - e * per_e;
                const int c0 = warp == 0 ? (in / a.tiles_k * 2 + rank) * kM : in % a.tiles_k * kWN + rank * (kWN / 2);
                const int count = seg.count(e), row0 = seg.begin[e];
                for (int p = 0; p < count; p += kBK) {
                    if (!ready && !ptx::bar_wait<false>(empty + r.bar, r.phase ^ 1, kWaitNs)) {
                        give_up(abort_flag);
                        ok = false;
                        break;
                    }
                    Stages next = r;
                    next.step(kWStageBytes, all);
                    ready = ptx::bar_try(empty + next.bar, next.phase ^ 1);
                    // a stage counts in the even CTA, for both; over one that
                    // runs into the next segment this CTA's warp 3 goes first
                    const bool over = runs_over(count - p);
                    const uint32_t bar = over ? tail + r.bar : full_pair + r.bar;
                    if (warp == 0) {
                        if (over) ptx::bar_expect(tail + r.bar, kWStageBytes);
                        else if (rank == 0) ptx::bar_expect(full + r.bar, 2 * kWStageBytes);
                    }
                    ptx::tma_load(part + r.at, tm, c0, row0 + p, bar);
                    ptx::tma_load(part + r.at + 8192, tm, c0 + 64, row0 + p, bar);
                    r = next;
                }
            }
            if (!ok) settle();
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            const uint32_t idesc = ptx::idesc_bf16_m256(kWN, true, true);
            Stages r;
            int s = 0;               // the tile's accumulator: its first part's
            uint32_t filled = 0;     // parity of each accumulator's uses
            // parity of each stage's uses, whole and cut (bit of its barrier's offset)
            uint32_t uses[2] = {0, 0};
            bool ok = true, ready = false;  // ready: the stage at r is known to be full
            const uint64_t ad0 = ptx::sdesc_sw128(ring_at, 8192, 1024);
            const uint64_t bd0 = ptx::sdesc_sw128(ring_at + kABytes, 8192, 1024);
            for (unsigned tile = pair; tile < tiles && ok; tile += pairs) {
                const int count = seg.count(tile / per_e);
                if (count == 0) continue;
                for (int p0 = 0, end; p0 < count && ok; p0 = end) {
                    end = part_end<T>(p0, count);
                    const int a_s = p0 == 0 ? s : s ^ 1;
                    if (!ptx::mbar_wait_cluster(&c->acc_empty[a_s], (filled >> a_s & 1) ^ 1, kWaitNs)) {
                        give_up(abort_flag);
                        ok = false;
                        break;
                    }
                    filled ^= 1u << a_s;
                    ptx::tc_fence_after();
                    const uint32_t d = tmem + a_s * kAccCols;
                    for (int p = p0; p < end; p += kBK) {
                        const uint32_t bit = r.bar >> 3;
                        const bool over = runs_over(count - p);
                        if (!ready) {
                            ok = over ? ptx::bar_wait<true>(cut + r.bar, uses[1] >> bit & 1, kWaitNs)
                                      : ptx::bar_wait<true>(full + r.bar, uses[0] >> bit & 1, kWaitNs);
                            if (!ok) {
                                give_up(abort_flag);
                                break;
                            }
                        }
                        if (over) uses[1] ^= 1u << bit;
                        else uses[0] ^= 1u << bit;
                        Stages next = r;
                        next.step(kWStageBytes, all);
                        // look ahead within the segment
                        ready = count - p > kBK && !runs_over(count - p - kBK) &&
                                ptx::bar_try_cluster(full + next.bar, uses[0] >> (next.bar >> 3) & 1);
                        ptx::tc_fence_after();
                        const uint64_t ad = ad0 + (r.at >> 4), bd = bd0 + (r.at >> 4);
                        const int steps = steps_of(count - p);
#pragma unroll
                        for (int kk = 0; kk < kBK / 16; ++kk)
                            if (kk < steps)
                                ptx::umma_bf16_pair(d, ad + kk * (2048 >> 4), bd + kk * (2048 >> 4), idesc,
                                                    p != p0 || kk != 0);
                        ptx::umma_commit_pair(empty + r.bar, 3);
                        r = next;
                    }
                    if (ok) ptx::umma_commit_pair(ptx::smem_u32(&c->acc_full[a_s]), 3);
                }
                s ^= 1;
            }
        }
    } else if (warp == 3) {
        // A stage that runs over a segment's end: zero the next segment's rows
        // in every box, then arrive for this CTA.
        Stages r;
        uint32_t uses = 0;    // parity of each stage's uses of its tail barrier
        uint64_t before = 0;  // stages up to the next wait, which lasts as long as they take
        for (unsigned tile = pair; tile < tiles; tile += pairs) {
            const int count = seg.count(tile / per_e), left = count % kBK;
            before += (count + kBK - 1) / kBK;
            for (int p = count / kBK; p > 0; --p) r.step(kWStageBytes, all);
            if (left == 0) continue;
            if (runs_over(left)) {
                const uint32_t bit = r.bar >> 3;
                if (!__all_sync(0xffffffffu,
                                ptx::bar_wait<false>(tail + r.bar, uses >> bit & 1, kWaitNs + before * kStageNs))) {
                    if (lane == 0) give_up(abort_flag);
                    break;
                }
                before = 0;
                uses ^= 1u << bit;
                const int end = steps_of(left) * 16 * 8;  // in 16-byte pieces of a 64-column box
#pragma unroll
                for (int box = 0; box < kWStageBytes / 8192; ++box) {
                    uint4* at = reinterpret_cast<uint4*>(ring + r.at + box * 8192);
                    for (int i = left * 8 + lane; i < end; i += 32) at[i] = make_uint4(0, 0, 0, 0);
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_to_rank(cut + r.bar, 0));
            }
            r.step(kWStageBytes, all);
        }
    } else if (warp >= 4) {
        const int ew = warp - 4, quarter = warp & 3, half = ew >> 2;
        uint8_t* stage = epi + ew * kWEpiBytes;
        int s = 0;
        uint32_t seen = 0;  // parity of each accumulator's uses
        for (unsigned tile = pair; tile < tiles; tile += pairs) {
            const int e = tile / per_e;
            const unsigned in = tile - e * per_e;
            const int row = (in / a.tiles_k * 2 + rank) * kM + quarter * 32;
            const int k0 = in % a.tiles_k * kWN + half * (kWN / 2);
            const bool some = seg.count(e) > 0;
            const uint32_t lanes = tmem + half * (kWN / 2) + (static_cast<uint32_t>(quarter * 32) << 16);
            const uint32_t base = lanes + s * kAccCols;
            bool whole = true;
            for (int p0 = 0, end, count = seg.count(e); p0 < count; p0 = end) {
                end = part_end<T>(p0, count);
                const int a_s = p0 == 0 ? s : s ^ 1;
                if (!ptx::mbar_wait(&c->acc_full[a_s], seen >> a_s & 1, kWaitNs + (end - p0) / kBK * kStageNs)) {
                    if (lane == 0) give_up(abort_flag);
                    *abort_flag = 1;
                }
                __syncwarp();
                if (__any_sync(0xffffffffu, *abort_flag)) {
                    whole = false;
                    break;
                }
                seen ^= 1u << a_s;
                ptx::tc_fence_after();
                if (p0 == 0) continue;
                ptx::tmem_add(base, lanes + a_s * kAccCols, kWN / 2);
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::bar_arrive_remote(ptx::map_to_rank(ptx::smem_u32(&c->acc_empty[a_s]), 0));
            }
            if (!whole) break;
            constexpr int COLS = 128 / (int)sizeof(T);  // of one tile store
#pragma unroll 1
            for (int j = 0; j < kWN / 2; j += COLS) {
                if (row >= a.N || k0 + j >= a.K) break;
                float v[COLS];
                if (!some) {
#pragma unroll
                    for (int i = 0; i < COLS; ++i) v[i] = 0.0f;
                } else if constexpr (COLS == 64) {
                    ptx::tmem_ld64(base + j, v);
                } else {
                    ptx::tmem_ld32(base + j, v);
                }
                if (lane == 0) ptx::tma_store_wait_read();
                __syncwarp();
                stage_row<T>(stage, v, lane);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::tma_store(&tmOut, ptx::smem_u32(stage), k0 + j, row, e);
            }
            if (some) {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::bar_arrive_remote(ptx::map_to_rank(ptx::smem_u32(&c->acc_empty[s]), 0));
                s ^= 1;
            }
        }
        if (lane == 0) ptx::tma_store_wait();
    }
    __syncwarp();
    end_block(tmem, warp);
}

// Column sums of the segments: a cluster of up to eight blocks per (expert, 256
// columns), its warps over the rows in turn, joined in warp and block order.
// (A second pass over grad_out.  Started beside expert_weight_kernel, one block
// an SM, it made both last longer: 1190 against 960 us for 32768 x 7168 rows.)
constexpr int kBiasBlocks = 8;

__global__ void __launch_bounds__(256)
    expert_bias_kernel(const bf16* dy, const int32_t* off, int64_t P, int N, int blocks, float* grad_bias) {
    __shared__ float part[8][256];
    __shared__ float joined[kBiasBlocks][256];  // the first block's is used
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)ptx::cluster_ctarank();
    const int e = blockIdx.y, c0 = blockIdx.x / blocks * 256, c = c0 + lane * 8;
    ptx::cluster_arrive();  // waited for before the first access to another block's shared memory
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t b = __ldg(off + e), t = __ldg(off + e + 1);
    const int64_t lo = b < 0 ? 0 : b > P ? P : b, hi = t > P ? P : t;
    float s[8] = {};
    if (c < N) {
#pragma unroll 8
        for (int64_t r = lo + rank * 8 + warp; r < hi; r += 8 * blocks) {
            const uint4 v = *reinterpret_cast<const uint4*>(dy + r * N + c);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack(w[i]);
                s[2 * i] += f.x;
                s[2 * i + 1] += f.y;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[warp][lane * 8 + i] = s[i];
    __syncthreads();
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += part[w][threadIdx.x];
    ptx::cluster_wait();
    ptx::st_cluster_u32(ptx::map_to_rank(ptx::smem_u32(&joined[rank][threadIdx.x]), 0), __float_as_uint(sum));
    ptx::cluster_sync();
    const int col = c0 + threadIdx.x;
    if (rank == 0 && col < N) {
        sum = 0.0f;
        for (int i = 0; i < blocks; ++i) sum += joined[i][threadIdx.x];
        grad_bias[(int64_t)e * N + col] = sum;
    }
}

// ---------------------------------------------------------------- host
// A bf16 (or fp32) tensor of `rank` dimensions, innermost first; strides in
// elements; 128 bytes of the innermost to a box.
cudaError_t encode(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                   const uint32_t* box, bool f32 = false) {
    using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::once_flag once;
    static EncodeFn fn = nullptr;
    static cudaError_t status = cudaSuccess;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        status = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
        if (status == cudaSuccess && q != cudaDriverEntryPointSuccess) status = cudaErrorNotSupported;
        fn = reinterpret_cast<EncodeFn>(p);
    });
    if (status != cudaSuccess || fn == nullptr) return status == cudaSuccess ? cudaErrorNotSupported : status;
    cuuint64_t d[5], st[5];
    cuuint32_t b[5], one[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        one[i] = 1;
        if (i > 0) st[i - 1] = strides[i - 1] * (f32 ? 4 : 2);
    }
    CUresult r = fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
                    const_cast<void*>(base), d, st, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t encode_rows(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int box_rows) {
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)cols};
    const uint32_t box[2] = {64, (uint32_t)box_rows};
    return encode(map, base, 2, dims, strides, box);
}

// Dynamic shared memory allowed for a kernel on the current device, once.
int allow_smem(const void* kern, int dev, size_t bytes) {
    static std::mutex mu;
    static std::unordered_map<int, std::unordered_map<const void*, bool>> done;  // device -> kernel
    std::lock_guard<std::mutex> lk(mu);
    bool& set = done[dev][kern];
    if (set) return MOE_OK;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (err != cudaSuccess) return set_cuda_error(err, "cudaFuncSetAttribute(expert matmul smem)");
    set = true;
    return MOE_OK;
}

template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), dim3 grid, int cluster, int threads, size_t smem, const char* who, void* stream,
           Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t err = cudaLaunchKernelEx(&cfg, kern, args...);
    return err == cudaSuccess ? MOE_OK : set_cuda_error(err, who);
}

int check_tiles(const char* who, int64_t tiles);

constexpr size_t kSmemMax = 232448;  // 227 KB
// Shared memory besides the stages: alignment, barriers, segments, staging.
size_t fixed_bytes(int E, size_t staging) { return 1024 + sizeof(Control) + segment_bytes(E) + staging; }
static_assert(1024 + 6 * (kABytes + 128 * kBK * 2) + sizeof(Control) + segment_bytes(kMaxE) + kEpiWarps * kEpiBytes <=
                  kSmemMax, "row products' shared memory");
static_assert(1024 + 5 * kWStageBytes + sizeof(Control) + segment_bytes(kMaxE) + kEpiWarps * kWEpiBytes <= kSmemMax,
              "weight gradient's shared memory");

int stages_of(size_t room, int stage_bytes) {
    const int fit = (int)(room / stage_bytes);
    return fit < kMaxStages ? fit : kMaxStages;
}

// Tokens per tile: enough for the experts' mean share of rows (narrow tiles
// leave room for more stages, which a product that waits for its weights
// needs), but no more than lets the tiles reach every pair of SMs: a call of
// few tiles takes as long as one of them.  (2-slot batch of 3373 tokens, one
// expert here, 200 x 232 with every part of the epilogue: 7.4 us with tiles of
// 32, 13.4 with tiles of 256.)
// The bounds on the mean, in us with tiles of 32 / 64 / 128 / 256 (uneven
// segments, 0.75 to 1.25 of the mean; 160 experts, 1544 by 1024, and 64, 7168 by
// 2048):  mean 16: 85 / 90 / 95 / 96, 277 / 272 / 273 / 272;  mean 32: 103 / 94 /
// 99 / 103, 307 / 278 / 283 / 285;  mean 56: 150 / 108 / 102 / 109, 404 / 295 /
// 291 / 304;  mean 128: 263 / 193 / 160 / 121, 714 / 509 / 409 / 339.  The rule is
// within 8% of the best width for means of 4 to 300.
void choose_tile(RowArgs& a, int pairs, int fit2, int fit4) {
    const int64_t mean = (a.P + a.E - 1) / a.E;
    a.tn_max = mean <= 16 ? 32 : mean <= 40 ? 64 : mean <= 80 ? 128 : 256;
    while (a.tn_max > 32 && (a.P + a.tn_max - 1) / a.tn_max * a.tiles_f < pairs) a.tn_max /= 2;
    // Where even tiles of 32 leave most SMs idle, 2 or 4 pairs share a tile's
    // reduction: a tile's time is then its weight's rows through one pair's
    // L2 ports (46 bytes a cycle and SM).  One token, 2 of 8 experts, 1024 by
    // 2 x 512: 6.7 us with four pairs, 7.3 with one; 16 rows of 20 experts,
    // 1888 by 248: 8.3 and 10.0; one row, 7168 by 256: 10.4 and 24.2.  Only where
    // all clusters run at once, so that each has at most one tile, whose sums need
    // no second buffer.
    a.split = 1;
    const int64_t most = (a.P / a.tn_max + (a.E < a.P ? a.E : a.P)) * a.tiles_f, blocks_k = (a.red + kBK - 1) / kBK;
    if (a.tn_max == 32 && most <= fit2)
        a.split = most <= fit4 && blocks_k >= 8 ? 4 : blocks_k >= 4 ? 2 : 1;
    a.stage_bytes = kABytes + a.tn_max / 2 * kBK * 2;
    a.stages = stages_of(kSmemMax - fixed_bytes(a.E, kEpiWarps * kEpiBytes + (a.split - 1) * kSumBytes), a.stage_bytes);
}

// Clusters of `split` pairs that run at once on the current device, looked up
// once (all forms of the kernel have a block to an SM).
int clusters_at_once(int dev, int split) {
    static std::mutex mu;
    static std::unordered_map<int, int> known;
    std::lock_guard<std::mutex> lk(mu);
    auto hit = known.find(dev * 8 + split);
    if (hit != known.end()) return hit->second;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * split);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemMax;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, expert_rows_kernel<kFwd>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    known[dev * 8 + split] = n;
    return n;
}

template <int MODE>
int run_rows(const char* who, const CUtensorMap& tmW, const void* x, int64_t x_cols, RowArgs& a, void* stream) {
    int dev = 0, sms = 0;
    int rc = sm_count(&dev, &sms);
    if (rc != MOE_OK) return rc;
    rc = allow_smem((const void*)expert_rows_kernel<MODE>, dev, kSmemMax);
    if (rc != MOE_OK) return rc;
    rc = allow_smem((const void*)expert_rows_kernel<kFwd>, dev, kSmemMax);
    if (rc != MOE_OK) return rc;
    const int fit2 = clusters_at_once(dev, 2), fit4 = clusters_at_once(dev, 4);
    choose_tile(a, sms / 2, fit2, fit4);
    rc = check_tiles(who, (a.P / a.tn_max + a.E) * a.tiles_f);
    if (rc != MOE_OK) return rc;
    CUtensorMap tmX, tmX16;  // boxes of 32 and of 16 tokens: a CTA's half of any number of units
    cudaError_t err = encode_rows(&tmX, x, a.P, x_cols, 32);
    if (err == cudaSuccess) err = encode_rows(&tmX16, x, a.P, x_cols, 16);
    if (err != cudaSuccess) return set_cuda_error(err, "cuTensorMapEncodeTiled(rows)");
    const size_t smem = (size_t)a.stages * a.stage_bytes +
                        fixed_bytes(a.E, kEpiWarps * kEpiBytes + (a.split - 1) * kSumBytes);
    // no more clusters than tiles
    const int64_t most = (a.P / a.tn_max + (a.E < a.P ? a.E : a.P)) * a.tiles_f;
    const int fit = a.split == 4 ? fit4 : a.split == 2 ? fit2 : sms / 2;
    const int blocks = (int)(most < fit ? most : fit) * 2 * a.split;
    return launch(expert_rows_kernel<MODE>, dim3(blocks), 2 * a.split, kThreads, smem, who, stream, tmW, tmX, tmX16, a);
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
    if (E > kMaxE || P >= (1ll << 31) - 256 || K > (1 << 24) || N > (1 << 24)) {
        snprintf(msg, sizeof msg, "%s: E=%d > 1024, P=%lld >= 2^31 - 256, or K=%d or N=%d > 2^24", who, E,
                 (long long)P, K, N);
        return set_error(MOE_ERR_UNSUPPORTED, msg);
    }
    return MOE_OK;
}

// Tiles are counted in 32 bits.
int check_tiles(const char* who, int64_t tiles) {
    if (tiles < (1ll << 31)) return MOE_OK;
    char msg[256];
    snprintf(msg, sizeof msg, "%s: %lld tiles of work are too many for one call", who, (long long)tiles);
    return set_error(MOE_ERR_UNSUPPORTED, msg);
}

int bad_pointer(const char* who) {
    char msg[256];
    snprintf(msg, sizeof msg, "%s: a pointer is null or not aligned (rows 16 bytes, offsets and bias 4)", who);
    return set_error(MOE_ERR_INVALID_ARG, msg);
}

}  // namespace

int read_expert_watchdog(unsigned int* count) {
    unsigned int v = 0;
    cudaError_t err = cudaMemcpyFromSymbol(&v, g_watchdog_trips_experts, sizeof(v));
    if (err != cudaSuccess) return set_cuda_error(err, "cudaMemcpyFromSymbol(expert watchdog)");
    *count = v;
    return MOE_OK;
}

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
    RowArgs a = {};
    a.off = expert_offsets;
    a.P = P;
    a.E = E;
    a.red = K;
    a.N = N;
    a.tiles_f = gated ? (N + kM - 1) / kM : (N + 2 * kM - 1) / (2 * kM);
    a.bias = bias;
    a.act = activation;
    a.extra = (const bf16*)residual;
    a.out = (bf16*)out;
    a.preact = (bf16*)preact_out;
    CUtensorMap tmW;
    cudaError_t err;
    const uint64_t k = K, n = N;
    if (gated) {
        // rows in the order (block of 8, gate or up, row of the block)
        const uint64_t dims[5] = {k, 8, 2, n / 8, (uint64_t)E}, strides[4] = {k, n * k, 8 * k, 2 * n * k};
        const uint32_t box[5] = {64, 8, 2, 8, 1};
        err = encode(&tmW, weight, 5, dims, strides, box);
    } else {
        const uint64_t dims[3] = {k, n, (uint64_t)E}, strides[2] = {k, n * k};
        const uint32_t box[3] = {64, kM, 1};
        err = encode(&tmW, weight, 3, dims, strides, box);
    }
    if (err != cudaSuccess) return set_cuda_error(err, "cuTensorMapEncodeTiled(weight)");
    return gated ? run_rows<kFwdGated>(who, tmW, x, K, a, stream) : run_rows<kFwd>(who, tmW, x, K, a, stream);
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
    RowArgs a = {};
    a.off = expert_offsets;
    a.P = P;
    a.E = E;
    a.red = N;
    a.N = K;
    a.tiles_f = (K + 2 * kM - 1) / (2 * kM);
    a.act = activation;
    a.extra = (const bf16*)preact;
    a.out = (bf16*)grad_x;
    const uint64_t dims[3] = {(uint64_t)K, (uint64_t)N, (uint64_t)E}, strides[2] = {(uint64_t)K, (uint64_t)N * K};
    const uint32_t box[3] = {64, kBK, 1};
    CUtensorMap tmW;
    cudaError_t err = encode(&tmW, weight, 3, dims, strides, box);
    if (err != cudaSuccess) return set_cuda_error(err, "cuTensorMapEncodeTiled(weight)");
    return gated ? run_rows<kGradGated>(who, tmW, grad_out, N, a, stream)
                 : run_rows<kGrad>(who, tmW, grad_out, N, a, stream);
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
    int dev = 0, sms = 0;
    int rc2 = sm_count(&dev, &sms);
    if (rc2 != MOE_OK) return rc2;
    WeightArgs a = {expert_offsets, P, E, N, K, (unsigned)(N + 2 * kM - 1) / (2 * kM),
                    (unsigned)(K + kWN - 1) / kWN, 0, grad_bias != nullptr};
    const size_t fixed = fixed_bytes(E, kEpiWarps * kWEpiBytes);
    a.stages = stages_of(kSmemMax - fixed, kWStageBytes);  // 6 up to 201 experts, else 5
    const size_t smem = fixed + (size_t)a.stages * kWStageBytes;
    const int64_t tiles = (int64_t)a.E * a.tiles_n * a.tiles_k;
    rc2 = check_tiles(who, tiles);
    if (rc2 != MOE_OK) return rc2;
    const dim3 grid(2 * (unsigned)(tiles < sms / 2 ? tiles : sms / 2));
    CUtensorMap tmY, tmX, tmOut;
    const bool f32 = dtype == MOE_DTYPE_F32;
    const uint64_t dims[3] = {(uint64_t)K, (uint64_t)N, (uint64_t)E}, strides[2] = {(uint64_t)K, (uint64_t)N * K};
    const uint32_t box[3] = {f32 ? 32u : 64u, 32, 1};
    // with P == 0 nothing is read through the maps; they still have to be valid ones
    cudaError_t err = encode_rows(&tmY, P ? grad_out : grad_weight, P ? P : 1, N, kBK);
    if (err == cudaSuccess) err = encode_rows(&tmX, P ? x : grad_weight, P ? P : 1, K, kBK);
    if (err == cudaSuccess) err = encode(&tmOut, grad_weight, 3, dims, strides, box, f32);
    if (err != cudaSuccess) return set_cuda_error(err, "cuTensorMapEncodeTiled(grad_weight)");
    if (f32) {
        rc2 = allow_smem((const void*)expert_weight_kernel<float>, dev, kSmemMax);
        if (rc2 == MOE_OK)
            rc2 = launch(expert_weight_kernel<float>, grid, 2, kThreads, smem, who, stream, tmY, tmX, tmOut,
                         a);
    } else {
        rc2 = allow_smem((const void*)expert_weight_kernel<bf16>, dev, kSmemMax);
        if (rc2 == MOE_OK)
            rc2 = launch(expert_weight_kernel<bf16>, grid, 2, kThreads, smem, who, stream, tmY, tmX, tmOut,
                         a);
    }
    if (rc2 != MOE_OK || !grad_bias) return rc2;
    int blocks = kBiasBlocks;  // with 16 rows to a warp or more
    while (blocks > 1 && P / E < 128 * blocks) blocks /= 2;
    return launch(expert_bias_kernel, dim3((N + 255) / 256 * blocks, E), blocks, 256, 0, who, stream,
                  (const bf16*)grad_out, expert_offsets, P, (int)N, blocks, grad_bias);
}

}  // extern "C"
