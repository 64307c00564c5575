// moe.hip -- a mixture-of-experts layer for a few tokens, on e4m3 experts.
//
//   l = x R^T, the top k of l, w = softmax, h_e = silu(G_e x) * (U_e x),
//   y = sum_e w_e D_e h_e.
//
// With few tokens the layer is as fast as the weights of the chosen experts
// come from memory, so each is read once per call for all tokens that chose
// it, and the activations keep their precision at no cost: a bfloat16 x is
// one matrix-core operand, a binary16 x the sum of two, a float32 value (x or
// h) of three, each the leading 8 mantissa bits of what the ones before left
// over.  The split is exact, and so is e4m3 in bfloat16, so the products are
// exact and are summed in float32.
//
// Three launches: the logits and the split of x; gate and up; down and the
// weighted sum; and a fourth that adds the parts where down is split.
#include <type_traits>

#include "fp8.h"

namespace sketch {
namespace {

constexpr int kWaves = 8;
constexpr int kMaxPairs = SKETCH_MOE_MAX_TOKENS * SKETCH_MOE_MAX_TOPK;

// Which tokens each chosen expert has: pairs (token * topk + slot) sorted by
// expert, then by pair, cut into the segments of the active experts.
struct Route {
    int32_t nact;
    int32_t expert[SKETCH_MOE_MAX_EXPERTS];
    int32_t begin[SKETCH_MOE_MAX_EXPERTS + 1];
    int32_t pair[kMaxPairs];
    float weight[kMaxPairs];   // by pair
};

struct MoeArgs {
    const void *router, *X;
    const uint8_t *gate, *up, *down;
    float* Y;
    int32_t* ids;
    float* weights;
    double* logits;      // [T][E]
    uint16_t* xs;        // [terms][T][ldh] bfloat16
    uint16_t* hs;        // [3][T * topk][ldi] bfloat16
    Route* route;
    float* parts;        // [splits][T][H], the down kernel's sums
    int64_t H, I, ldh, ldi;
    size_t gu_bytes, gu_scales, d_bytes, d_scales;   // one matrix, and its scales' offset
    int32_t gu_lds, d_lds;
    int32_t T, E, topk, renorm;
    int32_t splits, groups;   // of the down kernel
};

// An expert with few tokens has their NS terms in a tile's 16 columns, column
// NS t + s the term s of token t: one load and one matrix instruction for the
// terms of 16 / NS tokens, whose sums are added at the end.  With more tokens
// the terms follow one another.  (Down of 2 experts of 4096 x 11008 at 1 token:
// 25 -> 20 us; gate and up of 64 of 2048 x 1408 in binary16, 7 tokens: 39 ->
// 36 us.  Two tiles of columns at once for up to 10 tokens took more registers
// than two workgroups to a CU leave and lost: 20 -> 23 us.)
template <int NS> constexpr int kTokensOf = 16 / NS;

template <int DT> constexpr int x_terms() { return DT == SKETCH_BF16 ? 1 : DT == SKETCH_F16 ? 2 : 3; }

// Leading 8 mantissa bits of v as bfloat16; v becomes the rest (exact).
__device__ inline uint16_t take_bf16(float& v) {
    const uint32_t u = __float_as_uint(v) & 0xFFFF0000u;
    v -= __uint_as_float(u);
    return uint16_t(u >> 16);
}

__device__ inline u32x4 take8(float (&v)[8]) {
    uint32_t h[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) h[q] = take_bf16(v[q]);
    return u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
}

// Logits of expert blockIdx.x for NT tokens; the sums are float64,
// so that no two logits change places by rounding.  All workgroups also share
// out the split of x.
template <int DT, int NT>
__global__ __launch_bounds__(256) void moe_logits_kernel(MoeArgs a) {
    __shared__ double part[4][NT];
    const int tid = threadIdx.x, e = blockIdx.x, t0 = blockIdx.y * NT;
    double sum[NT] = {};
    for (int64_t j = tid * 8; j < a.H; j += 2048) {
        float w[8], x[NT][8];
        load_row8<DT>(a.router, e, a.H, j, w);
#pragma unroll
        for (int i = 0; i < NT; ++i) load_row8<DT>(a.X, min(t0 + i, a.T - 1), a.H, j, x[i]);
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
            for (int i = 0; i < NT; ++i) sum[i] += double(x[i][q]) * double(w[q]);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum[i] += __shfl_xor(sum[i], d);
        if ((tid & 63) == 0) part[tid >> 6][i] = sum[i];
    }
    const int64_t total = int64_t(a.T) * a.ldh, step = int64_t(gridDim.x) * gridDim.y * 2048;
    for (int64_t u = (int64_t(blockIdx.y) * gridDim.x + e) * 2048 + tid * 8; u < total; u += step) {
        const int64_t t = u / a.ldh, j = u % a.ldh;   // ldh is a multiple of 8
        float v[8];
        load_row8<DT>(a.X, t, a.H, j, v);
#pragma unroll
        for (int s = 0; s < x_terms<DT>(); ++s) *reinterpret_cast<u32x4*>(a.xs + s * total + u) = take8(v);
    }
    __syncthreads();
    if (tid < NT && t0 + tid < a.T)
        a.logits[int64_t(t0 + tid) * a.E + e] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
}

// Order of the logits as unsigned integers; NaN is the largest, 0 and the
// largest uint64 are free.
__device__ inline uint64_t order_key(double l) {
    if (l != l) return ~0ull - 1;
    const uint64_t u = uint64_t(__double_as_longlong(l + 0.0));   // -0 -> +0
    return u >> 63 ? ~u : u | (1ull << 63);
}

// The top k of one token, by one wave.
__device__ inline void top_k(const double* l, int E, int topk, int lane, int32_t* ids) {
    if (E <= 64) {   // each lane counts the experts before its own
        const uint64_t key = lane < E ? order_key(l[lane]) : 0;
        int rank = 0;
        for (int j0 = 0; j0 < E; j0 += 8)   // lanes past E have key 0, before nobody
#pragma unroll
            for (int j = j0; j < j0 + 8; ++j) {
                const uint64_t other = uint64_t(uint32_t(__builtin_amdgcn_readlane(int(key >> 32), j))) << 32 |
                                       uint32_t(__builtin_amdgcn_readlane(int(key), j));
                rank += other + (j < lane) > key;   // j's earlier than the lane's come before it when equal
            }
        if (lane < E && rank < topk) ids[rank] = lane;
        return;
    }
    constexpr int kPer = SKETCH_MOE_MAX_EXPERTS / 64;
    uint64_t key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = lane + 64 * i < E ? order_key(l[lane + 64 * i]) : 0;
    for (int s = 0; s < topk; ++s) {
        uint64_t best = key[0];
        int at = lane;
#pragma unroll
        for (int i = 1; i < kPer; ++i)
            if (key[i] > best) best = key[i], at = lane + 64 * i;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint64_t ob = __shfl_xor(best, d);
            const int oa = __shfl_xor(at, d);
            if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
        }
        if (lane == 0) ids[s] = at;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (at == lane + 64 * i) key[i] = 0;
    }
}

// The top k of every token and the segments, by a whole workgroup.  An
// expert's tokens are a bit mask: a token's place is the bits before its own.
static_assert(SKETCH_MOE_MAX_TOKENS <= 64, "one bit per token");

__device__ inline void build_route(const MoeArgs& a, const double* logits, Route& rt, int32_t* ids) {
    __shared__ uint64_t mask[SKETCH_MOE_MAX_EXPERTS];
    __shared__ int32_t start[SKETCH_MOE_MAX_EXPERTS];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, P = a.T * a.topk;
    for (int e = tid; e < a.E; e += kWaves * 64) mask[e] = 0;
    for (int t = wave; t < a.T; t += kWaves) top_k(logits + int64_t(t) * a.E, a.E, a.topk, lane, ids + t * a.topk);
    __syncthreads();
    for (int p = tid; p < P; p += kWaves * 64)
        atomicOr(reinterpret_cast<unsigned long long*>(&mask[ids[p]]), 1ull << (p / a.topk));
    __syncthreads();
    if (wave == 0) {
        int nact = 0, pairs = 0;
        for (int e0 = 0; e0 < a.E; e0 += 64) {
            const int e = e0 + lane, count = e < a.E ? __popcll(mask[e]) : 0;
            int before = count;   // inclusive sum over the lanes
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int up = __shfl_up(before, d);
                if (lane >= d) before += up;
            }
            const uint64_t active = __ballot(count > 0);
            if (count > 0) {
                const int i = nact + __popcll(active & ((1ull << lane) - 1));
                rt.expert[i] = e;
                rt.begin[i] = start[e] = pairs + before - count;
            }
            nact += __popcll(active);
            pairs += __shfl(before, 63);
        }
        if (lane == 0) {
            rt.nact = nact;
            rt.begin[nact] = P;
        }
    }
    __syncthreads();
    for (int p = tid; p < P; p += kWaves * 64) {
        const int e = ids[p];
        rt.pair[start[e] + __popcll(mask[e] & ((1ull << (p / a.topk)) - 1))] = p;
    }
    __syncthreads();
}

// The route and the weights to memory, for the caller and the next launch.
__device__ inline void publish_route(const MoeArgs& a, const double* logits, const Route& rt, const int32_t* ids) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, P = a.T * a.topk;
    for (int t = wave; t < a.T; t += kWaves) {
        const double* l = logits + int64_t(t) * a.E;
        const double top = l[ids[t * a.topk]];
        double sum = 0.0;
        if (!a.renorm)
            for (int e = lane; e < a.E; e += 64) sum += exp(l[e] - top);
        else if (lane < a.topk)
            sum = exp(l[ids[t * a.topk + lane]] - top);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
        if (lane < a.topk) {
            const int p = t * a.topk + lane;
            const float w = float(exp(l[ids[p]] - top) / sum);
            a.ids[p] = ids[p];
            a.weights[p] = w;
            a.route->weight[p] = w;
        }
    }
    for (int p = tid; p < P; p += kWaves * 64) a.route->pair[p] = rt.pair[p];
    for (int i = tid; i <= rt.nact; i += kWaves * 64) {
        if (i < rt.nact) a.route->expert[i] = rt.expert[i];
        a.route->begin[i] = rt.begin[i];
    }
    if (tid == 0) a.route->nact = rt.nact;
}

__device__ inline void load_w(const uint8_t* row, int c, u32x4 (&w)[2]) {
    w[0] = *reinterpret_cast<const u32x4*>(row + 16 * c);
    w[1] = *reinterpret_cast<const u32x4*>(row + 64 + 16 * c);
}

// A fragment of bfloat16 values.  Tokens past an expert's last one read another
// token's: no lane skips a load, and their products are not used.
__device__ inline void load_x(const uint16_t* row, int c, bf16x8 (&x)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const bf16x8*>(row + 64 * (j >> 1) + 16 * c + 8 * (j & 1));
}

// Loads issued so far stay before what follows.
__device__ inline void keep_order() { asm volatile("" ::: "memory"); }

// Gate and up: a workgroup takes kUpRows rows of one active expert at a time,
// its waves share out the blocks of 128 columns, and their sums meet in LDS.
// (16 rows, two blocks in flight: 41 us instead of 38 us for 2 experts of
// 4096 x 11008, 155 us instead of 132 us for 8 with 16 tokens: x is loaded for
// half the rows.)  The last workgroup only publishes the route.
//
// FEW (few tokens, a small router): every workgroup sums the logits for itself
// and splits x into LDS, instead of the launch before this one (1 token, 8
// experts of 512 x 256: 2.6 + 6.6 us in two launches, 7.9 us in one; with a
// router of 8 x 4096 4.7 + 43.5 us against 50.2 us, no gain any more).
constexpr int kUpTiles = 2, kUpRows = 16 * kUpTiles;
constexpr int kFewTokens = 4, kFewLogits = 4 * kWaves;
constexpr int64_t kFewTerms = 16384;   // tokens x experts x columns
constexpr size_t kFewLds = 32 * 1024;

template <int DT, bool FEW>
__global__ __launch_bounds__(kWaves * 64) void moe_up_kernel(MoeArgs a) {
    constexpr int NS = x_terms<DT>();
    extern __shared__ __attribute__((aligned(16))) uint16_t xlds[];   // FEW: [terms][T][ldh]
    __shared__ Route rt;
    __shared__ int32_t ids[kMaxPairs];
    __shared__ float part[kWaves][2][16][16 * kUpTiles + 1];
    __shared__ double logits[FEW ? kFewLogits : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4;
    const int64_t plane = int64_t(a.T) * a.ldh;
    if constexpr (FEW) {
        constexpr int kEach = kFewLogits / kWaves;   // (token, expert) wave + 8 i
        const int n = a.T * a.E;
        double sum[kEach] = {};
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = wave + kWaves * i;
            if (at >= n) break;
            for (int64_t j = lane * 8; j < a.H; j += 512) {
                float x[8], w[8];
                load_row8<DT>(a.X, at / a.E, a.H, j, x);
                load_row8<DT>(a.router, at % a.E, a.H, j, w);
#pragma unroll
                for (int q = 0; q < 8; ++q) sum[i] += double(x[q]) * double(w[q]);
            }
        }
        for (int64_t u = tid * 8; u < plane; u += kWaves * 64 * 8) {
            const int64_t t = u / a.ldh, j = u % a.ldh;
            float v[8];
            load_row8<DT>(a.X, t, a.H, j, v);
#pragma unroll
            for (int s = 0; s < NS; ++s) *reinterpret_cast<u32x4*>(xlds + s * plane + u) = take8(v);
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) sum[i] += __shfl_xor(sum[i], d);
            if (lane == 0 && wave + kWaves * i < n) logits[wave + kWaves * i] = sum[i];
        }
        __syncthreads();
    }
    const double* l = FEW ? logits : a.logits;
    build_route(a, l, rt, ids);
    if (blockIdx.x == gridDim.x - 1) {
        publish_route(a, l, rt, ids);
        return;
    }
    const int tiles = int(a.ldi / kUpRows), items = rt.nact * tiles, kbs = int(a.ldh / 128);
    const int64_t hplane = int64_t(a.T) * a.topk * a.ldi;
    for (int it = blockIdx.x; it < items; it += gridDim.x - 1) {
        const int act = it / tiles, m0 = it % tiles * kUpRows, e = __builtin_amdgcn_readfirstlane(rt.expert[act]);
        const int begin = __builtin_amdgcn_readfirstlane(rt.begin[act]), pend = __builtin_amdgcn_readfirstlane(rt.begin[act + 1]);
        const uint8_t *G = a.gate + e * a.gu_bytes, *U = a.up + e * a.gu_bytes;
        int64_t roff[kUpTiles];
#pragma unroll
        for (int i = 0; i < kUpTiles; ++i) roff[i] = min(int64_t(m0 + 16 * i + r), a.I - 1) * a.ldh;
        const int64_t srow = min(int64_t(m0), a.I - 1) / 128 * a.gu_lds;   // kUpRows rows lie in one block of 128
        const uint8_t *gs = G + a.gu_scales + srow, *us = U + a.gu_scales + srow;
        auto tokens = [&](auto in_columns, int first) {
            constexpr bool COLUMNS = decltype(in_columns)::value;
            constexpr int SEQ = COLUMNS ? 1 : NS, COL = COLUMNS ? NS : 1;   // terms one after the other, in columns
            const uint16_t* x = (FEW ? xlds : a.xs) + int64_t(rt.pair[min(first + r / COL, pend - 1)] / a.topk) * a.ldh +
                                r % COL * plane;
            f32x4 ga[kUpTiles], ua[kUpTiles];
#pragma unroll
            for (int i = 0; i < kUpTiles; ++i) ga[i] = ua[i] = f32x4{0, 0, 0, 0};
            for (int kb = wave; kb < kbs; kb += kWaves) {
                u32x4 gw[kUpTiles][2], uw[kUpTiles][2];
                bf16x8 xv[SEQ][4];
#pragma unroll
                for (int i = 0; i < kUpTiles; ++i) {
                    load_w(G + roff[i] + kb * 128, c, gw[i]);
                    load_w(U + roff[i] + kb * 128, c, uw[i]);
                }
#pragma unroll
                for (int s = 0; s < SEQ; ++s) load_x(x + s * plane + kb * 128, c, xv[s]);
                const float gsc = fp8_scale(gs[kb]), usc = fp8_scale(us[kb]);
                keep_order();
#pragma unroll
                for (int i = 0; i < kUpTiles; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bf16x8 gb = fp8_widen(gw[i][j >> 1][2 * (j & 1)], gw[i][j >> 1][2 * (j & 1) + 1], gsc);
                        const bf16x8 ub = fp8_widen(uw[i][j >> 1][2 * (j & 1)], uw[i][j >> 1][2 * (j & 1) + 1], usc);
#pragma unroll
                        for (int s = 0; s < SEQ; ++s) {
                            ga[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(gb, xv[s][j], ga[i], 0, 0, 0);
                            ua[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ub, xv[s][j], ua[i], 0, 0, 0);
                        }
                    }
            }
#pragma unroll
            for (int i = 0; i < kUpTiles; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    part[wave][0][r][16 * i + 4 * c + v] = ga[i][v];
                    part[wave][1][r][16 * i + 4 * c + v] = ua[i][v];
                }
            __syncthreads();
            for (int u = tid; u < 16 / COL * kUpRows; u += kWaves * 64) {
                const int tok = u / kUpRows, row = u % kUpRows;
                if (first + tok >= pend) break;
                float gv = 0.0f, uv = 0.0f;
#pragma unroll
                for (int s = 0; s < COL; ++s)
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) {
                        gv += part[w][0][tok * COL + s][row];
                        uv += part[w][1][tok * COL + s][row];
                    }
                float h = m0 + row < a.I ? gv / (1.0f + expf(-gv)) * uv : 0.0f;
                uint16_t* dst = a.hs + int64_t(rt.pair[first + tok]) * a.ldi + m0 + row;
#pragma unroll
                for (int s = 0; s < 3; ++s) dst[s * hplane] = take_bf16(h);
            }
            __syncthreads();
        };
        if constexpr (FEW) {
            static_assert(kFewTokens <= kTokensOf<NS>, "one tile of columns");
            tokens(std::true_type{}, begin);
        } else if (NS > 1 && pend - begin <= kTokensOf<NS>) {
            tokens(std::true_type{}, begin);
        } else {
            for (int p0 = begin; p0 < pend; p0 += 16) tokens(std::false_type{}, p0);
        }
    }
}

// Down and the weighted sum.  A workgroup owns 16 TILES outputs and a run of
// the active experts' blocks of 128 columns, which its waves take in turns;
// each wave sums into a tile of its own, the tiles are added in the order of
// the waves, and the runs in theirs by moe_add_kernel (the last workgroup of a
// row group adding them up was measured: the fences that takes cost 75 us).
// The loads of h, 4 or 12 to a block, serve 64 outputs (2 experts of 4096 x
// 11008 at 1 token: 20 us, 21 us with 32; 8 with 16 tokens 89 us and 100 us)
// and come with the weights' loads, not after them; layers too small to fill
// half the chip that way take 16 (512 x 256: 8.2 -> 5.9 us).
template <int TILES>
__global__ __launch_bounds__(kWaves * 64) void moe_down_kernel(MoeArgs a) {
    constexpr int kRows = 16 * TILES;
    extern __shared__ __attribute__((aligned(16))) float ytile[];   // [kWaves][T][kRows]
    __shared__ Route rt;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4;
    {   // all of the route at once: at most a segment per pair
        const int P = a.T * a.topk, A = min(P, a.E);
        for (int i = tid; i < P; i += kWaves * 64) {
            rt.pair[i] = a.route->pair[i];
            rt.weight[i] = a.route->weight[i];
        }
        for (int i = tid; i <= A; i += kWaves * 64) {
            if (i < A) rt.expert[i] = a.route->expert[i];
            rt.begin[i] = a.route->begin[i];
        }
        if (tid == 0) rt.nact = a.route->nact;
    }
    for (int u = tid; u < kWaves * a.T * kRows; u += kWaves * 64) ytile[u] = 0.0f;
    __syncthreads();
    float* y = ytile + wave * a.T * kRows;
    const int group = blockIdx.x % a.groups, split = blockIdx.x / a.groups;
    const int64_t m0 = int64_t(group) * kRows;
    const int kbs = int(a.ldi / 128), nact = __builtin_amdgcn_readfirstlane(rt.nact);
    const int u0 = int(int64_t(nact) * kbs * split / a.splits), u1 = int(int64_t(nact) * kbs * (split + 1) / a.splits);
    const int64_t hplane = int64_t(a.T) * a.topk * a.ldi;
    int64_t roff[TILES];
#pragma unroll
    for (int i = 0; i < TILES; ++i) roff[i] = min(m0 + 16 * i + r, a.H - 1) * a.ldi + 16 * c;
    // Tokens first .. pend - 1 of one expert, up to 5 with their terms in columns
    // of their own, or up to 16 with one term after the other.
    auto expert = [&](auto in_columns, int act, int first, int pend) {
        constexpr bool COLUMNS = decltype(in_columns)::value;
        constexpr int NS = COLUMNS ? 1 : 3;
        const int e = __builtin_amdgcn_readfirstlane(rt.expert[act]);
        const int kend = min(u1 - act * kbs, kbs), kfirst = max(u0 - act * kbs, 0) + wave;
        const uint8_t *D = a.down + e * a.d_bytes, *ds = D + a.d_scales + m0 / 128 * a.d_lds;
        const int tok = first + (COLUMNS ? r / 3 : r), pair = rt.pair[min(tok, pend - 1)];
        const uint16_t* h = a.hs + int64_t(pair) * a.ldi + (COLUMNS ? r % 3 * hplane : 0);
        f32x4 acc[TILES];
#pragma unroll
        for (int i = 0; i < TILES; ++i) acc[i] = f32x4{0, 0, 0, 0};
        for (int kb = kfirst; kb < kend; kb += kWaves) {
            u32x4 w[TILES][2];
            bf16x8 hv[NS][4];
#pragma unroll
            for (int i = 0; i < TILES; ++i) load_w(D + kb * 128 + roff[i], 0, w[i]);
#pragma unroll
            for (int s = 0; s < NS; ++s) load_x(h + s * hplane + kb * 128, c, hv[s]);
            const float scale = fp8_scale(ds[kb]);
            keep_order();
#pragma unroll
            for (int i = 0; i < TILES; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf16x8 wb = fp8_widen(w[i][j >> 1][2 * (j & 1)], w[i][j >> 1][2 * (j & 1) + 1], scale);
#pragma unroll
                    for (int s = 0; s < NS; ++s) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb, hv[s][j], acc[i], 0, 0, 0);
                }
        }
        if constexpr (COLUMNS) {
#pragma unroll
            for (int i = 0; i < TILES; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][v] = (acc[i][v] + __shfl_down(acc[i][v], 1)) + __shfl_down(acc[i][v], 2);
        }
        if (tok < pend && (!COLUMNS || r % 3 == 0)) {
            const float w = rt.weight[pair];
            f32x4* dst = reinterpret_cast<f32x4*>(y + pair / a.topk * kRows + 4 * c);
#pragma unroll
            for (int i = 0; i < TILES; ++i) dst[4 * i] += w * acc[i];
        }
    };
    for (int act = u0 / kbs; act * kbs < u1; ++act) {
        const int begin = __builtin_amdgcn_readfirstlane(rt.begin[act]), pend = __builtin_amdgcn_readfirstlane(rt.begin[act + 1]);
        if (pend - begin <= kTokensOf<3>)
            expert(std::true_type{}, act, begin, pend);
        else
            for (int p0 = begin; p0 < pend; p0 += 16) expert(std::false_type{}, act, p0, pend);
    }
    __syncthreads();
    float* out = a.splits > 1 ? a.parts + int64_t(split) * a.T * a.H : a.Y;
    for (int u = tid; u < a.T * kRows; u += kWaves * 64) {
        const int64_t m = m0 + u % kRows;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += ytile[w * a.T * kRows + u];
        if (m < a.H) out[int64_t(u / kRows) * a.H + m] = sum;
    }
}

__global__ __launch_bounds__(256) void moe_add_kernel(MoeArgs a) {
    const int64_t n = int64_t(a.T) * a.H, i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    float sum = 0.0f;
    for (int s0 = 0; s0 < a.splits; s0 += 8) {   // 8 loads in flight
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = a.parts[min(s0 + q, a.splits - 1) * n + i];
        keep_order();
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (s0 + q < a.splits) sum += v[q];
    }
    a.Y[i] = sum;
}

// How down is cut: 64 or 16 outputs to a row group, and the workgroups of a row
// group, about two per compute unit in all, each with some blocks to go through
// (every token has topk experts).
struct DownCut {
    int tiles, groups, splits;
};

DownCut down_cut(const sketch_moe_params* p, int64_t kbs) {
    const int64_t ncu = compute_units(), steps = (p->topk * kbs + kWaves / 2 - 1) / (kWaves / 2);
    DownCut d{};
    for (int tiles : {4, 1}) {
        const int64_t rows = 16 * tiles, groups = (p->H + rows - 1) / rows;
        int64_t s = (2 * ncu + groups - 1) / groups;
        if (s > steps) s = steps;
        d = {tiles, int(groups), int(s < 1 ? 1 : s)};
        if (groups * d.splits >= ncu / 2) break;
    }
    return d;
}

struct MoeLayout {
    sketch_fp8_shape gu, d;
    size_t xs, hs, route, parts, total;
    DownCut cut;
};

sketch_status moe_layout(const sketch_moe_params* p, int64_t tokens, MoeLayout* L) {
    if (!p || p->H < 1 || p->I < 1 || p->E < 1 || p->E > SKETCH_MOE_MAX_EXPERTS || p->topk < 1 ||
        p->topk > SKETCH_MOE_MAX_TOPK || p->topk > p->E)
        return SKETCH_EINVAL;
    if ((p->renorm != 0 && p->renorm != 1) ||
        (p->x_dtype != SKETCH_F32 && p->x_dtype != SKETCH_BF16 && p->x_dtype != SKETCH_F16))
        return SKETCH_EINVAL;
    if (tokens < 0 || tokens > SKETCH_MOE_MAX_TOKENS) return SKETCH_EINVAL;
    const sketch_fp8_params gu{p->I, p->H, 128, p->E}, d{p->H, p->I, 128, p->E};
    if (fp8_shape(&gu, &L->gu) != SKETCH_OK || fp8_shape(&d, &L->d) != SKETCH_OK) return SKETCH_EINVAL;
    const size_t terms = p->x_dtype == SKETCH_BF16 ? 1 : p->x_dtype == SKETCH_F16 ? 2 : 3;
    L->xs = align256(size_t(tokens) * p->E * sizeof(double));
    L->hs = align256(L->xs + terms * size_t(tokens) * L->gu.ld * 2);
    L->route = align256(L->hs + 3 * size_t(tokens) * p->topk * L->d.ld * 2);
    L->parts = align256(L->route + sizeof(Route));
    L->cut = down_cut(p, L->d.col_blocks);
    L->total = align256(L->parts + (L->cut.splits > 1 ? size_t(L->cut.splits) * size_t(tokens) * size_t(p->H) * 4 : 0));
    return SKETCH_OK;
}

}  // namespace
}  // namespace sketch

using namespace sketch;

extern "C" {

sketch_status sketch_moe_workspace_bytes(const sketch_moe_params* p, int64_t tokens, size_t* bytes) {
    MoeLayout L;
    const sketch_status rc = moe_layout(p, tokens, &L);
    if (rc != SKETCH_OK) return rc;
    if (!bytes) return SKETCH_EINVAL;
    *bytes = tokens == 0 ? 0 : L.total;
    return SKETCH_OK;
}

sketch_status sketch_moe(const sketch_moe_params* p, const void* router, const void* gate, const void* up,
                         const void* down, const void* X, int64_t tokens, float* Y, int32_t* ids, float* weights,
                         void* workspace, size_t workspace_bytes, void* stream) {
    MoeLayout L;
    const sketch_status rc = moe_layout(p, tokens, &L);
    if (rc != SKETCH_OK) return rc;
    if (tokens == 0) return SKETCH_OK;
    for (const void* q : {router, gate, up, down, X, static_cast<const void*>(Y), static_cast<const void*>(ids),
                          static_cast<const void*>(weights), static_cast<const void*>(workspace)})
        if (!q || !aligned16(q)) return SKETCH_EINVAL;
    if (workspace_bytes < L.total) return SKETCH_ESMALL;
    const size_t T = size_t(tokens), E = size_t(p->E), H = size_t(p->H), es = elem_bytes(p->x_dtype);
    const Range rx{X, T * H * es}, in[] = {{router, E * H * es}, {gate, E * L.gu.bytes}, {up, E * L.gu.bytes}, {down, E * L.d.bytes}},
                out[] = {{Y, T * H * 4}, {ids, T * p->topk * 4}, {weights, T * p->topk * 4}, {workspace, L.total}};
    for (int i = 0; i < 4; ++i) {
        if (i > 0 && overlap(out[i], rx)) return SKETCH_EINVAL;   // Y is written when X is done with
        for (int j = 0; j < 4; ++j)
            if (overlap(out[i], in[j]) || (j < i && overlap(out[i], out[j]))) return SKETCH_EINVAL;
    }
    const hipStream_t st = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    MoeArgs a;
    a.router = router;
    a.X = X;
    a.gate = static_cast<const uint8_t*>(gate);
    a.up = static_cast<const uint8_t*>(up);
    a.down = static_cast<const uint8_t*>(down);
    a.Y = Y;
    a.ids = ids;
    a.weights = weights;
    a.logits = reinterpret_cast<double*>(ws);
    a.xs = reinterpret_cast<uint16_t*>(ws + L.xs);
    a.hs = reinterpret_cast<uint16_t*>(ws + L.hs);
    a.route = reinterpret_cast<Route*>(ws + L.route);
    a.parts = reinterpret_cast<float*>(ws + L.parts);
    a.splits = L.cut.splits;
    a.groups = L.cut.groups;
    a.H = p->H;
    a.I = p->I;
    a.ldh = L.gu.ld;
    a.ldi = L.d.ld;
    a.gu_bytes = L.gu.bytes;
    a.gu_scales = L.gu.scales_offset;
    a.d_bytes = L.d.bytes;
    a.d_scales = L.d.scales_offset;
    a.gu_lds = int32_t(L.gu.lds);
    a.d_lds = int32_t(L.d.lds);
    a.T = int32_t(tokens);
    a.E = p->E;
    a.topk = p->topk;
    a.renorm = p->renorm;
    const int64_t ncu = compute_units();
    const int64_t items = (tokens * p->topk < p->E ? tokens * p->topk : int64_t(p->E)) * (L.d.ld / kUpRows);
    const unsigned up_grid = unsigned(items < 2 * ncu ? items : 2 * ncu) + 1;
    const size_t lds = size_t(kWaves) * tokens * 16 * L.cut.tiles * sizeof(float);
    // tokens of a workgroup that sums logits: 4 share the loads of the router, but one is sooner done
    // while all workgroups are in flight together (8 experts of 4096, 16 tokens: 7.8 us with 4, 4.7 us
    // with one; 256 of 2048, 64 tokens: 14 us and 17 us)
    const int nt = tokens * p->E <= 8 * ncu ? 1 : 4;
    auto go = [&](auto one, auto four, auto gate_up, auto gate_up_few, int terms) {
        const size_t xlds = size_t(terms) * tokens * L.gu.ld * 2;
        if (tokens <= kFewTokens && tokens * p->E <= kFewLogits && tokens * p->E * p->H <= kFewTerms && xlds <= kFewLds) {
            gate_up_few<<<up_grid, kWaves * 64, xlds, st>>>(a);
        } else {
            const auto logits = nt == 1 ? one : four;
            logits<<<dim3(unsigned(p->E), unsigned((tokens + nt - 1) / nt)), 256, 0, st>>>(a);
            if (hipGetLastError() != hipSuccess) return SKETCH_EDEVICE;
            gate_up<<<up_grid, kWaves * 64, 0, st>>>(a);
        }
        if (hipGetLastError() != hipSuccess) return SKETCH_EDEVICE;
        const unsigned grid = unsigned(L.cut.groups) * unsigned(L.cut.splits);
        if (L.cut.tiles == 4)
            moe_down_kernel<4><<<grid, kWaves * 64, lds, st>>>(a);
        else
            moe_down_kernel<1><<<grid, kWaves * 64, lds, st>>>(a);
        if (L.cut.splits == 1) return launch_status();
        if (hipGetLastError() != hipSuccess) return SKETCH_EDEVICE;
        moe_add_kernel<<<unsigned((tokens * p->H + 255) / 256), 256, 0, st>>>(a);
        return launch_status();
    };
    switch (p->x_dtype) {
        case SKETCH_F32:
            return go(moe_logits_kernel<SKETCH_F32, 1>, moe_logits_kernel<SKETCH_F32, 4>, moe_up_kernel<SKETCH_F32, false>,
                      moe_up_kernel<SKETCH_F32, true>, 3);
        case SKETCH_BF16:
            return go(moe_logits_kernel<SKETCH_BF16, 1>, moe_logits_kernel<SKETCH_BF16, 4>,
                      moe_up_kernel<SKETCH_BF16, false>, moe_up_kernel<SKETCH_BF16, true>, 1);
        default:
            return go(moe_logits_kernel<SKETCH_F16, 1>, moe_logits_kernel<SKETCH_F16, 4>, moe_up_kernel<SKETCH_F16, false>,
                      moe_up_kernel<SKETCH_F16, true>, 2);
    }
}

}  // extern "C"
