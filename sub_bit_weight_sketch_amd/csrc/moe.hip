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
// Three launches: the logits (one workgroup per expert) and the split of x;
// gate and up; down and the weighted sum.
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
    int64_t H, I, ldh, ldi;
    size_t gu_bytes, gu_scales, d_bytes, d_scales;   // one matrix, and its scales' offset
    int32_t gu_lds, d_lds;
    int32_t T, E, topk, renorm;
};

template <int DT> constexpr int x_terms() { return DT == SKETCH_BF16 ? 1 : DT == SKETCH_F16 ? 2 : 3; }

// Leading 8 mantissa bits of v as bfloat16; v becomes the rest (exact).
__device__ inline uint16_t take_bf16(float& v) {
    const uint32_t u = __float_as_uint(v) & 0xFFFF0000u;
    v -= __uint_as_float(u);
    return uint16_t(u >> 16);
}

template <int DT>
__global__ __launch_bounds__(256) void moe_logits_kernel(MoeArgs a) {
    __shared__ double part[4][SKETCH_MOE_MAX_TOKENS];
    const int tid = threadIdx.x, wave = tid >> 6, e = blockIdx.x;
    const int64_t total = int64_t(a.T) * a.ldh;
    for (int64_t u = int64_t(e) * 256 + tid; u < total; u += int64_t(a.E) * 256) {
        const int64_t t = u / a.ldh, j = u % a.ldh;
        float v = j < a.H ? load_elem<DT>(a.X, t * a.H + j) : 0.0f;
#pragma unroll
        for (int s = 0; s < x_terms<DT>(); ++s)
            a.xs[s * total + u] = DT == SKETCH_BF16 && j < a.H ? static_cast<const uint16_t*>(a.X)[t * a.H + j] : take_bf16(v);
    }
    for (int t = 0; t < a.T; ++t) {
        double sum = 0.0;
        for (int64_t j = tid; j < a.H; j += 256)
            sum += double(load_elem<DT>(a.X, t * a.H + j)) * double(load_elem<DT>(a.router, e * a.H + j));
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
        if ((tid & 63) == 0) part[wave][t] = sum;
    }
    __syncthreads();
    if (tid < a.T) a.logits[int64_t(tid) * a.E + e] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
}

// Order of the logits as unsigned integers; NaN is the largest, 0 is free.
__device__ inline uint64_t order_key(double l) {
    if (l != l) return ~0ull;
    const uint64_t u = uint64_t(__double_as_longlong(l + 0.0));   // -0 -> +0
    return u >> 63 ? ~u : u | (1ull << 63);
}

// The top k of every token and the segments, by all 512 threads of a
// workgroup.  Workgroup 0 also computes the weights and hands everything on.
__device__ void build_route(const MoeArgs& a, Route& rt, int32_t* ids, bool publish) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    constexpr int kPer = SKETCH_MOE_MAX_EXPERTS / 64;
    for (int t = wave; t < a.T; t += kWaves) {
        const double* l = a.logits + int64_t(t) * a.E;
        uint64_t key[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) key[i] = lane + 64 * i < a.E ? order_key(l[lane + 64 * i]) : 0;
        for (int s = 0; s < a.topk; ++s) {
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
            if (lane == 0) ids[t * a.topk + s] = at;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (at == lane + 64 * i) key[i] = 0;
        }
        if (publish) {
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
    }
    __syncthreads();
    const int P = a.T * a.topk;
    for (int p = tid; p < P; p += kWaves * 64) {
        const int e = ids[p];
        int pos = 0;
        for (int q = 0; q < P; ++q) pos += ids[q] < e || (ids[q] == e && q < p);
        rt.pair[pos] = p;
    }
    __syncthreads();
    if (wave == 0) {
        int n = 0;
        for (int p0 = 0; p0 < P; p0 += 64) {
            const int p = p0 + lane;
            const int e = p < P ? ids[rt.pair[p]] : -1;
            const bool head = p < P && (p == 0 || ids[rt.pair[p - 1]] != e);
            const uint64_t heads = __ballot(head);
            if (head) {
                const int i = n + __popcll(heads & ((1ull << lane) - 1));
                rt.expert[i] = e;
                rt.begin[i] = p;
            }
            n += __popcll(heads);
        }
        if (lane == 0) {
            rt.nact = n;
            rt.begin[n] = P;
        }
    }
    __syncthreads();
    if (publish) {
        for (int p = tid; p < P; p += kWaves * 64) a.route->pair[p] = rt.pair[p];
        for (int i = tid; i <= rt.nact; i += kWaves * 64) {
            if (i < rt.nact) a.route->expert[i] = rt.expert[i];
            a.route->begin[i] = rt.begin[i];
        }
        if (tid == 0) a.route->nact = rt.nact;
    }
}

__device__ inline void load_w(const uint8_t* row, int c, u32x4 (&w)[2]) {
    w[0] = *reinterpret_cast<const u32x4*>(row + 16 * c);
    w[1] = *reinterpret_cast<const u32x4*>(row + 64 + 16 * c);
}

__device__ inline void load_x(const uint16_t* row, int c, bool valid, bf16x8 (&x)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = bf16x8{};
        if (valid) x[j] = *reinterpret_cast<const bf16x8*>(row + 64 * (j >> 1) + 16 * c + 8 * (j & 1));
    }
}


// Gate and up: a workgroup takes 16 rows of one active expert at a time, its
// waves share out the blocks of 128 columns, and their sums meet in LDS.
template <int NS>
__global__ __launch_bounds__(kWaves * 64) void moe_up_kernel(MoeArgs a) {
    __shared__ Route rt;
    __shared__ int32_t ids[kMaxPairs];
    __shared__ float part[kWaves][2][16][17];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, c = lane >> 4;
    build_route(a, rt, ids, blockIdx.x == 0);
    const int tiles = int(a.ldi / 16), items = rt.nact * tiles, kbs = int(a.ldh / 128);
    const int64_t plane = int64_t(a.T) * a.ldh, hplane = int64_t(a.T) * a.topk * a.ldi;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const int act = it / tiles, m0 = it % tiles * 16, e = rt.expert[act];
        const int64_t m = min(int64_t(m0 + r), a.I - 1);
        const uint8_t *G = a.gate + e * a.gu_bytes, *U = a.up + e * a.gu_bytes;
        const uint8_t *g = G + m * a.ldh, *u = U + m * a.ldh;
        const int64_t srow = min(int64_t(m0), a.I - 1) / 128 * a.gu_lds;
        const uint8_t *gs = G + a.gu_scales + srow, *us = U + a.gu_scales + srow;
        for (int p0 = rt.begin[act]; p0 < rt.begin[act + 1]; p0 += 16) {
            const bool valid = p0 + r < rt.begin[act + 1];
            const uint16_t* x = a.xs + int64_t(valid ? rt.pair[p0 + r] / a.topk : 0) * a.ldh;
            f32x4 ga = {0, 0, 0, 0}, ua = {0, 0, 0, 0};
            for (int kb = wave; kb < kbs; kb += kWaves) {
                u32x4 gw[2], uw[2];
                load_w(g + kb * 128, c, gw);
                load_w(u + kb * 128, c, uw);
                const float gsc = fp8_scale(gs[kb]), usc = fp8_scale(us[kb]);
                bf16x8 xv[NS][4];
#pragma unroll
                for (int s = 0; s < NS; ++s) load_x(x + s * plane + kb * 128, c, valid, xv[s]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf16x8 gb = fp8_widen(gw[j >> 1][2 * (j & 1)], gw[j >> 1][2 * (j & 1) + 1], gsc);
                    const bf16x8 ub = fp8_widen(uw[j >> 1][2 * (j & 1)], uw[j >> 1][2 * (j & 1) + 1], usc);
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        ga = __builtin_amdgcn_mfma_f32_16x16x32_bf16(gb, xv[s][j], ga, 0, 0, 0);
                        ua = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ub, xv[s][j], ua, 0, 0, 0);
                    }
                }
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                part[wave][0][r][4 * c + v] = ga[v];
                part[wave][1][r][4 * c + v] = ua[v];
            }
            __syncthreads();
            if (tid < 256) {
                const int tok = tid >> 4, row = tid & 15;
                float gv = 0.0f, uv = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
                    gv += part[w][0][tok][row];
                    uv += part[w][1][tok][row];
                }
                float h = m0 + row < a.I ? gv / (1.0f + expf(-gv)) * uv : 0.0f;
                if (p0 + tok < rt.begin[act + 1]) {
                    uint16_t* dst = a.hs + int64_t(rt.pair[p0 + tok]) * a.ldi + m0 + row;
#pragma unroll
                    for (int s = 0; s < 3; ++s) dst[s * hplane] = take_bf16(h);
                }
            }
            __syncthreads();
        }
    }
}

// Down and the weighted sum: a workgroup owns 16 outputs of every token; its
// waves share out the (expert, block of 128 columns) units in order, each sums
// into its own tile, and the tiles are added in the order of the waves.
__global__ __launch_bounds__(kWaves * 64) void moe_down_kernel(MoeArgs a) {
    extern __shared__ float ytile[];   // [kWaves][T][16]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, c = lane >> 4;
    const Route& rt = *a.route;
    float* y = ytile + wave * a.T * 16;
    for (int u = lane; u < a.T * 16; u += 64) y[u] = 0.0f;
    const int64_t m0 = int64_t(blockIdx.x) * 16, m = min(m0 + r, a.H - 1);
    const int kbs = int(a.ldi / 128), units = rt.nact * kbs;
    const int64_t hplane = int64_t(a.T) * a.topk * a.ldi;
    const int u0 = int(int64_t(units) * wave / kWaves), u1 = int(int64_t(units) * (wave + 1) / kWaves);
    for (int u = u0; u < u1;) {
        const int act = u / kbs, kb0 = u % kbs, kb1 = min(kbs, kb0 + u1 - u), e = rt.expert[act];
        u += kb1 - kb0;
        const uint8_t* D = a.down + e * a.d_bytes;
        const uint8_t *d = D + m * a.ldi, *ds = D + a.d_scales + m0 / 128 * a.d_lds;
        for (int p0 = rt.begin[act]; p0 < rt.begin[act + 1]; p0 += 16) {
            const bool valid = p0 + r < rt.begin[act + 1];
            const int pair = valid ? rt.pair[p0 + r] : 0;
            const uint16_t* h = a.hs + int64_t(pair) * a.ldi;
            f32x4 acc = {0, 0, 0, 0};
            for (int kb = kb0; kb < kb1; ++kb) {
                u32x4 w[2];
                load_w(d + kb * 128, c, w);
                const float sc = fp8_scale(ds[kb]);
                bf16x8 hv[3][4];
#pragma unroll
                for (int s = 0; s < 3; ++s) load_x(h + s * hplane + kb * 128, c, valid, hv[s]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf16x8 wb = fp8_widen(w[j >> 1][2 * (j & 1)], w[j >> 1][2 * (j & 1) + 1], sc);
#pragma unroll
                    for (int s = 0; s < 3; ++s) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb, hv[s][j], acc, 0, 0, 0);
                }
            }
            if (valid) {
                const float w = rt.weight[pair];
                float* dst = y + pair / a.topk * 16 + 4 * c;
#pragma unroll
                for (int v = 0; v < 4; ++v) dst[v] += w * acc[v];
            }
        }
    }
    __syncthreads();
    for (int u = tid; u < a.T * 16; u += kWaves * 64) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += ytile[w * a.T * 16 + u];
        if (m0 + u % 16 < a.H) a.Y[int64_t(u / 16) * a.H + m0 + u % 16] = sum;
    }
}

struct MoeLayout {
    sketch_fp8_shape gu, d;
    size_t xs, hs, route, total;
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
    L->total = align256(L->route + sizeof(Route));
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
    const unsigned E = unsigned(p->E);
    const int64_t items = (tokens * p->topk < p->E ? tokens * p->topk : int64_t(p->E)) * (L.d.ld / 16);
    const int64_t room = 2 * int64_t(compute_units());
    const unsigned up_grid = unsigned(items < room ? items : room), down_grid = unsigned((p->H + 15) / 16);
    const size_t lds = size_t(kWaves) * tokens * 16 * sizeof(float);
    auto go = [&](auto logits, auto gate_up) {
        logits<<<E, 256, 0, st>>>(a);
        if (hipGetLastError() != hipSuccess) return SKETCH_EDEVICE;
        gate_up<<<up_grid, kWaves * 64, 0, st>>>(a);
        if (hipGetLastError() != hipSuccess) return SKETCH_EDEVICE;
        moe_down_kernel<<<down_grid, kWaves * 64, lds, st>>>(a);
        return launch_status();
    };
    if (p->x_dtype == SKETCH_F32) return go(moe_logits_kernel<SKETCH_F32>, moe_up_kernel<3>);
    if (p->x_dtype == SKETCH_BF16) return go(moe_logits_kernel<SKETCH_BF16>, moe_up_kernel<1>);
    return go(moe_logits_kernel<SKETCH_F16>, moe_up_kernel<2>);
}

}  // extern "C"
