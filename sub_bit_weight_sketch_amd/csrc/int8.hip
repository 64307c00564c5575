// int8.hip -- matrices held as 8-bit integers with a float32 scale for each
// row: their encoders, and the products Y = X8 * W8^T of few rows, for one weight
// or for a stack of them with the rows grouped by expert.
#include <type_traits>

#include "int8.h"

namespace sketch {
namespace {

// ---------------------------------------------------------------------------
// Rounding.  A code is the integer next to 127 x / amax, ties to even, of the
// exact quotient.  In b significant bits such a quotient is either the middle of
// two integers or at least 2^-(b + 8) of its size away from it: with x and amax
// integers X, A < 2^b (times a power of two) it differs from k + 1/2 by a multiple
// of 1 / (2 A).  So a quotient known well enough is rounded right once it is
// first brought to a grid that holds every middle and is finer than that distance.
// 16-bit types (b <= 11): the float32 product x * (127 / amax) is off by 2 steps
// of its last place at most; the grid is 8 of them, middles are 16 or more away.
// float32 (b = 24): in float64, on a grid of 2^-40 (middles: 2^-33 away, error
// 2^-45).
// ---------------------------------------------------------------------------
constexpr float kTiny = 7.88860905e-31f;   // 2^-100: below it 127 / amax may pass float32's range
constexpr double kGrid = 6144.0;           // 1.5 * 2^12: a float64 beside it has steps of 2^-40

__device__ inline int code64(double x, double inv) {
    const double q = __builtin_fma(x, inv, kGrid) - kGrid;
    return int(__builtin_rint(q));
}

template <int DT>
struct Rounder {   // 16-bit types
    float pre, inv;
    __device__ explicit Rounder(float amax) {
        pre = amax < kTiny ? 18446744073709551616.0f : 1.0f;   // 2^64
        inv = 127.0f / (amax * pre);
    }
    __device__ int code(float x) const {
        const float q = x * pre * inv;
        return int(__builtin_rintf(__uint_as_float((__float_as_uint(q) + 4u) & ~7u)));
    }
};

template <>
struct Rounder<SKETCH_F32> {
    double inv;
    __device__ explicit Rounder(float amax) : inv(127.0 / double(amax)) {}
    __device__ int code(float x) const { return code64(double(x), inv); }
};

__device__ inline uint32_t pack4(const int (&q)[8], int at) {
    return uint32_t(q[at] & 255) | uint32_t(q[at + 1] & 255) << 8 | uint32_t(q[at + 2] & 255) << 16 | uint32_t(q[at + 3]) << 24;
}

__device__ inline uint32_t max_bits(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    return m;
}

template <int DT>
__device__ inline uint2 codes8(const float (&v)[8], const Rounder<DT>& r) {
    int q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = r.code(v[e]);
    return make_uint2(pack4(q, 0), pack4(q, 4));
}

// Maximum over L lanes of a workgroup's row: a wave, or all four of them.
template <int L, typename T, typename Max>
__device__ inline T row_max(T m, T* red, Max larger) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = larger(m, __shfl_xor(m, d));
    if constexpr (L == 256) {
        __syncthreads();   // the last one's readers are done
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
        __syncthreads();
        m = larger(larger(red[0], red[1]), larger(red[2], red[3]));
    }
    return m;
}

// Scale of a row from the bits of its largest magnitude.
__device__ inline float row_scale(uint32_t bits) {
    return bits >= 0x7F800000u ? __builtin_nanf("") : __uint_as_float(bits) / 127.0f;
}

// K chunks of 8 columns of a row, L chunks apart, from chunk `at` on, zeros past
// its end.  All loads go out before any is used (each in a branch of its own, as in
// load_row8, they follow one another: 2048 rows of 8192 15.0 us, so 12.6); a chunk that
// does not lie in the row as a whole is loaded from its last 8 columns and read
// again by element.
template <int DT, int K, int L>
struct Chunks {
    typedef uint32_t loose __attribute__((ext_vector_type(4), aligned(2)));
    static constexpr int kWords = DT == SKETCH_F32 ? 2 : 1, es = DT == SKETCH_F32 ? 4 : 2;
    loose raw[K][kWords];

    __device__ inline void load(const char* x, int64_t N, int at) {
        if (N < 8) return;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            if (i * L * 8 >= N) break;   // the whole row's
            const loose* from = reinterpret_cast<const loose*>(x + min(int64_t(at + i * L) * 8, N - 8) * es);
#pragma unroll
            for (int u = 0; u < kWords; ++u) raw[i][u] = from[u];
        }
    }
    __device__ inline void get(const char* x, int64_t N, int at, int i, float (&v)[8]) const {
        if (i * L * 8 >= N) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
            return;
        }
        const int64_t c0 = int64_t(at + i * L) * 8;
        if (c0 + 8 <= N) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t h = (raw[i][0][e >> 1] >> ((e & 1) * 16)) & 0xFFFFu;
                v[e] = DT == SKETCH_F32    ? __uint_as_float(raw[i][e / 4 % kWords][e & 3])
                       : DT == SKETCH_BF16 ? bf16_bits_to_f32(h)
                                           : f16_bits_to_f32(h);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
            if (c0 < N) {
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (c0 + e < N) v[e] = load_elem<DT>(x, c0 + e);
            }
        }
    }
};

struct EncodeArgs {
    const void *a, *b;        // the matrix, or gate and up
    int64_t lda, ldb;
    uint8_t* buf;
    int32_t* status;
    int64_t M, N, ld, rows;   // rows of all matrices
    size_t scales_offset, bytes;
};

// SwiGLU of 8 elements in float32, times 2^24, and the least gate.  exp(-g) is a product in
// two parts, so that the error is that of a few roundings (h: under 6e-7 of its size) for
// gates from kLeastGate on.  The factor, which the sum 1 + exp(-g) takes on its way, keeps
// g / (1 + exp(-g)) of a subnormal gate normal: without it that quotient has lost its bits before
// a large `up` makes it count.  Infinities, NaN and h from 2^104 on show in the result.
constexpr float kLeastGate = -80.0f;
constexpr float kDown = 5.9604644775390625e-8f;   // 2^-24

__device__ inline void swiglu8(const float (&g)[8], const float (&u)[8], float (&h)[8], float& least) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.92596299112661746887e-8f;
        const float t = -g[e] * kLog2e;
        const float low = __builtin_fmaf(-g[e], kLog2e, -t) - g[e] * kLog2eLow;   // what t lacks
        const float ex = __builtin_amdgcn_exp2f(t) * __builtin_fmaf(low, 0.693147182f, 1.0f);
        h[e] = g[e] * __builtin_amdgcn_rcpf(__builtin_fmaf(ex, kDown, kDown)) * u[e];
        least = fminf(least, g[e]);
    }
}

__device__ inline double swiglu64(float g, float u) { return double(g) / (1.0 + exp(-double(g))) * double(u); }

// One row to L lanes (a workgroup of 256 has 256 / L rows), 8 elements to a
// lane at a time; kKept such chunks of a lane stay in registers between the
// maximum and the rounding, what a longer row has more is read again.
// HBM-bound: 28672 x 8192 bfloat16 126 us, 5.6 TB/s (vector units busy 84% of the cycles).
constexpr int kKept = 4;

template <int DT, int L>
__global__ __launch_bounds__(256) void int8_encode_kernel(EncodeArgs a) {
    __shared__ uint32_t red[4];
    const int at = threadIdx.x & (L - 1);
    const int64_t row = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * (256 / L) + threadIdx.x / L;
    if (row >= a.rows) return;   // a whole wave, or the whole workgroup
    const int64_t mat = row / a.M, m = row - mat * a.M;
    constexpr int es = DT == SKETCH_F32 ? 4 : 2;
    const char* W = static_cast<const char*>(a.a) + row * a.lda * es;
    uint8_t* buf = a.buf + mat * a.bytes;
    const int chunks = int(a.ld / 8);
    float v[kKept][8];
    uint32_t bits = 0;
    Chunks<DT, kKept, L> x;
    x.load(W, a.N, at);
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
        x.get(W, a.N, at, i, v[i]);
        bits = max(bits, max_bits(v[i]));
    }
    for (int c = at + kKept * L; c < chunks; c += L) {
        float x[8];
        load_row8<DT>(W, 0, a.N, int64_t(c) * 8, x);
        bits = max(bits, max_bits(x));
    }
    bits = row_max<L>(bits, red, [](uint32_t x, uint32_t y) { return max(x, y); });
    const bool bad = bits >= 0x7F800000u;
    const float amax = bad || bits == 0 ? 1.0f : __uint_as_float(bits);
    const Rounder<DT> r(amax);
    uint8_t* codes = buf + m * a.ld;
    auto put = [&](int c, const float (&x)[8]) {
        *reinterpret_cast<uint2*>(codes + int64_t(c) * 8) = bad ? make_uint2(0, 0) : codes8<DT>(x, r);
    };
#pragma unroll
    for (int i = 0; i < kKept; ++i)
        if (at + i * L < chunks) put(at + i * L, v[i]);
    for (int c = at + kKept * L; c < chunks; c += L) {
        float x[8];
        load_row8<DT>(W, 0, a.N, int64_t(c) * 8, x);
        put(c, x);
    }
    if (at == 0) {
        reinterpret_cast<float*>(buf + a.scales_offset)[m] = row_scale(bits);
        if (a.status && bad) atomicOr(a.status, SKETCH_FLAG_WEIGHT_RANGE);
    }
}

// The same of h = silu(gate) * up, K chunks of h kept.  The float32 h decides the
// codes where it is clear of the middle of two integers (by 1.2e-4 of a code; its
// error is under 7.6e-5), float64 the others, one in 4000, for which gate and up are
// read again; the largest magnitude is that of float64 among the elements within 2e-6
// of the largest in float32.  Rows that float32 cannot hold (a gate below
// kLeastGate, values from 2^104 on, or tiny ones throughout) are computed in float64,
// which alone tells those past float32's range.
// 2048 x 11008 bfloat16: 34 us, 3.4 TB/s.  Bound by neither alone: 36 instructions an
// element keep the vector units busy 68% of the cycles, and a workgroup's loads and arithmetic
// follow one another.  (Gate and up read three times, with nothing kept: 57 us.)
template <int DT, int L, int K>
__global__ __launch_bounds__(256) void int8_swiglu_kernel(EncodeArgs a) {
    __shared__ uint32_t red[4];
    __shared__ double red64[4];
    const int at = threadIdx.x & (L - 1);
    const int64_t row = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * (256 / L) + threadIdx.x / L;
    if (row >= a.rows) return;
    constexpr int es = DT == SKETCH_F32 ? 4 : 2;
    const char *G = static_cast<const char*>(a.a) + row * a.lda * es, *U = static_cast<const char*>(a.b) + row * a.ldb * es;
    const int chunks = int(a.ld / 8);
    auto load = [&](int c, float (&g)[8], float (&u)[8]) {   // past the row's end: zeros
        load_row8<DT>(G, 0, a.N, int64_t(c) * 8, g);
        load_row8<DT>(U, 0, a.N, int64_t(c) * 8, u);
    };
    auto precise = [&](int c, int e) { return swiglu64(load_elem<DT>(G, c * 8 + e), load_elem<DT>(U, c * 8 + e)); };
    auto umax = [](uint32_t x, uint32_t y) { return max(x, y); };
    auto dmax = [](double x, double y) { return x > y || x != x ? x : y; };   // NaN wins
    uint8_t* codes = a.buf + row * a.ld;
    float h[K][8], least = 0.0f;   // h and its bits: of 2^24 h
    uint32_t bits = 0;
    Chunks<DT, K, L> gates, ups;
    gates.load(G, a.N, at);
    ups.load(U, a.N, at);
#pragma unroll
    for (int i = 0; i < K; ++i) {
        float g[8], u[8];
        if (i * L >= chunks) {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = 0.0f;
            continue;
        }
        gates.get(G, a.N, at, i, g);
        ups.get(U, a.N, at, i, u);
        swiglu8(g, u, h[i], least);
        bits = max(bits, max_bits(h[i]));
    }
    for (int c = at + K * L; c < chunks; c += L) {
        float g[8], u[8], x[8];
        load(c, g, u);
        swiglu8(g, u, x, least);
        bits = max(bits, max_bits(x));
    }
    if (least < kLeastGate) bits = 0x7FFFFFFFu;
    bits = row_max<L>(bits, red, umax);
    const bool whole = bits >= 0x7F800000u || bits < __float_as_uint(kTiny);
    double big = 0.0;
    auto larger = [&](int c, const float (&x)[8]) {
        const float near = __uint_as_float(bits) * (1.0f - 2e-6f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (fabsf(x[e]) >= near) big = dmax(fabs(precise(c, e)), big);
    };
    if (whole) {
        for (int c = at; c < chunks; c += L) {
            float g[8], u[8];
            load(c, g, u);
            for (int e = 0; e < 8; ++e) big = dmax(fabs(swiglu64(g[e], u[e])), big);
        }
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (at + i * L < chunks) larger(at + i * L, h[i]);
        for (int c = at + K * L; c < chunks; c += L) {
            float g[8], u[8], x[8];
            load(c, g, u);
            swiglu8(g, u, x, least);
            larger(c, x);
        }
    }
    big = row_max<L>(big, red64, dmax);
    const bool bad = !(big <= 3.4028234663852886e38);   // NaN too
    const double per = bad || big == 0.0 ? 1.0 : big;
    auto code = [&](double x) { return bad ? 0 : int(__builtin_rint(x * 127.0 / per)); };
    const float inv = float(127.0 * double(kDown) / per);   // of 2^24 h
    auto put = [&](int c, const float (&x)[8]) {
        int q[8];
        uint32_t unsure = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = x[e] * inv, integer = __builtin_rintf(v);
            q[e] = int(integer);
            unsure |= fabsf(v - integer) > 0.5f - 1.2e-4f ? 1u << e : 0u;
        }
        if (unsure) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (unsure >> e & 1) q[e] = code(precise(c, e));
        }
        *reinterpret_cast<uint2*>(codes + int64_t(c) * 8) = make_uint2(pack4(q, 0), pack4(q, 4));
    };
    if (whole) {
        for (int c = at; c < chunks; c += L) {
            float g[8], u[8];
            int q[8];
            load(c, g, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = code(swiglu64(g[e], u[e]));
            *reinterpret_cast<uint2*>(codes + int64_t(c) * 8) = make_uint2(pack4(q, 0), pack4(q, 4));
        }
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (at + i * L < chunks) put(at + i * L, h[i]);
        for (int c = at + K * L; c < chunks; c += L) {
            float g[8], u[8], x[8];
            load(c, g, u);
            swiglu8(g, u, x, least);
            put(c, x);
        }
    }
    if (at == 0) {
        reinterpret_cast<float*>(a.buf + a.scales_offset)[row] = bad ? __builtin_nanf("") : float(big / 127.0);
        if (a.status && bad) atomicOr(a.status, SKETCH_FLAG_WEIGHT_RANGE);
    }
}

// ---------------------------------------------------------------------------
// Product of up to 16 terms at a time, bound by the codes of W coming from
// memory: 16 RT outputs to a workgroup, whose waves share out the columns in runs
// of 4 blocks of 128, all loads of a run in flight, both operands straight to
// registers.  A fragment is 16 rows x 128 columns, one row to a lane: lane l
// holds row l % 16 and the columns 16c..16c+15 and 64+16c..64+16c+15, c = l / 16,
// the same ones of outputs (A) and terms (B), so that a pair of loads covers 128
// contiguous bytes of a row.  D: term l % 16, outputs 4c..4c+3.  The waves' sums meet
// in LDS.  16 outputs to 8 waves for few rows of one weight (4096 x
// 4096 at 5 rows 6.2 us), 32 to 4 waves where many experts have a few terms each (64 experts of
// 2816 x 2048, 42 terms: 36 and 29 us).
// ---------------------------------------------------------------------------
struct Frag {
    i32x4 lo, hi;
    __device__ inline void load(const int8_t* row, uint32_t block, int c) {
        const int8_t* at = row + size_t(block) * 128 + 16 * c;
        lo = *reinterpret_cast<const i32x4*>(at);
        hi = *reinterpret_cast<const i32x4*>(at + 64);
    }
};

__device__ inline i32x4 multiply(const Frag& a, const Frag& b, i32x4 acc) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a.lo, b.lo, acc, 0, 0, 0);
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a.hi, b.hi, acc, 0, 0, 0);
}

constexpr int kRun = 4;

template <bool GROUP, int WAVES, int RT>
__global__ __launch_bounds__(WAVES * 64) void int8_rows_kernel(Int8Product p) {
    __shared__ __attribute__((aligned(16))) int part[WAVES][16][RT * 16 + 4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4;
    const int64_t tiles_o = (p.M + RT * 16 - 1) / (RT * 16);
    const int64_t id = int64_t(blockIdx.y) * gridDim.x + blockIdx.x, tile = id / tiles_o, m0 = (id - tile * tiles_o) * (RT * 16);
    Terms t{0, int(tile * 16), int(min(int64_t(16), p.T - tile * 16))};
    if (GROUP ? !find_terms<16>(p, [&](int) { return int(tile); }, t) : t.n <= 0) return;
    const int8_t* w = p.w + size_t(t.expert) * p.w_bytes;
    const int8_t* wrow[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) wrow[i] = w + min(m0 + i * 16 + r, p.M - 1) * p.ld;
    const int64_t mine = t.first + min(r, t.n - 1);
    const int8_t* xrow = p.x + (GROUP ? max(term_row(p, mine), int64_t(0)) : mine) * p.ld;
    i32x4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = i32x4{0, 0, 0, 0};
    for (uint32_t k = wave * kRun; k < p.kb; k += WAVES * kRun) {
        Frag a[kRun][RT], b[kRun];
#pragma unroll
        for (int u = 0; u < kRun; ++u) {   // blocks past the last are read as the last and not used
            const uint32_t block = min(k + u, p.kb - 1);
#pragma unroll
            for (int i = 0; i < RT; ++i) a[u][i].load(wrow[i], block, c);
            b[u].load(xrow, block, c);
        }
        asm volatile("" ::: "memory");   // all loads of the run before its first use
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            if (k + u >= p.kb) break;
#pragma unroll
            for (int i = 0; i < RT; ++i) acc[i] = multiply(a[u][i], b[u], acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) *reinterpret_cast<i32x4*>(&part[wave][r][i * 16 + 4 * c]) = acc[i];
    __syncthreads();
    // 16 terms x 16 RT outputs, 4 outputs to a thread
    constexpr int kAcross = RT * 4;
    static_assert(WAVES * 64 >= 16 * kAcross, "a thread for every 4 outputs");
    const int m = tid % kAcross * 4, n = tid / kAcross;
    if (n >= t.n || m0 + m >= p.M) return;
    const f32x4 sw = *reinterpret_cast<const f32x4*>(reinterpret_cast<const char*>(w) + p.w_scales + (m0 + m) * 4);
    i32x4 sum = *reinterpret_cast<const i32x4*>(&part[0][n][m]);
#pragma unroll
    for (int i = 1; i < WAVES; ++i) sum += *reinterpret_cast<const i32x4*>(&part[i][n][m]);
    const int64_t term = t.first + n, row = GROUP ? term_row(p, term) : term;
    const float sx = row < 0 ? __builtin_nanf("") : p.xs[row];
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = int8_value(sum[i], sx, sw[i]);
    const int64_t at = term * p.M + m0 + m;
    if (p.ydt == SKETCH_F32)
        store4_any<SKETCH_F32>(p.Y, at, v, m0 + m, p.M);
    else if (p.ydt == SKETCH_BF16)
        store4_any<SKETCH_BF16>(p.Y, at, v, m0 + m, p.M);
    else
        store4_any<SKETCH_F16>(p.Y, at, v, m0 + m, p.M);
}

// ---------------------------------------------------------------------------
// The same for up to 16 rows of X (p.x, of dtype XD) that every workgroup encodes for
// itself, which saves the launch that would encode them first: 16 outputs to a
// workgroup of 8 waves.  The loads of W go out first; while they are on their way the
// rows are encoded into LDS, a single one by the whole workgroup, several by a wave
// each, 8 columns to a lane at a time; what a row has more than the lanes keep is read
// again.
// ---------------------------------------------------------------------------
constexpr uint32_t kTokenCodes = 32768;   // bytes of codes that LDS holds, with 64 more for each row

template <int XD, bool GROUP, bool ONE>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(ONE ? 6 : 4))) void int8_tokens_kernel(Int8Product p, int64_t N) {
    extern __shared__ __attribute__((aligned(16))) uint8_t codes[];   // [min(16, T)][ld + 64]
    __shared__ uint32_t red[16];
    __shared__ __attribute__((aligned(16))) int part[8][16][20];
    constexpr int es = XD == SKETCH_F32 ? 4 : 2;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4, pitch = int(p.ld) + 64, chunks = int(p.ld / 8);
    const int64_t tiles_o = (p.M + 15) / 16, tile = GROUP ? blockIdx.x / tiles_o : 0;
    const int64_t m0 = (blockIdx.x - tile * tiles_o) * 16;
    Terms t{0, 0, int(p.T)};
    if (GROUP && !find_terms<16>(p, [&](int) { return int(tile); }, t)) return;
    const int8_t* w = p.w + size_t(t.expert) * p.w_bytes;
    const int8_t* wrow = w + min(m0 + r, p.M - 1) * p.ld;
    const uint32_t k0 = wave * kRun;
    Frag a[kRun];
#pragma unroll
    for (int u = 0; u < kRun; ++u) a[u].load(wrow, min(k0 + u, p.kb - 1), c);
    const float sw = reinterpret_cast<const float*>(reinterpret_cast<const char*>(w) + p.w_scales)[min(m0 + (tid & 15), p.M - 1)];
    asm volatile("" ::: "memory");   // on their way before X is asked for

    auto row_at = [&](int n) {
        const int64_t row = GROUP ? max(term_row(p, t.first + n), int64_t(0)) : n;
        return reinterpret_cast<const char*>(p.x) + row * N * es;
    };
    // row n by `lanes` threads, `at` this one's place among them, KEPT chunks of a thread kept
    auto encode = [&](int n, int at, auto lanes_c, auto kept_c, auto maximum) {
        constexpr int LANES = decltype(lanes_c)::value, KEPT = decltype(kept_c)::value;
        const char* x = row_at(n);
        float v[KEPT][8];
        uint32_t bits = 0;
        Chunks<XD, KEPT, LANES> kept;
        kept.load(x, N, at);
#pragma unroll
        for (int i = 0; i < KEPT; ++i) {
            kept.get(x, N, at, i, v[i]);
            bits = max(bits, max_bits(v[i]));
        }
        for (int q = at + KEPT * LANES; q < chunks; q += LANES) {
            float y[8];
            load_row8<XD>(x, 0, N, int64_t(q) * 8, y);
            bits = max(bits, max_bits(y));
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) bits = max(bits, uint32_t(__shfl_xor(int(bits), d)));
        bits = maximum(bits);
        const bool bad = bits >= 0x7F800000u;
        const Rounder<XD> round(bad || bits == 0 ? 1.0f : __uint_as_float(bits));
        auto put = [&](int q, const float (&y)[8]) {
            *reinterpret_cast<uint2*>(codes + n * pitch + q * 8) = bad ? make_uint2(0, 0) : codes8<XD>(y, round);
        };
#pragma unroll
        for (int i = 0; i < KEPT; ++i)
            if (at + i * LANES < chunks) put(at + i * LANES, v[i]);
        for (int q = at + KEPT * LANES; q < chunks; q += LANES) {
            float y[8];
            load_row8<XD>(x, 0, N, int64_t(q) * 8, y);
            put(q, y);
        }
        return bits;
    };
    if (ONE || t.n == 1) {
        const uint32_t bits = encode(0, tid, std::integral_constant<int, 512>(), std::integral_constant<int, 2>(), [&](uint32_t m) {
            if (lane == 0) red[wave + 8] = m;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, red[i + 8]);
            return m;
        });
        if (tid == 0) red[0] = bits;
    } else if constexpr (!ONE) {
        for (int n = wave; n < t.n; n += 8) {
            const uint32_t bits =
                encode(n, lane, std::integral_constant<int, 64>(), std::integral_constant<int, XD == SKETCH_F32 ? 2 : 4>(), [](uint32_t m) { return m; });
            if (lane == 0) red[n] = bits;
        }
    }
    __syncthreads();

    i32x4 acc = {0, 0, 0, 0};
    const int8_t* xrow = reinterpret_cast<const int8_t*>(codes) + min(r, t.n - 1) * pitch;   // terms past the last are not stored
    for (uint32_t k = k0; k < p.kb; k += 8 * kRun) {
        if (k != k0) {
#pragma unroll
            for (int u = 0; u < kRun; ++u) a[u].load(wrow, min(k + u, p.kb - 1), c);
        }
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            if (k + u >= p.kb) break;
            Frag b;
            b.load(xrow, k + u, c);
            acc = multiply(a[u], b, acc);
        }
    }
    *reinterpret_cast<i32x4*>(&part[wave][r][4 * c]) = acc;
    __syncthreads();
    const int m = tid & 15, n = tid >> 4;
    if (n >= t.n || m0 + m >= p.M) return;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += part[i][n][m];
    const int64_t term = t.first + n;
    const float sx = GROUP && term_row(p, term) < 0 ? __builtin_nanf("") : row_scale(red[n]);
    const float y = int8_value(sum, sx, sw);
    const int64_t at = term * p.M + m0 + m;
    if (p.ydt == SKETCH_F32)
        store1_val<SKETCH_F32>(p.Y, at, y);
    else if (p.ydt == SKETCH_BF16)
        store1_val<SKETCH_BF16>(p.Y, at, y);
    else
        store1_val<SKETCH_F16>(p.Y, at, y);
}

bool valid_dtype(int d) { return d == SKETCH_F32 || d == SKETCH_BF16 || d == SKETCH_F16; }

// A grid of `groups` workgroups of `threads` threads, over two dimensions where
// one does not hold them; false past that.
bool grid_of(int64_t groups, int threads, dim3* grid) {
    const int64_t line = kMaxThreads / threads, lines = (groups + line - 1) / line;
    if (lines > 65535) return false;
    *grid = dim3(unsigned(lines > 1 ? line : groups), unsigned(lines));
    return true;
}

sketch_status launch_encode8(const EncodeArgs& a, int dt, bool swiglu, hipStream_t st) {
    dim3 grid;
    // a wave to a row of up to 2048 columns, which it keeps, where there are rows for all compute units; a workgroup
    // to a row otherwise
    const bool narrow = a.ld <= 64 * 8 * kKept && a.rows >= 4 * int64_t(compute_units());
    if (!grid_of(narrow ? (a.rows + 3) / 4 : a.rows, 256, &grid)) return SKETCH_EINVAL;
    auto go = [&](auto one, auto all) {
        if (narrow)
            one<<<grid, 256, 0, st>>>(a);
        else
            all<<<grid, 256, 0, st>>>(a);
        return launch_status();
    };
    if (swiglu) {
        if (dt == SKETCH_F32) return go(int8_swiglu_kernel<SKETCH_F32, 64, 4>, int8_swiglu_kernel<SKETCH_F32, 256, 6>);
        if (dt == SKETCH_BF16) return go(int8_swiglu_kernel<SKETCH_BF16, 64, 4>, int8_swiglu_kernel<SKETCH_BF16, 256, 6>);
        return go(int8_swiglu_kernel<SKETCH_F16, 64, 4>, int8_swiglu_kernel<SKETCH_F16, 256, 6>);
    }
    if (dt == SKETCH_F32) return go(int8_encode_kernel<SKETCH_F32, 64>, int8_encode_kernel<SKETCH_F32, 256>);
    if (dt == SKETCH_BF16) return go(int8_encode_kernel<SKETCH_BF16, 64>, int8_encode_kernel<SKETCH_BF16, 256>);
    return go(int8_encode_kernel<SKETCH_F16, 64>, int8_encode_kernel<SKETCH_F16, 256>);
}

int64_t matrices(const sketch_int8_params* p) { return p->count > 1 ? p->count : 1; }

sketch_status launch_int8_encode(const sketch_int8_params* p, const sketch_int8_shape& s, const void* W, int dt,
                                 int64_t ldw, void* buf, int32_t* status, hipStream_t st) {
    return launch_encode8({W, nullptr, ldw, 0, static_cast<uint8_t*>(buf), status, p->M, p->N, s.ld,
                           p->M * matrices(p), s.scales_offset, s.bytes}, dt, false, st);
}

constexpr int64_t kMaxElements = int64_t(1) << 60;   // whose bytes an int64 counts

// Bytes from the first element of rows `ld` elements apart to behind the last.
size_t extent(int64_t rows, int64_t N, int64_t ld, int dtype) {
    return rows > 0 ? (size_t(rows - 1) * size_t(ld) + size_t(N)) * elem_bytes(dtype) : 0;
}

bool aligned_to_element(const void* p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (elem_bytes(dtype) - 1)) == 0; }

// What one product does and needs.
struct Plan {
    sketch_int8_shape w, x;   // one weight, the encoded rows
    bool encode;              // rows encoded by a launch of their own
    Int8Plan gemm;
    size_t workspace;
};

// Whether the workgroups of a product encode its raw rows themselves.  On the
// GPU that is faster where they are few, or long enough to hide it: a single row of
// 5179 x 3673 8.5 us, 11.1 with a launch of its own; 28672 x 8192 44 and 49; 28616 x 1385 19
// and 12.  2 to 16 rows, up to 16384 codes, where a compute unit has one workgroup at most, are
// 20% faster to 20% slower (1376 x 2048, 4 rows 5.7 and 7.1; 4096 x 4096, 2 rows 11.6 and
// 9.5), with more workgroups much slower (14601 x 356, 4 rows 18 and 7.4).  Those are
// replays of a graph; launched one by one a second kernel costs 4.5 us (16 rows of 256 x 512 12.1
// and 7.3 us), so the border lies where one launch takes what two of them take.
bool encodes_itself(int64_t M, int64_t terms, int64_t ld, int experts, bool group) {
    if (terms > 16 * (group ? experts : 1)) return false;   // more than a tile of each
    const int64_t rows = min(terms, int64_t(16)), tiles = group ? (terms + 15) / 16 + min(terms, int64_t(experts)) : 1;
    const int64_t groups = (M + 15) / 16 * tiles, ncu = compute_units();
    if (terms == 1) return ld <= int64_t(kTokenCodes) && (2 * groups <= 5 * ncu || ld * ncu >= 512 * groups);
    return rows * ld <= int64_t(kTokenCodes / 2) && groups <= ncu;
}

// Checks the parameters and fills the plan.  any_order: terms may take any rows of X.  The
// workspace does not depend on it (groups have no parts).
sketch_status make_plan(const sketch_int8_params* p, int64_t terms, int64_t x_rows, int x_dtype, int y_dtype,
                        bool group, bool any_order, Plan* plan) {
    sketch_status rc = int8_shape(p, &plan->w);
    if (rc != SKETCH_OK) return rc;
    const bool rows = x_dtype == SKETCH_INT8_ROWS;
    if (terms < 0 || terms > SKETCH_INT8_MAX_M || (!rows && !valid_dtype(x_dtype)) || !valid_dtype(y_dtype) ||
        matrices(p) > (group ? SKETCH_INT8_MAX_EXPERTS : 1))
        return SKETCH_EINVAL;
    const sketch_int8_params xp{x_rows, p->N, 1};
    rc = int8_shape(&xp, &plan->x);
    if (rc != SKETCH_OK) return rc;
    plan->workspace = 0;
    plan->encode = false;
    if (terms == 0 || p->M == 0) return SKETCH_OK;
    plan->encode = !rows && !encodes_itself(p->M, terms, plan->x.ld, int(matrices(p)), group);
    if (plan->encode) plan->workspace += plan->x.bytes;
    if (!plan->encode && !rows) return SKETCH_OK;   // encoded by the product's own workgroups
    const bool near = !any_order || x_rows * plan->x.ld <= int64_t(0xFFFFFFFF);
    rc = int8_plan(p->M, terms, uint32_t(plan->w.ld / 128), y_dtype, int(matrices(p)), group, near, &plan->gemm);
    plan->workspace += plan->gemm.workspace;
    return rc;
}

template <bool GROUP, int WAVES, int RT>
sketch_status launch_rows(const Int8Product& a, hipStream_t st) {
    const int64_t tiles = (a.T + 15) / 16 + (GROUP ? min(a.T, int64_t(a.experts)) : 0);
    dim3 grid;
    if (!grid_of((a.M + RT * 16 - 1) / (RT * 16) * tiles, WAVES * 64, &grid)) return SKETCH_EINVAL;
    int8_rows_kernel<GROUP, WAVES, RT><<<grid, WAVES * 64, 0, st>>>(a);
    return launch_status();
}

int64_t token_groups(const Int8Product& a) {
    return (a.M + 15) / 16 * (a.counts ? (a.T + 15) / 16 + min(a.T, int64_t(a.experts)) : 1);
}

sketch_status launch_tokens(const Int8Product& a, int x_dtype, int64_t N, hipStream_t st) {
    auto go = [&](auto kernel) {
        kernel<<<unsigned(token_groups(a)), 512, unsigned(min(a.T, int64_t(16)) * (a.ld + 64)), st>>>(a, N);
        return launch_status();
    };
    auto all = [&](auto f32, auto bf16, auto f16) { return x_dtype == SKETCH_F32 ? go(f32) : x_dtype == SKETCH_BF16 ? go(bf16) : go(f16); };
    if (a.counts)
        return all(int8_tokens_kernel<SKETCH_F32, true, false>, int8_tokens_kernel<SKETCH_BF16, true, false>,
                   int8_tokens_kernel<SKETCH_F16, true, false>);
    if (a.T == 1)
        return all(int8_tokens_kernel<SKETCH_F32, false, true>, int8_tokens_kernel<SKETCH_BF16, false, true>,
                   int8_tokens_kernel<SKETCH_F16, false, true>);
    return all(int8_tokens_kernel<SKETCH_F32, false, false>, int8_tokens_kernel<SKETCH_BF16, false, false>,
               int8_tokens_kernel<SKETCH_F16, false, false>);
}

sketch_status product(const sketch_int8_params* p, const void* buf, const void* X, int x_dtype, int64_t x_rows,
                      int64_t terms, const sketch_int8_groups* g, void* Y, int y_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
    Plan plan;
    const bool index = g && g->rows;
    sketch_status rc = make_plan(p, terms, x_rows, x_dtype, y_dtype, g != nullptr, index, &plan);
    if (rc != SKETCH_OK) return rc;
    if (g && ((g->counts_bits != 32 && g->counts_bits != 64) || (index && g->rows_bits != 32 && g->rows_bits != 64)))
        return SKETCH_EINVAL;
    if (terms == 0 || p->M == 0) return SKETCH_OK;
    if (!buf || !X || !Y || !aligned16(buf) || !aligned16(X) || !aligned16(Y)) return SKETCH_EINVAL;
    if (g && (x_rows < (index ? 1 : terms) || !g->counts ||
              (reinterpret_cast<uintptr_t>(g->counts) & (g->counts_bits / 8 - 1)) ||
              (index && (reinterpret_cast<uintptr_t>(g->rows) & (g->rows_bits / 8 - 1)))))
        return SKETCH_EINVAL;
    const size_t need = plan.workspace;
    if (need > 0) {
        if (!workspace || !aligned16(workspace)) return SKETCH_EINVAL;
        if (workspace_bytes < need) return SKETCH_ESMALL;
    }
    // workgroups that are done store Y while others still read
    const int64_t count = matrices(p);
    const Range ry{Y, size_t(terms) * size_t(p->M) * elem_bytes(y_dtype)}, rw{buf, size_t(count) * plan.w.bytes},
        rs{workspace, need}, rx{X, x_dtype == SKETCH_INT8_ROWS ? plan.x.bytes : extent(x_rows, p->N, p->N, x_dtype)},
        rcounts{g ? g->counts : nullptr, g ? size_t(count) * size_t(g->counts_bits / 8) : 0},
        rindex{index ? g->rows : nullptr, index ? size_t(terms) * size_t(g->rows_bits / 8) : 0};
    if (((g || !plan.encode || terms <= SKETCH_INT8_TOKENS) && overlap(ry, rx)) || overlap(rs, ry) || overlap(rs, rx)) return SKETCH_EINVAL;
    for (const Range& r : {rw, rcounts, rindex})
        if (overlap(ry, r) || overlap(rs, r)) return SKETCH_EINVAL;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int8_t *w8 = static_cast<const int8_t*>(buf), *x8 = static_cast<const int8_t*>(X);
    if (plan.encode) {
        const sketch_int8_params xp{x_rows, p->N, 1};
        rc = launch_int8_encode(&xp, plan.x, X, x_dtype, p->N, workspace, nullptr, st);
        if (rc != SKETCH_OK) return rc;
        x8 = static_cast<const int8_t*>(workspace);
        workspace = static_cast<char*>(workspace) + plan.x.bytes;
    }
    Int8Product a{};
    a.w = w8, a.w_bytes = plan.w.bytes, a.w_scales = plan.w.scales_offset;
    a.x = x8, a.xs = reinterpret_cast<const float*>(x8 + plan.x.scales_offset), a.x_rows = x_rows;
    a.Y = Y, a.M = p->M, a.T = terms, a.ld = plan.w.ld, a.kb = uint32_t(plan.w.ld / 128), a.ydt = y_dtype;
    a.experts = int(count);
    if (g) a.counts = g->counts, a.rows = g->rows, a.counts64 = g->counts_bits == 64, a.rows64 = g->rows_bits == 64;
    if (!plan.encode && x_dtype != SKETCH_INT8_ROWS)
        return launch_tokens(a, x_dtype, p->N, st);
    if (plan.gemm.kind == kInt8Rows1) return g ? launch_rows<true, 8, 1>(a, st) : launch_rows<false, 8, 1>(a, st);
    if (plan.gemm.kind == kInt8Rows2) return launch_rows<true, 4, 2>(a, st);   // groups alone
    return launch_int8_gemm(a, plan.gemm, workspace, st);
}

}  // namespace

sketch_status int8_shape(const sketch_int8_params* p, sketch_int8_shape* s) {
    if (!p || p->M < 0 || p->M > SKETCH_INT8_MAX_M || p->N < 1 || p->N > SKETCH_INT8_MAX_N) return SKETCH_EINVAL;
    if (p->count < 0 || p->count > SKETCH_INT8_MAX_COUNT) return SKETCH_EINVAL;
    s->ld = (p->N + 127) / 128 * 128;
    s->scales_offset = align256(size_t(p->M) * size_t(s->ld));
    s->bytes = align256(s->scales_offset + size_t(p->M) * 4);
    return SKETCH_OK;
}

}  // namespace sketch

using namespace sketch;

extern "C" {

sketch_status sketch_int8_layout(const sketch_int8_params* p, sketch_int8_shape* shape) {
    return shape ? int8_shape(p, shape) : SKETCH_EINVAL;
}

sketch_status sketch_int8_encode(const sketch_int8_params* p, const void* W, sketch_dtype w_dtype, int64_t ldw,
                                 void* buf, int32_t* status_dev, void* stream) {
    sketch_int8_shape s;
    const sketch_status rc = int8_shape(p, &s);
    if (rc != SKETCH_OK) return rc;
    if (!valid_dtype(w_dtype) || ldw < p->N || (reinterpret_cast<uintptr_t>(status_dev) & 3u))
        return SKETCH_EINVAL;
    if (p->M == 0) return SKETCH_OK;
    if (!W || !buf || !aligned_to_element(W, w_dtype) || !aligned16(buf)) return SKETCH_EINVAL;
    const int64_t count = matrices(p);
    if (ldw > kMaxElements / (count * p->M)) return SKETCH_EINVAL;
    if (overlap({W, extent(count * p->M, p->N, ldw, w_dtype)}, {buf, size_t(count) * s.bytes})) return SKETCH_EINVAL;
    return launch_int8_encode(p, s, W, w_dtype, ldw, buf, status_dev, static_cast<hipStream_t>(stream));
}

sketch_status sketch_int8_swiglu(const sketch_int8_params* p, const void* gate, int64_t ld_gate, const void* up,
                                 int64_t ld_up, sketch_dtype dtype, void* buf, int32_t* status_dev, void* stream) {
    sketch_int8_shape s;
    const sketch_status rc = int8_shape(p, &s);
    if (rc != SKETCH_OK) return rc;
    if (!valid_dtype(dtype) || p->count > 1 || (reinterpret_cast<uintptr_t>(status_dev) & 3u)) return SKETCH_EINVAL;
    if (ld_gate < p->N || ld_up < p->N) return SKETCH_EINVAL;
    if (p->M == 0) return SKETCH_OK;
    if (max(ld_gate, ld_up) > kMaxElements / p->M) return SKETCH_EINVAL;
    if (!buf || !aligned16(buf)) return SKETCH_EINVAL;
    for (const void* q : {gate, up})
        if (!q || !aligned_to_element(q, dtype)) return SKETCH_EINVAL;
    const Range out{buf, s.bytes};
    if (overlap({gate, extent(p->M, p->N, ld_gate, dtype)}, out) || overlap({up, extent(p->M, p->N, ld_up, dtype)}, out))
        return SKETCH_EINVAL;
    return launch_encode8({gate, up, ld_gate, ld_up, static_cast<uint8_t*>(buf), status_dev, p->M, p->N, s.ld, p->M,
                           s.scales_offset, s.bytes}, dtype, true, static_cast<hipStream_t>(stream));
}

sketch_status sketch_int8_workspace_bytes(const sketch_int8_params* p, int64_t batch, int x_dtype, int y_dtype,
                                          size_t* bytes) {
    Plan plan;
    const sketch_status rc = make_plan(p, batch, batch, x_dtype, y_dtype, false, false, &plan);
    if (rc != SKETCH_OK) return rc;
    if (!bytes) return SKETCH_EINVAL;
    *bytes = plan.workspace;
    return SKETCH_OK;
}

sketch_status sketch_int8_matmul(const sketch_int8_params* p, const void* buf, const void* X, int x_dtype,
                                 int64_t batch, void* Y, int y_dtype, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    return product(p, buf, X, x_dtype, batch, batch, nullptr, Y, y_dtype, workspace, workspace_bytes, stream);
}

sketch_status sketch_int8_group_workspace_bytes(const sketch_int8_params* p, int64_t terms, int64_t x_rows,
                                                int x_dtype, int y_dtype, size_t* bytes) {
    Plan plan;
    const sketch_status rc = make_plan(p, terms, x_rows, x_dtype, y_dtype, true, true, &plan);
    if (rc != SKETCH_OK) return rc;
    if (!bytes) return SKETCH_EINVAL;
    *bytes = plan.workspace;
    return SKETCH_OK;
}

sketch_status sketch_int8_matmul_group(const sketch_int8_params* p, const void* buf, const void* X, int x_dtype,
                                       int64_t x_rows, const sketch_int8_groups* g, void* Y, int y_dtype,
                                       void* workspace, size_t workspace_bytes, void* stream) {
    if (!g) return SKETCH_EINVAL;
    return product(p, buf, X, x_dtype, x_rows, g->terms, g, Y, y_dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
