// fp8.hip -- matrices held as e4m3 codes with a power-of-two scale for each
// block of 128 columns: their encoder and the product Y = X8 * W8^T.
//
// "Resumen Técnico" › Metodología §2 and §5: layers differ in how much
// compression they tolerate.  This is the format for those that are not
// sketched.  The scales are powers of two because gfx950 applies such a scale
// for nothing, in the matrix core as it multiplies e4m3 operands, or as it
// widens them: the sum over K runs on in one accumulator, with no pass over it
// per block of 128.
#include "fp8.h"

namespace sketch {
namespace {

// Largest magnitude's bits; magnitudes compare as their bits, NaN above infinity.
__device__ inline uint32_t max_bits(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    return m;
}

// The codes of 8 elements in a block of scale byte b (255: NaN).
__device__ inline uint2 codes8(const float (&v)[8], uint32_t b) {
    if (b == 255u) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    const float inv = fp8_inv_scale(b);
    return make_uint2(fp8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                      fp8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// The same at column c0 of a row of N: past the end the codes are zero.
__device__ inline uint2 codes8(const float (&v)[8], uint32_t b, int64_t c0, int64_t N) {
    uint2 q = codes8(v, b);
    if (b == 255u && c0 + 8 > N) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c0 + e >= N) (e < 4 ? q.x : q.y) &= ~(0xFFu << (8 * (e & 3)));
    }
    return q;
}

// Maximum over the 16 lanes of a row of a block.
__device__ inline uint32_t max16(uint32_t m) {
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) m = max(m, uint32_t(__shfl_xor(int(m), d)));
    return m;
}

// ---------------------------------------------------------------------------
// Encoder of 128 x 128 blocks.  One workgroup per block, 16 lanes to a row: a
// thread holds 8 columns of 8 rows, so the elements stay in registers between
// the maximum and the rounding and W is read once.  HBM-bound.
// ---------------------------------------------------------------------------
struct EncodeArgs {
    const void* W;
    uint8_t* buf;
    int32_t* status;
    int64_t M, N, ld, lds, row_blocks, col_blocks, count;
    size_t scales_offset, bytes;
};

template <int DT>
__global__ __launch_bounds__(256) void fp8_encode_kernel(EncodeArgs a) {
    __shared__ uint32_t red[4];
    const int tid = threadIdx.x;
    const int64_t id = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t cb = id % a.lds, rb = (id / a.lds) % a.row_blocks, mat = id / a.lds / a.row_blocks;
    if (mat >= a.count) return;
    uint8_t* codes = a.buf + mat * a.bytes;
    uint8_t* scale = codes + a.scales_offset + rb * a.lds + cb;
    if (cb >= a.col_blocks) {   // scale bytes that round a row of scales up to a dword
        if (tid == 0) *scale = 0;
        return;
    }
    constexpr int64_t es = DT == SKETCH_F32 ? 4 : 2;
    const unsigned char* W = static_cast<const unsigned char*>(a.W) + mat * a.M * a.N * es;
    const int64_t c0 = cb * 128 + (tid & 15) * 8, row0 = rb * 128 + (tid >> 4);
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (row0 + i * 16 < a.M) {
            load_row8<DT>(W, row0 + i * 16, a.N, c0, v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
        }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, max_bits(v[i]));
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = max(m, uint32_t(__shfl_xor(int(m), d)));
    if ((tid & 63) == 0) red[tid >> 6] = m;
    __syncthreads();
    const uint32_t b = fp8_scale_byte(max(max(red[0], red[1]), max(red[2], red[3])));
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (row0 + i * 16 < a.M)
            *reinterpret_cast<uint2*>(codes + (row0 + i * 16) * a.ld + c0) = codes8(v[i], b, c0, a.N);
    if (tid == 0) {
        *scale = uint8_t(b);
        if (a.status && b == 255u) atomicOr(a.status, SKETCH_FLAG_WEIGHT_RANGE);
    }
}

// Encoder of 1 x 128 blocks: 16 lanes per block, one block each.
template <int DT>
__global__ __launch_bounds__(256) void fp8_encode_rows_kernel(EncodeArgs a) {
    const uint64_t id = (uint64_t(blockIdx.y) * gridDim.x + blockIdx.x) * 16 + (threadIdx.x >> 4);   // (matrix, row, column block)
    const uint32_t lds = uint32_t(a.lds);
    const uint64_t grow = id / lds;
    const int64_t cb = int64_t(id - grow * lds), mat = int64_t(grow / uint64_t(a.M)), row = int64_t(grow) - mat * a.M;
    if (mat >= a.count) return;
    uint8_t* codes = a.buf + mat * a.bytes;
    uint8_t* scale = codes + a.scales_offset + row * a.lds + cb;
    const int64_t c0 = cb * 128 + (threadIdx.x & 15) * 8;
    constexpr int64_t es = DT == SKETCH_F32 ? 4 : 2;
    const unsigned char* W = static_cast<const unsigned char*>(a.W) + mat * a.M * a.N * es;
    float v[8];
    load_row8<DT>(W, row, a.N, c0, v);
    const uint32_t b = fp8_scale_byte(max16(max_bits(v)));
    if (cb < a.col_blocks) *reinterpret_cast<uint2*>(codes + row * a.ld + c0) = codes8(v, b, c0, a.N);
    if ((threadIdx.x & 15) == 0) {
        *scale = cb < a.col_blocks ? uint8_t(b) : uint8_t(0);
        if (a.status && b == 255u) atomicOr(a.status, SKETCH_FLAG_WEIGHT_RANGE);
    }
}

// ---------------------------------------------------------------------------
// Products of few rows.  Bound by the codes of W coming from memory, so every
// code is read once: a workgroup has 16 or 32 outputs, and its 8 waves share
// out the columns in runs of 4 blocks of 128.  A fragment is 16 rows x 128
// columns, one row to a lane: lane l holds row l % 16 and the columns
// 16c..16c+15 and 64+16c..64+16c+15, c = l / 16, the same ones of outputs (A)
// and tokens (B), so that each load covers 64 contiguous bytes of a row.
// D: token l % 16, outputs 4c..4c+3.  The waves' sums meet in LDS and are
// added in their order.
//
// Both fragments are widened to bfloat16 with their scales applied, four 16x16x32
// MFMAs, exact products, float32 sums.  (One 16x16x128 MFMA on the codes applies
// the scales itself, but its sums of 8 neighbouring products keep only 13 bits
// below the largest; it saves 0 to 3 us here: 11008 x 4096 at 4 rows 17.2 -> 14.4
// us, at 16 rows 17.9 -> 17.8 us.)
// ---------------------------------------------------------------------------
constexpr int kWaves = 8;
constexpr int kRun = 4;      // blocks of 128 columns in a wave's run
constexpr int kTokens = SKETCH_FP8_TOKENS;   // rows that fp8_tokens_kernel takes

__device__ inline i32x8 load_frag(const uint8_t* lo, const uint8_t* hi) {
    return __builtin_shufflevector(*reinterpret_cast<const i32x4*>(lo), *reinterpret_cast<const i32x4*>(hi), 0, 1, 2,
                                   3, 4, 5, 6, 7);
}

// acc += A B for a block: the fragments and their scale bytes.
__device__ inline f32x4 multiply(const i32x8& a, uint32_t as, const i32x8& b, uint32_t bs, f32x4 acc) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_widen(a[2 * q], a[2 * q + 1], fp8_scale(as)),
                                                      fp8_widen(b[2 * q], b[2 * q + 1], fp8_scale(bs)), acc, 0, 0, 0);
    return acc;
}

__device__ inline void store_y(const Fp8Product& p, int64_t t, int64_t m, float v) {
    const int64_t e = t * p.M + m;
    if (p.ydt == SKETCH_F32)
        store1_val<SKETCH_F32>(p.Y, e, v);
    else if (p.ydt == SKETCH_BF16)
        store1_val<SKETCH_BF16>(p.Y, e, v);
    else
        store1_val<SKETCH_F16>(p.Y, e, v);
}

// The codes of a run for RT x 16 outputs, and its scale bytes.  Blocks past
// the last are read as the last and not used.
template <int RT>
struct Run {
    i32x8 f[RT][kRun];
    uint32_t scales;

    __device__ inline void load(const uint8_t* const (&row)[RT], const uint8_t* srow, int c, uint32_t k0, uint32_t kb) {
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            const size_t at = size_t(min(k0 + u, kb - 1)) * 128;
#pragma unroll
            for (int i = 0; i < RT; ++i) f[i][u] = load_frag(row[i] + at + 16 * c, row[i] + at + 64 + 16 * c);
        }
        scales = *reinterpret_cast<const uint32_t*>(srow + k0);
    }
};

template <int RT>
__device__ inline void weight_rows(const Fp8Product& p, int64_t m0, int r, const uint8_t* (&row)[RT]) {
#pragma unroll
    for (int i = 0; i < RT; ++i) row[i] = p.w + min(m0 + i * 16 + r, p.M - 1) * p.ld;
}

template <int RT>
__device__ inline void add_and_store(const Fp8Product& p, float (*part)[16][RT * 16 + 1], const f32x4 (&acc)[RT],
                                     int64_t m0) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, c = lane >> 4;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) part[wave][r][i * 16 + 4 * c + v] = acc[i][v];
    __syncthreads();
    if (tid < RT * 256) {
        const int m = tid % (RT * 16), t = tid / (RT * 16);
        if (t >= p.T || m0 + m >= p.M) return;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += part[w][t][m];
        store_y(p, t, m0 + m, sum);
    }
}

// Up to NP rows of X (p.x, of dtype XD), encoded by every workgroup for itself,
// which saves the launch that would encode them first: a wave encodes the
// blocks of its own run, 16 lanes to a (block, row), into its own part of LDS.
// Repeated by all workgroups, this costs more than the launch beyond a few
// rows (28672 x 8192, 16 rows: 114 us against 66 us in two launches).
template <int XD, int NP>
__global__ __launch_bounds__(kWaves * 64) void fp8_tokens_kernel(Fp8Product p, int64_t N) {
    __shared__ __attribute__((aligned(16))) uint8_t codes[kWaves][4 * NP][128];
    __shared__ uint32_t scales[kWaves][4 * NP];
    __shared__ float part[kWaves][16][17];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4, T = int(p.T);
    const int64_t m0 = int64_t(blockIdx.x) * 16;
    const uint8_t* row[1];
    weight_rows<1>(p, m0, r, row);
    const uint8_t* srow = p.ws + m0 / 128 * p.lds;
    f32x4 acc[1] = {f32x4{0, 0, 0, 0}};
    for (uint32_t k = wave * kRun; k < p.kb; k += kWaves * kRun) {
        float x[NP][8] = {};
#pragma unroll
        for (int n = 0; n < NP; ++n) {   // (block, row) number 4 n + c of the run
            const int i = n * 4 + c;
            if (i < kRun * T) load_row8<XD>(p.x, i % T, N, int64_t(k + i / T) * 128 + r * 8, x[n]);
        }
        Run<1> w;
        w.load(row, srow, c, k, p.kb);
        asm volatile("" ::: "memory");   // all loads of the run before its first use
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const uint32_t b = fp8_scale_byte(max16(max_bits(x[n])));
            const int at = n * 4 + c;
            *reinterpret_cast<uint2*>(&codes[wave][at][(((r >> 1) ^ (at & 7)) << 4) + (r & 1) * 8]) = codes8(x[n], b);
            if (r == 0) scales[wave][at] = b;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            if (k + u >= p.kb) break;
            const int at = u * T + min(r, T - 1);   // tokens past the last are not stored
            const i32x8 xf = load_frag(&codes[wave][at][(c ^ (at & 7)) << 4], &codes[wave][at][((c + 4) ^ (at & 7)) << 4]);
            acc[0] = multiply(w.f[0][u], w.scales >> (8 * u) & 255u, xf, scales[wave][at], acc[0]);
        }
    }
    add_and_store<1>(p, part, acc, m0);
}

// Up to 16 encoded rows, read from memory (they stay in the caches).  The
// sums run in the same order as in fp8_tokens_kernel.
template <int RT>
__global__ __launch_bounds__(kWaves * 64) void fp8_rows_kernel(Fp8Product p) {
    __shared__ float part[kWaves][16][RT * 16 + 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4;
    const int64_t m0 = int64_t(blockIdx.x) * (RT * 16);
    const uint8_t* row[RT];
    weight_rows<RT>(p, m0, r, row);
    const uint8_t* srow = p.ws + m0 / 128 * p.lds;   // RT * 16 outputs lie in one block of 128
    const int64_t t = min(int64_t(r), p.T - 1);
    const uint8_t* x[1] = {p.x + t * p.ld};
    const uint8_t* xs = p.xs + t * p.lds;
    f32x4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = f32x4{0, 0, 0, 0};
    for (uint32_t k = wave * kRun; k < p.kb; k += kWaves * kRun) {
        Run<RT> w;
        Run<1> xr;
        w.load(row, srow, c, k, p.kb);
        xr.load(x, xs, c, k, p.kb);
        asm volatile("" ::: "memory");   // all loads of the run before its first use
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            if (k + u >= p.kb) break;
#pragma unroll
            for (int i = 0; i < RT; ++i)
                acc[i] = multiply(w.f[i][u], w.scales >> (8 * u) & 255u, xr.f[0][u], xr.scales >> (8 * u) & 255u, acc[i]);
        }
    }
    add_and_store<RT>(p, part, acc, m0);
}

sketch_status launch_few(const Fp8Product& p, int x_dtype, int64_t N, hipStream_t st) {
    auto tokens = [&](auto kernel) {
        kernel<<<unsigned((p.M + 15) / 16), kWaves * 64, 0, st>>>(p, N);
        return launch_status();
    };
    auto rows = [&](auto kernel, int64_t outputs) {
        kernel<<<unsigned((p.M + outputs - 1) / outputs), kWaves * 64, 0, st>>>(p);
        return launch_status();
    };
    if (x_dtype == SKETCH_F32)
        return p.T == 1 ? tokens(fp8_tokens_kernel<SKETCH_F32, 1>) : tokens(fp8_tokens_kernel<SKETCH_F32, 4>);
    if (x_dtype == SKETCH_BF16)
        return p.T == 1 ? tokens(fp8_tokens_kernel<SKETCH_BF16, 1>) : tokens(fp8_tokens_kernel<SKETCH_BF16, 4>);
    if (x_dtype == SKETCH_F16)
        return p.T == 1 ? tokens(fp8_tokens_kernel<SKETCH_F16, 1>) : tokens(fp8_tokens_kernel<SKETCH_F16, 4>);
    // 32 outputs to a workgroup halve the reads of X.  They pay from 64 outputs per compute unit on (16 rows, 16384 x
    // 4096: 20.5 us with 16 outputs, 19.1 us with 32; 28672 x 8192 61.6 and 56.1; 128256 x 1024 41.1 and 35.8; at 5 rows
    // 28672 x 8192 48.8 and 50.2), and below where a wave has several runs (16 rows, 5000 x 28672 61 and 48; 8192 x
    // 28672 68 and 57).  With one run (11008 x 4096: 15.2 and 17.0), or where those of 16 all have a compute unit to
    // themselves (4096 x 28672: 38 and 48), 16 have the shorter way.
    const int64_t ncu = compute_units();
    const bool two = p.M >= 64 * ncu || (p.M > 16 * ncu && p.kb > kWaves * kRun);
    return two ? rows(fp8_rows_kernel<2>, 32) : rows(fp8_rows_kernel<1>, 16);
}

bool valid_dtype(int d) { return d == SKETCH_F32 || d == SKETCH_BF16 || d == SKETCH_F16; }

// y_dtype of a product: the type of Y, and how the products are summed.  Only
// the rounding to bfloat16 (rms 1.7e-3 of an output) hides the e4m3 matrix
// cores' sums (up to 5e-5); that to binary16 (2.1e-4) does not, and up to
// SKETCH_FP8_EXACT_BATCH rows the product is bound by its bytes and gains
// nothing to speak of (11008 x 4096 at 64 rows 23.1 us either way; 28672 x 8192
// at 2048 rows 364 us, with float32 sums 740 us).
bool y_type(int y_dtype, int64_t batch, int* type, bool* exact) {
    const bool asked = y_dtype == (SKETCH_BF16 | SKETCH_FP8_F32_SUMS);
    *type = asked ? int(SKETCH_BF16) : y_dtype;
    *exact = *type != SKETCH_BF16 || asked || batch <= SKETCH_FP8_EXACT_BATCH;
    return valid_dtype(*type);
}

// What one product does and needs.
struct ProductPlan {
    sketch_fp8_shape w, x;   // the weight, the encoded rows
    int ydt;
    bool exact, encode;      // float32 sums; rows encoded by a launch of their own
    GemmPlan gemm;           // more than 16 rows
    size_t workspace;
};

// Checks the parameters (the rules of sketch_fp8_workspace_bytes) and fills the plan.
sketch_status product_plan(const sketch_fp8_params* p, int64_t batch, int x_dtype, int y_dtype, ProductPlan* plan) {
    sketch_status rc = fp8_shape(p, &plan->w);
    if (rc != SKETCH_OK) return rc;
    const bool rows = x_dtype == SKETCH_FP8_ROWS;
    if (batch < 0 || p->block_rows != 128 || p->count > 1 || (!rows && !valid_dtype(x_dtype)) ||
        !y_type(y_dtype, batch, &plan->ydt, &plan->exact))
        return SKETCH_EINVAL;
    const sketch_fp8_params xp{batch, p->N, 1, 1};
    rc = fp8_shape(&xp, &plan->x);
    if (rc != SKETCH_OK) return rc;
    plan->workspace = 0;
    if (batch == 0 || p->M == 0) return SKETCH_OK;
    plan->encode = !rows && batch > kTokens;
    if (plan->encode) plan->workspace += plan->x.bytes;
    if (batch <= 16) return SKETCH_OK;
    rc = fp8_gemm_plan(p->M, batch, uint32_t(plan->w.col_blocks), plan->exact, &plan->gemm);
    plan->workspace += plan->gemm.workspace;
    return rc;
}

}  // namespace

sketch_status fp8_shape(const sketch_fp8_params* p, sketch_fp8_shape* s) {
    if (!p || p->M < 0 || p->M > SKETCH_FP8_MAX_M || p->N < 1 || p->N > SKETCH_FP8_MAX_N) return SKETCH_EINVAL;
    if (p->block_rows != 1 && p->block_rows != 128) return SKETCH_EINVAL;
    if (p->count < 0 || p->count > SKETCH_FP8_MAX_COUNT) return SKETCH_EINVAL;
    s->ld = (p->N + 127) / 128 * 128;
    s->col_blocks = s->ld / 128;
    s->lds = (s->col_blocks + 3) / 4 * 4;
    s->row_blocks = (p->M + p->block_rows - 1) / p->block_rows;
    s->scales_offset = align256(size_t(p->M) * size_t(s->ld));
    s->bytes = align256(s->scales_offset + size_t(s->row_blocks) * size_t(s->lds));
    return SKETCH_OK;
}

sketch_status launch_fp8_encode(const sketch_fp8_params* p, const sketch_fp8_shape& s, const void* W,
                                sketch_dtype dt, void* buf, int32_t* status, hipStream_t st) {
    EncodeArgs a{W, static_cast<uint8_t*>(buf), status, p->M, p->N, s.ld, s.lds, s.row_blocks, s.col_blocks,
                 p->count > 1 ? p->count : 1, s.scales_offset, s.bytes};
    const bool rows = p->block_rows == 1;
    const int64_t blocks = a.lds * a.row_blocks * a.count, groups = rows ? (blocks + 15) / 16 : blocks;
    constexpr int64_t kLine = kMaxThreads / 256;
    const int64_t lines = (groups + kLine - 1) / kLine;
    if (lines > 65535) return SKETCH_EINVAL;
    const dim3 grid(unsigned(lines > 1 ? kLine : groups), unsigned(lines));
    auto go = [&](auto kernel) {
        kernel<<<grid, 256, 0, st>>>(a);
        return launch_status();
    };
    if (dt == SKETCH_F32) return rows ? go(fp8_encode_rows_kernel<SKETCH_F32>) : go(fp8_encode_kernel<SKETCH_F32>);
    if (dt == SKETCH_BF16) return rows ? go(fp8_encode_rows_kernel<SKETCH_BF16>) : go(fp8_encode_kernel<SKETCH_BF16>);
    return rows ? go(fp8_encode_rows_kernel<SKETCH_F16>) : go(fp8_encode_kernel<SKETCH_F16>);
}

}  // namespace sketch

using namespace sketch;

extern "C" {

sketch_status sketch_fp8_layout(const sketch_fp8_params* p, sketch_fp8_shape* shape) {
    return shape ? fp8_shape(p, shape) : SKETCH_EINVAL;
}

sketch_status sketch_fp8_encode(const sketch_fp8_params* p, const void* W, sketch_dtype w_dtype, void* buf,
                                int32_t* status_dev, void* stream) {
    sketch_fp8_shape s;
    const sketch_status rc = fp8_shape(p, &s);
    if (rc != SKETCH_OK) return rc;
    if (!valid_dtype(w_dtype) || (reinterpret_cast<uintptr_t>(status_dev) & 3u)) return SKETCH_EINVAL;
    if (p->M == 0) return SKETCH_OK;
    if (!W || !buf || !aligned16(W) || !aligned16(buf)) return SKETCH_EINVAL;
    const size_t count = p->count > 1 ? size_t(p->count) : 1;
    if (overlap({W, count * size_t(p->M) * size_t(p->N) * elem_bytes(w_dtype)}, {buf, count * s.bytes})) return SKETCH_EINVAL;
    return launch_fp8_encode(p, s, W, w_dtype, buf, status_dev, static_cast<hipStream_t>(stream));
}

sketch_status sketch_fp8_workspace_bytes(const sketch_fp8_params* p, int64_t batch, int x_dtype, int y_dtype,
                                         size_t* bytes) {
    ProductPlan plan;
    const sketch_status rc = product_plan(p, batch, x_dtype, y_dtype, &plan);
    if (rc != SKETCH_OK) return rc;
    if (!bytes) return SKETCH_EINVAL;
    *bytes = plan.workspace;
    return SKETCH_OK;
}

sketch_status sketch_fp8_matmul(const sketch_fp8_params* p, const void* buf, const void* X, int x_dtype,
                                int64_t batch, void* Y, int y_dtype, void* workspace,
                                size_t workspace_bytes, void* stream) {
    ProductPlan plan;
    sketch_status rc = product_plan(p, batch, x_dtype, y_dtype, &plan);
    if (rc != SKETCH_OK) return rc;
    if (batch == 0 || p->M == 0) return SKETCH_OK;
    const size_t need = plan.workspace;
    if (!buf || !X || !Y || !aligned16(buf) || !aligned16(X) || !aligned16(Y)) return SKETCH_EINVAL;
    if (need > 0) {
        if (!workspace || !aligned16(workspace)) return SKETCH_EINVAL;
        if (workspace_bytes < need) return SKETCH_ESMALL;
    }
    // workgroups that are done store Y while others still read
    const sketch_fp8_shape &s = plan.w, &xs = plan.x;
    const Range ry{Y, size_t(batch) * size_t(p->M) * elem_bytes(plan.ydt)}, rw{buf, s.bytes}, rs{workspace, need},
        rx{X, x_dtype == SKETCH_FP8_ROWS ? xs.bytes : size_t(batch) * size_t(p->N) * elem_bytes(x_dtype)};
    if (overlap(ry, rw) || overlap(ry, rs) || (!plan.encode && overlap(ry, rx)) || overlap(rs, rw) || overlap(rs, rx))
        return SKETCH_EINVAL;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const uint8_t *w8 = static_cast<const uint8_t*>(buf), *x8 = static_cast<const uint8_t*>(X);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (plan.encode) {
        const sketch_fp8_params xp{batch, p->N, 1, 1};
        rc = launch_fp8_encode(&xp, xs, X, sketch_dtype(x_dtype), ws, nullptr, st);
        if (rc != SKETCH_OK) return rc;
        x8 = ws;
        ws += xs.bytes;
    }
    const Fp8Product a{w8, w8 + s.scales_offset, x8, x8 + xs.scales_offset, Y, p->M, batch, s.ld, s.lds,
                       uint32_t(s.col_blocks), plan.ydt, plan.exact};
    if (batch > 16) return launch_fp8_gemm(a, plan.gemm, ws, st);
    return launch_few(a, plan.encode ? SKETCH_FP8_ROWS : x_dtype, p->N, st);
}

}  // extern "C"
