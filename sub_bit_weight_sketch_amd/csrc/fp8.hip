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

// ---------------------------------------------------------------------------
// Encoder.  One workgroup per 128 x 128 tile, 16 lanes to a row: a thread
// holds 8 columns of 8 rows, so the elements stay in registers between the
// maximum and the rounding and W is read once.  HBM-bound.
// ---------------------------------------------------------------------------
struct EncodeArgs {
    const void* W;
    uint8_t* buf;
    int32_t* status;
    int64_t M, N, ld, lds, tiles_m, col_blocks;
    size_t scales_offset, bytes;
};

template <int DT, bool ROWS>
__global__ __launch_bounds__(256) void fp8_encode_kernel(EncodeArgs a) {
    __shared__ uint32_t red[4];
    const int tid = threadIdx.x;
    const int64_t cb = blockIdx.x % a.lds, tm = (blockIdx.x / a.lds) % a.tiles_m,
                  mat = blockIdx.x / a.lds / a.tiles_m;
    uint8_t* codes = a.buf + mat * a.bytes;
    uint8_t* scales = codes + a.scales_offset;
    if (cb >= a.col_blocks) {   // scale bytes that round a row of scales up to a dword
        if (ROWS) {
            const int64_t row = tm * 128 + tid;
            if (tid < 128 && row < a.M) scales[row * a.lds + cb] = 0;
        } else if (tid == 0) {
            scales[tm * a.lds + cb] = 0;
        }
        return;
    }
    constexpr int64_t es = DT == SKETCH_F32 ? 4 : 2;
    const unsigned char* W = static_cast<const unsigned char*>(a.W) + mat * a.M * a.N * es;
    const int64_t c0 = cb * 128 + (tid & 15) * 8;
    const bool whole = a.N % 8 == 0 && c0 + 8 <= a.N;   // rows keep 16-byte alignment
    float v[8][8];
    uint32_t mx[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = tm * 128 + i * 16 + (tid >> 4);
        if (row < a.M && whole) {
            load8_f32<DT>(W, row * a.N + c0, v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] = row < a.M && c0 + e < a.N ? load_elem<DT>(W, row * a.N + c0 + e) : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        mx[i] = 0;   // magnitudes compare as their bits; NaN is above infinity
#pragma unroll
        for (int e = 0; e < 8; ++e) mx[i] = max(mx[i], __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
    }
    if constexpr (ROWS) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) mx[i] = max(mx[i], uint32_t(__shfl_xor(int(mx[i]), d)));
    } else {
        uint32_t m = mx[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max(m, mx[i]);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) m = max(m, uint32_t(__shfl_xor(int(m), d)));
        if ((tid & 63) == 0) red[tid >> 6] = m;
        __syncthreads();
        m = max(max(red[0], red[1]), max(red[2], red[3]));
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = m;
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = tm * 128 + i * 16 + (tid >> 4);
        if (row >= a.M) continue;
        const uint32_t b = fp8_scale_byte(mx[i]);
        const bool nan = b == 255u;
        bad |= nan;
        const float inv = fp8_inv_scale(nan ? 127u : b);
        uint2 q;
        q.x = nan ? 0x7F7F7F7Fu : fp8_pack4(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv);
        q.y = nan ? 0x7F7F7F7Fu : fp8_pack4(v[i][4] * inv, v[i][5] * inv, v[i][6] * inv, v[i][7] * inv);
        if (nan && c0 + 8 > a.N) {   // the padding stays zero
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c0 + e >= a.N) (e < 4 ? q.x : q.y) &= ~(0xFFu << (8 * (e & 3)));
        }
        *reinterpret_cast<uint2*>(codes + row * a.ld + c0) = q;
        if (ROWS && (tid & 15) == 0) scales[row * a.lds + cb] = uint8_t(b);
        if (!ROWS && tid == 0 && i == 0) scales[tm * a.lds + cb] = uint8_t(b);
    }
    if (a.status && __ballot(bad) != 0 && (tid & 63) == 0) atomicOr(a.status, SKETCH_FLAG_WEIGHT_RANGE);
}

// ---------------------------------------------------------------------------
// Product.  One wave per 16 outputs x 16 tokens, operands straight from
// memory, widened to bfloat16 with their scales applied (exact) and summed by
// 16x16x32 MFMAs.  A (weights): lane l holds output l % 16; B (tokens): token
// l % 16; the lane's 32 columns of a block are bytes 16c..16c+15 and
// 64+16c..64+16c+15, c = l / 16, in both, so that each load covers 64
// contiguous bytes of a row.  D: token l % 16, outputs 4c..4c+3.
// ---------------------------------------------------------------------------
__device__ inline i32x8 load_frag(const uint8_t* row, int c) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(row + 16 * c);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(row + 64 + 16 * c);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int YD>
__global__ __launch_bounds__(64) void fp8_simple_kernel(Fp8Product a) {
    const int lane = threadIdx.x, r = lane & 15, c = lane >> 4;
    const int64_t m0 = int64_t(blockIdx.x) * 16, t0 = int64_t(blockIdx.y) * 16;
    const int64_t m = min(m0 + r, a.M - 1), t = min(t0 + r, a.T - 1);
    const uint8_t *w = a.w + m * a.ld, *x = a.x + t * a.ld;
    const uint8_t *ws = a.ws + (m0 / 128) * a.lds, *xs = a.xs + t * a.lds;
    f32x4 acc = {0, 0, 0, 0};
    for (uint32_t k = 0; k < a.kb; ++k) {
        const i32x8 wf = load_frag(w + k * 128, c), xf = load_frag(x + k * 128, c);
        const float wsc = fp8_scale(ws[k]), xsc = fp8_scale(xs[k]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_widen(wf[2 * j], wf[2 * j + 1], wsc),
                                                          fp8_widen(xf[2 * j], xf[2 * j + 1], xsc), acc, 0, 0, 0);
    }
    if (t0 + r < a.T)
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (m0 + 4 * c + v < a.M) store1_val<YD>(a.Y, (t0 + r) * a.M + m0 + 4 * c + v, acc[v]);
}

bool valid_dtype(int d) { return d == SKETCH_F32 || d == SKETCH_BF16 || d == SKETCH_F16; }

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
    EncodeArgs a{W, static_cast<uint8_t*>(buf), status, p->M, p->N, s.ld, s.lds, (p->M + 127) / 128, s.col_blocks,
                 s.scales_offset, s.bytes};
    const int64_t grid = a.lds * a.tiles_m * (p->count > 1 ? p->count : 1);
    if (grid > 0x7FFFFFFF) return SKETCH_EINVAL;
    const bool rows = p->block_rows == 1;
    auto go = [&](auto kernel) {
        kernel<<<unsigned(grid), 256, 0, st>>>(a);
        return launch_status();
    };
    if (dt == SKETCH_F32)
        return rows ? go(fp8_encode_kernel<SKETCH_F32, true>) : go(fp8_encode_kernel<SKETCH_F32, false>);
    if (dt == SKETCH_BF16)
        return rows ? go(fp8_encode_kernel<SKETCH_BF16, true>) : go(fp8_encode_kernel<SKETCH_BF16, false>);
    return rows ? go(fp8_encode_kernel<SKETCH_F16, true>) : go(fp8_encode_kernel<SKETCH_F16, false>);
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
    return launch_fp8_encode(p, s, W, w_dtype, buf, status_dev, static_cast<hipStream_t>(stream));
}

sketch_status sketch_fp8_workspace_bytes(const sketch_fp8_params* p, int64_t batch, int x_dtype, sketch_dtype y_dtype,
                                         size_t* bytes) {
    sketch_fp8_shape s, xs;
    sketch_status rc = fp8_shape(p, &s);
    if (rc != SKETCH_OK) return rc;
    if (!bytes || batch < 0 || p->block_rows != 128 || p->count > 1 || (!valid_dtype(x_dtype) && x_dtype != SKETCH_FP8_ROWS) ||
        !valid_dtype(y_dtype))
        return SKETCH_EINVAL;
    const sketch_fp8_params xp{batch, p->N, 1, 1};
    rc = fp8_shape(&xp, &xs);
    if (rc != SKETCH_OK) return rc;
    *bytes = 0;
    if (batch == 0 || p->M == 0) return SKETCH_OK;
    if (x_dtype != SKETCH_FP8_ROWS) *bytes += xs.bytes;
    if (batch > SKETCH_FP8_EXACT_BATCH) *bytes += fp8_gemm_workspace(p->M, batch, uint32_t(s.col_blocks), y_dtype);
    return SKETCH_OK;
}

sketch_status sketch_fp8_matmul(const sketch_fp8_params* p, const void* buf, const void* X, int x_dtype,
                                int64_t batch, void* Y, sketch_dtype y_dtype, void* workspace,
                                size_t workspace_bytes, void* stream) {
    size_t need = 0;
    sketch_status rc = sketch_fp8_workspace_bytes(p, batch, x_dtype, y_dtype, &need);
    if (rc != SKETCH_OK) return rc;
    if (batch == 0 || p->M == 0) return SKETCH_OK;
    if (!buf || !X || !Y || !aligned16(buf) || !aligned16(X) || !aligned16(Y)) return SKETCH_EINVAL;
    if (need > 0) {
        if (!workspace || !aligned16(workspace)) return SKETCH_EINVAL;
        if (workspace_bytes < need) return SKETCH_ESMALL;
    }
    const hipStream_t st = static_cast<hipStream_t>(stream);
    sketch_fp8_shape s, xs;
    const sketch_fp8_params xp{batch, p->N, 1, 1};
    (void)fp8_shape(p, &s);
    (void)fp8_shape(&xp, &xs);
    const uint8_t *w8 = static_cast<const uint8_t*>(buf), *x8 = static_cast<const uint8_t*>(X);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (x_dtype != SKETCH_FP8_ROWS) {
        rc = launch_fp8_encode(&xp, xs, X, sketch_dtype(x_dtype), ws, nullptr, st);
        if (rc != SKETCH_OK) return rc;
        x8 = ws;
        ws += xs.bytes;
    }
    const Fp8Product a{w8, w8 + s.scales_offset, x8, x8 + xs.scales_offset, Y, p->M, batch, s.ld, s.lds,
                       uint32_t(s.col_blocks), int(y_dtype)};
    if (batch > SKETCH_FP8_EXACT_BATCH) return launch_fp8_gemm(a, ws, st);
    const dim3 grid(unsigned((p->M + 15) / 16), unsigned((batch + 15) / 16));
    auto go = [&](auto kernel) {
        kernel<<<grid, 64, 0, st>>>(a);
        return launch_status();
    };
    return y_dtype == SKETCH_F32    ? go(fp8_simple_kernel<SKETCH_F32>)
           : y_dtype == SKETCH_BF16 ? go(fp8_simple_kernel<SKETCH_BF16>)
                                    : go(fp8_simple_kernel<SKETCH_F16>);
}

}  // extern "C"
