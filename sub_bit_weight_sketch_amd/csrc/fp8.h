// fp8.h -- internal definitions of the e4m3 linears (fp8.hip) and of the
// mixture-of-experts layer that reads them (moe.hip).
#pragma once

#include <atomic>

#include "../../include/sketch_fp8.h"
#include "common.h"

namespace sketch {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp8Block = 128;   // columns of a block

// Checks the parameters and fills the layout (the rules of sketch_fp8_layout).
sketch_status fp8_shape(const sketch_fp8_params* p, sketch_fp8_shape* s);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Memory of a call, to refuse buffers that share it.
struct Range {
    const void* p;
    size_t bytes;
};

inline bool overlap(const Range& a, const Range& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.bytes > 0 && b.bytes > 0 && (x < y ? y - x < a.bytes : x - y < b.bytes);
}

inline size_t elem_bytes(int dtype) { return dtype == SKETCH_F32 ? 4 : 2; }

// Compute units of the current device, asked for once per device (256 when
// none answers).
inline int compute_units() {
    static std::atomic<int> known[64];
    int dev = 0, ncu = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    ncu = known[dev].load(std::memory_order_relaxed);
    if (ncu > 0) return ncu;
    if (hipDeviceGetAttribute(&ncu, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || ncu <= 0) return 256;
    known[dev].store(ncu, std::memory_order_relaxed);
    return ncu;
}

// Scale byte of a block from the bits of its largest magnitude.  With
// amax = m 2^p, 1 <= m < 2, the smallest e with amax <= 448 2^e = 1.75 2^(e+8)
// is p - 8, or p - 7 when m > 1.75.  NaN and infinities give 255.
__device__ inline uint32_t fp8_scale_byte(uint32_t amax_bits) {
    const uint32_t ex = amax_bits >> 23;
    if (ex == 255u) return 255u;
    const int b = int(ex) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return b < 0 ? 0u : uint32_t(b);
}

// 2^(127 - byte), the factor that takes an element to its code's range
// (byte <= 247; the exponent field is 254 - byte >= 7).
__device__ inline float fp8_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Four floats -> four e4m3 codes, ties to even.
__device__ inline uint32_t fp8_pack4(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
    return uint32_t(v);
}

// The byte as the exponent of a float32, the form in which the widening takes a
// scale: it reads that field alone, 0 as 2^-127 and 255 as NaN.
__device__ inline float fp8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// 8 codes (two dwords) -> 8 bfloat16 values times a power of two (exact).
__device__ inline bf16x8 fp8_widen(uint32_t lo, uint32_t hi, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 8 elements of a row from column c0 on, zeros past its end.  Rows of any
// length: the wide loads need only the alignment of an element (7.6 us
// element by element -> 4.1 us for 517 x 4001 float32).
template <int DT>
__device__ inline void load_row8(const void* W, int64_t row, int64_t N, int64_t c0, float (&v)[8]) {
    if (c0 + 8 <= N) {
        typedef uint32_t loose __attribute__((ext_vector_type(4), aligned(2)));
        constexpr int es = DT == SKETCH_F32 ? 4 : 2;
        const loose* at = reinterpret_cast<const loose*>(static_cast<const char*>(W) + (row * N + c0) * es);
        const loose a = at[0], b = DT == SKETCH_F32 ? at[1] : a;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t h = (a[e >> 1] >> ((e & 1) * 16)) & 0xFFFFu;
            v[e] = DT == SKETCH_F32    ? __uint_as_float(e < 4 ? a[e & 3] : b[e & 3])
                   : DT == SKETCH_BF16 ? bf16_bits_to_f32(h)
                                       : f16_bits_to_f32(h);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c0 + e < N ? load_elem<DT>(W, row * N + c0 + e) : 0.0f;
}

// Operands of one product: codes and scales of the weight [M] and of the
// encoded rows [T], both with row strides ld and lds.
struct Fp8Product {
    const uint8_t *w, *ws, *x, *xs;
    void* Y;
    int64_t M, T, ld, lds;
    uint32_t kb;   // blocks of 128 columns
    int ydt;
    bool exact;    // float32 sums
};

// Threads that one dimension of a grid holds.
constexpr int64_t kMaxThreads = 0xFFFFFFFF;

// Products of many rows (fp8_gemm.hip): which kernel one takes, and over how
// many workgroups K is split.
struct GemmPlan {
    bool big;          // fp8_gemm_big_kernel, or fp8_gemm_kernel
    int fa, fb;        // outputs and tokens of a tile, in units of 32
    uint32_t splits;
    int64_t tiles_o, tiles_t;
    size_t workspace;  // the parts of a split
};

// SKETCH_EINVAL when there are more tiles than a grid holds.
sketch_status fp8_gemm_plan(int64_t M, int64_t T, uint32_t kb, bool exact, GemmPlan* g);
sketch_status launch_fp8_gemm(const Fp8Product& p, const GemmPlan& g, void* ws, hipStream_t st);

sketch_status launch_fp8_encode(const sketch_fp8_params* p, const sketch_fp8_shape& s, const void* W,
                                sketch_dtype dt, void* buf, int32_t* status, hipStream_t st);

}  // namespace sketch
