// int8.h -- internal definitions of the 8-bit integer linears (int8.hip,
// int8_gemm.hip).
#pragma once

#include "../../include/sketch_int8.h"
#include "tile.h"

namespace sketch {

// Operands of one product: codes and scales of the weights (`experts` of them,
// w_bytes apart) and of the encoded rows, row strides ld.  Without `counts`,
// one weight and terms that are the rows in order.
struct Int8Product {
    const int8_t* w;
    size_t w_bytes, w_scales;   // from one weight to the next, from its codes to its scales
    const int8_t* x;
    const float* xs;
    int64_t x_rows;
    void* Y;
    int64_t M, T, ld;           // outputs, terms
    uint32_t kb;                // blocks of 128 columns
    int ydt;
    int experts;
    const void *counts, *rows;
    bool counts64, rows64;
};

// Terms of one expert that a workgroup multiplies: first, first + 1, .. (n of
// them).
struct Terms {
    int expert, first, n;
};

// Sum over the lanes up to this one (all lanes active).
__device__ inline int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // the last lane of a row of 16 to the next row
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // lane 31 to the upper half
    return v;
}

// Terms of expert e as its count says, within 0..T.
__device__ inline int expert_terms(const Int8Product& p, int e) {
    if (e >= p.experts) return 0;
    const int64_t c = p.counts64 ? static_cast<const int64_t*>(p.counts)[e] : int64_t(static_cast<const int32_t*>(p.counts)[e]);
    return int(c < 0 ? 0 : c > p.T ? p.T : c);
}

// The terms of 64 experts, one to a lane, cut into tiles of up to BT.  T <= 2^24,
// so 64 counts of up to T fit an int.
struct ExpertTiles {
    int begin, end;         // the lane's expert's terms
    int tiles, upto;        // its tiles, and those of all experts up to it
    int all_terms, all_tiles;

    // of experts base .., behind `terms` terms and `before` tiles
    template <int BT>
    __device__ inline void count(const Int8Product& p, int base, int terms, int before) {
        const int T = int(p.T), n = expert_terms(p, base + int(threadIdx.x & 63)), sum = wave_scan(n);
        begin = min(terms + sum - n, T);
        end = min(terms + sum, T);
        tiles = (end - begin + BT - 1) / BT;
        upto = before + wave_scan(tiles);
        all_terms = __builtin_amdgcn_readlane(end, 63);
        all_tiles = __builtin_amdgcn_readlane(upto, 63);
    }

    // whether `tile` is one of these, and which
    template <int BT>
    __device__ inline bool find(int base, int tile, Terms& t) const {
        const uint64_t hit = __ballot(tile >= upto - tiles && tile < upto);
        if (!hit) return false;
        const int src = __builtin_ctzll(hit);
        t.expert = base + src;
        t.first = __builtin_amdgcn_readlane(begin, src) + (tile - __builtin_amdgcn_readlane(upto - tiles, src)) * BT;
        t.n = min(BT, __builtin_amdgcn_readlane(end, src) - t.first);
        return true;
    }
};

// Tile `which(tiles)` of all `tiles` tiles of the experts' terms, or false where
// that is none of them.  Every wave works it out for itself from the counts.
template <int BT, typename Which>
__device__ inline bool find_terms(const Int8Product& p, Which which, Terms& t) {
    ExpertTiles x;
    x.count<BT>(p, 0, 0, 0);
    if (p.experts <= 64) return x.find<BT>(0, which(x.all_tiles), t);
    for (int base = 64; base < p.experts; base += 64) x.count<BT>(p, base, x.all_terms, x.all_tiles);
    const int tile = which(x.all_tiles);
    int terms = 0, before = 0;
    for (int base = 0; base < p.experts; base += 64) {
        x.count<BT>(p, base, terms, before);
        if (x.find<BT>(base, tile, t)) return true;
        terms = x.all_terms, before = x.all_tiles;
    }
    return false;
}

// Row of X of a term, or -1 where it lies outside.
__device__ inline int64_t term_row(const Int8Product& p, int64_t term) {
    if (!p.rows) return term;
    const int64_t r = p.rows64 ? static_cast<const int64_t*>(p.rows)[term] : int64_t(static_cast<const int32_t*>(p.rows)[term]);
    return r >= 0 && r < p.x_rows ? r : -1;
}

// What an exact sum stands for: rounded to float32, then by the scales.  The
// empty asm keeps the last product's rounding: without it the compiler may join it
// with a conversion to binary16 that follows, and round once.
__device__ inline float int8_value(int sum, float sx, float sw) {
    float v = float(sum) * sx * sw;
    asm("" : "+v"(v));
    return v;
}

// Which kernel a product takes, and over how many workgroups K is split.
enum Int8Kind {
    kInt8Rows1,   // int8_rows_kernel (int8.hip), 16 outputs to 8 waves
    kInt8Rows2,   // the same, 32 outputs to 4 waves (groups alone)
    kInt8Mid,     // int8_gemm_kernel (int8_gemm.hip)
    kInt8Big      // int8_gemm_big_kernel
};

struct Int8Plan {
    Int8Kind kind;
    int fa, fb;        // outputs and terms of a tile, in units of 32
    uint32_t splits;
    int64_t tiles_o, tiles_t;
    size_t workspace;  // the parts of a split
};

// near: terms that take rows of X in any order find each within 32 bits of bytes.  SKETCH_EINVAL when
// there are more tiles than a grid holds.
sketch_status int8_plan(int64_t M, int64_t T, uint32_t kb, int ydt, int experts, bool group, bool near, Int8Plan* g);
sketch_status launch_int8_gemm(const Int8Product& p, const Int8Plan& g, void* ws, hipStream_t st);

// Four outputs of a row from m on, at any alignment of an element.
template <int YD>
__device__ inline void store4_any(void* Y, int64_t e, f32x4 v, int64_t m, int64_t M) {
    typedef float loose4 __attribute__((ext_vector_type(4), aligned(4)));
    typedef uint32_t loose2 __attribute__((ext_vector_type(2), aligned(2)));
    if (m + 4 <= M) {
        if constexpr (YD == SKETCH_F32)
            *reinterpret_cast<loose4*>(static_cast<float*>(Y) + e) = v;
        else
            *reinterpret_cast<loose2*>(static_cast<uint16_t*>(Y) + e) = loose2{pack2<YD>(v[0], v[1]), pack2<YD>(v[2], v[3])};
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (m + i < M) store1_val<YD>(Y, e + i, v[i]);
}

sketch_status int8_shape(const sketch_int8_params* p, sketch_int8_shape* s);

}  // namespace sketch
