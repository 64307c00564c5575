// int8.h -- internal definitions of the 8-bit integer linears (int8.hip,
// int8_gemm.hip).
#pragma once

#include "../../include/sketch_int8.h"
#include "fp8.h"

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

// Tile `tile` of the experts' terms cut into tiles of up to BT, or false past
// the last one.  Every wave works it out for itself from the counts: 64 experts
// at a time, two sums over the lanes.  T <= 2^24, so 64 counts of up to T fit an int.
template <int BT>
__device__ inline bool find_terms(const Int8Product& p, int tile, Terms& t) {
    const int lane = threadIdx.x & 63, T = int(p.T);
    int terms = 0, tiles = 0;
    for (int base = 0; base < p.experts; base += 64) {
        const int n = expert_terms(p, base + lane);
        const int upto = wave_scan(n), begin = min(terms + upto - n, T), end = min(terms + upto, T);
        const int own = (end - begin + BT - 1) / BT, last = tiles + wave_scan(own);
        const uint64_t hit = __ballot(tile >= last - own && tile < last);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            t.expert = base + src;
            t.first = __builtin_amdgcn_readlane(begin, src) + (tile - __builtin_amdgcn_readlane(last - own, src)) * BT;
            t.n = min(BT, __builtin_amdgcn_readlane(end, src) - t.first);
            return true;
        }
        terms = min(terms + __builtin_amdgcn_readlane(upto, 63), T);
        tiles = __builtin_amdgcn_readlane(last, 63);
    }
    return false;
}

// Tiles of up to BT terms that the experts have.
template <int BT>
__device__ inline int count_tiles(const Int8Product& p) {
    const int lane = threadIdx.x & 63, T = int(p.T);
    int terms = 0, tiles = 0;
    for (int base = 0; base < p.experts; base += 64) {
        const int n = expert_terms(p, base + lane);
        const int upto = wave_scan(n), begin = min(terms + upto - n, T), end = min(terms + upto, T);
        tiles += __builtin_amdgcn_readlane(wave_scan((end - begin + BT - 1) / BT), 63);
        terms = min(terms + __builtin_amdgcn_readlane(upto, 63), T);
    }
    return tiles;
}

// Row of X of a term, or -1 where it lies outside.
__device__ inline int64_t term_row(const Int8Product& p, int64_t term) {
    if (!p.rows) return term;
    const int64_t r = p.rows64 ? static_cast<const int64_t*>(p.rows)[term] : int64_t(static_cast<const int32_t*>(p.rows)[term]);
    return r >= 0 && r < p.x_rows ? r : -1;
}

// What an exact sum stands for: rounded to float32, then by the scales.
__device__ inline float int8_value(int sum, float sx, float sw) { return float(sum) * sx * sw; }

// Products of many rows (int8_gemm.hip): which kernel one takes, and over how
// many workgroups K is split.
struct Int8Plan {
    bool big;          // int8_gemm_big_kernel, or int8_gemm_kernel
    int fa, fb;        // outputs and terms of a tile, in units of 32
    uint32_t splits;
    int64_t tiles_o, tiles_t;
    size_t workspace;  // the parts of a split
};

// near: row * ld of every row of X fits 32 bits, or its rows are the terms in
// order.  SKETCH_EINVAL when there are more tiles than a grid holds.
sketch_status int8_gemm_plan(int64_t M, int64_t T, uint32_t kb, int experts, bool group, bool near, Int8Plan* g);
sketch_status launch_int8_gemm(const Int8Product& p, const Int8Plan& g, void* ws, hipStream_t st);

sketch_status int8_shape(const sketch_int8_params* p, sketch_int8_shape* s);

}  // namespace sketch
