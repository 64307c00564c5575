// tile.h -- what the 8-bit tile kernels share: loads from memory straight into
// LDS, waits and barriers that the compiler does not move, and the stores of 4
// outputs.
#pragma once

#include "fp8.h"

namespace sketch {

// 16 (or 4) bytes per lane from base + off to LDS bytes lds + 16 i (4 i) of
// lane i.  Inline asm, because with the builtin the compiler waits for every
// outstanding load before each LDS read; here the waits that matter are
// written out.  There is no register result; M0 needs a wait state after its
// write.
__device__ inline void dma16(const uint8_t* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
                 : "memory", "m0");
}
__device__ inline void dma4(const uint8_t* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(lds)
                 : "memory", "m0");
}
__device__ inline void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ inline void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ inline void barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

__device__ inline uint32_t lds_address(const void* p) {
    return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)));
}

// Tile `block` of n = tiles_o * tiles_t.  Workgroups go round the 8 XCDs, so
// each XCD gets a contiguous run of tiles; a run goes through groups of G token
// tiles, so that the tiles in flight on an XCD share both operands in its L2.
template <uint32_t G>
__device__ inline void spread_tile(uint32_t block, uint32_t tiles_o, uint32_t tiles_t, uint32_t n, uint32_t& to, uint32_t& tt) {
    const uint32_t q = n / 8, rem = n % 8, xcd = block % 8;
    const uint32_t id = xcd * q + (xcd < rem ? xcd : rem) + block / 8;
    const uint32_t g = id / (G * tiles_o), gt = min(G, tiles_t - g * G), in = id - g * G * tiles_o;
    to = in / gt;
    tt = g * G + in % gt;
}

// Two floats in 16 bits each, ties to even.
template <int YD>
__device__ inline uint32_t pack2(float a, float b) {
    if constexpr (YD == SKETCH_BF16) {
        const bf16x2 h = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
        return __builtin_bit_cast(uint32_t, h);
    } else {
        return uint32_t(f32_to_f16_bits(a)) | (uint32_t(f32_to_f16_bits(b)) << 16);
    }
}

template <int YD>
__device__ inline void store4(void* Y, int64_t e, f32x4 v, int64_t m, int64_t M, bool vec) {
    if (vec && m + 4 <= M) {
        if constexpr (YD == SKETCH_F32) {
            *reinterpret_cast<f32x4*>(static_cast<float*>(Y) + e) = v;
        } else {
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(Y) + e) = make_uint2(pack2<YD>(v[0], v[1]), pack2<YD>(v[2], v[3]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (m + i < M) store1_val<YD>(Y, e + i, v[i]);
    }
}

}  // namespace sketch
