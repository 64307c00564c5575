// int8_gemm.hip -- the 8-bit integer product Y = X8 * W8^T for many rows, of one
// weight or of a stack with the rows grouped by expert.
//
// Both operands are staged in LDS one block of 128 columns at a time, straight
// from memory (no registers in between), 128 bytes to a row, the row's eight
// 16-byte pieces in the order piece ^ (row % 8), which lets the 16 rows of a
// fragment be read without bank conflicts.  A fragment is 16 rows x 128
// columns: lane l holds row l % 16 and the columns 16c..16c+15 and
// 64+16c..64+16c+15, c = l / 16, the same ones in both operands.
#include <math.h>

#include <type_traits>

#include "int8.h"

namespace sketch {
namespace {

struct GemmArgs {
    Int8Product p;
    uint32_t tiles_o, tiles_t;
    uint32_t splits;   // of K, over blockIdx.y (int8_gemm_kernel)
    int* parts;        // [splits][T][M] when splits > 1
};

// The same with an address of its own for each lane.
__device__ inline void dma16_at(const int8_t* at, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(at), "s"(lds) : "memory", "m0");
}

// Until at most N loads are on their way, the latest ones.
template <int N>
__device__ inline void wait_until() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// Tile of a workgroup: its first output and its terms; false where it has none.
// Tiles of experts differ in their number of terms, so each XCD gets a run of outputs, and all
// terms for them: runs of terms would give the XCDs uneven work (64 experts of 2048 x
// 1408, 3000 terms 55 -> 50 us, 8 of 22016 x 4096, 1600 terms 232 -> 216 us).
template <int ROWS, int BT, bool GROUP>
__device__ inline bool my_tile(const GemmArgs& a, int64_t& o0, Terms& t) {
    uint32_t to = 0, tt;
    if constexpr (GROUP) {
        const bool any = find_terms<BT>(a.p, [&](int tiles) {
            const uint32_t n = uint32_t(tiles) * a.tiles_o;
            if (blockIdx.x >= n) return -1;
            spread_tile<4>(blockIdx.x, uint32_t(tiles), a.tiles_o, n, tt, to);   // 4 tiles of outputs at a time
            return int(tt);
        }, t);
        o0 = int64_t(to) * ROWS;
        return any;
    }
    spread_tile<8>(blockIdx.x, a.tiles_o, a.tiles_t, gridDim.x, to, tt);
    o0 = int64_t(to) * ROWS;
    t.expert = 0;
    t.first = int(tt) * BT;
    t.n = int(min(int64_t(BT), a.p.T - t.first));
    return true;
}

// The scales of a tile: thread i loads that of output i, or of term i - ROWS, well
// before the sums are there; they meet in LDS behind the waves' parts.  (Asked for where they are
// used they cost a wait of two loads a tile: 28672 x 8192 at 2048 rows 374 -> 364 us.)
template <int ROWS, int BT, bool GROUP>
__device__ inline float tile_scale(const Int8Product& p, const Terms& t, int64_t o0) {
    const int i = threadIdx.x;
    if (i < ROWS) {
        const char* w = reinterpret_cast<const char*>(p.w) + size_t(t.expert) * p.w_bytes;
        return reinterpret_cast<const float*>(w + p.w_scales)[min(o0 + i, p.M - 1)];
    }
    const int64_t term = t.first + min(i - ROWS, t.n - 1), row = GROUP ? term_row(p, term) : term;
    return row < 0 ? __builtin_nanf("") : p.xs[row];
}

__device__ inline f32x4 values(i32x4 sum, float sx, f32x4 sw) {
    return f32x4{int8_value(sum[0], sx, sw[0]), int8_value(sum[1], sx, sw[1]), int8_value(sum[2], sx, sw[2]),
                 int8_value(sum[3], sx, sw[3])};
}

// The scaled sums of a wave's tile to Y: 16 FA outputs from o0 + wm on, strips of
// 16 terms, SPREAD apart, from wt on.  They go through the wave's own part of
// LDS (`mine`, JC strips at a time), so that a row's outputs leave in pieces of
// 16 bytes side by side, whatever M leaves of their alignment (8 experts of 15486 x
// 523, 3784 terms: 143 us with stores from registers; 24825 x 133 at 1101 rows, M odd:
// 40 us with stores by element, so 22).
template <int YD, int FA> constexpr uint32_t out_pitch() { return FA * 16 * (YD == SKETCH_F32 ? 4 : 2) + 16; }
template <int YD, int FA, int JC> constexpr uint32_t out_bytes() { return JC * 16 * out_pitch<YD, FA>(); }

template <int YD, int FA, int FB, int SPREAD, int JC>
__device__ inline void store_tile(const Int8Product& p, const Terms& t, const i32x4 (&acc)[FA][FB], int64_t o0, int wm,
                                  int wt, const float* scales, int rows, unsigned char* mine) {
    constexpr int es = YD == SKETCH_F32 ? 4 : 2;
    constexpr uint32_t pitch = out_pitch<YD, FA>();
    const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
    f32x4 so[FA];
#pragma unroll
    for (int i = 0; i < FA; ++i) so[i] = *reinterpret_cast<const f32x4*>(scales + wm + i * 16 + 4 * c);
    float sx[FB];
#pragma unroll
    for (int j = 0; j < FB; ++j) sx[j] = scales[rows + j * SPREAD + wt + r];
    const int left = int(min(p.M - o0 - wm, int64_t(FA * 16)));   // outputs that there are
    if (left <= 0) return;
    unsigned char* Y = static_cast<unsigned char*>(p.Y) + (int64_t(t.first) * p.M + o0 + wm) * es;
    // 16 bytes at a time, aligned to an element; by element where the row ends among them
    typedef uint32_t loose __attribute__((ext_vector_type(4), aligned(2)));
    typedef typename std::conditional<YD == SKETCH_F32, float, uint16_t>::type element;
    constexpr int per = FA * es, kIn = 16 / es;
    auto rows_out = [&](int j0) {
#pragma unroll 4
        for (int q = lane; q < JC * 16 * per; q += 64) {
            const int row = q / per, at = q % per * kIn, n = (j0 + row / 16) * SPREAD + wt + row % 16;
            if (n >= t.n || at >= left) continue;
            const element* from = reinterpret_cast<const element*>(mine + row * pitch) + at;
            element* to = reinterpret_cast<element*>(Y) + int64_t(n) * p.M + at;
            if (at + kIn <= left) {
                *reinterpret_cast<loose*>(to) = *reinterpret_cast<const u32x4*>(from);
            } else {
                for (int e = 0; at + e < left; ++e) to[e] = from[e];
            }
        }
    };
#pragma unroll
    for (int j0 = 0; j0 < FB; j0 += JC) {
        if (j0 * SPREAD + wt >= t.n) break;
#pragma unroll
        for (int j = j0; j < j0 + JC; ++j)
#pragma unroll
            for (int i = 0; i < FA; ++i) {
                const f32x4 v = values(acc[i][j], sx[j], so[i]);
                unsigned char* at = mine + ((j - j0) * 16 + r) * pitch + (i * 16 + 4 * c) * es;
                if constexpr (YD == SKETCH_F32)
                    *reinterpret_cast<f32x4*>(at) = v;
                else
                    *reinterpret_cast<uint2*>(at) = make_uint2(pack2<YD>(v[0], v[1]), pack2<YD>(v[2], v[3]));
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        rows_out(j0);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// ---------------------------------------------------------------------------
// 32 FA outputs x 256 terms (FA 8, or 7 where that fills the last round).  8 waves,
// two to a SIMD, each 16 FA x 64 by 16x16x64 MFMAs: 4 FA accumulators.  The waves work in two
// groups, one on each SIMD, half a step apart: while one group runs the MFMAs of its
// step from registers, the other reads its fragments from LDS, so the matrix
// cores always have one wave's work and LDS the other's.  Group g has the outputs
// 16 FA g .. of the tile.  In phase 2k group 0 reads step k, in phase 2k + 1 group
// 1 does; each multiplies in the phase after.
//
// A wave's terms are strips of 16, 64 apart, so that a tile of few terms leaves out whole
// strips, with their MFMAs and loads, and takes that much less (8 experts of 22016 x
// 4096, 600 terms: 198 -> 178 us).
//
// Loads go out between the MFMAs.  What a load overwrites has to have been
// read: group 0 loads its rows of W of step k + 2 in phase 2k + 1; group 1 its
// own and X, which both read, in phase 2k + 2.  The loads of steps past the
// last repeat it, into buffers that are done with, so that every phase has the
// same number of loads to count.
//
// 28672 x 8192 at 2048 rows: 370 us (350 to 395 from run to run), 2.6 POPS (the library's int8
// product: 530 us).  Bound by the card's power: the matrix cores are busy 72% of the cycles, at
// 1.8 of 2.4 GHz.
// 32x32x32 MFMAs, with half the instructions, took 3% to 24% longer.
// ---------------------------------------------------------------------------
constexpr uint32_t kBigStage = 512 * 128;   // 32 FA rows of W in the first half, 256 of X in the second
constexpr uint32_t kBigLds = 2 * kBigStage;

template <int YD, int FA, bool GROUP>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void int8_gemm_big_kernel(GemmArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const Int8Product& p = a.p;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4, group = wave >> 2, w4 = wave & 3, wm = group * FA * 16, wt = w4 * 16;
    constexpr int kRows = 32 * FA;
    constexpr int kTurns = (2 * FA + 3) / 4;   // loads of 8 rows that a wave has of its group's 16 FA rows of W
    int64_t o0;
    Terms t;
    if (!my_tile<kRows, 256, GROUP>(a, o0, t)) return;

    const uint8_t* wbase = reinterpret_cast<const uint8_t*>(p.w) + size_t(t.expert) * p.w_bytes + o0 * p.ld;
    const bool gather = GROUP && p.rows;
    const uint8_t* xbase = reinterpret_cast<const uint8_t*>(p.x) + (gather ? 0 : int64_t(t.first) * p.ld);
    const uint32_t wlast = uint32_t(min(int64_t(kRows - 1), p.M - 1 - o0));
    const uint32_t piece = uint32_t((lane & 7) ^ (lane >> 3)) * 16, ld = uint32_t(p.ld);
    uint32_t woff[kTurns], xoff[8];
#pragma unroll
    for (int i = 0; i < kTurns; ++i)   // a turn past the group's rows repeats its last 8
        woff[i] = min(uint32_t(wm + min(i * 4 + w4, 2 * FA - 1) * 8 + (lane >> 3)), wlast) * ld + piece;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t row = uint32_t(min((i * 4 + w4) * 8 + (lane >> 3), t.n - 1));
        if (gather) row = uint32_t(max(term_row(p, t.first + int(row)), int64_t(0)));   // x_rows * ld < 2^32 (the plan)
        xoff[i] = row * ld + piece;
    }
    const float scale = tile_scale<kRows, 512 - kRows, GROUP>(p, t, o0);
    const uint32_t lds0 = lds_address(lds), lx = lds0 + 32768 + w4 * 1024;
    uint32_t lw[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) lw[i] = lds0 + uint32_t(wm / 8 + min(i * 4 + w4, 2 * FA - 1)) * 1024;
    auto load_w = [&](uint32_t k, uint32_t buf, int i) { dma16(wbase + size_t(k) * 128, woff[i], lw[i] + buf * kBigStage); };
    auto load_x = [&](uint32_t k, uint32_t buf, int i) { dma16(xbase + size_t(k) * 128, xoff[i], lx + buf * kBigStage + i * 4096); };

    i32x4 acc[FA][4];
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    const unsigned char* frag = lds + r * 128 + ((c ^ (r & 7)) << 4);
    const unsigned char* frag2 = lds + r * 128 + (((c + 4) ^ (r & 7)) << 4);
    const uint32_t last = p.kb - 1;

    // the products of the first NJ strips of 64 terms
    auto run = [&](auto strips) {
        constexpr int NJ = decltype(strips)::value;
        i32x4 af[FA][2], bf[NJ][2];
        auto read_step = [&](uint32_t k) {
            const uint32_t st = (k & 1) * kBigStage;
            const unsigned char *f1 = frag + st + wm * 128, *f2 = frag2 + st + wm * 128;
            const unsigned char *g1 = frag + st + 32768 + wt * 128, *g2 = frag2 + st + 32768 + wt * 128;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                bf[j][0] = *reinterpret_cast<const i32x4*>(g1 + j * 8192);
                bf[j][1] = *reinterpret_cast<const i32x4*>(g2 + j * 8192);
            }
#pragma unroll
            for (int i = 0; i < FA; ++i) {
                af[i][0] = *reinterpret_cast<const i32x4*>(f1 + i * 2048);
                af[i][1] = *reinterpret_cast<const i32x4*>(f2 + i * 2048);
            }
        };
        // the step's MFMAs, with between(n) among them, n < 2 FA
        auto compute = [&](auto between) {
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int n = 0; n < 2 * FA; ++n) {
                const int i = n >> 1, h = n & 1;
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[i][h], bf[j][h], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                between(n);
                __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_s_setprio(0);
        };
        constexpr int kLoads = 2 * NJ + kTurns;   // of a wave of group 1
#pragma unroll
        for (uint32_t k = 0; k < 2; ++k) {
#pragma unroll
            for (int i = 0; i < kTurns; ++i) load_w(min(k, last), k, i);
            if (group == 1) {
#pragma unroll
                for (int i = 0; i < 2 * NJ; ++i) load_x(min(k, last), k, i);
            }
        }
        if (group == 0)   // step 0 is here
            wait_until<kTurns>();
        else
            wait_until<kLoads>();
        barrier();
        if (group == 0) {
            for (uint32_t k = 0; k < p.kb; ++k) {
                read_step(k);
                wait_lds();
                barrier();
                compute([&](int n) {
                    if (n % 2 == 0 && n / 2 < kTurns) load_w(min(k + 2, last), k & 1, n / 2);
                });
                wait_until<kTurns>();   // step k + 1 is here
                barrier();
            }
            barrier();
        } else {
            barrier();
            for (uint32_t k = 0; k < p.kb; ++k) {
                read_step(k);
                wait_lds();
                wait_loads();   // step k + 1 is here
                barrier();
                compute([&](int n) {
#pragma unroll
                    for (int i = n * kLoads / (2 * FA); i < (n + 1) * kLoads / (2 * FA); ++i) {
                        if (i < 2 * NJ)
                            load_x(min(k + 2, last), k & 1, i);
                        else
                            load_w(min(k + 2, last), k & 1, i - 2 * NJ);
                    }
                });
                barrier();
            }
        }
        wait_loads();
    };
    if (t.n > 192)
        run(std::integral_constant<int, 4>());
    else if (t.n > 128)
        run(std::integral_constant<int, 3>());
    else if (t.n > 64)
        run(std::integral_constant<int, 2>());
    else
        run(std::integral_constant<int, 1>());

    barrier();   // every wave is done reading its fragments
    constexpr int JC = YD == SKETCH_F32 ? 1 : 2;
    constexpr uint32_t parts = 8 * out_bytes<YD, FA, JC>();
    static_assert(parts + 2048 <= kBigLds, "the waves' parts of LDS and the scales");
    float* scales = reinterpret_cast<float*>(lds + parts);
    scales[tid] = scale;
    __syncthreads();
    store_tile<YD, FA, 4, 64, JC>(p, t, acc, o0, wm, wt, scales, kRows, lds + wave * out_bytes<YD, FA, JC>());
}

// ---------------------------------------------------------------------------
// 32 FA outputs x up to 32 FB terms, 4 waves of 16 FA x 16 FB, WGS workgroups to a CU,
// which share its LDS: for fewer terms than the big kernel needs, down to those
// whose time is the way of W from memory.  LDS holds as many steps of both
// operands as fit, all but one of them on their way: no registers are tied up by
// loads in flight, which is what operands straight to registers ran into (16 rows of 28672 x
// 8192: 59 us in int8_rows_kernel, here 45, 5.2 TB/s).  A wave's terms are strips of
// 16, 32 apart, so that a tile of few terms leaves out whole strips, with their loads, and
// has LDS for more steps instead.  Tiles of 32 or 64 outputs x 64 terms with 4 workgroups to a
// CU hide each other's beginnings and ends (two, with more steps each, were slower
// almost everywhere); three steps of 128 x 128, which leave a CU one workgroup, took
// 25% longer than two.
// K is split over blockIdx.y when the tiles alone leave compute units
// idle; the parts are the 32-bit sums, rows padded to 4 outputs, and
// int8_add_kernel adds them.
// ---------------------------------------------------------------------------
constexpr uint32_t mid_lds(int groups) { return 163840 / groups / 1024 * 1024; }   // of one of so many workgroups to a CU

// Steps of 32 NJ rows of X and of 32 FA rows of W that LDS holds: up to 4 of
// both, or one more of W, which comes from further away, where that fits.
template <int FA, int NJ, int WGS> constexpr int mid_steps_x() {
    return (FA + NJ) * 4 * 4096 <= int(mid_lds(WGS)) ? 4 : int(mid_lds(WGS)) / ((FA + NJ) * 4096);
}
template <int FA, int NJ, int WGS> constexpr int mid_steps_w() {
    constexpr int x = mid_steps_x<FA, NJ, WGS>();
    return x < 4 && (x * NJ + (x + 1) * FA) * 4096 <= int(mid_lds(WGS)) ? x + 1 : x;
}

template <int YD, int FA, int FB, int WGS, bool GROUP>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(WGS, WGS))) void int8_gemm_kernel(GemmArgs a) {
    constexpr int kRows = 32 * FA;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const Int8Product& p = a.p;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4, wm = (wave >> 1) * 16 * FA, wt = (wave & 1) * 16;
    int64_t o0;
    Terms t;
    if (!my_tile<kRows, 32 * FB, GROUP>(a, o0, t)) return;
    const uint32_t kend = uint32_t(uint64_t(p.kb) * (blockIdx.y + 1) / a.splits);
    const uint32_t kbeg = uint32_t(uint64_t(p.kb) * blockIdx.y / a.splits);

    const uint8_t* wbase = reinterpret_cast<const uint8_t*>(p.w) + size_t(t.expert) * p.w_bytes + o0 * p.ld;
    const uint32_t wlast = uint32_t(min(int64_t(kRows - 1), p.M - 1 - o0));
    const uint32_t piece = uint32_t((lane & 7) ^ (lane >> 3)) * 16, ld = uint32_t(p.ld);
    uint32_t woff[FA], xoff[FB];
    const int8_t* xat[FB];   // GROUP
#pragma unroll
    for (int i = 0; i < FA; ++i) woff[i] = min(uint32_t((i * 4 + wave) * 8 + (lane >> 3)), wlast) * ld + piece;
    const uint8_t* xbase = reinterpret_cast<const uint8_t*>(p.x) + int64_t(t.first) * p.ld;
#pragma unroll
    for (int i = 0; i < FB; ++i) {
        const int row = min((i * 4 + wave) * 8 + (lane >> 3), t.n - 1);
        if constexpr (GROUP)
            xat[i] = p.x + max(term_row(p, t.first + row), int64_t(0)) * p.ld + piece;
        else
            xoff[i] = uint32_t(row) * ld + piece;
    }
    const float scale = tile_scale<kRows, 256 - kRows, GROUP>(p, t, o0);
    const uint32_t lds0 = lds_address(lds) + wave * 1024;
    const uint32_t frag = r * 128 + ((c ^ (r & 7)) << 4), frag2 = r * 128 + (((c + 4) ^ (r & 7)) << 4);

    i32x4 acc[FA][FB];
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

    auto run = [&](auto strips) {
        constexpr int NJ = decltype(strips)::value, SX = mid_steps_x<FA, NJ, WGS>(), SW = mid_steps_w<FA, NJ, WGS>();
        static_assert(SX >= 2 && SX <= 4 && SW - SX <= 1 && (SW * FA + SX * NJ) * 4096 <= int(mid_lds(WGS)), "rings of steps");
        constexpr uint32_t w_step = FA * 4096, x_step = NJ * 4096, x0 = SW * w_step;
        auto next = [](uint32_t at, uint32_t step, uint32_t steps) { return at + step == steps * step ? 0 : at + step; };
        uint32_t w_to = 0, x_to = 0, w_from = 0, x_from = 0;   // where the next step goes, and the current one lies
        auto load_w = [&](uint32_t k) {
#pragma unroll
            for (int i = 0; i < FA; ++i) dma16(wbase + size_t(k) * 128, woff[i], lds0 + w_to + i * 4096);
            w_to = next(w_to, w_step, SW);
        };
        auto load_x = [&](uint32_t k) {
#pragma unroll
            for (int i = 0; i < NJ; ++i) {
                if constexpr (GROUP)
                    dma16_at(xat[i] + size_t(k) * 128, lds0 + x0 + x_to + i * 4096);
                else
                    dma16(xbase + size_t(k) * 128, xoff[i], lds0 + x0 + x_to + i * 4096);
            }
            x_to = next(x_to, x_step, SX);
        };
        // in the order of the steps, X of one before the W that goes out with it
        if (SW > SX && kbeg < kend) load_w(kbeg);
#pragma unroll
        for (uint32_t n = 0; n < SX - 1; ++n) {
            if (kbeg + n < kend) load_x(kbeg + n);
            if (kbeg + n + (SW - SX) < kend) load_w(kbeg + n + (SW - SX));
        }
        for (uint32_t k = kbeg; k < kend; ++k) {
            // what follows X of this step may stay on its way: W of the step that went out with it, and later steps
            constexpr int kAhead = SW > SX ? FA : 0;
            if (SX > 3 && k + 2 < kend)
                wait_until<2 * (FA + NJ)>();
            else if (SX > 2 && k + 1 + (SW - SX) < kend)
                wait_until<kAhead + FA + NJ>();
            else if (SX == 2 && SW > SX && k + 1 < kend)
                wait_until<kAhead>();
            else
                wait_loads();
            barrier();   // step k is here, and every wave is done with step k - 1
            if (k + SX - 1 < kend) load_x(k + SX - 1);
            if (k + SW - 1 < kend) load_w(k + SW - 1);
            const unsigned char *f = lds + w_from + wm * 128, *g = lds + x0 + x_from + wt * 128;
            w_from = next(w_from, w_step, SW), x_from = next(x_from, x_step, SX);
            i32x4 af[FA][2], bf[NJ][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = h ? frag2 : frag;
#pragma unroll
                for (int j = 0; j < NJ; ++j) bf[j][h] = *reinterpret_cast<const i32x4*>(g + at + j * 4096);
#pragma unroll
                for (int i = 0; i < FA; ++i) af[i][h] = *reinterpret_cast<const i32x4*>(f + at + i * 2048);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < FA; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[i][h], bf[j][h], acc[i][j], 0, 0, 0);
        }
    };
    if (FB == 4 && t.n > 96)
        run(std::integral_constant<int, FB>());
    else if (FB == 4 && t.n > 64)
        run(std::integral_constant<int, FB == 4 ? 3 : 1>());
    else if (t.n > 32)
        run(std::integral_constant<int, 2>());
    else
        run(std::integral_constant<int, 1>());

    if (!GROUP && a.splits > 1) {
        const int64_t ldy = (p.M + 3) / 4 * 4;
        int* part = a.parts + int64_t(blockIdx.y) * p.T * ldy;
#pragma unroll
        for (int j = 0; j < FB; ++j) {
            const int n = j * 32 + wt + r;
            if (n >= t.n) continue;
#pragma unroll
            for (int i = 0; i < FA; ++i) {
                const int64_t m = o0 + wm + i * 16 + 4 * c;
                if (m < p.M) *reinterpret_cast<i32x4*>(part + int64_t(t.first + n) * ldy + m) = acc[i][j];   // the padding too
            }
        }
        return;
    }
    barrier();   // every wave is done reading its fragments
    constexpr uint32_t parts = 4 * out_bytes<YD, FA, FB>();
    static_assert(parts + 1024 <= mid_lds(WGS) && kRows + 32 * FB <= 256, "the waves' parts of LDS and the scales");
    float* scales = reinterpret_cast<float*>(lds + parts);
    scales[tid] = scale;
    __syncthreads();
    store_tile<YD, FA, FB, 32, FB>(p, t, acc, o0, wm, wt, scales, kRows, lds + wave * out_bytes<YD, FA, FB>());
}

// Y from the parts, 4 outputs to a thread.
template <int YD>
__global__ __launch_bounds__(256) void int8_add_kernel(GemmArgs a) {
    const Int8Product& p = a.p;
    const int64_t ldy = (p.M + 3) / 4 * 4, m = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4, t = blockIdx.y;
    if (m >= p.M) return;
    const int* part = a.parts + t * ldy + m;
    i32x4 sum = *reinterpret_cast<const i32x4*>(part);
#pragma unroll 4
    for (uint32_t s = 1; s < a.splits; ++s) sum += *reinterpret_cast<const i32x4*>(part + s * p.T * ldy);
    const float* sw = reinterpret_cast<const float*>(reinterpret_cast<const char*>(p.w) + p.w_scales);
    store4_any<YD>(p.Y, t * p.M + m, values(sum, p.xs[t], *reinterpret_cast<const f32x4*>(sw + m)), m, p.M);
}

// What a product takes in us, by a model of the kernels: a sum of what one tile
// takes by itself (its steps of 128 columns one after another), of the rounds that
// the tiles make over the slots of the compute units, of the work that they add up to
// (tiles times steps, and strips of terms times steps), and of the bytes of W and
// Y in MB; parts cost the launch that adds them and their way to memory and back.  The
// figures are fitted to every kernel and split, timed on two thirds of 2000 products of one weight
// (64 x 64 to 28672 x 16384, 2 to 2100 rows) and of 1800 grouped ones (4 to 128 experts, 1 to
// 24000 terms).  What the model takes is 2.6% and 3.0% slower than the fastest kernel
// on average, at worst 45% and 43%; on the third that the fit has not seen 2.8% (61%) and 2.9%
// (37%).  Tiles of 128 x 128, unsplit or split as is best, in place of the set: 28% and 16%.
// The tiles of 256 terms were fitted to 477 large products of one weight; those of 224 outputs fill
// the last round where those of 256 leave it half empty (28672 x 8192 at 2048 rows: 1024
// tiles are 4 rounds, 896 are 3.5; 355 and 375 us in one run) and save 4% of these on average.
struct TileCost {
    int fa, fb;   // outputs and terms of a tile in units of 32
    double call, step, round_step, round, tile_step, strip_step, strip, parts, part_mb, mb, out_mb;   // one weight
    double g_call, g_step, g_round_step, g_round, g_strip_step, g_out_mb, g_mb;                      // grouped
};
constexpr TileCost kCost[] = {
    {1, 2, 3.22, 0.147, 0.092, 0.0, 0.045, 0.016, 0.218, 2.43, 1.44, 0.0325, 0.0, 4.47, 0.140, 0.084, 0.44, 0.064, 0.247, 0.0366},
    {2, 2, 3.34, 0.161, 0.055, 0.10, 0.065, 0.032, 0.112, 2.49, 1.52, 0.0657, 0.139, 4.45, 0.178, 0.178, 0.06, 0.078, 0.213, 0.0626},
    {2, 4, 3.75, 0.151, 0.211, 0.0, 0.094, 0.036, 0.160, 2.42, 1.45, 0.0417, 0.153, 0, 0, 0, 0, 0, 0, 0},
    {4, 2, 3.80, 0.188, 0.235, 0.0, 0.122, 0.034, 0.215, 2.57, 1.38, 0.0796, 0.178, 4.84, 0.174, 0.180, 0.47, 0.136, 0.279, 0.0831},
    {4, 4, 4.57, 0.182, 0.222, 0.0, 0.181, 0.055, 0.235, 1.98, 1.27, 0.0630, 0.115, 5.69, 0.172, 0.102, 1.02, 0.123, 0.233, 0.0920},
    {7, 8, 9.40, 0.735, 0.853, 3.06, 0.0, 0.097, 0.0, 0.0, 0.0, 0.0311, 0.124, 0, 0, 0, 0, 0, 0, 0},
    {8, 8, 8.66, 0.886, 0.991, 3.39, 0.0, 0.098, 0.0, 0.0, 0.0, 0.0233, 0.127, 6.21, 0.436, 0.492, 2.03, 0.263, 0.328, 0.0666}};
constexpr int64_t kMaxSplits = 16;
constexpr int64_t kFewRows = 32;      // rows up to which int8_rows_kernel was timed on one weight
constexpr double kFewPerExpert = 6;   // and terms per expert on groups

// Tiles of up to bt terms that an expert of `mean` terms has on average, where the
// numbers of terms fall off exponentially, as those of routed tokens about do.
double tiles_per_expert(double mean, int64_t bt) { return (1 - exp(-mean)) / (1 - exp(-double(bt) / mean)); }

struct Best {
    Int8Plan plan{};
    double us = 1e300;
    void consider(const Int8Plan& p, double t) {
        if (t < us) us = t, plan = p;
    }
};

Int8Plan choose_group(int64_t M, int64_t T, double kb, int experts, double out_mb, bool near) {
    const double ncu = double(compute_units()), mean = double(T) / experts;
    const double mb = 128e-6 * double(M) * kb * experts * (1 - exp(-mean));   // of the experts that have terms
    Best best;
    for (const TileCost& c : kCost) {
        const bool big = c.fb == 8;
        if (c.g_call == 0 || (big && !near)) continue;
        const double across = double((M + 32 * c.fa - 1) / (32 * c.fa)) * experts;
        const double tiles = across * tiles_per_expert(mean, 32 * c.fb), strips = across * tiles_per_expert(mean, big ? 64 : 32);
        const double rounds = fmax(tiles / ((big ? 1 : 2) * ncu), 1) - 1;
        best.consider({big ? kInt8Big : kInt8Mid, c.fa, c.fb, 1, 0, 0, 0},
                      c.g_call + c.g_step * kb + rounds * (c.g_round_step * kb + c.g_round) + c.g_strip_step * strips / ncu * kb +
                          c.g_out_mb * out_mb + c.g_mb * mb);
    }
    if (mean <= kFewPerExpert) {
        const double tiles = experts * tiles_per_expert(mean, 16) / ncu, one = double((M + 15) / 16) * tiles,
                     two = double((M + 31) / 32) * tiles;
        best.consider({kInt8Rows1, 0, 0, 1, 0, 0, 0}, 2.25 + 2.44 * ceil(kb / 32) + one * (2.42 * kb / 32 + 0.154) + 3.12 * out_mb);
        best.consider({kInt8Rows2, 0, 0, 1, 0, 0, 0}, 3.45 + 1.51 * ceil(kb / 16) + two * (4.21 * kb / 32 + 0.043) + 1.64 * out_mb);
    }
    return best.plan;
}

Int8Plan choose(int64_t M, int64_t T, uint32_t kb, double out_mb) {
    const int64_t ncu = compute_units();
    const double mb = 128e-6 * double(M) * double(kb);
    Best best;
    for (const TileCost& c : kCost) {
        const bool big = c.fb == 8;
        if (big && T <= 64) continue;
        const int64_t across = (M + 32 * c.fa - 1) / (32 * c.fa), bt = 32 * c.fb, down = (T + bt - 1) / bt, strip = big ? 64 : 32;
        for (int64_t n = 1; n <= kMaxSplits; ++n) {
            if (n > 1 && (big || 2 * n > int64_t(kb) || across * down * n > 4 * ncu || T > 65535)) break;   // T: a grid's second dimension
            const double tiles = double(across * down * n), strips = double(across * ((T + strip - 1) / strip) * n);
            const double steps = ceil(double(kb) / double(n)), rounds = ceil(tiles / double((big ? 1 : 2) * ncu)) - 1;
            double us = c.call + c.step * steps + rounds * (c.round_step * steps + c.round) +
                        (c.tile_step * tiles + c.strip_step * strips) / double(ncu) * steps + c.strip * strips / double(ncu) +
                        c.mb * mb + c.out_mb * out_mb;
            if (n > 1) us += c.parts + c.part_mb * 1e-6 * double(n) * double(T) * double(M);
            best.consider({big ? kInt8Big : kInt8Mid, c.fa, c.fb, uint32_t(n), 0, 0, 0}, us);
        }
    }
    if (T <= kFewRows) {
        const double w = double((M + 15) / 16 * ((T + 15) / 16)) / double(ncu), x = fmax(0, w - 1), k = kb / 32.0,
                     t = double(T < 16 ? T : 16) / 16;
        best.consider({kInt8Rows1, 0, 0, 1, 0, 0, 0},
                      2.87 + k * (2.36 + 1.45 * t) + x * (k * (2.59 + 1.17 * t) + 0.333) + (mb > 60 ? 0.0077 * mb : 0));
    }
    return best.plan;
}

template <int YD, bool GROUP>
sketch_status launch(const GemmArgs& a, const Int8Plan& g, hipStream_t st) {
    const int64_t tiles = g.tiles_o * g.tiles_t;
    if (g.kind == kInt8Big) {
        auto go = [&](auto kernel) { kernel<<<unsigned(tiles), 512, kBigLds, st>>>(a); };
        if (g.fa == 8)
            go(int8_gemm_big_kernel<YD, 8, GROUP>);
        else if constexpr (!GROUP)
            go(int8_gemm_big_kernel<YD, 7, false>);
        return launch_status();
    }
    const dim3 grid(unsigned(tiles), g.splits);
    auto go = [&](auto kernel, int slots) { kernel<<<grid, 256, mid_lds(slots), st>>>(a); };
    if (g.fa == 1)
        go(int8_gemm_kernel<YD, 1, 2, 4, GROUP>, 4);
    else if (g.fa == 2 && g.fb == 2)
        go(int8_gemm_kernel<YD, 2, 2, 4, GROUP>, 4);
    else if (g.fb == 2)
        go(int8_gemm_kernel<YD, 4, 2, 2, GROUP>, 2);
    else if (g.fa == 4)
        go(int8_gemm_kernel<YD, 4, 4, 2, GROUP>, 2);
    else if constexpr (!GROUP)
        go(int8_gemm_kernel<YD, 2, 4, 2, false>, 2);
    if (g.splits == 1) return launch_status();
    if (hipGetLastError() != hipSuccess) return SKETCH_EDEVICE;
    int8_add_kernel<YD><<<dim3(unsigned((a.p.M + 1023) / 1024), unsigned(a.p.T)), 256, 0, st>>>(a);
    return launch_status();
}

}  // namespace

sketch_status int8_plan(int64_t M, int64_t T, uint32_t kb, int ydt, int experts, bool group, bool near, Int8Plan* g) {
    const double out_mb = 1e-6 * double(T) * double(M) * double(elem_bytes(ydt));
    *g = group ? choose_group(M, T, kb, experts, out_mb, near) : choose(M, T, kb, out_mb);
    if (g->kind == kInt8Rows1 || g->kind == kInt8Rows2) return SKETCH_OK;   // their launch counts its own workgroups
    const int64_t rows = 32 * g->fa, cols = 32 * g->fb;
    g->tiles_o = (M + rows - 1) / rows;
    g->tiles_t = (T + cols - 1) / cols + (group ? min(T, int64_t(experts)) : 0);
    g->workspace = g->splits > 1 ? align256(size_t(g->splits) * size_t((M + 3) / 4 * 4) * size_t(T) * 4) : 0;
    return g->tiles_o * g->tiles_t > kMaxThreads / (g->kind == kInt8Big ? 512 : 256) ? SKETCH_EINVAL : SKETCH_OK;
}

sketch_status launch_int8_gemm(const Int8Product& p, const Int8Plan& g, void* ws, hipStream_t st) {
    const GemmArgs a{p, uint32_t(g.tiles_o), uint32_t(g.tiles_t), g.splits, static_cast<int*>(ws)};
    if (p.counts) {
        if (p.ydt == SKETCH_F32) return launch<SKETCH_F32, true>(a, g, st);
        return p.ydt == SKETCH_BF16 ? launch<SKETCH_BF16, true>(a, g, st) : launch<SKETCH_F16, true>(a, g, st);
    }
    if (p.ydt == SKETCH_F32) return launch<SKETCH_F32, false>(a, g, st);
    return p.ydt == SKETCH_BF16 ? launch<SKETCH_BF16, false>(a, g, st) : launch<SKETCH_F16, false>(a, g, st);
}

}  // namespace sketch
