// int8_gemm.hip -- the 8-bit integer product Y = X8 * W8^T for many rows, of one
// weight or of a stack with the rows grouped by expert.
//
// Both operands are staged in LDS one block of 128 columns at a time, straight
// from memory (no registers in between), 128 bytes to a row, the row's eight
// 16-byte pieces in the order piece ^ (row % 8), which lets the 16 rows of a
// fragment be read without bank conflicts.  A fragment is 16 rows x 128
// columns: lane l holds row l % 16 and the columns 16c..16c+15 and
// 64+16c..64+16c+15, c = l / 16, the same ones in both operands.
#include "int8.h"
#include "tile.h"

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

// Tile of a workgroup: its first output and its terms; false where it has none.
template <int ROWS, int BT, bool GROUP>
__device__ inline bool my_tile(const GemmArgs& a, int64_t& o0, Terms& t) {
    uint32_t to, tt, n = gridDim.x, tiles_t = a.tiles_t;
    if constexpr (GROUP) {
        tiles_t = uint32_t(count_tiles<BT>(a.p));
        n = tiles_t * a.tiles_o;
        if (blockIdx.x >= n) return false;
    }
    spread_tile(blockIdx.x, a.tiles_o, tiles_t, n, to, tt);
    o0 = int64_t(to) * ROWS;
    if constexpr (GROUP) return find_terms<BT>(a.p, int(tt), t);
    t.expert = 0;
    t.first = int(tt) * BT;
    t.n = int(min(int64_t(BT), a.p.T - t.first));
    return true;
}

__device__ inline float term_scale(const Int8Product& p, bool group, int64_t term) {
    const int64_t row = group ? term_row(p, term) : term;
    return row < 0 ? __builtin_nanf("") : p.xs[row];
}

__device__ inline f32x4 values(i32x4 sum, float sx, f32x4 sw) {
    return f32x4{int8_value(sum[0], sx, sw[0]), int8_value(sum[1], sx, sw[1]), int8_value(sum[2], sx, sw[2]),
                 int8_value(sum[3], sx, sw[3])};
}

// ---------------------------------------------------------------------------
// 32 FA outputs x 256 terms.  8 waves, two to a SIMD, each 16 FA x 64: 4 FA
// accumulators of 16x16.  The waves work in two groups, one on each SIMD, half
// a step apart: while one group runs the MFMAs of its step from registers, the
// other reads its fragments from LDS.  Group g has the outputs 16 FA g .. of the
// tile.  In phase 2k group 0 reads step k, in phase 2k + 1 group 1 does; each
// multiplies in the phase after.
//
// Loads go out between the MFMAs.  What a load overwrites has to have been
// read: group 0 loads its rows of W of step k + 2 in phase 2k + 1; group 1 its
// own and X, which both read, in phase 2k + 2.  The loads of steps past the
// last repeat it, into buffers that are done with, so that every phase has the
// same number of loads to count.
// ---------------------------------------------------------------------------
constexpr uint32_t kBigStage = 512 * 128;   // 32 FA rows of W in the first half, 256 of X in the second
constexpr uint32_t kBigLds = 2 * kBigStage;

template <int YD, int FA, bool GROUP>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void int8_gemm_big_kernel(GemmArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const Int8Product& p = a.p;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4, group = wave >> 2, w4 = wave & 3, wm = group * FA * 16, wt = w4 * 64;
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
    i32x4 af[FA][2], bf[4][2];
    const unsigned char* frag = lds + r * 128 + ((c ^ (r & 7)) << 4);
    const unsigned char* frag2 = lds + r * 128 + (((c + 4) ^ (r & 7)) << 4);

    auto read_step = [&](uint32_t k) {
        const uint32_t st = (k & 1) * kBigStage;
        const unsigned char *f1 = frag + st + wm * 128, *f2 = frag2 + st + wm * 128;
        const unsigned char *g1 = frag + st + 32768 + wt * 128, *g2 = frag2 + st + 32768 + wt * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bf[j][0] = *reinterpret_cast<const i32x4*>(g1 + j * 2048);
            bf[j][1] = *reinterpret_cast<const i32x4*>(g2 + j * 2048);
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
            for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[i][h], bf[j][h], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            between(n);
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_setprio(0);
    };

    const uint32_t last = p.kb - 1;
    constexpr int kLoads = 8 + kTurns;   // of a wave of group 1
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) load_w(min(k, last), k, i);
        if (group == 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) load_x(min(k, last), k, i);
        }
    }
    wait_loads();
    barrier();
    if (group == 0) {
        for (uint32_t k = 0; k < p.kb; ++k) {
            read_step(k);
            wait_lds();
            barrier();
            compute([&](int n) {
                if (n % 2 == 0 && n / 2 < kTurns) load_w(min(k + 2, last), k & 1, n / 2);
            });
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kTurns) : "memory");   // step k + 1 is here
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
                    if (i < 8)
                        load_x(min(k + 2, last), k & 1, i);
                    else
                        load_w(min(k + 2, last), k & 1, i - 8);
                }
            });
            barrier();
        }
    }
    wait_loads();

    const float* sw = reinterpret_cast<const float*>(reinterpret_cast<const char*>(p.w) + size_t(t.expert) * p.w_bytes + p.w_scales);
    f32x4 so[FA];
    const int64_t m_last = (p.M - 1) & ~int64_t(3);
#pragma unroll
    for (int i = 0; i < FA; ++i) so[i] = *reinterpret_cast<const f32x4*>(sw + min(o0 + wm + i * 16 + 4 * c, m_last));
    float sx[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) sx[j] = term_scale(p, GROUP, t.first + min(wt + j * 16 + r, t.n - 1));
    // 16-bit rows go out through LDS, 256 contiguous bytes of a term's row and
    // more at a time, where their pieces are aligned
    if (YD != SKETCH_F32 && p.M % 8 == 0) {
        constexpr uint32_t kRow = FA * 32;   // bytes of a term's outputs in the wave's tile
        unsigned char* mine = lds + wave * (64 * kRow);
        barrier();   // every wave is done reading its fragments
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < FA; ++i) {
                const f32x4 v = values(acc[i][j], sx[j], so[i]);
                *reinterpret_cast<uint2*>(mine + (j * 16 + r) * kRow + i * 32 + c * 8) =
                    make_uint2(pack2<YD>(v[0], v[1]), pack2<YD>(v[2], v[3]));
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        uint16_t* Y = static_cast<uint16_t*>(p.Y) + int64_t(t.first + wt) * p.M + o0 + wm;
        const int64_t left = p.M - o0 - wm;
#pragma unroll
        for (uint32_t n = 0; n < 64 * kRow / 1024; ++n) {
            const uint32_t at = n * 1024 + lane * 16, row = at / kRow, m = at % kRow / 2;
            if (wt + int(row) < t.n && int64_t(m) < left)
                *reinterpret_cast<u32x4*>(Y + int64_t(row) * p.M + m) = *reinterpret_cast<const u32x4*>(mine + at);
        }
        return;
    }
    const bool vec = p.M % 4 == 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int n = wt + j * 16 + r;
        if (n >= t.n) continue;
#pragma unroll
        for (int i = 0; i < FA; ++i) {
            const int64_t m = o0 + wm + i * 16 + 4 * c;
            store4<YD>(p.Y, int64_t(t.first + n) * p.M + m, values(acc[i][j], sx[j], so[i]), m, p.M, vec);
        }
    }
}

// ---------------------------------------------------------------------------
// 32 FA outputs x 32 FB terms, 4 waves of 16 FA x 16 FB, two workgroups to a CU:
// for fewer tiles than the big kernel needs.  The loads of the next step go out
// first.  K is split over blockIdx.y when the tiles alone leave compute units
// idle; the parts are the 32-bit sums, rows padded to 4 outputs, and
// int8_add_kernel adds them.
// ---------------------------------------------------------------------------
template <int FA, int FB> constexpr uint32_t mid_stage() { return (32 * FA + 32 * FB) * 128; }
template <int FA, int FB> constexpr uint32_t mid_lds() { return 2 * mid_stage<FA, FB>(); }

template <int YD, int FA, int FB, bool GROUP>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void int8_gemm_kernel(GemmArgs a) {
    static_assert(FA <= 4 && FB <= 4, "a wave loads FA times 8 rows of W and FB times 8 of X");
    constexpr int kRows = 32 * FA;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const Int8Product& p = a.p;
    constexpr uint32_t stage = mid_stage<FA, FB>();
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4, wm = (wave >> 1) * 16 * FA, wt = (wave & 1) * 16 * FB;
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
    const uint32_t lds0 = lds_address(lds), lw = lds0 + wave * 1024, lx = lw + kRows * 128;
    auto load_part = [&](uint32_t k, int i) {   // i < 4
        const uint32_t st = ((k - kbeg) & 1) * stage;
        if (i < FA) dma16(wbase + size_t(k) * 128, woff[i], lw + st + i * 4096);
        if (i < FB) {
            if constexpr (GROUP)
                dma16_at(xat[i] + size_t(k) * 128, lx + st + i * 4096);
            else
                dma16(xbase + size_t(k) * 128, xoff[i], lx + st + i * 4096);
        }
    };

    i32x4 acc[FA][FB];
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    const unsigned char* frag = lds + r * 128 + ((c ^ (r & 7)) << 4);
    const unsigned char* frag2 = lds + r * 128 + (((c + 4) ^ (r & 7)) << 4);

    if (kbeg < kend)
#pragma unroll
        for (int i = 0; i < 4; ++i) load_part(kbeg, i);
    for (uint32_t k = kbeg; k < kend; ++k) {
        wait_loads();
        barrier();   // step k is here, and every wave is done with step k - 1
        if (k + 1 < kend)
#pragma unroll
            for (int i = 0; i < 4; ++i) load_part(k + 1, i);
        const uint32_t st = ((k - kbeg) & 1) * stage;
        const unsigned char* f[2] = {frag + st + wm * 128, frag2 + st + wm * 128};
        const unsigned char* g[2] = {frag + st + (kRows + wt) * 128, frag2 + st + (kRows + wt) * 128};
        i32x4 af[FA][2], bf[FB][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < FB; ++j) bf[j][h] = *reinterpret_cast<const i32x4*>(g[h] + j * 2048);
#pragma unroll
            for (int i = 0; i < FA; ++i) af[i][h] = *reinterpret_cast<const i32x4*>(f[h] + i * 2048);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < FA; ++i)
#pragma unroll
                for (int j = 0; j < FB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[i][h], bf[j][h], acc[i][j], 0, 0, 0);
    }

    if (!GROUP && a.splits > 1) {
        const int64_t ldy = (p.M + 3) / 4 * 4;
        int* part = a.parts + int64_t(blockIdx.y) * p.T * ldy;
#pragma unroll
        for (int j = 0; j < FB; ++j) {
            const int n = wt + j * 16 + r;
            if (n >= t.n) continue;
#pragma unroll
            for (int i = 0; i < FA; ++i) {
                const int64_t m = o0 + wm + i * 16 + 4 * c;
                if (m < p.M) *reinterpret_cast<i32x4*>(part + int64_t(t.first + n) * ldy + m) = acc[i][j];   // the padding too
            }
        }
        return;
    }
    const float* sw = reinterpret_cast<const float*>(reinterpret_cast<const char*>(p.w) + size_t(t.expert) * p.w_bytes + p.w_scales);
    const int64_t m_last = (p.M - 1) & ~int64_t(3);
    f32x4 so[FA];
#pragma unroll
    for (int i = 0; i < FA; ++i) so[i] = *reinterpret_cast<const f32x4*>(sw + min(o0 + wm + i * 16 + 4 * c, m_last));
    const bool vec = p.M % 4 == 0;
#pragma unroll
    for (int j = 0; j < FB; ++j) {
        const int n = wt + j * 16 + r;
        if (n >= t.n) continue;
        const float sx = term_scale(p, GROUP, t.first + n);
#pragma unroll
        for (int i = 0; i < FA; ++i) {
            const int64_t m = o0 + wm + i * 16 + 4 * c;
            store4<YD>(p.Y, int64_t(t.first + n) * p.M + m, values(acc[i][j], sx, so[i]), m, p.M, vec);
        }
    }
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
    store4<YD>(p.Y, t * p.M + m, values(sum, p.xs[t], *reinterpret_cast<const f32x4*>(sw + m)), m, p.M, p.M % 4 == 0);
}

template <int YD, bool GROUP>
sketch_status launch(const GemmArgs& a, const Int8Plan& g, hipStream_t st) {
    const int64_t tiles = g.tiles_o * g.tiles_t;
    if (g.big) {
        auto go = [&](auto kernel) { kernel<<<unsigned(tiles), 512, kBigLds, st>>>(a); };
        g.fa == 8   ? go(int8_gemm_big_kernel<YD, 8, GROUP>)
        : g.fa == 7 ? go(int8_gemm_big_kernel<YD, 7, GROUP>)
                    : go(int8_gemm_big_kernel<YD, 6, GROUP>);
        return launch_status();
    }
    const dim3 grid(unsigned(tiles), g.splits);
    if (g.fb == 2)
        int8_gemm_kernel<YD, 4, 2, GROUP><<<grid, 256, mid_lds<4, 2>(), st>>>(a);
    else if (g.fa == 4)
        int8_gemm_kernel<YD, 4, 4, GROUP><<<grid, 256, mid_lds<4, 4>(), st>>>(a);
    else
        int8_gemm_kernel<YD, 3, 4, GROUP><<<grid, 256, mid_lds<3, 4>(), st>>>(a);
    if (g.splits == 1) return launch_status();
    if (hipGetLastError() != hipSuccess) return SKETCH_EDEVICE;
    int8_add_kernel<YD><<<dim3(unsigned((a.p.M + 1023) / 1024), unsigned(a.p.T)), 256, 0, st>>>(a);
    return launch_status();
}

}  // namespace

sketch_status int8_gemm_plan(int64_t M, int64_t T, uint32_t kb, int experts, bool group, bool near, Int8Plan* g) {
    *g = Int8Plan{};
    const int64_t ncu = compute_units();
    g->big = (M + 255) / 256 * ((T + 255) / 256) >= ncu / 2 && near;
    g->fa = g->big ? 8 : 4, g->fb = g->big ? 8 : 4, g->splits = 1;
    const int64_t rows = 32 * g->fa, cols = 32 * g->fb;
    g->tiles_o = (M + rows - 1) / rows;
    g->tiles_t = (T + cols - 1) / cols + (group ? min(T, int64_t(experts)) : 0);
    g->workspace = g->splits > 1 ? align256(size_t(g->splits) * size_t((M + 3) / 4 * 4) * size_t(T) * 4) : 0;
    return g->tiles_o * g->tiles_t > kMaxThreads / (g->big ? 512 : 256) ? SKETCH_EINVAL : SKETCH_OK;
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
