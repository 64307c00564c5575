// fp8_gemm.hip -- the e4m3 product Y = X8 * W8^T for many rows.
//
// Both operands are staged in LDS one block of 128 columns at a time, straight
// from memory (no registers in between), 128 bytes to a row, the row's eight
// 16-byte pieces in the order piece ^ (row % 8), which lets the 16 rows of a
// fragment be read without bank conflicts.  A fragment is 16 rows x 128
// columns: lane l holds row l % 16 and the columns 16c..16c+15 and
// 64+16c..64+16c+15, c = l / 16, the same ones in both operands.
#include "tile.h"

namespace sketch {
namespace {

struct GemmArgs {
    Fp8Product p;
    uint32_t tiles_o, tiles_t;
    uint32_t splits;   // of K, over blockIdx.y (fp8_gemm_kernel)
    float* parts;      // [splits][T][M] when splits > 1
};

// Tile of a workgroup.
__device__ inline void tile_of(const GemmArgs& a, uint32_t& to, uint32_t& tt) {
    spread_tile<8>(blockIdx.x, a.tiles_o, a.tiles_t, gridDim.x, to, tt);
}

// ---------------------------------------------------------------------------
// 32 FA outputs x 256 tokens.  8 waves, two to a SIMD, each 16 FA x 64: 4 FA
// accumulators of 16x16.  FA is 8, or 7 or 6 where that many more tiles fill
// their last round over the compute units better (28672 outputs x 2048 tokens:
// 896 tiles are 3.5 rounds, 1024 are 4).  The e4m3 matrix cores take the codes, or,
// for float32 sums (EXACT, FA 4 or 3), both fragments are widened
// to bfloat16 with their scales applied, a quarter of a block at a time, between
// the MFMAs (28672 x 8192 at 2048 tokens: 758 us, 803 us without the two groups).
//
// The waves work in two groups, one on each SIMD, half a step apart: while one
// group runs the MFMAs of its step from registers, the other reads its
// fragments from LDS, so the matrix cores always have one wave's work and LDS
// the other's.  Group g has the outputs 16 FA g .. of the tile.  In phase 2k
// group 0 reads step k, in phase 2k + 1 group 1 does; each multiplies in the
// phase after.
//
// Loads go out between the MFMAs, not before them: 64 of them at the start of
// a phase held up the phase's MFMAs by as long as these take (443 -> 359 us
// for 28672 x 8192 at 2048 tokens).  What a load overwrites has to have been
// read: group 0 loads its rows of W of step k + 2 in phase 2k + 1; group 1 its
// own and X, which both read, in phase 2k + 2.  The loads of steps past the
// last repeat it, into buffers that are done with, so that every phase has the
// same number of loads to count.
// ---------------------------------------------------------------------------
constexpr uint32_t kBigStage = 512 * 128;           // 32 FA rows of W in the first half, 256 of X in the second
constexpr uint32_t kBigScales = (256 + 16) * 4;     // dwords of 4 steps: one per token, one per 16 outputs
constexpr uint32_t kBigLds = 2 * kBigStage + 2 * kBigScales;

template <int YD, int FA, bool EXACT>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void fp8_gemm_big_kernel(GemmArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const Fp8Product& p = a.p;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4, group = wave >> 2, w4 = wave & 3, wm = group * FA * 16, wt = w4 * 64;
    uint32_t to, tt;
    tile_of(a, to, tt);
    constexpr int kRows = 32 * FA;
    constexpr int kTurns = (2 * FA + 3) / 4;   // loads of 8 rows that a wave has of its group's 16 FA rows of W
    const int64_t o0 = int64_t(to) * kRows, t0 = int64_t(tt) * 256;

    const uint8_t *wbase = p.w + o0 * p.ld, *xbase = p.x + t0 * p.ld;
    const uint32_t wlast = uint32_t(min(int64_t(kRows - 1), p.M - 1 - o0)), xlast = uint32_t(min(int64_t(255), p.T - 1 - t0));
    const uint32_t piece = uint32_t((lane & 7) ^ (lane >> 3)) * 16, ld = uint32_t(p.ld);
    uint32_t woff[kTurns], xoff[8];
#pragma unroll
    for (int i = 0; i < kTurns; ++i)   // a turn past the group's rows repeats its last 8
        woff[i] = min(uint32_t(wm + min(i * 4 + w4, 2 * FA - 1) * 8 + (lane >> 3)), wlast) * ld + piece;
#pragma unroll
    for (int i = 0; i < 8; ++i) xoff[i] = min(uint32_t((i * 4 + w4) * 8 + (lane >> 3)), xlast) * ld + piece;
    // scales, by group 1: each wave 64 tokens', and all of them the outputs' (16 outputs lie in one block of 128)
    const uint8_t *xsbase = p.xs + t0 * p.lds;
    const uint32_t xsoff = min(uint32_t(w4 * 64 + lane), xlast) * uint32_t(p.lds);
    const uint32_t wsoff = uint32_t(min(o0 + min(lane, 2 * FA - 1) * 16, p.M - 1) / 128) * uint32_t(p.lds);
    const uint32_t lds0 = lds_address(lds), lx = lds0 + 32768 + w4 * 1024, lsc = lds0 + 2 * kBigStage;
    uint32_t lw[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) lw[i] = lds0 + uint32_t(wm / 8 + min(i * 4 + w4, 2 * FA - 1)) * 1024;

    auto load_w = [&](uint32_t k, uint32_t buf, int i) { dma16(wbase + size_t(k) * 128, woff[i], lw[i] + buf * kBigStage); };
    auto load_x = [&](uint32_t k, uint32_t buf, int i) { dma16(xbase + size_t(k) * 128, xoff[i], lx + buf * kBigStage + i * 4096); };
    auto load_scales = [&](uint32_t k) {   // of steps k .. k + 3
        const uint32_t to_lds = lsc + ((k >> 2) & 1) * kBigScales;
        dma4(xsbase + k, xsoff, to_lds + w4 * 256);
        if (lane < 16) dma4(p.ws + k, wsoff, to_lds + 1024);
    };

    f32x4 acc[FA][4];
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    i32x8 af[FA], bf[4];
    constexpr int kScales = FA == 8 ? 1 : FA;   // 128 outputs lie in one block
    int as[kScales], bs[4];
    const unsigned char* frag = lds + r * 128 + ((c ^ (r & 7)) << 4);
    const unsigned char* frag2 = lds + r * 128 + (((c + 4) ^ (r & 7)) << 4);

    auto read_step = [&](uint32_t k) {
        const uint32_t st = (k & 1) * kBigStage;
        const unsigned char *f1 = frag + st + wm * 128, *f2 = frag2 + st + wm * 128;
        const unsigned char *g1 = frag + st + 32768 + wt * 128, *g2 = frag2 + st + 32768 + wt * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            bf[j] = __builtin_shufflevector(*reinterpret_cast<const i32x4*>(g1 + j * 2048),
                                            *reinterpret_cast<const i32x4*>(g2 + j * 2048), 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int i = 0; i < FA; ++i)
            af[i] = __builtin_shufflevector(*reinterpret_cast<const i32x4*>(f1 + i * 2048),
                                            *reinterpret_cast<const i32x4*>(f2 + i * 2048), 0, 1, 2, 3, 4, 5, 6, 7);
        if ((k & 3) == 0) {
            const int* sc = reinterpret_cast<const int*>(lds + 2 * kBigStage + ((k >> 2) & 1) * kBigScales);
#pragma unroll
            for (int j = 0; j < 4; ++j) bs[j] = sc[wt + j * 16 + r];
#pragma unroll
            for (int i = 0; i < kScales; ++i) as[i] = sc[256 + wm / 16 + i];
        } else {   // the next byte to the low end
#pragma unroll
            for (int j = 0; j < 4; ++j) bs[j] = int(uint32_t(bs[j]) >> 8);
#pragma unroll
            for (int i = 0; i < kScales; ++i) as[i] = int(uint32_t(as[i]) >> 8);
        }
    };
    // the step's MFMAs, with between(n) among them, n < kBetween
    constexpr int kBetween = EXACT ? 4 * FA : 2 * FA;
    auto compute = [&](auto between) {
        __builtin_amdgcn_s_setprio(1);
        if constexpr (EXACT) {
            // quarters of the block; what the next 4 MFMAs need is widened before the 4 that
            // run meanwhile
            float asf[kScales], bsf[4];
#pragma unroll
            for (int i = 0; i < kScales; ++i) asf[i] = fp8_scale(uint32_t(as[i]) & 255u);
#pragma unroll
            for (int j = 0; j < 4; ++j) bsf[j] = fp8_scale(uint32_t(bs[j]) & 255u);
            bf16x8 aw[2], bw[2][4];
            auto widen_a = [&](int n) {   // n = q FA + i
                const int i = n % FA, q = n / FA;
                aw[n & 1] = fp8_widen(af[i][2 * q], af[i][2 * q + 1], asf[i % kScales]);
            };
            auto widen_b = [&](int q, int j) { bw[q & 1][j] = fp8_widen(bf[j][2 * q], bf[j][2 * q + 1], bsf[j]); };
            widen_a(0);
#pragma unroll
            for (int j = 0; j < 4; ++j) widen_b(0, j);
#pragma unroll
            for (int n = 0; n < 4 * FA; ++n) {
                const int i = n % FA, q = n / FA;
                if (n + 1 < 4 * FA) widen_a(n + 1);
                if (q < 3) {
#pragma unroll
                    for (int j = i * 4 / FA; j < (i + 1) * 4 / FA; ++j) widen_b(q + 1, j);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(aw[n & 1], bw[q & 1][j], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                between(n);
                __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_s_setprio(0);
            return;
        }
#pragma unroll
        for (int n = 0; n < 2 * FA; ++n) {
            const int i = n >> 1, j = 2 * (n & 1);
#pragma unroll
            for (int q = j; q < j + 2; ++q)
                acc[i][q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af[i], bf[q], acc[i][q], 0, 0, 0,
                                                                              as[i % kScales], 0, bs[q]);
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
            if (k == 0) load_scales(0);
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
            if (((k + 2) & 3) == 0 && k + 2 < p.kb) load_scales(k + 2);
            compute([&](int n) {
#pragma unroll
                for (int i = n * kLoads / kBetween; i < (n + 1) * kLoads / kBetween; ++i) {
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

    // Whole tiles go out through LDS, 256 contiguous bytes of a token's row and
    // more at a time; the others element by element where they have to.
    if (YD != SKETCH_F32 && o0 + kRows <= p.M && t0 + 256 <= p.T && p.M % 8 == 0) {
        constexpr uint32_t kRow = FA * 32;   // bytes of a token's outputs in the wave's tile
        unsigned char* mine = lds + wave * (64 * kRow);
        barrier();   // every wave is done reading its fragments
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < FA; ++i)
                *reinterpret_cast<uint2*>(mine + (j * 16 + r) * kRow + i * 32 + c * 8) =
                    make_uint2(pack2<YD>(acc[i][j][0], acc[i][j][1]), pack2<YD>(acc[i][j][2], acc[i][j][3]));
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        uint16_t* Y = static_cast<uint16_t*>(p.Y) + (t0 + wt) * p.M + o0 + wm;
#pragma unroll
        for (uint32_t n = 0; n < 64 * kRow / 1024; ++n) {
            const uint32_t at = n * 1024 + lane * 16, t = at / kRow, m = at % kRow;
            *reinterpret_cast<u32x4*>(Y + int64_t(t) * p.M + m / 2) = *reinterpret_cast<const u32x4*>(mine + at);
        }
        return;
    }
    const bool vec = p.M % 4 == 0;
    for (int j = 0; j < 4; ++j) {
        const int64_t t = t0 + wt + j * 16 + r;
        if (t >= p.T) continue;
#pragma unroll
        for (int i = 0; i < FA; ++i) {
            const int64_t m = o0 + wm + i * 16 + 4 * c;
            f32x4 v = acc[i][0];
#pragma unroll
            for (int q = 1; q < 4; ++q)
                if (j == q) v = acc[i][q];
            store4<YD>(p.Y, t * p.M + m, v, m, p.M, vec);
        }
    }
}

// ---------------------------------------------------------------------------
// 32 FA outputs x 32 FB tokens (128 or 96 x 128 or 64), 4 waves of 16 FA x 16 FB,
// two workgroups to a CU: for fewer tiles than the big kernel needs.  EXACT is as
// above.  The loads of the next step go out first: between the MFMAs, as above,
// they came too late for a step this short (4096 x 4096 at 2048 tokens 49 -> 53
// us).  Loads two steps ahead, and widening between the MFMAs, changed nothing.
// K is split over blockIdx.y when the tiles alone leave compute units idle; the parts are float32, rows padded to 4
// outputs, and fp8_add_kernel adds them in their order.
// ---------------------------------------------------------------------------
template <int FA, int FB> constexpr uint32_t mid_stage() { return (32 * FA + 32 * FB) * 128; }
constexpr uint32_t kMidScales = (128 + 64) * 4;   // dwords of 4 steps: one per token, one per 16 outputs
template <int FA, int FB> constexpr uint32_t mid_lds() { return 2 * mid_stage<FA, FB>() + 2 * kMidScales; }

template <int YD, bool EXACT, int FA, int FB>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void fp8_gemm_kernel(GemmArgs a) {
    static_assert(FA <= 4 && FB <= 4, "a wave loads FA times 8 rows of W and FB times 8 of X");
    constexpr int kRows = 32 * FA;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const Fp8Product& p = a.p;
    constexpr uint32_t stage = mid_stage<FA, FB>();
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4, wm = (wave >> 1) * 16 * FA, wt = (wave & 1) * 16 * FB;
    uint32_t to, tt;
    tile_of(a, to, tt);
    const int64_t o0 = int64_t(to) * kRows, t0 = int64_t(tt) * (32 * FB);
    const uint32_t kend = uint32_t(uint64_t(p.kb) * (blockIdx.y + 1) / a.splits);
    const uint32_t kbeg = uint32_t(uint64_t(p.kb) * blockIdx.y / a.splits);

    // loads of this wave: 8 FA rows of W and 8 FB of X per step; waves 0 and 1 the
    // tokens' scales, wave 2 the outputs' (16 outputs lie in one block of 128)
    const uint8_t *wbase = p.w + o0 * p.ld, *xbase = p.x + t0 * p.ld;
    const uint32_t wlast = uint32_t(min(int64_t(kRows - 1), p.M - 1 - o0)),
                   xlast = uint32_t(min(int64_t(32 * FB - 1), p.T - 1 - t0));
    const uint32_t piece = uint32_t((lane & 7) ^ (lane >> 3)) * 16, ld = uint32_t(p.ld);
    uint32_t woff[FA], xoff[FB];
#pragma unroll
    for (int i = 0; i < FA; ++i) woff[i] = min(uint32_t((i * 4 + wave) * 8 + (lane >> 3)), wlast) * ld + piece;
#pragma unroll
    for (int i = 0; i < FB; ++i) xoff[i] = min(uint32_t((i * 4 + wave) * 8 + (lane >> 3)), xlast) * ld + piece;
    const uint8_t* sbase = wave < 2 ? p.xs + t0 * p.lds : p.ws;
    const uint32_t soff = (wave < 2 ? min(uint32_t(wave * 64 + lane), xlast)
                                    : uint32_t(min(o0 + min(lane, 2 * FA - 1) * 16, p.M - 1) / 128)) * uint32_t(p.lds);
    const uint32_t lds0 = lds_address(lds), lw = lds0 + wave * 1024, lx = lw + kRows * 128;
    const uint32_t lsc = lds0 + 2 * stage + wave * 256;
    auto load_part = [&](uint32_t k, int i) {   // i < 4
        const uint32_t st = ((k - kbeg) & 1) * stage;
        if (i < FA) dma16(wbase + size_t(k) * 128, woff[i], lw + st + i * 4096);
        if (i < FB) dma16(xbase + size_t(k) * 128, xoff[i], lx + st + i * 4096);
        if (i == 0 && ((k & 3) == 0 || k == kbeg) && wave < 3)
            dma4(sbase + (k & ~3u), soff, lsc + ((k >> 2) & 1) * kMidScales);
    };

    f32x4 acc[FA][FB];
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
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
        const unsigned char *f1 = frag + st + wm * 128, *f2 = frag2 + st + wm * 128;
        const unsigned char *g1 = frag + st + (kRows + wt) * 128, *g2 = frag2 + st + (kRows + wt) * 128;
        const int* sc = reinterpret_cast<const int*>(lds + 2 * stage + ((k >> 2) & 1) * kMidScales);
        constexpr int kScales = FA == 4 ? 1 : FA;   // 128 outputs lie in one block
        i32x8 af[FA], bf[FB];
        uint32_t as[kScales], bs[FB];
#pragma unroll
        for (int i = 0; i < kScales; ++i) as[i] = uint32_t(sc[128 + wm / 16 + i]) >> (8 * (k & 3)) & 255u;
#pragma unroll
        for (int j = 0; j < FB; ++j) {
            bf[j] = __builtin_shufflevector(*reinterpret_cast<const i32x4*>(g1 + j * 2048),
                                            *reinterpret_cast<const i32x4*>(g2 + j * 2048), 0, 1, 2, 3, 4, 5, 6, 7);
            bs[j] = uint32_t(sc[wt + j * 16 + r]) >> (8 * (k & 3)) & 255u;
        }
#pragma unroll
        for (int i = 0; i < FA; ++i)
            af[i] = __builtin_shufflevector(*reinterpret_cast<const i32x4*>(f1 + i * 2048),
                                            *reinterpret_cast<const i32x4*>(f2 + i * 2048), 0, 1, 2, 3, 4, 5, 6, 7);
        if constexpr (EXACT) {
            bf16x8 bw[FB][4];
#pragma unroll
            for (int j = 0; j < FB; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) bw[j][q] = fp8_widen(bf[j][2 * q], bf[j][2 * q + 1], fp8_scale(bs[j]));
#pragma unroll
            for (int i = 0; i < FA; ++i) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const bf16x8 aw = fp8_widen(af[i][2 * q], af[i][2 * q + 1], fp8_scale(as[i % kScales]));
#pragma unroll
                    for (int j = 0; j < FB; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(aw, bw[j][q], acc[i][j], 0, 0, 0);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < FA; ++i) {
#pragma unroll
                for (int j = 0; j < FB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af[i], bf[j], acc[i][j], 0, 0, 0,
                                                                                  int(as[i % kScales]), 0, int(bs[j]));
            }
        }
    }

    const int64_t ldy = a.splits > 1 ? (p.M + 3) / 4 * 4 : p.M;
    float* part = a.parts + int64_t(blockIdx.y) * p.T * ldy;
    const bool vec = p.M % 4 == 0;
#pragma unroll
    for (int j = 0; j < FB; ++j) {
        const int64_t t = t0 + wt + j * 16 + r;
        if (t >= p.T) continue;
#pragma unroll
        for (int i = 0; i < FA; ++i) {
            const int64_t m = o0 + wm + i * 16 + 4 * c;
            if (a.splits > 1) {
                if (m < p.M) *reinterpret_cast<f32x4*>(part + t * ldy + m) = acc[i][j];   // the padding too
            } else {
                store4<YD>(p.Y, t * p.M + m, acc[i][j], m, p.M, vec);
            }
        }
    }
}

// Y from the parts, 4 outputs to a thread.
template <int YD>
__global__ __launch_bounds__(256) void fp8_add_kernel(GemmArgs a) {
    const int64_t ldy = (a.p.M + 3) / 4 * 4, m = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4, t = blockIdx.y;
    if (m >= a.p.M) return;
    const float* part = a.parts + t * ldy + m;
    f32x4 sum = *reinterpret_cast<const f32x4*>(part);
#pragma unroll 4
    for (uint32_t s = 1; s < a.splits; ++s) sum += *reinterpret_cast<const f32x4*>(part + s * a.p.T * ldy);
    store4<YD>(a.p.Y, t * a.p.M + m, sum, m, a.p.M, a.p.M % 4 == 0);
}

// What a product takes in us, by a model of the kernels: a block of 128 columns
// takes a tile a time of its own, more where two workgroups share a compute
// unit; tiles of the big kernel go in rounds over the units, each as long as two
// blocks more to begin and end, the smaller ones follow one another, half a
// round lost at the end; parts cost the launch that adds them and their way to
// memory and back.  The figures are fitted to every kernel and split timed on
// 512 products (58 x 20935 to 128256 x 2048, 17 to 70000 tokens): what the model
// takes is 1.2% slower than the fastest one on average, at worst 20%; on 163
// others that the fit has not seen 1.7%, at worst 30%.  (Tiles of 256 tokens
// wherever they make 3/4 of a round, and parts by one figure for all kinds of
// tiles, as simpler rules, took 10% more than the fastest on average, and
// 28672 x 8192 in float32 at 17 tokens 112 us, now 59, 128256 x 2048 129 us, now 55.)
struct TileCost {
    int fa, fb;         // outputs and tokens of a tile, in units of 32
    double one, two;    // us per block: a workgroup alone on its compute unit, or one of two
};
constexpr TileCost kCost[2][3] = {   // [exact]
    {{4, 4, 0.83, 1.05}, {3, 4, 0.67, 0.85}, {4, 2, 0.56, 0.77}},
    {{4, 4, 1.07, 1.70}, {3, 4, 0.92, 1.36}, {4, 2, 0.68, 1.04}}};
constexpr TileCost kBigCost[2][3] = {{{8, 8, 1.50, 0}, {7, 8, 1.15, 0}, {6, 8, 1.01, 0}},
                                     {{4, 8, 1.55, 0}, {3, 8, 1.24, 0}, {3, 8, 1.24, 0}}};
constexpr int64_t kMaxSplits = 16, kNarrowTokens = 192;   // most tokens that tiles of 64 were timed with

GemmPlan choose(int64_t M, int64_t T, uint32_t kb, bool exact) {
    const int64_t ncu = compute_units();
    GemmPlan best{};
    double least = 1e300;
    auto consider = [&](const GemmPlan& g, double us) {
        if (us < least) least = us, best = g;
    };
    auto tiles_of = [&](const TileCost& c) { return (M + 32 * c.fa - 1) / (32 * c.fa) * ((T + 32 * c.fb - 1) / (32 * c.fb)); };
    for (const TileCost& c : kBigCost[exact])
        consider({true, c.fa, c.fb, 1, 0, 0, 0}, (exact ? 3.9 : 5.8) + double((tiles_of(c) + ncu - 1) / ncu) * double(kb + 2) * c.one);
    for (const TileCost& c : kCost[exact]) {
        if (c.fb == 2 && T > kNarrowTokens) continue;
        const int64_t tiles = tiles_of(c);
        for (int64_t n = 1; n <= kMaxSplits; ++n) {
            if (n > 1 && (2 * n > int64_t(kb) || tiles * n > 4 * ncu || T > 65535)) break;   // T: a grid's second dimension
            const int64_t w = tiles * n, slots = 2 * ncu;
            const double steps = double(kb) / double(n) + 0.5, rounds = double(w) / double(slots);
            double us = 4.8 + steps * (w <= ncu     ? c.one
                                       : w <= slots ? c.two
                                                    : c.two * 0.5 * (rounds + double((w + slots - 1) / slots)));
            if (n > 1) us += 1.3 + 1.5e-6 * double(n) * double(T) * double(M);
            consider({false, c.fa, c.fb, uint32_t(n), 0, 0, 0}, us);
        }
    }
    return best;
}

void launch_big(const GemmArgs& a, int fa, unsigned grid, hipStream_t st) {
    auto go = [&](auto kernel) { kernel<<<grid, 512, kBigLds, st>>>(a); };
    if (!a.p.exact)
        fa == 8   ? go(fp8_gemm_big_kernel<SKETCH_BF16, 8, false>)
        : fa == 7 ? go(fp8_gemm_big_kernel<SKETCH_BF16, 7, false>)
                  : go(fp8_gemm_big_kernel<SKETCH_BF16, 6, false>);
    else if (a.p.ydt == SKETCH_F32)
        fa == 4 ? go(fp8_gemm_big_kernel<SKETCH_F32, 4, true>) : go(fp8_gemm_big_kernel<SKETCH_F32, 3, true>);
    else if (a.p.ydt == SKETCH_BF16)
        fa == 4 ? go(fp8_gemm_big_kernel<SKETCH_BF16, 4, true>) : go(fp8_gemm_big_kernel<SKETCH_BF16, 3, true>);
    else
        fa == 4 ? go(fp8_gemm_big_kernel<SKETCH_F16, 4, true>) : go(fp8_gemm_big_kernel<SKETCH_F16, 3, true>);
}

}  // namespace

sketch_status fp8_gemm_plan(int64_t M, int64_t T, uint32_t kb, bool exact, GemmPlan* g) {
    *g = choose(M, T, kb, exact);
    const int64_t rows = 32 * g->fa, cols = 32 * g->fb;
    g->tiles_o = (M + rows - 1) / rows;
    g->tiles_t = (T + cols - 1) / cols;
    g->workspace = g->splits > 1 ? align256(size_t(g->splits) * size_t((M + 3) / 4 * 4) * size_t(T) * 4) : 0;
    return g->tiles_o * g->tiles_t > kMaxThreads / (g->big ? 512 : 256) ? SKETCH_EINVAL : SKETCH_OK;
}

sketch_status launch_fp8_gemm(const Fp8Product& p, const GemmPlan& g, void* ws, hipStream_t st) {
    const GemmArgs a{p, uint32_t(g.tiles_o), uint32_t(g.tiles_t), g.splits, static_cast<float*>(ws)};
    const int64_t tiles = g.tiles_o * g.tiles_t;
    if (g.big) {
        launch_big(a, g.fa, unsigned(tiles), st);
        return launch_status();
    }
    auto go = [&](auto four, auto three, auto two, auto add) {
        const dim3 grid(unsigned(tiles), g.splits);
        if (g.fb == 2)
            two<<<grid, 256, mid_lds<4, 2>(), st>>>(a);
        else if (g.fa == 4)
            four<<<grid, 256, mid_lds<4, 4>(), st>>>(a);
        else
            three<<<grid, 256, mid_lds<3, 4>(), st>>>(a);
        if (g.splits == 1) return launch_status();
        if (hipGetLastError() != hipSuccess) return SKETCH_EDEVICE;
        add<<<dim3(unsigned((p.M + 1023) / 1024), unsigned(p.T)), 256, 0, st>>>(a);
        return launch_status();
    };
    if (p.ydt == SKETCH_F32)
        return go(fp8_gemm_kernel<SKETCH_F32, true, 4, 4>, fp8_gemm_kernel<SKETCH_F32, true, 3, 4>,
                  fp8_gemm_kernel<SKETCH_F32, true, 4, 2>, fp8_add_kernel<SKETCH_F32>);
    if (p.ydt == SKETCH_F16)
        return go(fp8_gemm_kernel<SKETCH_F16, true, 4, 4>, fp8_gemm_kernel<SKETCH_F16, true, 3, 4>,
                  fp8_gemm_kernel<SKETCH_F16, true, 4, 2>, fp8_add_kernel<SKETCH_F16>);
    if (p.exact)
        return go(fp8_gemm_kernel<SKETCH_BF16, true, 4, 4>, fp8_gemm_kernel<SKETCH_BF16, true, 3, 4>,
                  fp8_gemm_kernel<SKETCH_BF16, true, 4, 2>, fp8_add_kernel<SKETCH_BF16>);
    return go(fp8_gemm_kernel<SKETCH_BF16, false, 4, 4>, fp8_gemm_kernel<SKETCH_BF16, false, 3, 4>,
              fp8_gemm_kernel<SKETCH_BF16, false, 4, 2>, fp8_add_kernel<SKETCH_BF16>);
}

}  // namespace sketch
