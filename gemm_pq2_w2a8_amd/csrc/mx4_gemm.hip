// mx4_gemm.hip -- the product of two MX4 matrices, and the gated feed-forward
// block on it (gfx950).
//
//   y[m][n] = sum_k a[m][k] w[n][k],          h = act(a Wg^T) * (a Wu^T)
//
// Both operands are 4-bit floats with one power-of-two scale per 32 values
// along k, which is what one lane of the scaled matrix instruction takes: 16
// bytes and a scale byte. Products and scales are exact there, sums float32.
// The gated block takes its gate and up rows as alternating runs of 16 rows, so
// both values of an output meet in the same registers of the same lane: the
// activation, the product, and the next quantisation need no exchange but the
// one among the four lanes of a block of 32.
#include <type_traits>

#include "mx4_device.hpp"
#include "mx4_launch.hpp"
#include "mx4_plan.hpp"

namespace pq2 {
namespace {

// Results of a block of 32 gated columns and one token: h[p][i] is column 16 p
// + 4 (lane / 16) + i. Quantised into the token's codes and scale byte.
__device__ __forceinline__ void store_quantised(const v4f32 (&h)[2], uint8_t *codes, uint8_t *scale,
                                                bool live, int lane) {
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            top = max(top, bits_of(h[p][i]) & 0x7fffffffu);
    top = max(top, (uint32_t)swizzle_xor16((int)top));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    const uint32_t byte = mx_scale_byte(top);
    const float s = mx_scale(byte);
    uint32_t c = 0;
    c = mx_encode2<0>(c, h[0][0], h[0][1], s);
    c = mx_encode2<1>(c, h[0][2], h[0][3], s);
    c = mx_encode2<2>(c, h[1][0], h[1][1], s);
    c = mx_encode2<3>(c, h[1][2], h[1][3], s);
    if (byte == 255u) c = 0;
    if (!live) return;
    const int lg = lane >> 4;
    *reinterpret_cast<uint16_t *>(codes + 2 * lg) = (uint16_t)c;
    *reinterpret_cast<uint16_t *>(codes + 8 + 2 * lg) = (uint16_t)(c >> 16);
    if (lg == 0) *scale = (uint8_t)byte;
}

// Four consecutive columns of one row: `whole` where all of them exist and the
// address is aligned to the four.
__device__ __forceinline__ void store4(void *y, int fmt, int64_t at, v4f32 v, int left, bool whole) {
    if (whole) {
        if (fmt == kF32) {
            *reinterpret_cast<v4f32 *>(static_cast<float *>(y) + at) = v;
        } else {
            const v2u two = {pack16(fmt, v[0], v[1]), pack16(fmt, v[2], v[3])};
            *reinterpret_cast<v2u *>(static_cast<uint16_t *>(y) + at) = two;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < left) store_fmt(y, fmt, at + i, v[i]);
}

// Whether every run of four columns from a multiple of four on is aligned, and of
// eight.
__device__ __forceinline__ bool aligned4(const void *y, int fmt, int64_t n) {
    return (n & 3) == 0 && (reinterpret_cast<uintptr_t>(y) & (fmt == kF32 ? 15 : 7)) == 0;
}
__device__ __forceinline__ bool aligned8(const void *y, int64_t n) {
    return (n & 7) == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
}

// 32 columns of one row from element `at` on, which is a multiple of 16 columns
// into it: a lane's four of the first 16 and of the second. 16-bit rows exchange
// every other 16 lanes' second halves, so that a lane has eight columns in a row
// and the four lanes of a token write 64 contiguous bytes at once (eight bytes a
// lane, 32 contiguous, took the gated batch of 2048 x 17408 with g and u 305 us
// instead of 279). `left`: columns that exist; live: the lane's row does.
__device__ __forceinline__ void store_pair(void *y, int fmt, int64_t at, v4f32 a, v4f32 b, int64_t left,
                                           bool live, int lg, bool four, bool eight) {
    if (fmt != kF32 && eight && left >= 32) {
        const auto lo = __builtin_amdgcn_permlane16_swap(pack16(fmt, a[0], a[1]), pack16(fmt, b[0], b[1]), false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(pack16(fmt, a[2], a[3]), pack16(fmt, b[2], b[3]), false, false);
        const v4u v = {lo[0], hi[0], lo[1], hi[1]};
        if (live) *reinterpret_cast<v4u *>(static_cast<uint16_t *>(y) + at + 16 * (lg & 1) + 8 * (lg >> 1)) = v;
        return;
    }
    if (!live) return;
    const int la = (int)(left - 4 * lg < 4 ? left - 4 * lg : 4);
    if (la > 0) store4(y, fmt, at + 4 * lg, a, la, four && la == 4);
    const int lb = (int)(left - 16 - 4 * lg < 4 ? left - 16 - 4 * lg : 4);
    if (lb > 0) store4(y, fmt, at + 16 + 4 * lg, b, lb, four && lb == 4);
}

// The end of a product: acc[i][j] are four consecutive rows of w (from 4 (lane /
// 16) on) of instruction tile i against token m + 16 j. Plain: tile i's columns
// of y start at n + 16 i. Gated: tiles alternate between gate and up, tiles 2 p
// and 2 p + 1 make the columns from n + 16 p on, and NI is a multiple of four,
// so that blocks of 32 columns are whole.
template <int NI, int WM, bool GATED>
__device__ __forceinline__ void finish(const Mx4Args &a, const v4f32 (&acc)[NI][WM], int64_t n,
                                       int64_t m, int64_t end, int lane) {
    const int lg = lane >> 4;
    const bool wide = aligned4(a.y, a.y_format, a.N);
    if constexpr (!GATED) {
        const bool eight = aligned8(a.y, a.N);
#pragma unroll
        for (int j = 0; j < WM; ++j) {
            const int64_t t = m + 16 * j;
            if constexpr (NI % 2 == 0) {
#pragma unroll
                for (int i = 0; i < NI; i += 2) {
                    const int64_t c = n + 16 * i;
                    store_pair(a.y, a.y_format, t * a.N + c, acc[i][j], acc[i + 1][j], end - c, t < a.M, lg,
                               wide, eight);
                }
            } else {
                const int64_t c = n + 4 * lg;
                const int left = (int)(end - c < 4 ? end - c : 4);
                if (t < a.M && left > 0) store4(a.y, a.y_format, t * a.N + c, acc[0][j], left, wide && left == 4);
            }
        }
    } else {
        constexpr int P = NI < 4 ? NI / 2 : 2;               // pairs of tiles at a time
        const bool wide_gu = aligned4(a.gu, a.y_format, a.N);
        const bool eight = aligned8(a.y, a.N), eight_gu = aligned8(a.gu, a.N);
        auto run = [&](auto act) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < WM; ++j) {
                const int64_t t = m + 16 * j;
                const bool live = t < a.M;
#pragma unroll
                for (int b = 0; b < NI / (2 * P); ++b) {
                    v4f32 g[2], u[2], h[2];
                    const int64_t c = n + 16 * P * b;
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const int q = p < P ? p : 0;                // one pair: its columns end after 16
                        g[p] = acc[2 * (P * b + q)][j];
                        u[p] = acc[2 * (P * b + q) + 1][j];
#pragma unroll
                        for (int i = 0; i < 4; ++i) h[p][i] = p < P ? gate_act<act.value>(g[p][i]) * u[p][i] : 0.0f;
                    }
                    const int64_t left = P == 2 || end - c < 16 ? end - c : 16;
                    if (a.y) store_pair(a.y, a.y_format, t * a.N + c, h[0], h[1], left, live, lg, wide, eight);
                    if (a.gu) {
                        store_pair(a.gu, a.y_format, 2 * t * a.N + c, g[0], g[1], left, live, lg, wide_gu, eight_gu);
                        store_pair(a.gu, a.y_format, (2 * t + 1) * a.N + c, u[0], u[1], left, live, lg, wide_gu, eight_gu);
                    }
                    if constexpr (P == 2) {
                        if (a.hq)
                            store_quantised(h, a.hq + (t * a.N + c) / 2, a.hs + (t * a.N + c) / 32,
                                            live && c < end, lane);
                    }
                    __builtin_amdgcn_sched_barrier(0);   // one block's registers at a time
                }
            }
        };
        if (a.act == kSilu)
            run(std::integral_constant<int, kSilu>());
        else if (a.act == kGelu)
            run(std::integral_constant<int, kGelu>());
        else
            run(std::integral_constant<int, kGeluTanh>());
    }
}

// First column of a tile (gated: of h).
template <class L, bool GATED>
__device__ __forceinline__ int64_t first_column(int tn) {
    return (int64_t)tn * (GATED ? L::BN / 2 : L::BN);
}

// The end of a block's work: the tile's results, or a split tile's sums. Waves
// past the last token have none.
template <class L, bool GATED>
__device__ __forceinline__ void end_share(const Mx4Args &a, const MxPlan &p, const MxShare &s,
                                          const v4f32 (&acc)[L::WN][L::WM], int wave, int lane) {
    const int wn = wave % L::NWN, wm = wave / L::NWN;
    const int64_t m = (int64_t)s.tm * L::BM + 16 * L::WM * wm;
    if (!s.split) {
        finish<L::WN, L::WM, GATED>(a, acc, first_column<L, GATED>(s.tn) + (GATED ? 8 : 16) * L::WN * wn, m + (lane & 15), a.N, lane);
        return;
    }
    if (m < a.M) store_share<L::WN, L::WM, L::T>(p, s.item, wave * kWave + lane, L::WM, acc);
}

// The split tiles' sums and their end: a block for every two instruction tiles of a
// wave's rows (gated: four, a block of 32 columns).
template <class L, bool GATED>
__global__ __launch_bounds__(L::T) void mx4_sum_kernel(Mx4Args a, MxPlan p) {
    constexpr int NI = GATED ? 4 : 2, WM = L::WM, kCuts = L::WN / NI;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;
    const int index = (int)blockIdx.x / kCuts, cut = (int)blockIdx.x % kCuts;
    const int wn = wave % L::NWN, wm = wave / L::NWN;
    int tn, tm;
    tile_at(p, p.full + index, tn, tm);
    const int64_t m = (int64_t)tm * L::BM + 16 * WM * wm;
    if (m >= a.M) return;
    v4f32 acc[NI][WM];
    sum_shares<L::WN, WM, L::T>(p, index, NI * cut, 0, tid, acc);
    const int64_t n = first_column<L, GATED>(tn) + (GATED ? 8 : 16) * (L::WN * wn + NI * cut);
    finish<NI, WM, GATED>(a, acc, n, m + (lane & 15), a.N, lane);
}

// ---------------------------------------------------------------- tiles
//
// A block owns BN weight rows x BM tokens, NWN x NWM waves of WN x WM
// instruction tiles of 16 x 16. Weights are the instruction's first operand, so
// a lane's four results are consecutive columns of y. K advances in stages of
// 256 (two instructions), copied into a ring of two LDS slots by 16-byte buffer
// -> LDS copies, a whole 128-byte line of a row per eight lanes; the copies of
// stage s + 1 fly while stage s is multiplied. Inside a row the 16-byte unit c
// lies at place c ^ swizzle(row), so the reads of 16 rows' unit c are free of
// bank conflicts. Scales travel four instructions (16 bytes a row) at a time in
// two slots of their own.
// Rows past the end lie outside the buffer resources: they read zeros.
template <int WN_, int WM_, int NWN_, int NWM_>
struct MxTile {
    static constexpr int WN = WN_, WM = WM_, NWN = NWN_, NWM = NWM_;
    static constexpr int W = NWN * NWM, T = kWave * W;
    static constexpr int BN = 16 * WN * NWN, BM = 16 * WM * NWM;
    static constexpr int kStageBytes = (BN + BM) * 128;
    static constexpr int kScaleBytes = (BN + BM) * 16;
    static constexpr int kLdsBytes = 2 * kStageBytes + 2 * kScaleBytes;
    static constexpr int kCopiesN = BN / 8 / W, kCopiesM = BM / 8 / W;   // per wave and stage
    static constexpr int kBlocks = 160 * 1024 / kLdsBytes;               // a compute unit holds
    static constexpr int kRun = BN == 64 ? 1050 : 1550, kMore = BN == 64 ? 1050 : 750,
                         kEnds = BN == 64 ? 1500 : 3000;                 // plan_tiles's times, ns
    static_assert(BN % (8 * W) == 0 && BM % (8 * W) == 0 && BN % 64 == 0 && BM % 64 == 0, "copies");
};

__device__ __forceinline__ int mx_swizzle(int row) { return row & 6; }

// SPAN: rows of scales are copied 16 bytes at a time (K a multiple of 512 and
// 16-byte bases); else 4 bytes at a time.
template <class L, bool GATED, bool SPAN>
__global__ __launch_bounds__(L::T) void mx4_tile_kernel(Mx4Args a, MxPlan plan) {
    constexpr int WN = L::WN, WM = L::WM, W = L::W;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % L::NWN, wm = wave / L::NWN;
    const int r = lane & 15, lg = lane >> 4;

    const MxShare share = share_of(plan);
    if (!share.live) return;
    const int64_t m0 = (int64_t)share.tm * L::BM, n0 = first_column<L, GATED>(share.tn);
    const int kb = (int)(a.K / 2), sb = (int)(a.K / kMxBlock);   // bytes of a row
    // where the block's steps end: a run is four
    const int steps = share.q1 == plan.runs ? (int)(a.K / 128) : 4 * share.q1, stages = (steps + 1) / 2;
    const int rows_n = (int)(a.N - n0 < L::BN ? a.N - n0 : L::BN);
    const int rows_m = (int)(a.M - m0 < L::BM ? a.M - m0 : L::BM);

    // copy i of a wave fills rows 8 (i W + wave) ..; in the gated block runs of
    // 16 rows alternate between gate and up, which for a wave is one or the other
    const bool up = GATED && ((wave >> 1) & 1);
    const __amdgpu_buffer_rsrc_t rs_w = make_rsrc(a.w + (n0 + (up ? a.N : 0)) * kb, (int64_t)rows_n * kb);
    const __amdgpu_buffer_rsrc_t rs_a = make_rsrc(a.a + m0 * kb, (int64_t)rows_m * kb);
    const __amdgpu_buffer_rsrc_t rs_ws =
        make_rsrc(a.ws + n0 * sb, (GATED ? a.N * sb : 0) + (int64_t)rows_n * sb);
    const __amdgpu_buffer_rsrc_t rs_as = make_rsrc(a.as + m0 * sb, (int64_t)rows_m * sb);

    int woff[L::kCopiesN], aoff[L::kCopiesM];
    const int sub = lane >> 3;
#pragma unroll
    for (int i = 0; i < L::kCopiesN; ++i) {
        const int row = 8 * (i * W + wave) + sub;
        const int unit = (lane & 7) ^ mx_swizzle(row);
        const int src = GATED ? 16 * (row >> 5) + (row & 15) : row;
        woff[i] = src < rows_n ? src * kb + 16 * unit : kCopyOob;
    }
#pragma unroll
    for (int i = 0; i < L::kCopiesM; ++i) {
        const int row = 8 * (i * W + wave) + sub;
        const int unit = (lane & 7) ^ mx_swizzle(row);
        aoff[i] = row < rows_m ? row * kb + 16 * unit : kCopyOob;
    }
    // the last stage of an odd number of steps has only the first half of its units
    const int last = steps & 1 ? stages - 1 : -1;

    auto issue_stage = [&](int s) __attribute__((always_inline)) {
        uint8_t *st = smem + (s & 1) * L::kStageBytes;
        const int at = s * 128;
#pragma unroll
        for (int i = 0; i < L::kCopiesN; ++i) {
            const int row = 8 * (i * W + wave) + sub;
            const bool live = woff[i] != kCopyOob && !(s == last && (((lane & 7) ^ mx_swizzle(row)) & 4));
            copy16_to_lds(rs_w, st + (i * W + wave) * 1024, live ? woff[i] + at : kCopyOob);
        }
#pragma unroll
        for (int i = 0; i < L::kCopiesM; ++i) {
            const int row = 8 * (i * W + wave) + sub;
            const bool live = aoff[i] != kCopyOob && !(s == last && (((lane & 7) ^ mx_swizzle(row)) & 4));
            copy16_to_lds(rs_a, st + L::BN * 128 + (i * W + wave) * 1024, live ? aoff[i] + at : kCopyOob);
        }
    };
    // scale rows: first the weights' BN, then the tokens' BM, 16 bytes each
    auto scale_source = [&](int row, int &off) __attribute__((always_inline)) {
        if (row < L::BN) {
            const int src = GATED ? 16 * (row >> 5) + (row & 15) : row;
            off = src < rows_n ? src * sb + (GATED && (row & 16) ? (int)(a.N * sb) : 0) : kCopyOob;
        } else {
            off = row - L::BN < rows_m ? (row - L::BN) * sb : kCopyOob;
        }
    };
    auto issue_scales = [&](int q) __attribute__((always_inline)) {   // steps 4 q .. 4 q + 3
        uint8_t *sc = smem + 2 * L::kStageBytes + (q & 1) * L::kScaleBytes;
        constexpr int kRows = SPAN ? 64 : 16;                         // rows of one copy
        constexpr int kAll = (L::BN + L::BM) / kRows;
#pragma unroll
        for (int i = 0; i < (kAll + W - 1) / W; ++i) {
            const int c = i * W + wave;
            if (kAll % W != 0 && c >= kAll) break;
            int off;
            scale_source(c * kRows + (SPAN ? lane : lane >> 2), off);
            const __amdgpu_buffer_rsrc_t rs = c * kRows < L::BN ? rs_ws : rs_as;
            if constexpr (SPAN) {
                const bool live = off != kCopyOob && 4 * q < steps;
                copy16_to_lds(rs, sc + c * 1024, live ? off + 16 * q : kCopyOob);
            } else {
                const int step = 4 * q + (lane & 3);
                const bool live = off != kCopyOob && step < steps;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t *)(sc + c * 256), 4,
                                                         live ? off + 4 * step : kCopyOob, 0, 0, 0);
            }
        }
    };

    v4f32 acc[WN][WM];
#pragma unroll
    for (int i = 0; i < WN; ++i)
#pragma unroll
        for (int j = 0; j < WM; ++j) acc[i][j] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};

    const int row_n = 16 * WN * wn + r, row_m = L::BN + 16 * WM * wm + r;
    issue_scales(share.q0);
    issue_stage(2 * share.q0);
    for (int s = 2 * share.q0; s < stages; ++s) {
        wait_vmem<0>();                         // this wave's copies of stage s
        ring_barrier();                         // everyone's; and stage s - 1 is read
        if (s + 1 < stages) issue_stage(s + 1);
        if ((s & 1) == 0 && 2 * s + 4 < steps) issue_scales((s >> 1) + 1);
        const uint8_t *st = smem + (s & 1) * L::kStageBytes;
        const uint8_t *sc = smem + 2 * L::kStageBytes + ((s >> 1) & 1) * L::kScaleBytes + 8 * (s & 1);
        v2u sw[WN], sa[WM];
#pragma unroll
        for (int i = 0; i < WN; ++i) sw[i] = *reinterpret_cast<const v2u *>(sc + 16 * (row_n + 16 * i));
#pragma unroll
        for (int j = 0; j < WM; ++j) sa[j] = *reinterpret_cast<const v2u *>(sc + 16 * (row_m + 16 * j));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (2 * s + half >= steps) break;
            const int place = 16 * ((4 * half + lg) ^ mx_swizzle(r));
            v4i fw[WN], fa[WM];
#pragma unroll
            for (int i = 0; i < WN; ++i)
                fw[i] = *reinterpret_cast<const v4i *>(st + 128 * (row_n + 16 * i) + place);
#pragma unroll
            for (int j = 0; j < WM; ++j)
                fa[j] = *reinterpret_cast<const v4i *>(st + 128 * (row_m + 16 * j) + place);
#pragma unroll
            for (int i = 0; i < WN; ++i)
#pragma unroll
                for (int j = 0; j < WM; ++j)
                    acc[i][j] = mfma_mx4(fw[i], fa[j], acc[i][j], sw[i][half] >> (8 * lg),
                                         sa[j][half] >> (8 * lg));
        }
    }

    end_share<L, GATED>(a, plan, share, acc, wave, lane);
}

// ---------------------------------------------------------------- wide tiles
//
// 256 weight rows x 256 tokens, eight waves (two a SIMD) of 128 x 64. Stages of
// 256 along K in two slots of 64 KB, scales of four steps (512) in one of 8 KB.
// A step is one instruction's 128. What a step multiplies was read from LDS
// during the step before: tokens into the other of two register sets, weights
// and their scales rolling, each tile's registers taking the next step's as soon
// as its four products are issued. After a stage's last read a barrier frees its
// slot; the copies of the next stage but one are dealt over the products that
// follow.
// Each copy has a resource of its own, the eight rows that it fills as far as
// they exist, so that one lane offset serves all of them.
// 4096 x 5120 x 17408 185 to 194 us by the clock (3.9 PFLOP/s) and 11 of sums; gated
// 2048 x 17408 x 5120 212 us (3.4), 280 with g and u written. With 128 x 128 tiles 276 and 310. The same
// loop without its copies reaches 4.9, matrix instructions alone on random operands
// 6.2 to 6.9 (the clock falls to 1.7 GHz; 8.6 on constant ones): the copies' share of
// the issue and the clock bound it. An epilogue overlaps nothing, a unit has one block.
struct MxWide {
    static constexpr int W = 8, T = 512, BN = 256, BM = 256, WN = 8, WM = 4, NWN = 2;
    static constexpr int kStageBytes = (BN + BM) * 128;
    static constexpr int kScaleBytes = (BN + BM) * 16;
    static constexpr int kLdsBytes = 2 * kStageBytes + kScaleBytes;
    static constexpr int kBlocks = 1, kRun = 2300, kMore = 1700, kEnds = 6000;
};

template <bool GATED, bool SPAN>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void mx4_wide_kernel(Mx4Args a, MxPlan plan) {
    typedef MxWide L;
    constexpr int WN = L::WN, WM = L::WM, W = L::W;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint8_t *const sc = smem + 2 * L::kStageBytes;
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % L::NWN, wm = wave / L::NWN;
    const int r = lane & 15, lg = lane >> 4;

    const MxShare share = share_of(plan);
    if (!share.live) return;
    const int64_t m0 = (int64_t)share.tm * L::BM, n0 = first_column<L, GATED>(share.tn);
    const int kb = (int)(a.K / 2), sb = (int)(a.K / kMxBlock);   // bytes of a row
    const int q0 = share.q0, q1 = share.q1;
    const int steps = q1 == plan.runs ? (int)(a.K / 128) : 4 * q1;   // where the block's end
    const int rows_n = (int)(a.N - n0 < L::BN ? a.N - n0 : L::BN);
    const int rows_m = (int)(a.M - m0 < L::BM ? a.M - m0 : L::BM);

    // copy k < 4 of a wave: weight rows 64 k + 8 wave .. of the tile, else tokens'.
    // In the gated block runs of 16 tile rows alternate between gate and up.
    const bool up = GATED && ((wave >> 1) & 1);
    const int first_n = GATED ? 16 * (wave >> 2) + 8 * (wave & 1) : 8 * wave, first_m = 8 * wave;
    const uint8_t *const base_n = a.w + (n0 + (up ? a.N : 0) + first_n) * kb;
    const uint8_t *const base_m = a.a + (m0 + first_m) * kb;
    auto bytes = [&](int rows) __attribute__((always_inline)) {
        return __builtin_amdgcn_readfirstlane((rows < 0 ? 0 : rows > 8 ? 8 : rows) * kb);
    };
    constexpr int kNext = GATED ? 32 : 64;           // weight rows between two copies
    const int bytes_n[4] = {bytes(rows_n - first_n), bytes(rows_n - first_n - kNext),
                            bytes(rows_n - first_n - 2 * kNext), bytes(rows_n - first_n - 3 * kNext)};
    const int bytes_m[4] = {bytes(rows_m - first_m), bytes(rows_m - first_m - 64),
                            bytes(rows_m - first_m - 128), bytes(rows_m - first_m - 192)};
    const int sub = lane >> 3, unit = (lane & 7) ^ mx_swizzle(sub);
    const int off = sub * kb + 16 * unit;
    int stage_off = kCopyOob;                        // of the stage being copied
    auto open_stage = [&](int s) __attribute__((always_inline)) {
        stage_off = 2 * s + (unit >> 2) < steps ? off : kCopyOob;
    };
    auto copy = [&](int s, int k) __attribute__((always_inline)) {
        const __amdgpu_buffer_rsrc_t rs = k < 4 ? make_rsrc(base_n + (int64_t)k * kNext * kb, bytes_n[k & 3])
                                                : make_rsrc(base_m + (int64_t)(k & 3) * 64 * kb, bytes_m[k & 3]);
        copy16_to_lds_at(rs, smem + (s & 1) * L::kStageBytes + (k * W + wave) * 1024, stage_off, 128 * s);
    };
    // scale rows of the tile: the weights' 256, then the tokens'
    auto scale_off = [&](int row) __attribute__((always_inline)) {
        if (row < L::BN) {
            const int src = GATED ? 16 * (row >> 5) + (row & 15) : row;
            return src < rows_n ? src * sb + (GATED && (row & 16) ? (int)(a.N * sb) : 0) : kCopyOob;
        }
        return row - L::BN < rows_m ? (row - L::BN) * sb : kCopyOob;
    };
    const __amdgpu_buffer_rsrc_t rs_ws =
        make_rsrc(a.ws + n0 * sb, (GATED ? a.N * sb : 0) + (int64_t)rows_n * sb);
    const __amdgpu_buffer_rsrc_t rs_as = make_rsrc(a.as + m0 * sb, (int64_t)rows_m * sb);
    constexpr int NS = SPAN ? 1 : 4;                 // scale copies of a wave
    int soff[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i)
        soff[i] = scale_off(SPAN ? 64 * wave + lane : 16 * (i * W + wave) + (lane >> 2));
    auto copy_scales = [&](int q) __attribute__((always_inline)) {
        if constexpr (SPAN) {
            copy16_to_lds_at(wave < W / 2 ? rs_ws : rs_as, sc + wave * 1024, q < q1 ? soff[0] : kCopyOob, 16 * q);
        } else {
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int step = 4 * q + (lane & 3);
                const int at = soff[i] != kCopyOob && step < steps ? soff[i] + 4 * step : kCopyOob;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(i < NS / 2 ? rs_ws : rs_as,
                                                         (lds_void_t *)(sc + (i * W + wave) * 256), 4, at, 0, 0, 0);
            }
        }
    };

    v4f32 acc[WN][WM];
#pragma unroll
    for (int i = 0; i < WN; ++i)
#pragma unroll
        for (int j = 0; j < WM; ++j) acc[i][j] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};

    const int row_n = 16 * WN * wn + r, row_m = L::BN + 16 * WM * wm + r;
    v4i w[WN], x[2][WM];
    uint32_t sw[WN], sa[WM], sa_next[WM];
    // step u of four: stage u / 2 of two slots, half u % 2
    const uint8_t *const at0 = smem + 128 * row_n + 16 * (lg ^ mx_swizzle(r));
    const uint8_t *const at1 = smem + 128 * row_n + 16 * ((4 + lg) ^ mx_swizzle(r));
    const uint8_t *const at2 = at0 + L::kStageBytes, *const at3 = at1 + L::kStageBytes;
    const int over = 128 * (row_m - row_n);
    const uint8_t *const xt0 = at0 + over, *const xt1 = at1 + over, *const xt2 = at2 + over, *const xt3 = at3 + over;
    auto read_w = [&](int u, int i) __attribute__((always_inline)) {
        const uint8_t *p = u == 0 ? at0 : u == 1 ? at1 : u == 2 ? at2 : at3;
        w[i] = *reinterpret_cast<const v4i *>(p + 2048 * i);
    };
    auto read_x = [&](int u, int j) __attribute__((always_inline)) {
        const uint8_t *p = u == 0 ? xt0 : u == 1 ? xt1 : u == 2 ? xt2 : xt3;
        x[u & 1][j] = *reinterpret_cast<const v4i *>(p + 2048 * j);
    };
    // byte lg of a row's four words: the lane's scales of four steps
    const uint32_t pick = 0x0c0c0400u + 0x0101u * lg;
    auto read_scale = [&](int row) __attribute__((always_inline)) {
        const v4u v = *reinterpret_cast<const v4u *>(sc + 16 * row);
        const uint32_t lo = __builtin_amdgcn_perm(v[1], v[0], pick);
        const uint32_t hi = __builtin_amdgcn_perm(v[3], v[2], pick);
        return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
    };

    // the slots go by the stage's parity: start on an even one
    const int s0 = 2 * q0;
    copy_scales(q0);
    open_stage(s0);
#pragma unroll
    for (int k = 0; k < 8; ++k) copy(s0, k);
    open_stage(s0 + 1);
#pragma unroll
    for (int k = 0; k < 6; ++k) copy(s0 + 1, k);
    wait_vmem<6>();
    ring_barrier();
#pragma unroll
    for (int i = 0; i < WN; ++i) read_w(0, i);
#pragma unroll
    for (int j = 0; j < WM; ++j) read_x(0, j);
#pragma unroll
    for (int i = 0; i < WN; ++i) sw[i] = read_scale(row_n + 16 * i);
#pragma unroll
    for (int j = 0; j < WM; ++j) sa[j] = read_scale(row_m + 16 * j);

    constexpr int kLead = 2;                         // tiles multiplied before a step's barrier
    for (int q = q0; q < q1; ++q) {
        auto step = [&](auto number) __attribute__((always_inline)) {
            constexpr int U = decltype(number)::value, V = (U + 1) & 3;
            auto products = [&](int i) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < WM; ++j)
                    acc[i][j] = mfma_mx4<U>(w[i], x[U & 1][j], acc[i][j], sw[i], sa[j]);
            };
            auto next = [&](int i) __attribute__((always_inline)) {
                read_w(V, i);
                if (U == 3) sw[i] = read_scale(row_n + 16 * i);
            };
#pragma unroll
            for (int i = 0; i < kLead; ++i) {
                products(i);
                if ((U & 1) == 0) copy(2 * q + 1 + U / 2, 6 + i);
            }
            if (U & 1) {
                __builtin_amdgcn_sched_barrier(0);
                wait_vmem<0>();                      // the next stage, and at U = 3 its scales
                ring_barrier();                      // for all waves; this stage is read
                if (U == 1) copy_scales(q + 1);
                open_stage(2 * q + U / 2 + 2);
            }
#pragma unroll
            for (int j = 0; j < WM; ++j) read_x(V, j);
            if (U == 3) {
#pragma unroll
                for (int j = 0; j < WM; ++j) sa_next[j] = read_scale(row_m + 16 * j);
            }
#pragma unroll
            for (int i = 0; i < kLead; ++i) next(i);
#pragma unroll
            for (int i = kLead; i < WN; ++i) {
                products(i);
                next(i);
                if (U & 1) copy(2 * q + U / 2 + 2, i - kLead);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        step(std::integral_constant<int, 0>());
        step(std::integral_constant<int, 1>());
        step(std::integral_constant<int, 2>());
        step(std::integral_constant<int, 3>());
#pragma unroll
        for (int j = 0; j < WM; ++j) sa[j] = sa_next[j];
    }
    wait_vmem<0>();                                  // no copy may land after the block ends

    end_share<L, GATED>(a, plan, share, acc, wave, lane);
}

// ---------------------------------------------------------------- few tokens
//
// Up to 16 TT tokens in all: bound by the weights' bytes. A block takes `rows`
// weight rows (gated: that many of gate and of up), a multiple of four chosen so
// that the blocks fill the compute units evenly, and its waves share the runs of
// 512 along K: their sums meet in LDS and are added in the order of K. A wave
// copies a run's codes, of the weights and of the tokens, into a piece of LDS of
// its own, 256 contiguous bytes a row and four rows a copy (loaded straight into
// the instruction's registers, 64 bytes a row, every line is requested twice),
// and waits for no other wave; the waves of a unit keep about 100 KB in flight.
// The 16-byte unit c of row r lies at place c ^ (r % 16): reads of 16 rows are
// free of bank conflicts.
// An instruction's rows do not mix: tiles' rows past `rows`, whose reads are
// clamped to the last one, and tokens past M make results that are not stored.
// Rows past the end of an array lie outside its resource and read zeros.
// Bound by HBM from some 20 MB of weights on: 16 x 5120 x 17408 10.0 us (4.7 TB/s; 64 x
// 64 tiles 36.5), gated 1 x 17408 x 5120 22.3 (4.2 TB/s); 1 x 5120 x 6144 5.0, where
// start and end of the blocks count as much.
struct MxThin {
    int rows;                         // of a block
    int tokens4;                      // copies that hold the tokens, four each
};

template <int NI, int TT, bool GATED>
__global__ __launch_bounds__(1024) void mx4_thin_kernel(Mx4Args a, MxThin plan) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x >> 6;
    const int r = lane & 15, lg = lane >> 4;
    constexpr int kHalves = GATED ? 2 : 1;
    const int64_t n0 = (int64_t)blockIdx.x * plan.rows;
    const int kb = (int)(a.K / 2), sb = (int)(a.K / kMxBlock);
    const int steps = (int)(a.K / 128), runs = (steps + 3) / 4;
    const int q0 = __builtin_amdgcn_readfirstlane((int)((uint32_t)runs * wave / waves));
    const int q1 = __builtin_amdgcn_readfirstlane((int)((uint32_t)runs * (wave + 1) / waves));
    const int rows_n = (int)(a.N - n0 < plan.rows ? a.N - n0 : plan.rows);
    const int rows_m = (int)a.M;
    uint8_t *const mine = smem + wave * 256 * (kHalves * plan.rows + 4 * plan.tokens4);
    uint8_t *const mine_x = mine + 256 * kHalves * plan.rows;

    v4f32 acc[NI][TT];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[i][j] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
    // where the lane's row of tile i lies (gated: gate, up, gate, ...), and its token's
    const uint8_t *from[NI], *from_x[TT];
    int turn[NI], turn_x[TT];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int row = 16 * (i / kHalves) + r, in = row < plan.rows ? row : plan.rows - 1;
        from[i] = mine + 256 * ((i % kHalves) * plan.rows + in);
        turn[i] = in & 15;
    }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int t = 16 * j + r, in = t < 4 * plan.tokens4 ? t : 4 * plan.tokens4 - 1;
        from_x[j] = mine_x + 256 * in;
        turn_x[j] = in & 15;
    }
    const uint32_t pick = 0x0c0c0400u + 0x0101u * lg;
    auto own = [&](v4u v) __attribute__((always_inline)) {      // byte lg of the row's four words
        const uint32_t lo = __builtin_amdgcn_perm(v[1], v[0], pick);
        const uint32_t hi = __builtin_amdgcn_perm(v[3], v[2], pick);
        return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
    };
    // rows 4 p .. 4 p + 3 of an array's `rows` rows into `to`
    auto copies = [&](const uint8_t *base, int rows, int pieces, uint8_t *to, int q) __attribute__((always_inline)) {
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(base, (int64_t)rows * kb);
        for (int p = 0; p < pieces; ++p) {
            const int row = 4 * p + lg, unit = r ^ (row & 15);
            copy16_to_lds(rs, to + p * 1024,
                          4 * q + (unit >> 2) < steps && row < rows ? row * kb + 16 * unit + 256 * q : kCopyOob);
        }
    };
    for (int q = q0; q < q1; ++q) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
            copies(a.w + (n0 + h * a.N) * kb, rows_n, plan.rows / 4, mine + 256 * h * plan.rows, q);
        copies(a.a, rows_m, plan.tokens4, mine_x, q);
        v4u sw[NI], sx[TT];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int row = 16 * (i / kHalves) + r;
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.ws + (n0 + (i % kHalves) * a.N) * sb, (int64_t)rows_n * sb);
            sw[i] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(
                rs, row < rows_n ? row * sb + 16 * q : kCopyOob, 0, 0));
        }
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.as, (int64_t)rows_m * sb);
#pragma unroll
        for (int j = 0; j < TT; ++j)
            sx[j] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(
                rs, 16 * j + r < rows_m ? (16 * j + r) * sb + 16 * q : kCopyOob, 0, 0));
        wait_vmem<0>();
        asm volatile("" ::: "memory");                           // no LDS read moves up
        uint32_t ow[NI], ox[TT];
#pragma unroll
        for (int i = 0; i < NI; ++i) ow[i] = own(sw[i]);
#pragma unroll
        for (int j = 0; j < TT; ++j) ox[j] = own(sx[j]);
        // a step past K would take other rows' scales: it is left out
        auto step = [&](auto u) __attribute__((always_inline)) {
            if (4 * q + u.value >= steps) return;
            v4i w[NI], x[TT];
#pragma unroll
            for (int i = 0; i < NI; ++i)
                w[i] = *reinterpret_cast<const v4i *>(from[i] + 16 * ((4 * u.value + lg) ^ turn[i]));
#pragma unroll
            for (int j = 0; j < TT; ++j)
                x[j] = *reinterpret_cast<const v4i *>(from_x[j] + 16 * ((4 * u.value + lg) ^ turn_x[j]));
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < TT; ++j)
                    acc[i][j] = mfma_mx4<u.value>(w[i], x[j], acc[i][j], ow[i], ox[j]);
        };
        step(std::integral_constant<int, 0>());
        step(std::integral_constant<int, 1>());
        step(std::integral_constant<int, 2>());
        step(std::integral_constant<int, 3>());
        // the piece is read before the next run's copies into it
        __builtin_amdgcn_s_waitcnt(0xC07F);                      // lgkmcnt(0)
        asm volatile("" ::: "memory");
    }
    __syncthreads();
    v4f32 *const sums = reinterpret_cast<v4f32 *>(smem);         // [waves][NI][TT][64]
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) sums[((wave * NI + i) * TT + j) * kWave + lane] = acc[i][j];
    __syncthreads();
    // a wave ends one tile (gated: all of them, which a block of 32 columns may
    // span) of one token tile at a time
    constexpr int kEnds = GATED ? 1 : NI, kEach = NI / kEnds;
    for (int e = wave; e < kEnds * TT; e += waves) {
        const int i0 = e / TT, j = e % TT;
        v4f32 v[kEach][1];
#pragma unroll
        for (int i = 0; i < kEach; ++i) v[i][0] = sums[((i0 + i) * TT + j) * kWave + lane];
        for (int o = 1; o < waves; ++o)
#pragma unroll
            for (int i = 0; i < kEach; ++i) v[i][0] += sums[((o * NI + i0 + i) * TT + j) * kWave + lane];
        finish<kEach, 1, GATED>(a, v, n0 + 16 * i0, 16 * j + r, n0 + rows_n, lane);
    }
}

template <class L, bool GATED>
hipError_t launch_tiles(const Mx4Args &a, MxPlan p, void *work, hipStream_t stream) {
    p.part = static_cast<float *>(work);
    const int rest = p.tiles_n * p.tiles_m - p.full;
    const bool span = a.K % 512 == 0 &&
                      ((reinterpret_cast<uintptr_t>(a.as) | reinterpret_cast<uintptr_t>(a.ws)) & 15) == 0;
    const dim3 grid(plan_blocks(p)), block(L::T);
    const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, L::kLdsBytes, stream, a, p);
        return hipGetLastError();
    };
    hipError_t e;
    if constexpr (std::is_same<L, MxWide>::value)
        e = span ? go(mx4_wide_kernel<GATED, true>) : go(mx4_wide_kernel<GATED, false>);
    else
        e = span ? go(mx4_tile_kernel<L, GATED, true>) : go(mx4_tile_kernel<L, GATED, false>);
    if (e != hipSuccess || rest == 0) return e;
    hipLaunchKernelGGL((mx4_sum_kernel<L, GATED>), dim3((unsigned)(rest * (L::WN / (GATED ? 4 : 2)))), block, 0, stream, a, p);
    return hipGetLastError();
}

template <class L>
hipError_t run_tiles(const Mx4Args &a, bool gated, const MxPlan &p, void *work, hipStream_t stream) {
    return gated ? launch_tiles<L, true>(a, p, work, stream) : launch_tiles<L, false>(a, p, work, stream);
}

template <int NI, int TT, bool GATED>
hipError_t launch_thin(const Mx4Args &a, int rows, hipStream_t stream) {
    const int64_t blocks = (a.N + rows - 1) / rows;
    MxThin plan;
    plan.rows = rows;
    plan.tokens4 = (int)(a.M + 3) / 4;
    // as many waves as LDS holds (two blocks a unit unless each has its own),
    // the runs dealt evenly
    const int64_t bytes = 256 * ((GATED ? 2 : 1) * rows + 4 * plan.tokens4);
    const int64_t sums = NI * TT * 1024, piece = bytes > sums ? bytes : sums;
    const int64_t runs = (a.K + 511) / 512;
    int64_t most = (blocks > 256 ? 80 * 1024 : 160 * 1024) / piece;
    most = most > 16 ? 16 : most;
    const int64_t each = (runs + most - 1) / most;
    const int waves = (int)((runs + each - 1) / each);
    hipLaunchKernelGGL((mx4_thin_kernel<NI, TT, GATED>), dim3((unsigned)blocks), dim3((unsigned)(kWave * waves)),
                       (size_t)(waves * piece), stream, a, plan);
    return hipGetLastError();
}

// Rows of a block: those with which the busiest of the compute units reads the
// fewest, each block counted as four more. Quantised columns go by whole blocks.
int thin_rows(int64_t N, bool blocks32) {
    const int64_t cus = device_cus() > 0 ? device_cus() : 256;
    int best = 32;
    int64_t least = INT64_MAX;
    for (int rows = blocks32 ? 32 : 4; rows <= 32; rows += 4) {
        const int64_t blocks = (N + rows - 1) / rows;
        const int64_t cost = (blocks + cus - 1) / cus * (rows + 4);
        if (cost < least) {
            least = cost;
            best = rows;
        }
    }
    return best;
}

template <int TT>
hipError_t run_thin(const Mx4Args &a, bool gated, hipStream_t stream) {
    const int rows = thin_rows(a.N, gated && a.hq);
    if (!gated)
        return rows <= 16 ? launch_thin<1, TT, false>(a, rows, stream) : launch_thin<2, TT, false>(a, rows, stream);
    return rows <= 16 ? launch_thin<2, TT, true>(a, rows, stream) : launch_thin<4, TT, true>(a, rows, stream);
}

typedef MxTile<4, 1, 1, 4> MxSmall;    // 64 x 64
typedef MxTile<4, 4, 2, 2> MxMid;      // 128 x 128

// The tile for a shape: the least of plan_tiles's counts. (Measured at 33 to 4096
// tokens, N x K 5120 x 17408, 17408 x 5120, plain and gated, 6144 x 5120, 17408 x 1024
// and 1411 x 896, each tile in 1 to 16 ways: what the count takes is within 8 % of the
// fastest but at 1024 x 5120 x 17408, 74.5 us whole in 128 x 128 where 256 x 256 in two
// ways takes 64.7.)
enum class MxKind { kSmall, kMid, kWide };
MxKind choose_tile(int64_t M, int64_t N, int64_t K, bool gated, size_t bytes, MxPlan &plan) {
    const int64_t rows = gated ? 2 * N : N, runs = (K + 511) / 512;
    const MxCost s = plan_tiles<MxSmall>(M, rows, runs, bytes), m = plan_tiles<MxMid>(M, rows, runs, bytes),
                 w = plan_tiles<MxWide>(M, rows, runs, bytes);
    const MxKind kind = w.ns <= s.ns && w.ns <= m.ns ? MxKind::kWide : m.ns <= s.ns ? MxKind::kMid : MxKind::kSmall;
    plan = kind == MxKind::kWide ? w.plan : kind == MxKind::kMid ? m.plan : s.plan;
    return kind;
}

// Up to 16 tokens, and up to 32 where 64 x 64 tiles are fewer than two a compute
// unit. Both ways at 17 and 32 tokens, 1411 to 65536 rows and K of 896, 5120 and 17408
// (us at 32): 5120 x 17408 13.8 this way and 18.1 in tiles, 17408 x 5120 15.6 and 16.6,
// 24576 x 17408 61.5 and 55.7, 34816 x 5120 23.5 and 21.7 (gated 29.4 and 31.6), 65536 x
// 17408 143 and 128; the rule takes the faster one or one within 17 %.
bool takes_thin(int64_t M, int64_t N, bool gated) {
    return M <= 16 || (M <= 32 && (gated ? 2 * N : N) < 64 * 512);
}

}  // namespace

size_t mx4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, bool gated) {
    if (takes_thin(M, N, gated)) return 0;
    MxPlan p;
    switch (choose_tile(M, N, K, gated, SIZE_MAX, p)) {
        case MxKind::kSmall: return part_bytes<MxSmall>(p);
        case MxKind::kMid: return part_bytes<MxMid>(p);
        default: return part_bytes<MxWide>(p);
    }
}

hipError_t launch_mx4_gemm(const Mx4Args &a, bool gated, void *work, size_t work_bytes,
                           hipStream_t stream) {
    if (takes_thin(a.M, a.N, gated)) return a.M <= 16 ? run_thin<1>(a, gated, stream) : run_thin<2>(a, gated, stream);
    MxPlan p;
    switch (choose_tile(a.M, a.N, a.K, gated, work ? work_bytes : 0, p)) {
        case MxKind::kSmall: return run_tiles<MxSmall>(a, gated, p, work, stream);
        case MxKind::kMid: return run_tiles<MxMid>(a, gated, p, work, stream);
        default: return run_tiles<MxWide>(a, gated, p, work, stream);
    }
}

}  // namespace pq2
