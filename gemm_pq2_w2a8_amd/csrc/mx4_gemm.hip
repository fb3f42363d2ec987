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
#include "pq2_launch.hpp"

namespace pq2 {
namespace {

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
    static_assert(BN % (8 * W) == 0 && BM % (8 * W) == 0 && BN % 64 == 0 && BM % 64 == 0, "copies");
};

__device__ __forceinline__ int mx_swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

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

// Whether every run of four columns from a multiple of four on is aligned.
__device__ __forceinline__ bool aligned4(const void *y, int fmt, int64_t n) {
    return (n & 3) == 0 && (reinterpret_cast<uintptr_t>(y) & (fmt == kF32 ? 15 : 7)) == 0;
}

// SPAN: rows of scales are copied 16 bytes at a time (K a multiple of 512 and
// 16-byte bases); else 4 bytes at a time.
template <class L, bool GATED, bool SPAN>
__global__ __launch_bounds__(L::T) void mx4_tile_kernel(Mx4Args a, int tiles_n, int tiles) {
    constexpr int WN = L::WN, WM = L::WM, W = L::W;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % L::NWN, wm = wave / L::NWN;
    const int r = lane & 15, lg = lane >> 4;

    // each XCD takes a contiguous run of tiles
    const int per = (tiles + 7) / 8;
    const int tile = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if (tile >= tiles) return;
    const int64_t m0 = (int64_t)(tile / tiles_n) * L::BM;
    const int64_t n0 = (int64_t)(tile % tiles_n) * (GATED ? L::BN / 2 : L::BN);

    const int kb = (int)(a.K / 2), sb = (int)(a.K / kMxBlock);   // bytes of a row
    const int steps = (int)(a.K / 128), stages = (steps + 1) / 2;
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
    issue_scales(0);
    issue_stage(0);
    for (int s = 0; s < stages; ++s) {
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

    const int64_t mt = m0 + 16 * WM * wm + r;
    if constexpr (!GATED) {
        const bool wide = aligned4(a.y, a.y_format, a.N);
#pragma unroll
        for (int j = 0; j < WM; ++j) {
            const int64_t m = mt + 16 * j;
            if (m >= a.M) continue;
#pragma unroll
            for (int i = 0; i < WN; ++i) {
                const int64_t n = n0 + 16 * WN * wn + 16 * i + 4 * lg;
                const int left = (int)(a.N - n < 4 ? a.N - n : 4);
                if (left > 0) store4(a.y, a.y_format, m * a.N + n, acc[i][j], left, wide && left == 4);
            }
        }
    } else {
        const bool wide = aligned4(a.y, a.y_format, a.N);
        const bool wide_gu = aligned4(a.gu, a.y_format, a.N);
        auto finish = [&](auto act) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < WM; ++j) {
                const int64_t m = mt + 16 * j;
                const bool live = m < a.M;
#pragma unroll
                for (int b = 0; b < WN / 4; ++b) {
                    v4f32 h[2];
                    const int64_t n = n0 + 8 * WN * wn + 32 * b;   // the block of 32 columns
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const v4f32 g = acc[4 * b + 2 * p][j], u = acc[4 * b + 2 * p + 1][j];
#pragma unroll
                        for (int i = 0; i < 4; ++i) h[p][i] = gate_act<act.value>(g[i]) * u[i];
                        const int64_t c = n + 16 * p + 4 * lg;
                        const int left = (int)(a.N - c < 4 ? a.N - c : 4);
                        if (live && left > 0) {
                            if (a.y) store4(a.y, a.y_format, m * a.N + c, h[p], left, wide && left == 4);
                            if (a.gu) {
                                const bool whole = wide_gu && left == 4;
                                store4(a.gu, a.y_format, 2 * m * a.N + c, g, left, whole);
                                store4(a.gu, a.y_format, (2 * m + 1) * a.N + c, u, left, whole);
                            }
                        }
                    }
                    if (a.hq)
                        store_quantised(h, a.hq + (m * a.N + n) / 2, a.hs + (m * a.N + n) / 32,
                                        live && n < a.N, lane);
                    __builtin_amdgcn_sched_barrier(0);   // one block's registers at a time
                }
            }
        };
        if (a.act == kSilu)
            finish(std::integral_constant<int, kSilu>());
        else if (a.act == kGelu)
            finish(std::integral_constant<int, kGelu>());
        else
            finish(std::integral_constant<int, kGeluTanh>());
    }
}

template <class L, bool GATED>
hipError_t run_tiles(const Mx4Args &a, hipStream_t stream) {
    constexpr int cols = GATED ? L::BN / 2 : L::BN;
    const int64_t tn = (a.N + cols - 1) / cols, tm = (a.M + L::BM - 1) / L::BM;
    const int64_t per = (tn * tm + 7) / 8;
    const bool span = a.K % 512 == 0 &&
                      ((reinterpret_cast<uintptr_t>(a.as) | reinterpret_cast<uintptr_t>(a.ws)) & 15) == 0;
    const auto go = [&](auto kernel) -> hipError_t {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(8 * per)), dim3(L::T), L::kLdsBytes, stream, a,
                           (int)tn, (int)(tn * tm));
        return hipGetLastError();
    };
    return span ? go(mx4_tile_kernel<L, GATED, true>) : go(mx4_tile_kernel<L, GATED, false>);
}

}  // namespace

size_t mx4_gemm_workspace_bytes(int64_t, int64_t, int64_t, bool) { return 0; }

hipError_t launch_mx4_gemm(const Mx4Args &a, bool gated, void *, size_t, hipStream_t stream) {
    typedef MxTile<8, 4, 2, 4> Big;
    typedef MxTile<4, 1, 1, 4> Small;
    const int64_t rows = gated ? 2 * a.N : a.N;
    const int64_t big = ((rows + 255) / 256) * ((a.M + 255) / 256);
    if (big >= 192) return gated ? run_tiles<Big, true>(a, stream) : run_tiles<Big, false>(a, stream);
    return gated ? run_tiles<Small, true>(a, stream) : run_tiles<Small, false>(a, stream);
}

}  // namespace pq2
