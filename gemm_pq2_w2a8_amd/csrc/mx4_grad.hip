// mx4_grad.hip -- gradients through MX4 weights (gfx950): the input's gradient
// of the product, and the gated feed-forward block's backward pass.
//
//   dx[m][k] = sum_n d[m][n] w[n][k]
//   gated:  du = dh act(g),  dg = dh u act'(g),  d = (dg | du), n over 2 F
//
// The sum runs along n, across the weights' blocks of scales, so the weights
// are expanded to bfloat16, in which every one of them is exact, and multiplied
// by bfloat16 matrix instructions with float32 sums. d enters without a
// rounding of its own: bfloat16 as it is, float16 and float32 split into two
// and three bfloat16 parts that add up to it exactly (truncated, so that no
// part overflows), which run through the same loop as two or three passes over
// d's tiles beside one expansion of the weights.
#include <type_traits>

#include "mx4_launch.hpp"
#include "mx4_plan.hpp"

namespace pq2 {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));

constexpr int kStep = 64;             // n of a stage: two matrix instructions

int parts_of(int format) { return format == kBf16 ? 1 : format == kF16 ? 2 : 3; }

// ---------------------------------------------------------------- parts of d

// d's parts [parts][M][cols] (cols: N rounded up to a stage, zeros past N), or
// d itself where it can be read in place.
struct GradRows {
    const uint16_t *d;
    int64_t cols, plane;              // elements between rows, and between parts
    int parts;
    int64_t n;                        // columns that exist
};

__device__ __forceinline__ uint16_t take_part(float &v) {
    const uint32_t b = bits_of(v);
    const uint32_t top = b & 0xffff0000u;
    if ((b & 0x7f800000u) == 0x7f800000u) {      // infinite, NaN: whole, nothing left
        v = 0.0f;
        return (uint16_t)(b & 0x007fffffu ? (top >> 16) | 0x40u : top >> 16);
    }
    v -= as_float(top);         // exact
    return (uint16_t)(top >> 16);
}

__device__ __forceinline__ void store_parts(uint16_t *out, int64_t at, int64_t plane, int parts,
                                            float v) {
    if (parts == 1) {
        out[at] = bf16_rne(v);                   // a bfloat16 value: exact
        return;
    }
    for (int p = 0; p < parts; ++p) out[at + p * plane] = take_part(v);
}

// One thread per column of d (and of its padding). GATED: per column of dh,
// whose two columns of dgu (dgu may be gu) and of the parts it writes.
template <int FMT, bool GATED>
__global__ __launch_bounds__(256) void grad_rows_kernel(const void *dy, const void *gu, void *dgu,
                                                        int act, uint16_t *out, int64_t M,
                                                        int64_t N, int64_t cols, int parts) {
    typedef typename MxType<FMT>::T T;
    const int64_t F = GATED ? N / 2 : N;         // columns of dy
    const int64_t width = F + (out ? cols - N : 0);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < M * width;
         i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / width, c = i % width;
        if (c >= F) {                                // padding
            for (int p = 0; p < parts; ++p) out[p * M * cols + m * cols + N + (c - F)] = 0;
            continue;
        }
        float v = widen<FMT>(static_cast<const T *>(dy)[m * F + c]);
        if constexpr (GATED) {
            const float g = widen<FMT>(static_cast<const T *>(gu)[2 * m * F + c]);
            const float u = widen<FMT>(static_cast<const T *>(gu)[(2 * m + 1) * F + c]);
            float a, s;
            gate_act_slope(act, g, a, s);
            const T dg = narrow<FMT>(v * u * s), du = narrow<FMT>(v * a);
            if (dgu) {
                static_cast<T *>(dgu)[2 * m * F + c] = dg;
                static_cast<T *>(dgu)[(2 * m + 1) * F + c] = du;
            }
            if (out) {
                store_parts(out, m * cols + c, M * cols, parts, widen<FMT>(dg));
                store_parts(out, m * cols + F + c, M * cols, parts, widen<FMT>(du));
            }
        } else {
            store_parts(out, m * cols + c, M * cols, parts, v);
        }
    }
}

// ---------------------------------------------------------------- product
//
// A block owns BK columns of dx x BM tokens. Stage s covers 64 n: d's tile (one
// part) and the weights' 4-bit rows come by buffer -> LDS copies, and while
// stage s is multiplied the weights of stage s + 1 are expanded into the other
// of two bfloat16 tiles, rows n of BK values. The instruction wants, for a
// column k, eight consecutive n: the transposing LDS read takes them out of
// four rows at a time. The 32-byte segment of 16 columns seg of row n lies at
// place seg ^ turn(n), so that the four (and eight) rows of such a read are in
// different banks.
template <int WK_, int WM_, int NWK_, int NWM_>
struct GradTile {
    static constexpr int WK = WK_, WM = WM_, NWK = NWK_, NWM = NWM_;
    static constexpr int W = NWK * NWM, T = kWave * W;
    static constexpr int BN = 16 * WK * NWK, BM = 16 * WM * NWM;       // BN: columns of dx
    static constexpr int kD = BM * 128;                  // bytes of a tile of d
    static constexpr int kRaw = kStep * BN / 2;
    static constexpr int kWide = kStep * BN * 2;
    static constexpr int kLdsBytes = 2 * (kD + kRaw + kWide);
    static constexpr int kCopiesM = BM / 8 / W;          // per wave
    static constexpr int kCopiesW = kRaw / 1024 / W;
    static constexpr int kUnits = BN / 32;               // blocks of scales in a row of the tile
    static constexpr int kItems = kStep * kUnits / T;    // expanded by a thread
    static constexpr int kBlocks = 160 * 1024 / kLdsBytes;  // a compute unit holds
    static constexpr int kRun = 700, kMore = 400, kEnds = 2500;        // plan_tiles's times
    static_assert(kCopiesM * W * 8 == BM && kCopiesW * W * 1024 == kRaw && kItems * T == kStep * kUnits,
                  "whole copies");
};

__device__ __forceinline__ int grad_turn(int n) { return (n & 3) | (((n >> 3) & 1) << 2); }
__device__ __forceinline__ int grad_swizzle(int row) { return row & 6; }

__device__ __forceinline__ uint32_t expand2(uint32_t word, float scale, int byte) {
    switch (byte) {
        case 0: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 0));
        case 1: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 1));
        case 2: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 2));
        default: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 3));
    }
}

// Sixteen columns of four rows, transposed: lane i of 16 gives the address of
// four columns of row i / 4 and gets column i of all four rows.
__device__ __forceinline__ v4s read_turned(const uint8_t *p) {
    typedef __attribute__((address_space(3))) v4s lds_v4s;
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)p);
}

// Four results of one row of dx from column k on, which is a multiple of four.
__device__ __forceinline__ void store_dx(void *dx, int format, int64_t at, v4f32 v, bool wide) {
    if (wide && format == kF32) {
        *reinterpret_cast<v4f32 *>(static_cast<float *>(dx) + at) = v;
    } else if (wide) {
        *reinterpret_cast<v2u *>(static_cast<uint16_t *>(dx) + at) =
            v2u{pack16(format, v[0], v[1]), pack16(format, v[2], v[3])};
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) store_fmt(dx, format, at + e, v[e]);
    }
}

// acc[i][j]: four columns from k + 16 i + 4 (lane / 16) on of token m + 16 j.
template <int NI, int WM>
__device__ __forceinline__ void finish_dx(const v4f32 (&acc)[NI][WM], void *dx, int format, int64_t k, int64_t m,
                                          int64_t M, int64_t K, int lane) {
    const bool wide = (reinterpret_cast<uintptr_t>(dx) & (format == kF32 ? 15 : 7)) == 0;
#pragma unroll
    for (int j = 0; j < WM; ++j) {
        const int64_t t = m + 16 * j;
        if (t >= M) continue;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int64_t c = k + 16 * i + 4 * (lane >> 4);
            if (c < K) store_dx(dx, format, t * K + c, acc[i][j], wide);     // K is a multiple of four
        }
    }
}

struct GradOut {
    void *dx;
    int format;
    int64_t M, N, K;
};

// The end of a block's work: the tile's results, or a split tile's sums.
template <class L>
__device__ __forceinline__ void end_grad(const GradOut &o, const MxPlan &p, const MxShare &s,
                                         const v4f32 (&acc)[L::WK][L::WM], int wave, int lane) {
    const int wk = wave % L::NWK, wm = wave / L::NWK;
    const int64_t m = (int64_t)s.tm * L::BM + 16 * L::WM * wm;
    if (!s.split)
        finish_dx<L::WK, L::WM>(acc, o.dx, o.format, (int64_t)s.tn * L::BN + 16 * L::WK * wk, m + (lane & 15), o.M,
                                o.K, lane);
    else if (m < o.M)
        store_share<L::WK, L::WM, L::T>(p, s.item, wave * kWave + lane, acc);
}

template <class L>
__global__ __launch_bounds__(L::T) void grad_sum_kernel(GradOut o, MxPlan p) {
    constexpr int NI = 4, kCuts = L::WK / NI;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;
    const int index = (int)blockIdx.x / kCuts, cut = (int)blockIdx.x % kCuts;
    const int wk = wave % L::NWK, wm = wave / L::NWK;
    int tn, tm;
    tile_at(p, p.full + index, tn, tm);
    const int64_t m = (int64_t)tm * L::BM + 16 * L::WM * wm;
    if (m >= o.M) return;
    v4f32 acc[NI][L::WM];
    sum_shares<NI, L::WK, L::WM, L::T>(p, index, NI * cut, tid, acc);
    finish_dx<NI, L::WM>(acc, o.dx, o.format, (int64_t)tn * L::BN + 16 * (L::WK * wk + NI * cut), m + (lane & 15), o.M,
                         o.K, lane);
}

template <class L>
__global__ __launch_bounds__(L::T) void grad_kernel(GradRows d, const uint8_t *__restrict__ w,
                                                    const uint8_t *__restrict__ ws, GradOut o, MxPlan plan) {
    constexpr int WK = L::WK, WM = L::WM, W = L::W;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint8_t *const raw0 = smem + 2 * L::kD, *const wide0 = raw0 + 2 * L::kRaw;
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % L::NWK, wm = wave / L::NWK;
    const int r = lane & 15, lg = lane >> 4;
    const MxShare share = share_of(plan);
    if (!share.live) return;
    const int64_t M = o.M, N = o.N, K = o.K, m0 = (int64_t)share.tm * L::BM;
    const int k0 = share.tn * L::BN, s0 = share.q0, s1 = share.q1;
    const int parts = d.parts;

    const int rows_m = (int)(M - m0 < L::BM ? M - m0 : L::BM);
    const int cols = (int)(K - k0 < L::BN ? K - k0 : L::BN);
    const int sub = lane >> 3;

    // stage s of d's rows, part p
    auto issue_d = [&](int s, int p, int slot) __attribute__((always_inline)) {
        const __amdgpu_buffer_rsrc_t rs =
            make_rsrc(d.d + p * d.plane + m0 * d.cols + (int64_t)s * kStep,
                      ((int64_t)(rows_m - 1) * d.cols + kStep) * 2);
        uint8_t *to = smem + slot * L::kD;
        const int64_t left = d.n - (int64_t)s * kStep;           // columns that exist from here on
#pragma unroll
        for (int i = 0; i < L::kCopiesM; ++i) {
            const int row = 8 * (i * W + wave) + sub;
            const int unit = (lane & 7) ^ grad_swizzle(row);
            const bool live = row < rows_m && 8 * unit < left;
            copy16_to_lds(rs, to + (i * W + wave) * 1024,
                          live ? (int)(row * d.cols * 2) + 16 * unit : kCopyOob);
        }
    };
    // 4-bit rows n of stage s, unit u (32 columns) of row n at place u
    auto issue_w = [&](int s) __attribute__((always_inline)) {
        const int64_t n0 = (int64_t)s * kStep;
        const int rows = (int)(N - n0 < kStep ? N - n0 : kStep);
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(w + (n0 * K + k0) / 2, ((int64_t)(rows - 1) * K + cols) / 2);
        uint8_t *to = raw0 + (s & 1) * L::kRaw;
#pragma unroll
        for (int i = 0; i < L::kCopiesW; ++i) {
            const int item = (i * W + wave) * 64 + lane;
            const int row = item / L::kUnits, u = item % L::kUnits;
            const bool live = row < rows && 32 * u < cols;
            copy16_to_lds(rs, to + (i * W + wave) * 1024, live ? (int)(row * (K / 2)) + 16 * u : kCopyOob);
        }
    };
    uint32_t scale_byte[L::kItems];
    auto load_scales = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < L::kItems; ++i) {
            const int item = i * L::T + tid;
            const int64_t n = (int64_t)s * kStep + item / L::kUnits;
            const int u = item % L::kUnits;
            scale_byte[i] = n < N && 32 * u < cols ? ws[n * (K / kMxBlock) + k0 / kMxBlock + u] : 0u;
        }
    };
    auto expand = [&](int s) __attribute__((always_inline)) {
        const uint8_t *from = raw0 + (s & 1) * L::kRaw;
        uint8_t *to = wide0 + (s & 1) * L::kWide;
#pragma unroll
        for (int i = 0; i < L::kItems; ++i) {
            const int item = i * L::T + tid;
            const int n = item / L::kUnits, u = item % L::kUnits;
            const v4u c = *reinterpret_cast<const v4u *>(from + 16 * item);
            const float scale = mx_scale(scale_byte[i]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v4u o;
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = expand2(c[q], scale, j);
                const int seg = (2 * u + (q >> 1)) ^ grad_turn(n);
                *reinterpret_cast<v4u *>(to + n * (2 * L::BN) + 32 * seg + 16 * (q & 1)) = o;
            }
        }
    };

    v4f32 acc[WK][WM];
#pragma unroll
    for (int i = 0; i < WK; ++i)
#pragma unroll
        for (int j = 0; j < WM; ++j) acc[i][j] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};

    if (s0 < s1) {
        issue_w(s0);
        load_scales(s0);
        issue_d(s0, 0, 0);
        wait_vmem<0>();
        ring_barrier();
        expand(s0);
        if (s0 + 1 < s1) {
            issue_w(s0 + 1);
            load_scales(s0 + 1);
        }
    }
    for (int s = s0, p = 0, slot = 0; s < s1; slot ^= 1) {
        wait_vmem<0>();
        ring_barrier();                  // d's tile, the 4-bit rows s + 1, the bfloat16 rows s
        const bool turn = p + 1 == parts;
        if (!turn)
            issue_d(s, p + 1, slot ^ 1);
        else if (s + 1 < s1)
            issue_d(s + 1, 0, slot ^ 1);
        if (p == 0 && s + 1 < s1) {
            // the 4-bit rows' other slot was read a stage ago
            expand(s + 1);
            if (s + 2 < s1) {
                issue_w(s + 2);
                load_scales(s + 2);
            }
        }
        const uint8_t *dt = smem + slot * L::kD;
        const uint8_t *wt = wide0 + (s & 1) * L::kWide;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            v8bf fw[WK], fd[WM];
#pragma unroll
            for (int j = 0; j < WM; ++j) {
                const int row = 16 * (WM * wm + j) + r;
                fd[j] = *reinterpret_cast<const v8bf *>(dt + 128 * row + 16 * ((4 * half + lg) ^ grad_swizzle(r)));
            }
#pragma unroll
            for (int i = 0; i < WK; ++i) {
                const int n = 32 * half + 8 * lg + (r >> 2);
                const int seg = WK * wk + i;
                const v4s lo = read_turned(wt + n * (2 * L::BN) + 32 * (seg ^ grad_turn(n)) + 8 * (r & 3));
                const v4s hi = read_turned(wt + (n + 4) * (2 * L::BN) + 32 * (seg ^ grad_turn(n + 4)) + 8 * (r & 3));
                fw[i] = __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
#pragma unroll
            for (int i = 0; i < WK; ++i)
#pragma unroll
                for (int j = 0; j < WM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[i], fd[j], acc[i][j], 0, 0, 0);
        }
        p = turn ? 0 : p + 1;
        s += turn;
    }

    end_grad<L>(o, plan, share, acc, wave, lane);
}

// ---------------------------------------------------------------- wide tiles
//
// 256 columns x 256 tokens, eight waves (two a SIMD) of 128 x 64; d's tiles, the
// 4-bit rows and the bfloat16 rows in two slots each, 144 KB. A step is one
// instruction's 32 n, two a stage. What a step multiplies was read from LDS during
// the step before, tokens into the other of two register sets, weights rolling.
// In a stage's first step the next stage's weights are expanded; in its second a
// barrier frees d's slot and shows the others' expansion, and the copies of the
// next tile but one are dealt over the products that follow.
// TODO figures
struct GradWide {
    static constexpr int W = 8, T = 512, BN = 256, BM = 256, WK = 8, WM = 4, NWK = 2;
    static constexpr int kD = BM * 128, kRaw = kStep * BN / 2, kWide = kStep * BN * 2;
    static constexpr int kLdsBytes = 2 * (kD + kWide + kRaw);
    static constexpr int kBlocks = 1, kRun = 1500, kMore = 600, kEnds = 6000;   // plan_tiles's times
};

__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void grad_wide_kernel(GradRows d, const uint8_t *__restrict__ w, const uint8_t *__restrict__ ws, GradOut o,
                      MxPlan plan) {
    typedef GradWide L;
    constexpr int WK = L::WK, WM = L::WM, W = L::W;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint8_t *const wide0 = smem + 2 * L::kD, *const raw0 = wide0 + 2 * L::kWide;
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % L::NWK, wm = wave / L::NWK;
    const int r = lane & 15, lg = lane >> 4;
    const MxShare share = share_of(plan);
    if (!share.live) return;
    const int64_t M = o.M, N = o.N, K = o.K, m0 = (int64_t)share.tm * L::BM;
    const int k0 = share.tn * L::BN, s0 = share.q0, s1 = share.q1;
    const int parts = d.parts;
    const int rows_m = (int)(M - m0 < L::BM ? M - m0 : L::BM);
    const int cols = (int)(K - k0 < L::BN ? K - k0 : L::BN);

    // d: copy i of a wave fills rows 64 i + 8 wave .., each copy with a resource
    // of the rows that exist and one lane offset for all
    const int sub = lane >> 3, unit = (lane & 7) ^ grad_swizzle(sub);
    const int row_bytes = (int)(d.cols * 2);
    auto bytes = [&](int i) __attribute__((always_inline)) {
        const int rows = rows_m - 64 * i - 8 * wave;
        return __builtin_amdgcn_readfirstlane((rows < 0 ? 0 : rows > 8 ? 8 : rows) * row_bytes);
    };
    const int bytes_d[4] = {bytes(0), bytes(1), bytes(2), bytes(3)};
    const int off = sub * row_bytes + 16 * unit;
    const uint16_t *const base_d = d.d + (m0 + 8 * wave) * d.cols;
    const uint16_t *from_d = base_d;                 // of the tile being copied
    int off_d = kCopyOob;
    auto open_d = [&](int s, int p) __attribute__((always_inline)) {
        from_d = base_d + p * d.plane + (int64_t)s * kStep;
        off_d = s < s1 && (int64_t)s * kStep + 8 * unit < d.n ? off : kCopyOob;
    };
    auto copy_d = [&](int slot, int i) __attribute__((always_inline)) {
        copy16_to_lds(make_rsrc(from_d + (int64_t)i * 64 * d.cols, bytes_d[i]),
                      smem + slot * L::kD + (i * W + wave) * 1024, off_d);
    };
    // 4-bit rows: wave's copy fills rows 8 wave .. of the stage, eight units each
    const int kb = (int)(K / 2);
    const int row_w = 8 * wave + sub, unit_w = lane & 7;
    const bool live_w = 32 * unit_w < cols;
    auto copy_w = [&](int s) __attribute__((always_inline)) {
        const int64_t n0 = (int64_t)s * kStep;
        const int rows = (int)(N - n0 < kStep ? N - n0 : kStep);
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(w + n0 * kb + k0 / 2, (int64_t)(rows - 1) * kb + cols / 2);
        copy16_to_lds(rs, raw0 + (s & 1) * L::kRaw + wave * 1024,
                      live_w && row_w < rows ? row_w * kb + 16 * unit_w : kCopyOob);
    };
    // the thread expands unit unit_w of row row_w
    auto scale_of = [&](int s) __attribute__((always_inline)) {
        const int64_t n = (int64_t)s * kStep + row_w;
        return live_w && n < N ? (uint32_t)ws[n * (K / kMxBlock) + k0 / kMxBlock + unit_w] : 0u;
    };
    uint8_t *const to_wide = wide0 + row_w * 512 + 32 * ((2 * unit_w) ^ grad_turn(row_w));
    const int other = 32 - 64 * (((2 * unit_w) ^ grad_turn(row_w)) & 1);         // to the unit's second half
    auto expand = [&](int slot, uint32_t byte) __attribute__((always_inline)) {
        const v4u c = *reinterpret_cast<const v4u *>(raw0 + slot * L::kRaw + 16 * tid);
        const float scale = mx_scale(byte);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v4u v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = expand2(c[q], scale, j);
            *reinterpret_cast<v4u *>(to_wide + slot * L::kWide + (q >> 1) * other + 16 * (q & 1)) = v;
        }
    };

    v4f32 acc[WK][WM];
#pragma unroll
    for (int i = 0; i < WK; ++i)
#pragma unroll
        for (int j = 0; j < WM; ++j) acc[i][j] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
    v8bf fw[WK], fd[2][WM];
    // weights: segment 8 wk + i of row 8 lg + r / 4 of a step, and of the row four on
    const uint32_t turned = 32 * ((8 * wk) ^ grad_turn(8 * lg + (r >> 2))) + 8 * (r & 3) + 512 * (8 * lg + (r >> 2));
    auto read_w = [&](int slot, int half, int i) __attribute__((always_inline)) {
        const uint8_t *p = wide0 + (turned ^ (32 * i)) + slot * L::kWide + half * (32 * 512);
        const v4s lo = read_turned(p), hi = read_turned(p + 4 * 512);
        fw[i] = __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    const uint8_t *const at_d0 = smem + 128 * (16 * WM * wm + r) + 16 * (lg ^ grad_swizzle(r));
    const uint8_t *const at_d1 = smem + 128 * (16 * WM * wm + r) + 16 * ((4 + lg) ^ grad_swizzle(r));
    auto read_d = [&](int slot, int half, int j) __attribute__((always_inline)) {
        fd[half][j] = *reinterpret_cast<const v8bf *>((half ? at_d1 : at_d0) + slot * L::kD + 2048 * j);
    };

    // prologue: d's tiles 0 and 1 (but two copies), 4-bit rows of stages s0 .. s0 + 2
    const int tiles = (s1 - s0) * parts;
    copy_w(s0);
    uint32_t byte = scale_of(s0);
    open_d(s0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) copy_d(0, i);
    wait_vmem<0>();
    ring_barrier();
    expand(s0 & 1, byte);
    byte = 0;
    uint32_t byte_next = 0;
    if (s0 + 1 < s1) {
        copy_w(s0 + 1);
        byte = scale_of(s0 + 1);
    }
    wait_vmem<0>();
    ring_barrier();                                  // expanded, and stage s0's 4-bit rows read
    if (s0 + 2 < s1) {
        copy_w(s0 + 2);
        byte_next = scale_of(s0 + 2);
    }
    int ahead_s = parts > 1 ? s0 : s0 + 1, ahead_p = parts > 1 ? 1 : 0;          // the tile after this one
    open_d(ahead_s, ahead_p);
#pragma unroll
    for (int i = 0; i < 4; ++i) copy_d(1, i);
#pragma unroll
    for (int i = 0; i < WK; ++i) read_w(s0 & 1, 0, i);
#pragma unroll
    for (int j = 0; j < WM; ++j) read_d(0, 0, j);

    constexpr int kLead = 2;                         // column tiles multiplied before the barrier
    int s = s0, p = 0;
    for (int t = 0; t < tiles; ++t) {
        const int slot = t & 1, ws_slot = s & 1;
        auto products = [&](int half, int i) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < WM; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[i], fd[half][j], acc[i][j], 0, 0, 0);
        };
        // first step: the second's fragments, and the next stage's weights
#pragma unroll
        for (int j = 0; j < WM; ++j) read_d(slot, 1, j);
#pragma unroll
        for (int i = 0; i < WK; ++i) {
            products(0, i);
            read_w(ws_slot, 1, i);
            if (i == 0 && p == 0 && s + 1 < s1) expand(ws_slot ^ 1, byte);
        }
        __builtin_amdgcn_sched_barrier(0);
        // second step
#pragma unroll
        for (int i = 0; i < kLead; ++i) products(1, i);
        __builtin_amdgcn_sched_barrier(0);
        const bool turn = p + 1 == parts;
        const int s_next = turn ? s + 1 : s;
        wait_vmem<0>();                              // the next tile of d, 4-bit rows s + 2
        ring_barrier();                              // for all waves; d's slot is read, s + 1 expanded
        if (turn) {
            byte = byte_next;
            if (s + 3 < s1) {
                copy_w(s + 3);
                byte_next = scale_of(s + 3);
            }
        }
        ++ahead_p;
        if (ahead_p == parts) {
            ahead_p = 0;
            ++ahead_s;
        }
        open_d(ahead_s, ahead_p);
#pragma unroll
        for (int j = 0; j < WM; ++j) read_d(slot ^ 1, 0, j);
#pragma unroll
        for (int i = 0; i < kLead; ++i) read_w(s_next & 1, 0, i);
#pragma unroll
        for (int i = kLead; i < WK; ++i) {
            products(1, i);
            read_w(s_next & 1, 0, i);
            if (i - kLead < 4) copy_d(slot, i - kLead);
        }
        __builtin_amdgcn_sched_barrier(0);
        s = s_next;
        p = turn ? 0 : p + 1;
    }
    wait_vmem<0>();                                  // no copy may land after the block ends
    end_grad<L>(o, plan, share, acc, wave, lane);
}

// A launch holds fewer than 2^32 threads: the kernels go round again.
unsigned blocks_of(int64_t threads) {
    const int64_t b = (threads + 255) / 256;
    return (unsigned)(b < (1 << 22) ? b : 1 << 22);
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Whether d is read where it lies: bfloat16 rows of whole 16-byte units.
bool in_place(int64_t N, int format) { return format == kBf16 && N % 8 == 0; }

typedef GradTile<4, 2, 2, 2> GradSmall;    // 128 x 64

// The tile for a shape: the least of plan_tiles's counts.
bool choose_wide(int64_t M, int64_t N, int64_t K, int parts, size_t bytes, MxPlan &plan) {
    const int64_t stages = (N + kStep - 1) / kStep;
    const MxCost s = plan_tiles<GradSmall>(M, K, stages, bytes, parts), w = plan_tiles<GradWide>(M, K, stages, bytes, parts);
    plan = w.ns <= s.ns ? w.plan : s.plan;
    return w.ns <= s.ns;
}

template <class L>
hipError_t run_grad(const GradRows &d, const Mx4GradArgs &a, MxPlan p, void *work, hipStream_t stream) {
    p.part = static_cast<float *>(work);
    const GradOut o{a.dx, a.format, a.M, a.N, a.K};
    if constexpr (std::is_same<L, GradWide>::value)
        hipLaunchKernelGGL(grad_wide_kernel, dim3(plan_blocks(p)), dim3(L::T), L::kLdsBytes, stream, d, a.w, a.ws, o, p);
    else
        hipLaunchKernelGGL(grad_kernel<L>, dim3(plan_blocks(p)), dim3(L::T), L::kLdsBytes, stream, d, a.w, a.ws, o, p);
    const hipError_t e = hipGetLastError();
    const int rest = p.tiles_n * p.tiles_m - p.full;
    if (e != hipSuccess || rest == 0) return e;
    hipLaunchKernelGGL(grad_sum_kernel<L>, dim3((unsigned)(rest * (L::WK / 4))), dim3(L::T), 0, stream, o, p);
    return hipGetLastError();
}

template <int FMT>
hipError_t run_rows(const Mx4GradArgs &a, void *dgu, uint16_t *out, int64_t cols, hipStream_t stream) {
    const int64_t F = a.gu ? a.N / 2 : a.N;
    const int64_t n = a.M * (F + (out ? cols - a.N : 0));
    const dim3 grid(blocks_of(n)), block(256);
    if (a.gu)
        hipLaunchKernelGGL((grad_rows_kernel<FMT, true>), grid, block, 0, stream, a.dy, a.gu, dgu,
                           a.act, out, a.M, a.N, cols, parts_of(FMT));
    else
        hipLaunchKernelGGL((grad_rows_kernel<FMT, false>), grid, block, 0, stream, a.dy, nullptr,
                           nullptr, 0, out, a.M, a.N, cols, parts_of(FMT));
    return hipGetLastError();
}

}  // namespace

size_t mx4_grad_least_bytes(int64_t M, int64_t N, int format, bool gated, bool keeps_dgu) {
    if (in_place(N, format)) return gated && !keeps_dgu ? (size_t)round_up(M * N * 2, 256) : 0;
    return (size_t)round_up(parts_of(format) * M * round_up(N, kStep) * 2, 256);
}

size_t mx4_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int format, bool gated,
                                bool keeps_dgu) {
    MxPlan p;
    const bool wide = choose_wide(M, N, K, parts_of(format), SIZE_MAX, p);
    return mx4_grad_least_bytes(M, N, format, gated, keeps_dgu) + (wide ? part_bytes<GradWide>(p) : part_bytes<GradSmall>(p));
}

hipError_t launch_mx4_grad(const Mx4GradArgs &a, void *work, size_t work_bytes, hipStream_t stream) {
    const size_t least = mx4_grad_least_bytes(a.M, a.N, a.format, a.gu != nullptr, a.dgu != nullptr);
    uint16_t *const rows = static_cast<uint16_t *>(work);
    GradRows d;
    d.parts = parts_of(a.format);
    d.n = a.N;
    hipError_t e = hipSuccess;
    if (in_place(a.N, a.format)) {
        d.cols = a.N;
        d.plane = 0;
        d.d = static_cast<const uint16_t *>(a.dy);
        if (a.gu) {
            void *dgu = a.dgu ? a.dgu : rows;
            e = run_rows<kBf16>(a, dgu, nullptr, a.N, stream);
            d.d = static_cast<const uint16_t *>(dgu);
        }
    } else {
        d.cols = round_up(a.N, kStep);
        d.plane = a.M * d.cols;
        d.d = rows;
        d.n = d.cols;
        e = a.format == kF32 ? run_rows<kF32>(a, a.dgu, rows, d.cols, stream)
          : a.format == kBf16 ? run_rows<kBf16>(a, a.dgu, rows, d.cols, stream)
                              : run_rows<kF16>(a, a.dgu, rows, d.cols, stream);
    }
    if (e != hipSuccess) return e;
    MxPlan p;
    const bool wide = choose_wide(a.M, a.N, a.K, d.parts, work_bytes - least, p);
    void *const sums = p.ways > 1 ? static_cast<uint8_t *>(work) + least : nullptr;
    return wide ? run_grad<GradWide>(d, a, p, sums, stream) : run_grad<GradSmall>(d, a, p, sums, stream);
}

}  // namespace pq2
