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

constexpr int parts_of(int format) { return format == kBf16 ? 1 : format == kF16 ? 2 : 3; }

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

// V columns of one row of d as its parts, from element `at` of the first on.
template <int FMT, int V>
__device__ __forceinline__ void store_parts(uint16_t *out, int64_t at, int64_t plane, float (&v)[V]) {
#pragma unroll
    for (int p = 0; p < parts_of(FMT); ++p) {
        uint16_t h[V];
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = FMT == kBf16 ? bf16_rne(v[i]) : take_part(v[i]);   // one part: exact
        uint16_t *to = out + at + p * plane;
        if constexpr (V == 8) {
            v4u o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = (uint32_t)h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
            *reinterpret_cast<v4u *>(to) = o;
        } else {
            *to = h[0];
        }
    }
}

// V values of a row (V = 8: from a 16-byte address on).
template <int FMT, int V>
__device__ __forceinline__ void load_values(const void *x, int64_t at, float (&v)[V]) {
    typedef typename MxType<FMT>::T T;
    const T *from = static_cast<const T *>(x) + at;
    if constexpr (V == 1) {
        v[0] = widen<FMT>(*from);
    } else if constexpr (FMT == kF32) {
        const v4f32 lo = *reinterpret_cast<const v4f32 *>(from), hi = *reinterpret_cast<const v4f32 *>(from + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = lo[i];
            v[4 + i] = hi[i];
        }
    } else {
        const v4u two = *reinterpret_cast<const v4u *>(from);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = widen<FMT>((uint16_t)(two[i] & 0xffffu));
            v[2 * i + 1] = widen<FMT>((uint16_t)(two[i] >> 16));
        }
    }
}

// Rounds v to the format, and stores it where x is given.
template <int FMT, int V>
__device__ __forceinline__ void round_values(void *x, int64_t at, float (&v)[V]) {
    typedef typename MxType<FMT>::T T;
    T t[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        t[i] = narrow<FMT>(v[i]);
        v[i] = widen<FMT>(t[i]);
    }
    if (!x) return;
    T *to = static_cast<T *>(x) + at;
    if constexpr (V == 1) {
        *to = t[0];
    } else if constexpr (FMT == kF32) {
        *reinterpret_cast<v4f32 *>(to) = v4f32{t[0], t[1], t[2], t[3]};
        *reinterpret_cast<v4f32 *>(to + 4) = v4f32{t[4], t[5], t[6], t[7]};
    } else {
        v4u o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = (uint32_t)t[2 * i] | ((uint32_t)t[2 * i + 1] << 16);
        *reinterpret_cast<v4u *>(to) = o;
    }
}

// What multiplies the weights: d's parts, for a gated block from dh, g and u, whose
// dgu it writes too (dgu may be gu). V columns a thread: eight where rows of F
// columns keep 16-byte addresses (2048 x 17408 bfloat16 116 us one by one, TODO by
// eight); the columns behind d's last, up to a whole stage, are zeros. A block is
// 2^span threads wide, the others of its 256 take rows below.
template <int FMT, bool GATED, int V>
__global__ __launch_bounds__(256) void grad_rows_kernel(const void *dy, const void *gu, void *dgu,
                                                        int act, uint16_t *out, int64_t M,
                                                        int64_t N, int64_t cols, int span) {
    const int64_t F = GATED ? N / 2 : N;         // columns of dy
    const int64_t c = (((int64_t)blockIdx.x << span) + (threadIdx.x & ((1 << span) - 1))) * V;
    if (c >= F + (out ? cols - N : 0)) return;
    const int64_t rows = 256 >> span;
    for (int64_t m = (int64_t)blockIdx.y * rows + (threadIdx.x >> span); m < M; m += gridDim.y * rows) {
        float v[V];
        if (c >= F) {                            // padding
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = 0.0f;
            store_parts<FMT, V>(out, m * cols + N + (c - F), M * cols, v);
            continue;
        }
        load_values<FMT, V>(dy, m * F + c, v);
        if constexpr (GATED) {
            float g[V], u[V], dg[V], du[V];
            load_values<FMT, V>(gu, 2 * m * F + c, g);
            load_values<FMT, V>(gu, (2 * m + 1) * F + c, u);
            auto run = [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float a, s;
                    gate_act_slope<kind.value>(g[e], a, s);
                    dg[e] = v[e] * u[e] * s;
                    du[e] = v[e] * a;
                }
            };
            if (act == kSilu)
                run(std::integral_constant<int, kSilu>());
            else if (act == kGelu)
                run(std::integral_constant<int, kGelu>());
            else
                run(std::integral_constant<int, kGeluTanh>());
            round_values<FMT, V>(dgu, 2 * m * F + c, dg);
            round_values<FMT, V>(dgu, (2 * m + 1) * F + c, du);
            if (out) {
                store_parts<FMT, V>(out, m * cols + c, M * cols, dg);
                store_parts<FMT, V>(out, m * cols + F + c, M * cols, du);
            }
        } else {
            store_parts<FMT, V>(out, m * cols + c, M * cols, v);
        }
    }
}

// ---------------------------------------------------------------- product
//
// A block owns BN columns of dx x BM tokens, NWK x NWM waves of WK x WM
// instruction tiles. A stage is 64 n of one part of d: d's tile and the weights
// as bfloat16, rows n of BN values, in two LDS slots each. Both come through
// registers, loaded a stage before they are stored: a thread expands 32 values
// under one scale (sixteen conversions) while others multiply. (Buffer -> LDS
// copies do not go with the transposing LDS reads: the compiler waits for every
// copy in flight before such a read; 4096 x 5120 x 17408 in 1009 us instead of
// TODO.) The instruction wants, for a column k, eight consecutive n: the
// transposing read takes them out of four rows at a time. The 32-byte segment seg
// of row n lies at place seg ^ turn(n), so that the four (and eight) rows of such a
// read are in different banks.
// A step is one instruction's 32 n, two a stage. What a step multiplies was read
// from LDS during the step before, tokens into the other of two register sets,
// weights rolling, each tile's registers taking the next step's as soon as its
// products are issued. In the first step of a stage the next stage's tile is
// stored and the one after requested; a barrier in the second shows it to all.
// TODO figures
template <int WK_, int WM_, int NWK_, int NWM_>
struct GradTile {
    static constexpr int WK = WK_, WM = WM_, NWK = NWK_, NWM = NWM_;
    static constexpr int W = NWK * NWM, T = kWave * W;
    static constexpr int BN = 16 * WK * NWK, BM = 16 * WM * NWM;
    static constexpr int kD = BM * 128;                  // bytes of a tile of d
    static constexpr int kWide = kStep * BN * 2;
    static constexpr int kLdsBytes = 2 * (kD + kWide);
    static constexpr int kRows = BM / 8 / W;             // 16-byte pieces of d's tile a thread moves
    static constexpr int kUnits = BN / 32;               // blocks of scales in a row of the tile
    static constexpr bool kTwo = W == 8;                 // two waves a SIMD (wide)
    static constexpr int kBlocks = kTwo ? 1 : 3;         // a compute unit holds
    static constexpr int kRun = kTwo ? 1770 : 640, kMore = kTwo ? 80 : 540,
                         kEnds = kTwo ? 5000 : 2500;               // plan_tiles's times
    static_assert(kRows * W * 8 == BM && kStep * kUnits == T, "a thread expands one block");
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
    constexpr int NI = 1, kCuts = L::WK / NI;
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
__global__ __launch_bounds__(L::T) __attribute__((amdgpu_waves_per_eu(2)))
void grad_kernel(GradRows d, const uint8_t *__restrict__ w, const uint8_t *__restrict__ ws, GradOut o, MxPlan plan) {
    constexpr int WK = L::WK, WM = L::WM, W = L::W, NR = L::kRows;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint8_t *const wide0 = smem + 2 * L::kD;
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

    // d: piece i of a wave is rows 8 (i W + wave) .., each with a resource of the
    // rows that exist and one lane offset for all
    const int sub = lane >> 3, unit = (lane & 7) ^ grad_swizzle(sub);
    const int row_bytes = (int)(d.cols * 2);
    int bytes_d[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int rows = rows_m - 8 * (i * W + wave);
        bytes_d[i] = __builtin_amdgcn_readfirstlane((rows < 0 ? 0 : rows > 8 ? 8 : rows) * row_bytes);
    }
    const int off = sub * row_bytes + 16 * unit;
    const uint16_t *const base_d = d.d + (m0 + 8 * wave) * d.cols;
    v4u held[NR];                                    // the tile of d after the next
    auto load_d = [&](int s, int p) __attribute__((always_inline)) {
        const uint16_t *from = base_d + p * d.plane + (int64_t)s * kStep;
        const int at = s < s1 && (int64_t)s * kStep + 8 * unit < d.n ? off : kCopyOob;
#pragma unroll
        for (int i = 0; i < NR; ++i)
            held[i] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(
                make_rsrc(from + (int64_t)i * (8 * W) * d.cols, bytes_d[i]), at, 0, 0));
    };
    auto store_d = [&](int slot) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NR; ++i)
            *reinterpret_cast<v4u *>(smem + slot * L::kD + (i * W + wave) * 1024 + 16 * lane) = held[i];
    };
    // weights: the thread expands block unit_w of row row_w of a stage
    const int kb = (int)(K / 2), row_w = tid / L::kUnits, unit_w = tid % L::kUnits;
    const bool live_w = 32 * unit_w < cols;
    v4u codes;
    uint32_t byte;
    auto load_w = [&](int s) __attribute__((always_inline)) {
        const int64_t n0 = (int64_t)s * kStep;
        const int rows = s < s1 ? (int)(N - n0 < kStep ? N - n0 : kStep) : 0;
        const bool live = live_w && row_w < rows;
        const int64_t first = rows ? n0 : 0;
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(w + first * kb + k0 / 2, rows ? (int64_t)(rows - 1) * kb + cols / 2 : 0);
        codes = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(
            rs, live ? row_w * kb + 16 * unit_w : kCopyOob, 0, 0));
        const int sb = kb / 16;
        const __amdgpu_buffer_rsrc_t rss =
            make_rsrc(ws + first * sb + k0 / kMxBlock, rows ? (int64_t)(rows - 1) * sb + cols / kMxBlock : 0);
        byte = __builtin_amdgcn_raw_buffer_load_b8(rss, live ? row_w * sb + unit_w : kCopyOob, 0, 0);
    };
    // 16-byte piece q of the block goes to place q ^ turn of its 64 bytes in the
    // row; the lanes write their pieces in the order q ^ order, so that eight of
    // them fill 128 bytes at a time (in one order 32 clocks a store, so 14)
    const int order = (unit_w >> 1) & 3, turn_w = grad_turn(row_w);
    const uint32_t to_wide = row_w * (2 * L::BN) + 64 * (unit_w ^ (turn_w >> 1)) + 16 * (order ^ (2 * (turn_w & 1)));
    auto expand = [&](int slot) __attribute__((always_inline)) {
        const float scale = mx_scale(byte & 0xffu);
        const bool odd = order & 1, high = order & 2;
        const uint32_t c0 = odd ? codes[1] : codes[0], c1 = odd ? codes[0] : codes[1];
        const uint32_t c2 = odd ? codes[3] : codes[2], c3 = odd ? codes[2] : codes[3];
        const v4u c = {high ? c2 : c0, high ? c3 : c1, high ? c0 : c2, high ? c1 : c3};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v4u v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = expand2(c[q], scale, j);
            *reinterpret_cast<v4u *>(wide0 + slot * L::kWide + (to_wide ^ (16 * q))) = v;
        }
    };

    v4f32 acc[WK][WM];
#pragma unroll
    for (int i = 0; i < WK; ++i)
#pragma unroll
        for (int j = 0; j < WM; ++j) acc[i][j] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
    v8bf fw[WK], fd[2][WM];
    // weights: segment WK wk + i of row 8 lg + r / 4 of a step, and of the row four
    // on; WK wk + i and i differ in bits that turn() leaves alone or by an XOR too
    const int row_t = 8 * lg + (r >> 2);
    const uint32_t turned = 32 * ((WK * wk) ^ grad_turn(row_t)) + 8 * (r & 3) + 2 * L::BN * row_t;
    auto read_w = [&](int slot, int half, int i) __attribute__((always_inline)) {
        const uint8_t *p = wide0 + (turned ^ (32 * i)) + slot * L::kWide + half * (64 * L::BN);
        const v4s lo = read_turned(p), hi = read_turned(p + 8 * L::BN);
        fw[i] = __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    const uint8_t *const at_d0 = smem + 128 * (16 * WM * wm + r) + 16 * (lg ^ grad_swizzle(r));
    const uint8_t *const at_d1 = smem + 128 * (16 * WM * wm + r) + 16 * ((4 + lg) ^ grad_swizzle(r));
    auto read_d = [&](int slot, int half, int j) __attribute__((always_inline)) {
        fd[half][j] = *reinterpret_cast<const v8bf *>((half ? at_d1 : at_d0) + slot * L::kD + 2048 * j);
    };

    load_d(s0, 0);
    load_w(s0);
    store_d(0);
    expand(s0 & 1);
    int ahead_s = parts > 1 ? s0 : s0 + 1, ahead_p = parts > 1 ? 1 : 0;          // the tile that is held
    load_d(ahead_s, ahead_p);
    load_w(s0 + 1);
    ring_barrier();
#pragma unroll
    for (int i = 0; i < WK; ++i) read_w(s0 & 1, 0, i);
#pragma unroll
    for (int j = 0; j < WM; ++j) read_d(0, 0, j);

    constexpr int kLead = WK / 4;                    // column tiles multiplied before the barrier
    int s = s0, p = 0;
    for (int t = 0; s < s1; ++t) {
        const int slot = t & 1, slot_w = s & 1;
        auto products = [&](int half, int i) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < WM; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[i], fd[half][j], acc[i][j], 0, 0, 0);
        };
        // first step
#pragma unroll
        for (int j = 0; j < WM; ++j) read_d(slot, 1, j);
#pragma unroll
        for (int i = 0; i < WK; ++i) {
            products(0, i);
            read_w(slot_w, 1, i);
            // wide: the two waves of a SIMD, wave and wave + W / 2, not at once (684 -> 645
            // us at 2048 x 34816 x 5120). Small: a block has one wave on each
            if (i == 0 ? !L::kTwo || wave < W / 2 : L::kTwo && i == WK / 2 && wave >= W / 2) {
                __builtin_amdgcn_sched_barrier(0);
                store_d(slot ^ 1);
                ++ahead_p;
                if (ahead_p == parts) {
                    ahead_p = 0;
                    ++ahead_s;
                }
                load_d(ahead_s, ahead_p);
                // in a stage's first tile or in its last, as measured: wide 616 us at 4096 x
                // 5120 x 17408 (628 in the last), small 116 at 128 x 5120 x 17408 float32 (134)
                if (L::kTwo ? p == 0 : p + 1 == parts) {
                    expand(slot_w ^ 1);
                    load_w(s + 2);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // second step
#pragma unroll
        for (int i = 0; i < kLead; ++i) products(1, i);
        __builtin_amdgcn_sched_barrier(0);
        ring_barrier();                              // the next tile is there, this one is read
        const bool turn = p + 1 == parts;
        const int next_w = (turn ? s + 1 : s) & 1;
#pragma unroll
        for (int j = 0; j < WM; ++j) read_d(slot ^ 1, 0, j);
#pragma unroll
        for (int i = 0; i < kLead; ++i) read_w(next_w, 0, i);
#pragma unroll
        for (int i = kLead; i < WK; ++i) {
            products(1, i);
            read_w(next_w, 0, i);
        }
        __builtin_amdgcn_sched_barrier(0);
        s += turn;
        p = turn ? 0 : p + 1;
    }
    end_grad<L>(o, plan, share, acc, wave, lane);
}

// A launch holds fewer than 2^32 threads: the kernels go round again.
int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Whether d is read where it lies: bfloat16 rows of whole 16-byte units.
bool in_place(int64_t N, int format) { return format == kBf16 && N % 8 == 0; }

typedef GradTile<8, 4, 2, 4> GradWide;     // 256 x 256
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
    hipLaunchKernelGGL(grad_kernel<L>, dim3(plan_blocks(p)), dim3(L::T), L::kLdsBytes, stream, d, a.w, a.ws, o, p);
    const hipError_t e = hipGetLastError();
    const int rest = p.tiles_n * p.tiles_m - p.full;
    if (e != hipSuccess || rest == 0) return e;
    hipLaunchKernelGGL(grad_sum_kernel<L>, dim3((unsigned)(rest * L::WK)), dim3(L::T), 0, stream, o, p);
    return hipGetLastError();
}

template <int FMT, bool GATED, int V>
hipError_t launch_rows(const Mx4GradArgs &a, void *dgu, uint16_t *out, int64_t cols, hipStream_t stream) {
    const int64_t F = GATED ? a.N / 2 : a.N, width = (F + (out ? cols - a.N : 0)) / V;
    int span = 0;
    while (span < 8 && (1 << span) < width) ++span;
    const int64_t across = (width + (1 << span) - 1) >> span, down = (a.M + (256 >> span) - 1) / (256 >> span);
    int64_t most = (1 << 22) / across;               // a launch holds fewer than 2^32 threads: rows go round again
    most = most < 65535 ? most : 65535;
    hipLaunchKernelGGL((grad_rows_kernel<FMT, GATED, V>),
                       dim3((unsigned)across, (unsigned)(down < most ? down : most)), dim3(256), 0, stream, a.dy,
                       a.gu, dgu, a.act, out, a.M, a.N, cols, span);
    return hipGetLastError();
}

template <int FMT>
hipError_t run_rows(const Mx4GradArgs &a, void *dgu, uint16_t *out, int64_t cols, hipStream_t stream) {
    const bool eight = (a.gu ? a.N / 2 : a.N) % 8 == 0;     // bases are 16-byte aligned, cols whole stages
    if (a.gu)
        return eight ? launch_rows<FMT, true, 8>(a, dgu, out, cols, stream)
                     : launch_rows<FMT, true, 1>(a, dgu, out, cols, stream);
    return eight ? launch_rows<FMT, false, 8>(a, dgu, out, cols, stream)
                 : launch_rows<FMT, false, 1>(a, dgu, out, cols, stream);
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
