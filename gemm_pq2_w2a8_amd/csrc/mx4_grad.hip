// mx4_grad.hip -- gradients through MX4 weights (gfx950): the input's gradient
// of the product, and the gated feed-forward block's backward pass.
//
//   dx[m][k] = sum_n d[m][n] w[n][k]
//   gated:  du = dh act(g),  dg = dh u act'(g),  d = (dg | du), n over 2 F
//
// The sum runs along n, across the weights' blocks of scales, so the weights
// are expanded to bfloat16, in which every one of them is exact (subnormal ones
// too; those beyond its range lend d a factor, see split_scale), and multiplied
// by bfloat16 matrix instructions with float32 sums. d enters without a
// rounding of its own: bfloat16 as it is, float16 and float32 split into two
// and three bfloat16 parts that add up to it exactly (truncated, so that no
// part overflows; of a float32 below 2^-110 the bits below bfloat16's last, 2^-133,
// are lost), which run through the same loop as two or three passes over
// d's tiles beside one expansion of the weights.
#include <type_traits>

#include "mx4_launch.hpp"
#include "mx4_plan.hpp"

namespace pq2 {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

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

// v u s with a slope s (at most 1.13): where the first product overflows although its
// factors are finite, both exceed 1, and with s near 0 the whole may still be finite.
__device__ __forceinline__ float times_slope(float v, float u, float s) {
    const float p = v * u;
    return fabsf(p) == INFINITY && fabsf(v) != INFINITY ? v * (u * s) : p * s;
}

// What multiplies the weights: d's parts, for a gated block from dh, g and u, whose
// dgu it writes too (dgu may be gu). dg and du are rounded to the format before they
// multiply, returned or not, so that dx is the product of the dgu that adapters are
// trained with, the same bits whether a caller keeps it. Unrounded they would be further
// parts: 2048 x 17408 x 5120 bfloat16 takes 688 us, with a second part, as float16 has,
// 1237; dx is off by 0.0023 relative instead of 0.0017, its own rounding's. V columns a
// thread: eight where rows of F columns keep 16-byte addresses (2048 x 17408 bfloat16
// 116 us one by one, 55 by eight, 6.5 TB/s); the columns behind d's last, up to a whole
// stage, are zeros. A block is 2^span threads wide, the others of its 256 take rows below.
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
                    dg[e] = times_slope(v[e], u[e], s);
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
// A block owns BN columns of dx x BM tokens, a wave 32 of the columns (one block of
// scales) and all tokens, so that no two waves expand the same weights. A stage is
// 64 n of one part of d, in two LDS slots: d's tile, and the weights' codes and
// scales (as float32) as they are, rows n of BN codes. All come through registers,
// loaded a stage before they are stored. The instruction wants, for a column k,
// eight consecutive n: the transposing read gives a lane eight rows' bytes of one
// place, which are two columns, 2 r and 2 r + 1, of each row; a conversion makes
// the two bfloat16 values of a byte under its row's scale, a permutation of two
// conversions a pair of n of one column. So an instruction tile holds the 16 even
// columns of a block and the next one the odd, and a lane's results are eight
// columns in a row. The 16-byte unit u of row n lies at place(u, n), so that the 16
// rows that half a wave reads at a time are in different banks.
// A step is one instruction's 32 n, two a stage. What a step multiplies was read
// from LDS during the step before: weights into the other of two register sets,
// tokens rolling, each tile's registers taking the next step's as soon as its
// products are issued. In the first step of a stage the next stage's tile is
// stored and the one after requested; a barrier in the second shows it to all.
// 4096 x 5120 x 17408 bfloat16 576 to 600 us by the clock with 256 x 256 tiles (1.2 to
// 1.27 PFLOP/s; a library product of bfloat16 matrices 1.37 to 1.44); 128 x 34816 x 5120
// 82 with 128 x 64. Every
// other instruction shares the SIMD's issue with the matrix instructions: the loop of
// waves of 64 columns x half the tokens, with parts left out, took 358 us for those
// alone, 99 more with the conversions, 31 with the reads of d, 40 with the stores to
// LDS, 73 with the requests, 17 with their latency, 619 in all. From there scales as
// float32 instead of bytes (no shifts: 608), the waves of 32 columns (half the
// conversions, twice the reads of d: 591), addresses stepped instead of formed anew
// (580) and products at a higher priority (573). Before it, weights expanded to bfloat16 in
// LDS once a block and read transposed from there: 616 and 92 us, LDS and conversions;
// and buffer -> LDS copies, which the compiler waits for before a transposing read:
// 1009 us instead of 708.
template <int WM_, int W_>
struct GradTile {
    static constexpr int WM = WM_, W = W_, T = kWave * W;
    static constexpr int BN = 32 * W, BM = 16 * WM;
    static constexpr int kD = BM * 128;                  // bytes of a tile of d
    static constexpr int kRow = BN / 2;                  // bytes of a row n of codes
    static constexpr int kScales = 4 * kStep + 32;    // bytes of a block's scales, one for each n
    static constexpr int kSlot = kStep * kRow + W * kScales;
    static constexpr int kOver = 2 * (kD + kSlot);       // whether the block met a scale beyond 2^125
    static constexpr int kLdsBytes = kOver + 16;
    static constexpr int kRows = BM / 8 / W;             // 16-byte pieces of d's tile a thread moves
    static constexpr bool kTwo = W == 8;                 // two waves a SIMD (wide)
    static constexpr int kBlocks = kTwo ? 1 : WM == 4 ? 3 : 5;    // a compute unit holds
    static constexpr int kRun = kTwo ? 1450 : WM == 4 ? 490 : 440, kMore = kTwo ? 170 : WM == 4 ? 390 : 900,
                         kEnds = kTwo ? 5000 : 2500;     // plan_tiles's times
    static constexpr int kNJ = WM < 4 ? 1 : WM / 4;     // instruction tiles of tokens a block sums
    static_assert(kRows * W * 8 == BM && kStep * W == T && kSlot % 16 == 0, "a thread moves one block");

    // where unit u of row n of the codes lies in the row
    static __device__ __forceinline__ int place(int u, int n) { return u ^ (W == 8 ? (n >> 1) & 7 : (n >> 2) & 3); }
};

__device__ __forceinline__ int grad_swizzle(int row) { return row & 6; }

// Eight codes of one place 2 c, 2 c + 1 of eight rows (byte j: row j's pair), under
// the rows' scales (byte j: row j's): the column of the even places and of the odd.
// The conversion takes its scale's exponent bits alone.
template <int J>
__device__ __forceinline__ uint32_t expand2(v2u codes, const v4f32 (&scales)[2]) {
    const float scale = scales[J / 4][J % 4];
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[J / 4], scale, J % 4));
}

template <int J>
__device__ __forceinline__ void expand4(v2u codes, const v4f32 (&scales)[2], v4u &even, v4u &odd) {
    const uint32_t a = expand2<2 * J>(codes, scales), b = expand2<2 * J + 1>(codes, scales);
    even[J] = __builtin_amdgcn_perm(b, a, 0x05040100u);
    odd[J] = __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// Scales beyond 2^125 make weights that bfloat16 does not hold. A wave's weights of a
// row n are one block, so such a row can be expanded under 2^125 and the rest of its
// scale, 2 or 4, multiply the row's values of d. The exponent of that rest lies in the
// low bits of the scale, which the conversions do not read. 255 (NaN) stays.
constexpr uint32_t kTopByte = 252;
__device__ __forceinline__ bool is_over(uint32_t byte) { return byte - (kTopByte + 1) < 2u; }
__device__ __forceinline__ uint32_t split_scale(uint32_t byte) {
    return is_over(byte) ? kTopByte << 23 | (byte - kTopByte) : byte << 23;
}

// The exponents of the rests of eight rows' scales, two bits each.
__device__ __forceinline__ uint32_t rests_of(const v4f32 (&scales)[2]) {
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) all |= (bits_of(scales[i / 4][i % 4]) & 3u) << (2 * i);
    return all;
}

// Eight values of d by their rows' rests. A finite one that overflows becomes the
// largest finite one: by a weight of 2^124 or more it is infinite all the same, by 0
// it is 0.
__device__ __forceinline__ v8bf lifted(v8bf d, uint32_t rests) {
    v4u w = __builtin_bit_cast(v4u, d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t out = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float x = as_float(h ? w[i] & 0xffff0000u : w[i] << 16);
            uint32_t b = bits_of(ldexpf(x, (int)(rests >> (2 * (2 * i + h)) & 3u)));
            if ((b & 0x7fffffffu) == 0x7f800000u && fabsf(x) != INFINITY) b = (b & 0x80000000u) | 0x7f7f0000u;
            out |= h ? b & 0xffff0000u : b >> 16;
        }
        w[i] = out;
    }
    return __builtin_bit_cast(v8bf, w);
}

// Sixteen bytes of eight rows, transposed: lane i of 16 gives the address of eight
// bytes of row i / 2 and gets byte i of all eight rows.
__device__ __forceinline__ v2u read_turned(const uint8_t *p) {
    typedef int v2i __attribute__((ext_vector_type(2)));
    typedef __attribute__((address_space(3))) v2i lds_v2i;
    return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)p));
}

// acc[0][j], acc[1][j]: the even and the odd ones of eight columns from
// k + 8 (lane / 16) on, token m + 16 j.
template <int NJ>
__device__ __forceinline__ void finish_dx(const v4f32 (&acc)[2][NJ], void *dx, int format, int64_t k, int64_t m,
                                          int64_t M, int64_t K, int lane) {
    const bool wide = (reinterpret_cast<uintptr_t>(dx) & 15) == 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int64_t t = m + 16 * j;
        if (t >= M) continue;
        const int64_t c = k + 8 * (lane >> 4), at = t * K + c;
        if (c >= K) continue;                        // K is a multiple of 32
        const v4f32 e = acc[0][j], o = acc[1][j];
        if (wide && format == kF32) {
            *reinterpret_cast<v4f32 *>(static_cast<float *>(dx) + at) = v4f32{e[0], o[0], e[1], o[1]};
            *reinterpret_cast<v4f32 *>(static_cast<float *>(dx) + at + 4) = v4f32{e[2], o[2], e[3], o[3]};
        } else if (wide) {
            *reinterpret_cast<v4u *>(static_cast<uint16_t *>(dx) + at) =
                v4u{pack16(format, e[0], o[0]), pack16(format, e[1], o[1]), pack16(format, e[2], o[2]),
                    pack16(format, e[3], o[3])};
        } else {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                store_fmt(dx, format, at + 2 * x, e[x]);
                store_fmt(dx, format, at + 2 * x + 1, o[x]);
            }
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
                                         const v4f32 (&acc)[2][L::WM], int wave, int lane) {
    const int64_t m = (int64_t)s.tm * L::BM;
    if (!s.split)
        finish_dx(acc, o.dx, o.format, (int64_t)s.tn * L::BN + 32 * wave, m + (lane & 15), o.M, o.K, lane);
    else
        store_share<2, L::WM, L::T>(p, s.item, wave * kWave + lane, (int)(o.M - m < L::BM ? (o.M - m + 15) / 16 : L::WM),
                                    acc);
}

template <class L>
__global__ __launch_bounds__(L::T) void grad_sum_kernel(GradOut o, MxPlan p) {
    constexpr int NJ = L::kNJ, kCuts = L::WM / NJ;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;
    const int index = (int)blockIdx.x / kCuts, j0 = (int)blockIdx.x % kCuts * NJ;
    int tn, tm;
    tile_at(p, p.full + index, tn, tm);
    const int64_t m = (int64_t)tm * L::BM + 16 * j0;
    if (m >= o.M) return;
    v4f32 acc[2][NJ];
    sum_shares<2, L::WM, L::T>(p, index, 0, j0, tid, acc);
    finish_dx(acc, o.dx, o.format, (int64_t)tn * L::BN + 32 * wave, m + (lane & 15), o.M, o.K, lane);
}

template <class L>
__global__ __launch_bounds__(L::T) __attribute__((amdgpu_waves_per_eu(2)))
void grad_kernel(GradRows d, const uint8_t *__restrict__ w, const uint8_t *__restrict__ ws, GradOut o, MxPlan plan) {
    constexpr int WM = L::WM, W = L::W, NR = L::kRows;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint8_t *const codes0 = smem + 2 * L::kD;
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, lg = lane >> 4;
    const MxShare share = share_of(plan);
    if (!share.live) return;
    int *const met = reinterpret_cast<int *>(smem + L::kOver);
    if (tid == 0) *met = 0;
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
    const uint16_t *next_d = base_d + (int64_t)s0 * kStep;       // the tile that is loaded next
    const int64_t turn_d = kStep - (parts - 1) * d.plane;
    auto load_d = [&](int s, int p) __attribute__((always_inline)) {
        const uint16_t *from = next_d;
        next_d += p + 1 == parts ? turn_d : d.plane;
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
    // weights: the thread moves block unit_w of row row_w of a stage, and its scale
    const int kb = (int)(K / 2), row_w = tid / W, unit_w = tid % W;
    const bool live_w = 32 * unit_w < cols;
    v4u codes;
    uint32_t byte;
    bool over = false;                               // a scale of the thread's was
    const uint8_t *next_w = w + (int64_t)s0 * kStep * kb + k0 / 2;
    const uint8_t *next_s = ws + (int64_t)s0 * kStep * (kb / 16) + k0 / kMxBlock;
    auto load_w = [&](int s) __attribute__((always_inline)) {
        const int64_t n0 = (int64_t)s * kStep;
        const int rows = s < s1 ? (int)(N - n0 < kStep ? N - n0 : kStep) : 0;
        const bool live = live_w && row_w < rows;
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(next_w, rows * kb);
        codes = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(
            rs, live ? row_w * kb + 16 * unit_w : kCopyOob, 0, 0));
        const int sb = kb / 16;
        const __amdgpu_buffer_rsrc_t rss = make_rsrc(next_s, rows * sb);
        next_w += kStep * kb;
        next_s += kStep * sb;
        byte = __builtin_amdgcn_raw_buffer_load_b8(rss, live ? row_w * sb + unit_w : kCopyOob, 0, 0);
    };
    const uint32_t to_codes = row_w * L::kRow + 16 * L::place(unit_w, row_w);
    const uint32_t to_scale = kStep * L::kRow + unit_w * L::kScales + 4 * row_w;
    auto store_w = [&](int slot) __attribute__((always_inline)) {
        *reinterpret_cast<v4u *>(codes0 + slot * L::kSlot + to_codes) = codes;
        *reinterpret_cast<uint32_t *>(codes0 + slot * L::kSlot + to_scale) = byte << 23;
        over |= is_over(byte);
    };

    v4f32 acc[2][WM];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < WM; ++j) acc[i][j] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
    v4u fw[2][2];                                    // of a step, and of the next
    v8bf fd[WM];
    // weights: rows 8 lg .. of a step, columns of block `wave`
    v2u raw;
    v4f32 scales[2];
    const int row_t = 8 * lg + (r >> 1);
    const uint8_t *const at_w = codes0 + row_t * L::kRow + 16 * L::place(wave, row_t) + 8 * (r & 1);
    const uint8_t *const at_s = codes0 + kStep * L::kRow + wave * L::kScales + 32 * lg;
    auto read_w = [&](int slot, int half) __attribute__((always_inline)) {
        raw = read_turned(at_w + slot * L::kSlot + half * (32 * L::kRow));
        scales[0] = *reinterpret_cast<const v4f32 *>(at_s + slot * L::kSlot + 128 * half);
        scales[1] = *reinterpret_cast<const v4f32 *>(at_s + slot * L::kSlot + 128 * half + 16);
    };
    auto expand = [&](int half) __attribute__((always_inline)) {
        expand4<0>(raw, scales, fw[half][0], fw[half][1]);
        expand4<1>(raw, scales, fw[half][0], fw[half][1]);
        expand4<2>(raw, scales, fw[half][0], fw[half][1]);
        expand4<3>(raw, scales, fw[half][0], fw[half][1]);
    };
    const uint8_t *const at_d0 = smem + 128 * r + 16 * (lg ^ grad_swizzle(r));
    const uint8_t *const at_d1 = smem + 128 * r + 16 * ((4 + lg) ^ grad_swizzle(r));
    auto read_d = [&](int slot, int half, int j) __attribute__((always_inline)) {
        fd[j] = *reinterpret_cast<const v8bf *>((half ? at_d1 : at_d0) + slot * L::kD + 2048 * j);
    };

    load_d(s0, 0);
    load_w(s0);
    store_d(0);
    store_w(s0 & 1);
    int ahead_s = parts > 1 ? s0 : s0 + 1, ahead_p = parts > 1 ? 1 : 0;          // the tile that is held
    load_d(ahead_s, ahead_p);
    load_w(s0 + 1);
    ring_barrier();
    read_w(s0 & 1, 0);
#pragma unroll
    for (int j = 0; j < WM; ++j) read_d(0, 0, j);
    expand(0);

    constexpr int kLead = WM / 4;                 // token tiles multiplied before the barrier
    int s = s0, p = 0;
    for (int t = 0; s < s1; ++t) {
        const int slot = t & 1, slot_w = s & 1;
        const bool turn = p + 1 == parts;            // the next tile is of the next stage
        auto products = [&](int half, int j) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, fw[half][i]), fd[j],
                                                                    acc[i][j], 0, 0, 0);
        };
        // first step
        read_w(slot_w, 1);
#pragma unroll
        for (int j = 0; j < WM; ++j) {
            __builtin_amdgcn_s_setprio(1);           // this wave's products before the other's rest
            products(0, j);
            __builtin_amdgcn_s_setprio(0);
            read_d(slot, 1, j);
            // wide: the two waves of a SIMD, wave and wave + W / 2, not at once. Small: a
            // block has one wave on each
            if (j == 0 ? !L::kTwo || wave < W / 2 : L::kTwo && j == WM / 2 && wave >= W / 2) {
                __builtin_amdgcn_sched_barrier(0);
                store_d(slot ^ 1);
                ++ahead_p;
                if (ahead_p == parts) {
                    ahead_p = 0;
                    ++ahead_s;
                }
                load_d(ahead_s, ahead_p);
                if (turn) {
                    store_w(slot_w ^ 1);
                    load_w(s + 2);
                }
            }
        }
        expand(1);
        __builtin_amdgcn_sched_barrier(0);
        // second step
#pragma unroll
        for (int j = 0; j < kLead; ++j) products(1, j);
        __builtin_amdgcn_sched_barrier(0);
        ring_barrier();                              // the next tile is there, this one is read
        read_w((turn ? s + 1 : s) & 1, 0);
#pragma unroll
        for (int j = 0; j < kLead; ++j) read_d(slot ^ 1, 0, j);
#pragma unroll
        for (int j = kLead; j < WM; ++j) {
            __builtin_amdgcn_s_setprio(1);
            products(1, j);
            __builtin_amdgcn_s_setprio(0);
            read_d(slot ^ 1, 0, j);
        }
        expand(0);
        __builtin_amdgcn_sched_barrier(0);
        s += turn;
        p = turn ? 0 : p + 1;
    }
    // A scale beyond 2^125, which the quantiser does not write: the whole sum again, one
    // tile at a time, with the rests on d. The loop above only notes that there was one
    // (4096 x 5120 x 17408 594 -> 599 us; lifting d in that loop, in a branch, spilled 64
    // of its registers).
    if (__any(over) && lane == 0) *met = 1;          // cleared before the first barrier
    ring_barrier();
    if (__builtin_amdgcn_readfirstlane(*met)) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < WM; ++j) acc[i][j] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
        next_d = base_d + (int64_t)s0 * kStep;
        next_w = w + (int64_t)s0 * kStep * kb + k0 / 2;
        next_s = ws + (int64_t)s0 * kStep * (kb / 16) + k0 / kMxBlock;
        for (s = s0; s < s1; ++s) {
            load_w(s);
            for (p = 0; p < parts; ++p) {
                load_d(s, p);
                ring_barrier();                      // the last tile is read
                store_d(0);
                if (p == 0) {
                    *reinterpret_cast<v4u *>(codes0 + to_codes) = codes;
                    *reinterpret_cast<uint32_t *>(codes0 + to_scale) = split_scale(byte);
                }
                ring_barrier();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    read_w(0, half);
                    expand(half);
                    const uint32_t rests = rests_of(scales);
#pragma unroll
                    for (int j = 0; j < WM; ++j) {
                        read_d(0, half, j);
                        fd[j] = lifted(fd[j], rests);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(v8bf, fw[half][i]), fd[j], acc[i][j], 0, 0, 0);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
        }
    }
    end_grad<L>(o, plan, share, acc, wave, lane);
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Whether d is read where it lies: bfloat16 rows of whole 16-byte units.
bool in_place(int64_t N, int format) { return format == kBf16 && N % 8 == 0; }

typedef GradTile<16, 8> GradWide;     // 256 x 256
typedef GradTile<4, 4> GradSmall;    // 128 x 64
typedef GradTile<2, 4> GradFew;      // 128 x 32

// f(a tile's type, its plan) for a shape's tile: the small one's or the wide one's,
// the less of plan_tiles's counts; where 32 tokens are all, the one that holds no
// more, five blocks a unit instead of three (16 x 5120 x 17408 float32 38 us instead of
// 50; bfloat16 16 x 34816 x 5120 36 instead of 42 with weights in the caches, 47 instead
// of 48 without; 64 x 5120 x 17408, two tiles down, 33 instead of 29).
template <class F>
auto with_tile(int64_t M, int64_t N, int64_t K, int parts, size_t bytes, F f) {
    const int64_t stages = (N + kStep - 1) / kStep;
    if (M <= GradFew::BM) return f(GradFew(), plan_tiles<GradFew>(M, K, stages, bytes, parts).plan);
    const MxCost small = plan_tiles<GradSmall>(M, K, stages, bytes, parts),
                 wide = plan_tiles<GradWide>(M, K, stages, bytes, parts);
    return wide.ns <= small.ns ? f(GradWide(), wide.plan) : f(GradSmall(), small.plan);
}

template <class L>
hipError_t run_grad(const GradRows &d, const Mx4GradArgs &a, MxPlan p, void *work, hipStream_t stream) {
    p.part = static_cast<float *>(work);
    const GradOut o{a.dx, a.format, a.M, a.N, a.K};
    hipLaunchKernelGGL(grad_kernel<L>, dim3(plan_blocks(p)), dim3(L::T), L::kLdsBytes, stream, d, a.w, a.ws, o, p);
    const hipError_t e = hipGetLastError();
    const int rest = p.tiles_n * p.tiles_m - p.full;
    if (e != hipSuccess || rest == 0) return e;
    hipLaunchKernelGGL(grad_sum_kernel<L>, dim3((unsigned)(rest * (L::WM / L::kNJ))), dim3(L::T), 0, stream, o, p);
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
    const bool eight = (a.gu ? a.N / 2 : a.N) % 8 == 0;     // then bases are 16-byte aligned; cols are whole stages
    if (a.gu)
        return eight ? launch_rows<FMT, true, 8>(a, dgu, out, cols, stream)
                     : launch_rows<FMT, true, 1>(a, dgu, out, cols, stream);
    if constexpr (FMT != kBf16)                      // such rows of bfloat16 are read in place
        if (eight) return launch_rows<FMT, false, 8>(a, dgu, out, cols, stream);
    return launch_rows<FMT, false, 1>(a, dgu, out, cols, stream);
}

}  // namespace

size_t mx4_grad_least_bytes(int64_t M, int64_t N, int format, bool gated, bool keeps_dgu) {
    if (in_place(N, format)) return gated && !keeps_dgu ? (size_t)round_up(M * N * 2, 256) : 0;
    return (size_t)round_up(parts_of(format) * M * round_up(N, kStep) * 2, 256);
}

size_t mx4_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int format, bool gated,
                                bool keeps_dgu) {
    return mx4_grad_least_bytes(M, N, format, gated, keeps_dgu) +
           with_tile(M, N, K, parts_of(format), SIZE_MAX, [](auto tile, const MxPlan &p) { return part_bytes<decltype(tile)>(p); });
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
    return with_tile(a.M, a.N, a.K, d.parts, work_bytes - least, [&](auto tile, const MxPlan &p) {
        return run_grad<decltype(tile)>(d, a, p, p.ways > 1 ? static_cast<uint8_t *>(work) + least : nullptr, stream);
    });
}

}  // namespace pq2
