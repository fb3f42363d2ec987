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
#include "mx4_device.hpp"
#include "mx4_launch.hpp"
#include "pq2_launch.hpp"

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
    static constexpr int BK = 16 * WK * NWK, BM = 16 * WM * NWM;
    static constexpr int kD = BM * 128;                  // bytes of a tile of d
    static constexpr int kRaw = kStep * BK / 2;
    static constexpr int kWide = kStep * BK * 2;
    static constexpr int kLdsBytes = 2 * (kD + kRaw + kWide);
    static constexpr int kCopiesM = BM / 8 / W;          // per wave
    static constexpr int kCopiesW = kRaw / 1024 / W;
    static constexpr int kUnits = BK / 32;               // blocks of scales in a row of the tile
    static constexpr int kItems = kStep * kUnits / T;    // expanded by a thread
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

// chunks: the n range is dealt to that many blocks per tile; with more than one
// their float32 sums go to part [chunks][M][K].
template <class L>
__global__ __launch_bounds__(L::T) void grad_kernel(GradRows d, const uint8_t *__restrict__ w,
                                                    const uint8_t *__restrict__ ws, void *dx,
                                                    int format, float *part, int64_t M, int64_t N,
                                                    int64_t K, int tiles_k, int tiles, int chunks) {
    constexpr int WK = L::WK, WM = L::WM, W = L::W;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint8_t *const raw0 = smem + 2 * L::kD, *const wide0 = raw0 + 2 * L::kRaw;
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % L::NWK, wm = wave / L::NWK;
    const int r = lane & 15, lg = lane >> 4;

    const int all = tiles * chunks;
    const int per = (all + 7) / 8;
    const int at = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if (at >= all) return;
    const int tile = at / chunks, chunk = at % chunks;
    const int64_t m0 = (int64_t)(tile / tiles_k) * L::BM;
    const int k0 = (tile % tiles_k) * L::BK;

    // this chunk's stages
    const int stages = (int)((N + kStep - 1) / kStep);
    const int s0 = (int)((int64_t)stages * chunk / chunks), s1 = (int)((int64_t)stages * (chunk + 1) / chunks);
    const int parts = d.parts;

    const int rows_m = (int)(M - m0 < L::BM ? M - m0 : L::BM);
    const int cols = (int)(K - k0 < L::BK ? K - k0 : L::BK);
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
                *reinterpret_cast<v4u *>(to + n * (2 * L::BK) + 32 * seg + 16 * (q & 1)) = o;
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
                const v4s lo = read_turned(wt + n * (2 * L::BK) + 32 * (seg ^ grad_turn(n)) + 8 * (r & 3));
                const v4s hi = read_turned(wt + (n + 4) * (2 * L::BK) + 32 * (seg ^ grad_turn(n + 4)) + 8 * (r & 3));
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

    const bool wide = (reinterpret_cast<uintptr_t>(dx) & (format == kF32 ? 15 : 7)) == 0;
#pragma unroll
    for (int j = 0; j < WM; ++j) {
        const int64_t m = m0 + 16 * (WM * wm + j) + r;
        if (m >= M) continue;
#pragma unroll
        for (int i = 0; i < WK; ++i) {
            const int k = k0 + 16 * (WK * wk + i) + 4 * lg;
            if (k >= K) continue;                // K is a multiple of four
            if (chunks > 1)
                *reinterpret_cast<v4f32 *>(part + ((int64_t)chunk * M + m) * K + k) = acc[i][j];
            else if (wide && format == kF32)
                *reinterpret_cast<v4f32 *>(static_cast<float *>(dx) + m * K + k) = acc[i][j];
            else if (wide)
                *reinterpret_cast<v2u *>(static_cast<uint16_t *>(dx) + m * K + k) =
                    v2u{pack16(format, acc[i][j][0], acc[i][j][1]), pack16(format, acc[i][j][2], acc[i][j][3])};
            else
#pragma unroll
                for (int e = 0; e < 4; ++e) store_fmt(dx, format, m * K + k + e, acc[i][j][e]);
        }
    }
}

// dx of the chunks' sums, added in chunk order.
__global__ __launch_bounds__(256) void grad_sum_kernel(const float *__restrict__ part, void *dx,
                                                       int format, int64_t n, int chunks) {
    for (int64_t i = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x); i < n;
         i += (int64_t)gridDim.x * 1024) {
        v4f32 v = *reinterpret_cast<const v4f32 *>(part + i);
        for (int c = 1; c < chunks; ++c) v += *reinterpret_cast<const v4f32 *>(part + c * n + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) store_fmt(dx, format, i + e, v[e]);
    }
}

// A launch holds fewer than 2^32 threads: the kernels go round again.
unsigned blocks_of(int64_t threads) {
    const int64_t b = (threads + 255) / 256;
    return (unsigned)(b < (1 << 22) ? b : 1 << 22);
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Whether d is read where it lies: bfloat16 rows of whole 16-byte units.
bool in_place(int64_t N, int format) { return format == kBf16 && N % 8 == 0; }

struct GradPlan {
    bool big;
    int chunks;
    int64_t sums;                     // bytes of the chunks' sums
};

GradPlan plan_grad(int64_t M, int64_t N, int64_t K, size_t bytes) {
    GradPlan p;
    const int64_t tiles_big = ((K + 255) / 256) * ((M + 255) / 256);
    p.big = tiles_big >= 192;
    const int64_t tiles = p.big ? tiles_big : ((K + 127) / 128) * ((M + 63) / 64);
    const int64_t stages = (N + kStep - 1) / kStep;
    int64_t c = p.big ? 1 : 512 / tiles;
    c = c < stages / 4 ? c : stages / 4;
    c = c < 16 ? c : 16;
    const int64_t fits = (int64_t)(bytes / ((size_t)M * (size_t)K * sizeof(float)));
    c = c < fits ? c : fits;
    p.chunks = c < 1 ? 1 : (int)c;
    p.sums = p.chunks > 1 ? p.chunks * M * K * (int64_t)sizeof(float) : 0;
    return p;
}

template <class L>
hipError_t run_grad(const GradRows &d, const Mx4GradArgs &a, float *part, int chunks, hipStream_t stream) {
    const int64_t tk = (a.K + L::BK - 1) / L::BK, tm = (a.M + L::BM - 1) / L::BM;
    const int64_t per = (tk * tm * chunks + 7) / 8;
    hipLaunchKernelGGL(grad_kernel<L>, dim3((unsigned)(8 * per)), dim3(L::T), L::kLdsBytes, stream, d,
                       a.w, a.ws, a.dx, a.format, part, a.M, a.N, a.K, (int)tk, (int)(tk * tm), chunks);
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
    return mx4_grad_least_bytes(M, N, format, gated, keeps_dgu) + (size_t)plan_grad(M, N, K, SIZE_MAX).sums;
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
    const GradPlan p = plan_grad(a.M, a.N, a.K, work_bytes - least);
    float *part = p.chunks > 1 ? reinterpret_cast<float *>(static_cast<uint8_t *>(work) + least) : nullptr;
    typedef GradTile<8, 4, 2, 4> Big;
    typedef GradTile<4, 2, 2, 2> Small;
    e = p.big ? run_grad<Big>(d, a, part, p.chunks, stream) : run_grad<Small>(d, a, part, p.chunks, stream);
    if (e != hipSuccess || p.chunks == 1) return e;
    const int64_t n = a.M * a.K;
    hipLaunchKernelGGL(grad_sum_kernel, dim3(blocks_of(n / 4)), dim3(256), 0, stream,
                       part, a.dx, a.format, n, p.chunks);
    return hipGetLastError();
}

}  // namespace pq2
