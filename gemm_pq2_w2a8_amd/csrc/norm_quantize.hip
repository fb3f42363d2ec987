// norm_quantize.hip -- the norms after and before a block, with the block's
// gate and residual scale, ending in the per-128-group int8 quantiser.
//
// Per row m (rms(v) = v / sqrt(mean(v^2) + eps)):
//   p = w_post ? rms(x) * w_post : x
//   h = residual + alpha * gate * p          (residual and gate optional)
//   n = w_pre ? rms(h) * w_pre : h
//   q, s, t = the quantiser's rule on n      (quantize_groups8)
// Everything between the loads and the stores is float32: h is rounded to x's
// type only where it is stored and n is formed from the unrounded h, so the
// stored h costs the norm behind it no accuracy.
//
// One block per row; 8 lanes per group, lane j holding elements
// 16 j .. 16 j + 15 (the quantiser's 8-lane layout), so the row stays in
// registers between the two norms and every array is read and written once.
// Rows too long for that (K > 32768) are read again in each of three sweeps,
// each element always by the thread that stores it.
// 4096 x 5120 bfloat16 with both norms and a residual: 45 us, where its 148 MB
// need 30 at a large copy's rate. Neither memory nor issue is full: 648 vector
// instructions a wave keep the SIMDs 56 % busy, and the waves wait for 59 % of
// their time, since a row's phases follow one another -- its loads, the first
// reduction, w_post, the second reduction, w_pre (whose wait, behind the
// conditional store of h, is for that store too), the quantiser -- and a block
// requests nothing of a next row meanwhile. A single row is the latency of one
// block, two reductions deep (5120: 4.4 us).
#include "pq2_device.hpp"
#include "pq2_launch.hpp"

namespace pq2 {

namespace {

constexpr int kNormMaxThreads = 1024;
constexpr int64_t kNormMaxBlocks = int64_t(1) << 22;   // rows beyond: blocks loop

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// 16 consecutive elements as loaded (float32: four 16-byte words; bfloat16 or
// binary16: two).
template <int FMT>
struct Raw16 {
    v4u w[FMT == 0 ? 4 : 2];
};

template <int FMT>
__device__ __forceinline__ void load16(const void *p, int64_t i, Raw16<FMT> &r) {
    const v4u *src = reinterpret_cast<const v4u *>(static_cast<const char *>(p) + i * (FMT == 0 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < (FMT == 0 ? 4 : 2); ++k) r.w[k] = src[k];
}

template <int FMT>
__device__ __forceinline__ float element(const Raw16<FMT> &r, int e) {
    if constexpr (FMT == 0) {
        const uint32_t u = r.w[e >> 2][e & 3];   // (a bit cast of the vector element itself reads element 0)
        return __builtin_bit_cast(float, u);
    } else {
        const uint32_t u = r.w[e >> 3][(e >> 1) & 3];
        if constexpr (FMT == 1)
            return __builtin_bit_cast(float, (e & 1) ? (u & 0xffff0000u) : (u << 16));
        else
            return half_bits_to_float((uint16_t)((e & 1) ? (u >> 16) : (u & 0xffffu)));
    }
}

// v rounded to nearest even in the format, stored at element i.
template <int FMT>
__device__ __forceinline__ void store16(void *p, int64_t i, const float (&v)[16]) {
    v4u *dst = reinterpret_cast<v4u *>(static_cast<char *>(p) + i * (FMT == 0 ? 4 : 2));
    if constexpr (FMT == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v4u o;
#pragma unroll
            for (int c = 0; c < 4; ++c) o[c] = __builtin_bit_cast(uint32_t, v[4 * k + c]);
            dst[k] = o;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            v4u o;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float a = v[8 * k + 2 * c], b = v[8 * k + 2 * c + 1];
                if constexpr (FMT == 1) {
                    const v2bf t = {(__bf16)a, (__bf16)b};   // v_cvt_pk_bf16_f32
                    o[c] = __builtin_bit_cast(uint32_t, t);
                } else {
                    const v2h t = {(_Float16)a, (_Float16)b};
                    o[c] = __builtin_bit_cast(uint32_t, t);
                }
            }
            dst[k] = o;
        }
    }
}

// Sum over the block, the same bits on every thread: waves by lane exchange,
// their sums through LDS in wave order. `red` is not reused before every
// thread has passed another barrier.
__device__ __forceinline__ float block_sum(float v, float *red) {
    v = segment_sum<64>(v);
    const int waves = blockDim.x / kWave;
    if (waves == 1) return v;
    if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = v;
    __syncthreads();
    float s = red[0];
    for (int w = 1; w < waves; ++w) s += red[w];
    return s;
}

// 16 elements of value 1, or -0, in a format.
template <int FMT>
__device__ __forceinline__ void fill(Raw16<FMT> &r, uint32_t w) {
#pragma unroll
    for (int k = 0; k < (FMT == 0 ? 4 : 2); ++k) r.w[k] = v4u{w, w, w, w};
}
template <int FMT>
__device__ __forceinline__ void ones(Raw16<FMT> &r) {
    fill(r, FMT == 0 ? 0x3f800000u : FMT == 1 ? 0x3f803f80u : 0x3c003c00u);
}
template <int FMT>
__device__ __forceinline__ void minus_zeros(Raw16<FMT> &r) {
    fill(r, FMT == 0 ? 0x80000000u : 0x80008000u);
}

// h of 16 elements: residual + alpha * gate * (x * scale * w_post). What the
// call leaves out is 1 (weights, gate, scale) or -0 (residual) here, which
// changes no bit of what is left (+0 would turn a -0 into a +0) and keeps the
// elements free of branches.
template <int FMT>
__device__ __forceinline__ void form_h(float alpha, const Raw16<FMT> &x, const Raw16<FMT> &r,
                                       const Raw16<FMT> &gt, const Raw16<0> &wp, float scale,
                                       float (&h)[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
        h[e] = fmaf(alpha, element<FMT>(x, e) * scale * element<0>(wp, e) * element<FMT>(gt, e),
                    element<FMT>(r, e));
}

// Stores of one group's 16 elements: h, n and the quantised group. Called by
// every lane (the quantiser exchanges lanes); `live` lanes store.
template <int FMT>
__device__ __forceinline__ void finish(const NormArgs &a, int64_t m, int g, int j, bool live,
                                       const float (&h)[16], const Raw16<0> &wq, float scale) {
    const int64_t at = m * a.K + (int64_t)g * kGroup + 16 * j;
    if (a.h && live) store16<FMT>(a.h, at, h);
    float n[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) n[e] = h[e] * scale * element<0>(wq, e);
    if (a.n && live) store16<FMT>(a.n, at, n);
    if (!a.q) return;
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float4(n[4 * i], n[4 * i + 1], n[4 * i + 2], n[4 * i + 3]);
    uint32_t word[4];
    float sc;
    int sum;
    quantize_groups8(v, word, sc, sum);
    if (!live) return;
    int8_t *q = a.q + m * a.K + (int64_t)g * kGroup;
#pragma unroll
    for (int p = 0; p < 4; ++p) *reinterpret_cast<uint32_t *>(q + 32 * p + 4 * j) = word[p];
    if (j == 0) {
        const int64_t gg = m * (a.K / kGroup) + g;
        a.s[gg] = sc;
        a.t[gg] = sum;
    }
}

// NR groups per 8-lane slot held in registers; NR = 0: any K, re-reading.
template <int FMT, int NR>
__global__ __launch_bounds__(kNormMaxThreads) void norm_quantize_kernel(NormArgs a) {
    __shared__ float red_post[kNormMaxThreads / kWave], red_pre[kNormMaxThreads / kWave];
    const int slots = blockDim.x / 8, slot = threadIdx.x / 8, j = threadIdx.x & 7;
    const int G = (int)(a.K / kGroup);
    const float inv_k = 1.0f / (float)a.K;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const int64_t row = m * a.K;
        const int64_t gate_row = a.gate ? m / a.rows_per_gate * a.K : 0;
        float scale_post = 1.0f, scale_pre = 1.0f;
        // what the row needs beside x, of group g
        auto load_rest = [&](int g, Raw16<FMT> &r, Raw16<FMT> &gt) __attribute__((always_inline)) {
            const int64_t k = (int64_t)g * kGroup + 16 * j;
            if (a.residual) load16<FMT>(a.residual, row + k, r);
            if (a.gate) load16<FMT>(a.gate, gate_row + k, gt);
        };
        auto load_weights = [&](const float *w, int g, Raw16<0> &o) __attribute__((always_inline)) {
            if (w) load16<0>(w, (int64_t)g * kGroup + 16 * j, o);
        };
        if constexpr (NR > 0) {
            // The row goes out at once, the weights where they are used: 86
            // registers leave five waves a SIMD, with the weights among the first
            // loads it is 109 and four (4096 x 5120 bfloat16, both norms and a
            // residual: 45.5 us against 55.5; one row: 5.0 both ways). With two
            // groups per slot only x fits in registers beside h.
            Raw16<FMT> x[NR] = {}, r, gt;
            Raw16<0> wp, wq;
            minus_zeros(r);
            ones<FMT>(gt);
            ones<0>(wp);
            ones<0>(wq);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int g = slot + i * slots;
                if (g >= G) continue;
                load16<FMT>(a.x, row + (int64_t)g * kGroup + 16 * j, x[i]);
                if (NR == 1) load_rest(g, r, gt);
            }
            if (a.w_post) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < NR; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) ss = fmaf(element<FMT>(x[i], e), element<FMT>(x[i], e), ss);
                scale_post = 1.0f / sqrtf(block_sum(ss, red_post) * inv_k + a.eps);
            }
            float h[NR][16];
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int g = slot + i * slots;
                if (NR > 1) {
                    minus_zeros(r);
                    if (g < G) load_rest(g, r, gt);
                }
                if (g < G) load_weights(a.w_post, g, wp);
                form_h<FMT>(a.alpha, x[i], r, gt, wp, scale_post, h[i]);
                if (g < G) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) ss = fmaf(h[i][e], h[i][e], ss);
                }
            }
            if (a.w_pre) scale_pre = 1.0f / sqrtf(block_sum(ss, red_pre) * inv_k + a.eps);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int g = slot + i * slots;
                if (g < G) load_weights(a.w_pre, g, wq);
                finish<FMT>(a, m, g, j, g < G, h[i], wq, scale_pre);
            }
        } else {
            if (a.w_post) {
                float ss = 0.0f;
                for (int g = slot; g < G; g += slots) {
                    Raw16<FMT> x;
                    load16<FMT>(a.x, row + (int64_t)g * kGroup + 16 * j, x);
#pragma unroll
                    for (int e = 0; e < 16; ++e) ss = fmaf(element<FMT>(x, e), element<FMT>(x, e), ss);
                }
                scale_post = 1.0f / sqrtf(block_sum(ss, red_post) * inv_k + a.eps);
            }
            // sweep 0 sums h^2, sweep 1 stores; slots walk together (the
            // quantiser exchanges lanes), those past the end idle along
            float ss = 0.0f;
            for (int sweep = a.w_pre ? 0 : 1; sweep < 2; ++sweep) {
                for (int g0 = 0; g0 < G; g0 += slots) {
                    const int g = g0 + slot;
                    const bool live = g < G;
                    const int at = live ? g : G - 1;
                    Raw16<FMT> x, r, gt;
                    Raw16<0> wp, wq;
                    minus_zeros(r);
                    ones<FMT>(gt);
                    ones<0>(wp);
                    ones<0>(wq);
                    load16<FMT>(a.x, row + (int64_t)at * kGroup + 16 * j, x);
                    load_rest(at, r, gt);
                    load_weights(a.w_post, at, wp);
                    float h[16];
                    form_h<FMT>(a.alpha, x, r, gt, wp, scale_post, h);
                    if (sweep == 0) {
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) ss = fmaf(h[e], h[e], ss);
                        }
                    } else {
                        load_weights(a.w_pre, at, wq);
                        finish<FMT>(a, m, g, j, live, h, wq, scale_pre);
                    }
                }
                if (sweep == 0) scale_pre = 1.0f / sqrtf(block_sum(ss, red_pre) * inv_k + a.eps);
            }
        }
        if (m + gridDim.x < a.M) __syncthreads();   // red_* are written again
    }
}

template <int FMT>
hipError_t launch_norm(const NormArgs &a, hipStream_t stream) {
    const int64_t G = a.K / kGroup;
    const int max_slots = kNormMaxThreads / 8;
    const int nr = G <= max_slots ? 1 : G <= 2 * max_slots ? 2 : 0;
    const int64_t slots = nr ? (G + nr - 1) / nr : max_slots;
    const unsigned threads = (unsigned)((slots * 8 + kWave - 1) / kWave * kWave);
    const dim3 grid((unsigned)(a.M < kNormMaxBlocks ? a.M : kNormMaxBlocks));
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, stream, a);
    };
    if (nr == 0)
        launch(norm_quantize_kernel<FMT, 0>);
    else if (nr == 2)
        launch(norm_quantize_kernel<FMT, 2>);
    else
        launch(norm_quantize_kernel<FMT, 1>);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_quantize(const NormArgs &a, int format, hipStream_t stream) {
    if (format == 1) return launch_norm<1>(a, stream);
    if (format == 2) return launch_norm<2>(a, stream);
    return launch_norm<0>(a, stream);
}

}  // namespace pq2
