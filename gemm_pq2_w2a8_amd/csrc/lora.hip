// lora.hip -- low-rank adapters of many requests beside a shared projection.
//
// Row m uses adapter l = adapter[m] (none when outside [0, L)):
//   v[m] = A[l] x[m]                      (shrink: K -> rank)
//   y[m] = base[m] + scale[l] * B[l] v[m] (expand: rank -> N)
// Two launches: the shrink leaves its sums in the caller's workspace (float32,
// one copy per K chunk), the expand adds the chunks in order, multiplies by B
// and adds to the base.
//
// Both products run on the matrix cores in 16 x 16 tiles, 16 consecutive rows
// at a time. Rows of a tile may have different adapters: the tile's distinct
// adapters are walked one by one, each with all 16 rows as operand, and only
// the results of the adapter's own rows are kept (selected, not multiplied by
// zero: another adapter's infinities or NaN stay with its rows).
//
// Operands that are not both bfloat16 (or both binary16) are split exactly into
// bfloat16 parts of 8 significant bits -- a binary16 value into two, a float32
// into three -- and the parts' products added; products of parts below 2^-24 of
// the whole are left out. v stays float32 this way, so the rank dimension costs
// no accuracy.
#include "pq2_device.hpp"
#include "pq2_launch.hpp"

namespace pq2 {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kShrinkRanks = 64;         // ranks of one shrink block (4 tiles)

enum { kF32 = 0, kBf16 = 1, kF16 = 2 };  // PQ2_ACT_*

// Parts an operand of a type is split into for bfloat16 products.
template <int FMT>
constexpr int kParts = FMT == kF32 ? 3 : FMT == kF16 ? 2 : 1;

__device__ __forceinline__ v4f mfma_bf16(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma_f16(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Eight float32 values as N exact bfloat16 parts, largest first: each part is
// the upper half of what is left, the rest an exact difference.
template <int N>
__device__ __forceinline__ void split8(const float (&v)[8], v4u (&part)[N]) {
    float rest[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) rest[e] = v[e];
#pragma unroll
    for (int p = 0; p < N; ++p) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const uint32_t lo = __builtin_bit_cast(uint32_t, rest[2 * d]);
            const uint32_t hi = __builtin_bit_cast(uint32_t, rest[2 * d + 1]);
            part[p][d] = (lo >> 16) | (hi & 0xffff0000u);
            if (p + 1 < N) {
                rest[2 * d] -= __builtin_bit_cast(float, lo & 0xffff0000u);
                rest[2 * d + 1] -= __builtin_bit_cast(float, hi & 0xffff0000u);
            }
        }
    }
}

// Eight consecutive 16-bit values as bfloat16 parts.
template <int FMT>
__device__ __forceinline__ void parts_of(v4u raw, v4u (&part)[kParts<FMT>]) {
    if constexpr (FMT == kBf16) {
        part[0] = raw;
    } else {
        float v[8];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const uint32_t u = raw[d];
            v[2 * d] = half_bits_to_float((uint16_t)(u & 0xffffu));
            v[2 * d + 1] = half_bits_to_float((uint16_t)(u >> 16));
        }
        split8(v, part);
    }
}

// Sum of the parts' products (a's parts times b's), without those below 2^-24.
template <int NA, int NB>
__device__ __forceinline__ v4f mfma_parts(const v4u (&a)[NA], const v4u (&b)[NB], v4f c) {
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (i + j < 3) c = mfma_bf16(a[i], b[j], c);
    return c;
}

// The adapters of the 16 rows from m0: this lane's row lane % 16 (-1: none, or
// past M).
__device__ __forceinline__ int row_adapter(const LoraArgs &p, int64_t m0, int r) {
    if (m0 + r >= p.M) return -1;
    const int id = p.adapter[m0 + r];
    return id >= 0 && id < p.L ? id : -1;
}

// Takes the next distinct adapter off `left` (a bit per row): its id, and the
// rows that have it.
__device__ __forceinline__ int next_adapter(int id_of_row, uint32_t &left, uint32_t &mine) {
    const int id = __builtin_amdgcn_readlane(id_of_row, __builtin_ctz(left));
    mine = (uint32_t)__ballot(id_of_row == id) & 0xffffu;
    left &= ~mine;
    return id;
}

__device__ __forceinline__ int rank_of(const LoraArgs &p, int id) {
    const int R = (int)p.R;
    return p.ranks ? min(max(p.ranks[id], 0), R) : R;
}

// Shrink: a block sums one K chunk of 16 rows x 64 ranks; its four waves take a
// quarter of the chunk each and meet in LDS, added in wave order.
template <int XF, int WF>
__global__ __launch_bounds__(256) void lora_shrink_kernel(LoraArgs p, float *__restrict__ v,
                                                          int64_t chunk) {
    constexpr int T = kShrinkRanks / 16;
    __shared__ v4f part[4][T][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int r = lane & 15, c = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * 16;
    const int r0 = (int)blockIdx.z * kShrinkRanks;
    const int64_t k0 = (int64_t)blockIdx.y * chunk;
    const int64_t k1 = k0 + chunk < p.K ? k0 + chunk : p.K;
    const int64_t quarter = (k1 - k0) / 4;                 // a multiple of 32
    const int64_t kw = k0 + wave * quarter + 8 * c;
    const int64_t m = m0 + r < p.M ? m0 + r : p.M - 1;
    const int id_of_row = row_adapter(p, m0, r);
    uint32_t left = (uint32_t)__ballot(id_of_row >= 0) & 0xffffu, mine;
    v += (int64_t)blockIdx.y * p.M * p.R;
    while (left) {
        const int id = next_adapter(id_of_row, left, mine);
        const int rank = rank_of(p, id);
        if (r0 >= rank) continue;
        v4f acc[T] = {};
        for (int64_t k = kw; k < kw + quarter; k += 32) {
            v4u xr[XF == kF32 ? 2 : 1];
            const char *xs = static_cast<const char *>(p.x) + (m * p.K + k) * (XF == kF32 ? 4 : 2);
#pragma unroll
            for (int i = 0; i < (XF == kF32 ? 2 : 1); ++i)
                xr[i] = *reinterpret_cast<const v4u *>(xs + 16 * i);
            v4u xp[kParts<XF>];
            if constexpr (XF == kF32) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t u = xr[e >> 2][e & 3];
                    f[e] = __builtin_bit_cast(float, u);
                }
                split8(f, xp);
            } else if constexpr (XF != WF) {
                parts_of<XF>(xr[0], xp);
            }
#pragma unroll
            for (int j = 0; j < T; ++j) {
                if (r0 + 16 * j >= rank) continue;
                // ranks past R are read from the last one; their sums are not kept
                const int row = min(r0 + 16 * j + r, (int)p.R - 1);
                const v4u w = *reinterpret_cast<const v4u *>(
                    static_cast<const uint16_t *>(p.a) + ((int64_t)id * p.R + row) * p.K + k);
                if constexpr (XF == WF && WF == kBf16) {
                    acc[j] = mfma_bf16(xr[0], w, acc[j]);
                } else if constexpr (XF == WF) {
                    acc[j] = mfma_f16(xr[0], w, acc[j]);
                } else {
                    v4u wp[kParts<WF>];
                    parts_of<WF>(w, wp);
                    acc[j] = mfma_parts(xp, wp, acc[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < T; ++j) part[wave][j][lane] = acc[j];
        __syncthreads();
        // wave j stores rank tile j: rank r0 + 16 j + r of rows 4 c + i
        v4f sum = part[0][wave][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) sum += part[w][wave][lane];
        const int rk = r0 + 16 * wave + r;
        if (rk < rank) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (mine >> (4 * c + i) & 1) v[(m0 + 4 * c + i) * p.R + rk] = sum[i];
        }
        __syncthreads();
    }
}

// Drops the values of a vector of eight from element `keep` on.
__device__ __forceinline__ v4u keep_first(v4u w, int keep) {
#pragma unroll
    for (int d = 0; d < 4; ++d)
        w[d] = keep >= 2 * d + 2 ? w[d] : keep == 2 * d + 1 ? (w[d] & 0xffffu) : 0u;
    return w;
}

// Expand: a wave forms 16 rows x 16 columns of y.
template <int WF, int YF>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs p, const float *__restrict__ v,
                                                          int chunks) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int r = lane & 15, c = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * 16;
    const int64_t n0 = ((int64_t)blockIdx.y * 4 + wave) * 16;
    if (n0 >= p.N) return;
    const int64_t n = n0 + r < p.N ? n0 + r : p.N - 1;
    const int64_t m = m0 + r < p.M ? m0 + r : p.M - 1;
    const int id_of_row = row_adapter(p, m0, r);
    uint32_t left = (uint32_t)__ballot(id_of_row >= 0) & 0xffffu, mine;
    const uint32_t some = left;
    v4f out = {};
    while (left) {
        const int id = next_adapter(id_of_row, left, mine);
        const int rank = rank_of(p, id);
        const float scale = p.scale ? p.scale[id] : 1.0f;
        const bool own = mine >> r & 1;
        v4f acc = {};
        for (int k0 = 0; k0 < rank; k0 += 32) {
            const int k = k0 + 8 * c;
            const int keep = rank - k;                     // ranks of this lane's vector
            float f[8] = {};
            v4u w = {};
            if (keep > 0) {
                w = *reinterpret_cast<const v4u *>(
                    static_cast<const uint16_t *>(p.b) + ((int64_t)id * p.N + n) * p.R + k);
                w = keep_first(w, keep);
                if (own) {
                    const float *src = v + m * p.R + k;
                    for (int s = 0; s < chunks; ++s, src += p.M * p.R) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float4 u = *reinterpret_cast<const float4 *>(src + 4 * h);
                            f[4 * h] += u.x;
                            f[4 * h + 1] += u.y;
                            f[4 * h + 2] += u.z;
                            f[4 * h + 3] += u.w;
                        }
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = e < keep ? f[e] * scale : 0.0f;
            v4u vp[3], wp[kParts<WF>];
            split8(f, vp);
            parts_of<WF>(w, wp);
            acc = mfma_parts(vp, wp, acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (mine >> (4 * c + i) & 1) out[i] = acc[i];
    }
    if (n0 + r >= p.N) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (m0 + 4 * c + i >= p.M) continue;
        const int64_t at = (m0 + 4 * c + i) * p.N + n0 + r;
        const bool add = some >> (4 * c + i) & 1;
        if (!add && p.base == p.y) continue;
        if constexpr (YF == kF32) {
            const float b = static_cast<const float *>(p.base)[at];
            static_cast<float *>(p.y)[at] = add ? b + out[i] : b;
        } else {
            const uint16_t u = static_cast<const uint16_t *>(p.base)[at];
            const float b = __builtin_bit_cast(float, (uint32_t)u << 16);
            static_cast<uint16_t *>(p.y)[at] = add ? bf16_rne(b + out[i]) : u;
        }
    }
}

// K chunks of the shrink: about 512 blocks in all, at least 512 of K each.
int plan_chunks(int64_t M, int64_t K) {
    const int64_t tiles = (M + 15) / 16;
    int64_t s = 512 / tiles;
    const int64_t most = (K + 511) / 512 < 16 ? (K + 511) / 512 : 16;
    if (s > most) s = most;
    return s < 1 ? 1 : (int)s;
}

template <int XF, int WF>
void launch_shrink(const LoraArgs &a, float *v, int64_t chunk, dim3 grid, hipStream_t stream) {
    hipLaunchKernelGGL((lora_shrink_kernel<XF, WF>), grid, dim3(256), 0, stream, a, v, chunk);
}

template <int WF, int YF>
void launch_expand(const LoraArgs &a, const float *v, int chunks, hipStream_t stream) {
    const dim3 grid((unsigned)((a.M + 15) / 16), (unsigned)((a.N + 63) / 64));
    hipLaunchKernelGGL((lora_expand_kernel<WF, YF>), grid, dim3(256), 0, stream, a, v, chunks);
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t R) {
    return (size_t)plan_chunks(M, K) * (size_t)M * (size_t)R * sizeof(float);
}

hipError_t launch_lora(const LoraArgs &a, int x_format, int w_format, int y_format, float *work,
                       size_t work_bytes, hipStream_t stream) {
    const size_t per = (size_t)a.M * (size_t)a.R * sizeof(float);
    int64_t chunks = plan_chunks(a.M, a.K);
    if ((uint64_t)chunks > work_bytes / per) chunks = (int64_t)(work_bytes / per);
    // chunks are whole groups of 128 (a quarter is whole MFMA steps of 32)
    const int64_t chunk = (a.K / 128 + chunks - 1) / chunks * 128;
    chunks = (a.K + chunk - 1) / chunk;
    const dim3 grid((unsigned)((a.M + 15) / 16), (unsigned)chunks,
                    (unsigned)((a.R + kShrinkRanks - 1) / kShrinkRanks));
    const bool wb = w_format == kBf16;
    if (x_format == kF32)
        wb ? launch_shrink<kF32, kBf16>(a, work, chunk, grid, stream)
           : launch_shrink<kF32, kF16>(a, work, chunk, grid, stream);
    else if (x_format == kBf16)
        wb ? launch_shrink<kBf16, kBf16>(a, work, chunk, grid, stream)
           : launch_shrink<kBf16, kF16>(a, work, chunk, grid, stream);
    else
        wb ? launch_shrink<kF16, kBf16>(a, work, chunk, grid, stream)
           : launch_shrink<kF16, kF16>(a, work, chunk, grid, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (y_format == kF32)
        wb ? launch_expand<kBf16, kF32>(a, work, (int)chunks, stream)
           : launch_expand<kF16, kF32>(a, work, (int)chunks, stream);
    else
        wb ? launch_expand<kBf16, kBf16>(a, work, (int)chunks, stream)
           : launch_expand<kF16, kBf16>(a, work, (int)chunks, stream);
    return hipGetLastError();
}

}  // namespace pq2
