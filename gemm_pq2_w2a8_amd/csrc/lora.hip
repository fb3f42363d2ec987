// lora.hip -- low-rank adapters of many requests beside a shared projection.
//
// Row m uses adapter l = adapter[m] (none when outside [0, L)):
//   v[m] = A[l] x[m]                      (shrink: K -> rank)
//   y[m] = base[m] + scale[l] * B[l] v[m] (expand: rank -> N)
// Two launches: the shrink leaves its sums in the caller's workspace (float32,
// one copy per K chunk), the expand adds the chunks in order, multiplies by B
// and adds to the base.
//
// Both products run on the matrix cores in 16 x 16 tiles. A block takes up to
// 128 consecutive rows, walks the distinct adapters among them and gathers each
// one's rows into tiles, so an adapter is read once per block however its rows
// are spread, and rows of different adapters never share an MFMA.
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

// The rows m0 .. m0 + rows - 1 (at most 128) of a block and their adapters, two
// rows to a lane. next() gives the distinct adapters one by one, take() lists
// the rows that have one; every wave of a block sees the same sequence.
constexpr int kWindow = 128;

struct Rows {
    int64_t m0;
    int id0, id1;            // adapters of rows lane and 64 + lane; -1: none, -2: past the end
    uint64_t left0, left1;   // rows whose adapter has not been taken
    uint8_t *list;           // the wave's own list in LDS

    __device__ __forceinline__ Rows(const LoraArgs &p, int64_t first, int64_t rows, uint8_t *own)
        : m0(first), list(own) {
        const int lane = threadIdx.x & (kWave - 1);
        auto adapter = [&](int i) __attribute__((always_inline)) {
            if (i >= rows || m0 + i >= p.M) return -2;
            const int id = p.adapter[m0 + i];
            return id >= 0 && id < p.L ? id : -1;
        };
        id0 = adapter(lane);
        id1 = adapter(kWave + lane);
        left0 = __ballot(id0 >= 0);
        left1 = __ballot(id1 >= 0);
    }

    // Lists the rows with this id; their number.
    __device__ __forceinline__ int take(int id) {
        const int lane = threadIdx.x & (kWave - 1);
        const uint64_t a = __ballot(id0 == id), b = __ballot(id1 == id);
        const uint64_t below = (uint64_t(1) << lane) - 1;
        const int n = __popcll(a);
        __builtin_amdgcn_wave_barrier();
        if (id0 == id) list[__popcll(a & below)] = (uint8_t)lane;
        if (id1 == id) list[n + __popcll(b & below)] = (uint8_t)(kWave + lane);
        __builtin_amdgcn_wave_barrier();
        return n + __popcll(b);
    }

    __device__ __forceinline__ bool any() const { return (left0 | left1) != 0; }

    // The next distinct adapter.
    __device__ __forceinline__ int next() {
        const int id = left0 ? __builtin_amdgcn_readlane(id0, __builtin_ctzll(left0))
                             : __builtin_amdgcn_readlane(id1, __builtin_ctzll(left1));
        left0 &= ~__ballot(id0 == id);
        left1 &= ~__ballot(id1 == id);
        return id;
    }

    // Row of entry i of the list (the first one past its end).
    __device__ __forceinline__ int64_t row(int i, int count) const {
        return m0 + list[i < count ? i : 0];
    }
};

__device__ __forceinline__ int rank_of(const LoraArgs &p, int id) {
    const int R = (int)p.R;
    return p.ranks ? min(max(p.ranks[id], 0), R) : R;
}

// Shrink: a block sums one K chunk of its rows x 64 ranks, adapter by adapter,
// 16 * TR rows at a time; its eight waves share the chunk's steps and meet in
// LDS, added in wave order.
constexpr int kShrinkWaves = 8;

// One wave's part of TR x T tiles: rows x (16 * TR), ranks w (16 * T), from k to
// k1, the operands of kSteps MFMA steps of 32 loaded together.
template <int TR>
constexpr int kSteps = TR == 1 ? 4 : 2;

template <int XF, int WF, int TR, int T>
__device__ __forceinline__ void shrink_steps(const char *const (&xrow)[TR],
                                             const uint16_t *const (&wrow)[4], int64_t k, int64_t k1,
                                             v4f (&acc)[TR][4]) {
    constexpr int XV = XF == kF32 ? 2 : 1;     // 16-byte vectors of eight x
    constexpr int S = kSteps<TR>;
    for (; k < k1; k += 32 * S) {
        v4u w[S][T], xr[S][TR][XV];
#pragma unroll
        for (int i = 0; i < S; ++i) {
#pragma unroll
            for (int j = 0; j < T; ++j) w[i][j] = *reinterpret_cast<const v4u *>(wrow[j] + k + 32 * i);
#pragma unroll
            for (int u = 0; u < TR; ++u)
#pragma unroll
                for (int h = 0; h < XV; ++h)
                    xr[i][u][h] = *reinterpret_cast<const v4u *>(xrow[u] + (k + 32 * i) * (2 * XV) + 16 * h);
        }
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
            for (int u = 0; u < TR; ++u) {
                v4u xp[kParts<XF>];
                if constexpr (XF == kF32) {
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t b = xr[i][u][e >> 2][e & 3];
                        f[e] = __builtin_bit_cast(float, b);
                    }
                    split8(f, xp);
                } else if constexpr (XF != WF) {
                    parts_of<XF>(xr[i][u][0], xp);
                }
#pragma unroll
                for (int j = 0; j < T; ++j) {
                    if constexpr (XF == WF && WF == kBf16) {
                        acc[u][j] = mfma_bf16(xr[i][u][0], w[i][j], acc[u][j]);
                    } else if constexpr (XF == WF) {
                        acc[u][j] = mfma_f16(xr[i][u][0], w[i][j], acc[u][j]);
                    } else {
                        v4u wp[kParts<WF>];
                        parts_of<WF>(w[i][j], wp);
                        acc[u][j] = mfma_parts(xp, wp, acc[u][j]);
                    }
                }
            }
    }
}

template <int XF, int WF, int TR>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(LoraArgs p,
                                                                        float *__restrict__ v,
                                                                        int64_t chunk, int window,
                                                                        int turns) {
    __shared__ v4f part[kShrinkWaves][4][kWave];
    __shared__ uint8_t lists[kShrinkWaves][kWindow];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int r = lane & 15, c = lane >> 4;
    const int turn = (int)blockIdx.z % turns;
    const int r0 = (int)blockIdx.z / turns * kShrinkRanks;
    const int64_t k0 = (int64_t)blockIdx.y * chunk;
    const int64_t k1 = k0 + chunk < p.K ? k0 + chunk : p.K;
    constexpr int kBatch = 32 * kSteps<TR>;    // divides 128, and so the chunk
    const int64_t each = ((k1 - k0) / kBatch + kShrinkWaves - 1) / kShrinkWaves * kBatch;
    const int64_t kw = k0 + wave * each + 8 * c;
    const int64_t kw1 = k0 + (wave + 1) * each < k1 ? k0 + (wave + 1) * each : k1;
    Rows rows(p, (int64_t)blockIdx.x * window, window, lists[wave]);
    v += (int64_t)blockIdx.y * p.M * p.R;
    for (int at = 0; rows.any(); ++at) {
        const int id = rows.next();
        if (at % turns != turn) continue;
        const int rank = rank_of(p, id);
        if (r0 >= rank) continue;
        const int count = rows.take(id);
        // ranks past R are read from the last one; their sums are not kept
        const uint16_t *wrow[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            wrow[j] = static_cast<const uint16_t *>(p.a) +
                      ((int64_t)id * p.R + min(r0 + 16 * j + r, (int)p.R - 1)) * p.K;
        const int tiles = min((rank - r0 + 15) / 16, 4);
        for (int i0 = 0; i0 < count; i0 += 16 * TR) {
            const char *xrow[TR];
#pragma unroll
            for (int u = 0; u < TR; ++u)
                xrow[u] = static_cast<const char *>(p.x) +
                          rows.row(i0 + 16 * u + r, count) * p.K * (XF == kF32 ? 4 : 2);
            v4f acc[TR][4] = {};
            if (tiles == 1)
                shrink_steps<XF, WF, TR, 1>(xrow, wrow, kw, kw1, acc);
            else if (tiles == 2)
                shrink_steps<XF, WF, TR, 2>(xrow, wrow, kw, kw1, acc);
            else
                shrink_steps<XF, WF, TR, 4>(xrow, wrow, kw, kw1, acc);
#pragma unroll
            for (int u = 0; u < TR; ++u) {
                if (u > 0 && i0 + 16 * u >= count) break;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < tiles) part[wave][j][lane] = acc[u][j];
                __syncthreads();
                // wave j stores rank tile j: rank r0 + 16 j + r of entries 4 c + i
                if (wave < tiles) {
                    v4f sum = part[0][wave][lane];
#pragma unroll
                    for (int w = 1; w < kShrinkWaves; ++w) sum += part[w][wave][lane];
                    const int rk = r0 + 16 * wave + r;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int e = i0 + 16 * u + 4 * c + i;
                        if (e < count && rk < rank) v[rows.row(e, count) * p.R + rk] = sum[i];
                    }
                }
                __syncthreads();
            }
        }
    }
}

// Drops the values of a vector of eight from element `keep` on.
__device__ __forceinline__ v4u keep_first(v4u w, int keep) {
#pragma unroll
    for (int d = 0; d < 4; ++d)
        w[d] = keep >= 2 * d + 2 ? w[d] : keep == 2 * d + 1 ? (w[d] & 0xffffu) : 0u;
    return w;
}

// 16 consecutive values of a row, as loaded.
template <int YF>
struct Raw16 {
    uint32_t w[YF == kF32 ? 16 : 8];
};

// Four words that are aligned like an element only (rows of an odd N).
template <int YF>
struct __attribute__((packed, aligned(YF == kF32 ? 4 : 2))) Words4 {
    uint32_t w[4];
};

// base of row m from column n on; `wide`: all 16 columns exist.
template <int YF>
__device__ __forceinline__ void load16(const LoraArgs &p, int64_t m, int64_t n, bool wide, Raw16<YF> &o) {
    constexpr int V = YF == kF32 ? 4 : 2;
    const int64_t at = m * p.N + n;
    if (wide) {
        const Words4<YF> *b = reinterpret_cast<const Words4<YF> *>(
            static_cast<const char *>(p.base) + at * (YF == kF32 ? 4 : 2));
#pragma unroll
        for (int a = 0; a < V; ++a) {
            const Words4<YF> u = b[a];
#pragma unroll
            for (int k = 0; k < 4; ++k) o.w[4 * a + k] = u.w[k];
        }
    } else if constexpr (YF == kF32) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            o.w[e] = n + e < p.N ? static_cast<const uint32_t *>(p.base)[at + e] : 0;
    } else {
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const uint16_t *b = static_cast<const uint16_t *>(p.base) + at + e;
            o.w[e / 2] = (n + e < p.N ? b[0] : 0) | (n + e + 1 < p.N ? (uint32_t)b[1] << 16 : 0);
        }
    }
}

// y of row m from column n on: the loaded base, plus d (ADD) rounded once.
template <int YF, bool ADD>
__device__ __forceinline__ void store16(const LoraArgs &p, int64_t m, int64_t n, bool wide,
                                        const Raw16<YF> &base, const v4f (&d)[4]) {
    const int64_t at = m * p.N + n;
    uint32_t o[YF == kF32 ? 16 : 8];
#pragma unroll
    for (int i = 0; i < (YF == kF32 ? 16 : 8); ++i) {
        const uint32_t u = base.w[i];
        if constexpr (!ADD) {
            o[i] = u;
        } else if constexpr (YF == kF32) {
            const float f = d[i >> 2][i & 3];
            o[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, u) + f);
        } else {
            const float lo = d[i >> 1][2 * i & 3], hi = d[i >> 1][(2 * i & 3) + 1];
            o[i] = (uint32_t)bf16_rne(__builtin_bit_cast(float, u << 16) + lo) |
                   ((uint32_t)bf16_rne(__builtin_bit_cast(float, u & 0xffff0000u) + hi) << 16);
        }
    }
    if (wide) {
        Words4<YF> *y = reinterpret_cast<Words4<YF> *>(static_cast<char *>(p.y) + at * (YF == kF32 ? 4 : 2));
#pragma unroll
        for (int a = 0; a < (YF == kF32 ? 4 : 2); ++a)
            y[a] = Words4<YF>{{o[4 * a], o[4 * a + 1], o[4 * a + 2], o[4 * a + 3]}};
    } else if constexpr (YF == kF32) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (n + e < p.N) static_cast<uint32_t *>(p.y)[at + e] = o[e];
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (n + e < p.N)
                static_cast<uint16_t *>(p.y)[at + e] = (uint16_t)(e & 1 ? o[e / 2] >> 16 : o[e / 2]);
    }
}

// Expand: a block forms its rows x 256 columns of y, adapter by adapter, 16 rows
// and 64 ranks at a time: the block's threads add the K chunks' sums of v,
// apply the adapter's scale and leave v's three bfloat16 parts in LDS, then each
// wave multiplies them by B's rows of its 64 columns (in registers; kept from
// tile to tile up to rank 64). Operand A is B's rows (columns of y), operand B
// the rows' v: row 4 c + i of MFMA tile a is column 16 c + 4 a + i, so that the
// four tiles leave a lane with 16 consecutive columns of one row, and four
// lanes with 64.
constexpr int kExpandRows = 16;
constexpr int kExpandStride = 144;             // LDS bytes of a row's 64 ranks (128 + pad)

template <int WF, int YF>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs p, const float *__restrict__ v,
                                                          int chunks, int window, int turns) {
    __shared__ uint8_t lists[4][kWindow];
    __shared__ __attribute__((aligned(16))) uint8_t vparts[3][kExpandRows * kExpandStride];
    constexpr int U = kExpandRows / 16;
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1), wave = tid / kWave;
    const int r = lane & 15, c = lane >> 4;
    const int64_t n0 = ((int64_t)blockIdx.y * 4 + wave) * 64;
    const int64_t n = n0 + 16 * c;             // this lane's columns
    const bool wide = n + 16 <= p.N;
    const uint16_t *wrow[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const int64_t col = n0 + 16 * (r >> 2) + 4 * a + (r & 3);
        wrow[a] = static_cast<const uint16_t *>(p.b) + (col < p.N ? col : p.N - 1) * p.R + 8 * c;
    }
    Rows rows(p, (int64_t)blockIdx.x * window, window, lists[wave]);
    for (int at = 0; rows.any(); ++at) {
        const int id = rows.next();
        if (at % turns != (int)blockIdx.z) continue;
        const int count = rows.take(id);
        const int rank = rank_of(p, id);
        const float scale = p.scale ? p.scale[id] : 1.0f;
        const int64_t wbase = (int64_t)id * p.N * p.R;
        v4u w[2][4] = {};
        for (int i0 = 0; i0 < count; i0 += kExpandRows) {
            const int live = min(count - i0, kExpandRows);
            // the base, B's vectors and v are requested together
            int64_t m[U];
            Raw16<YF> base[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                m[u] = rows.row(i0 + 16 * u + r, count);
                if (16 * u + r < live && n < p.N) load16<YF>(p, m[u], n, wide, base[u]);
            }
            v4f acc[U][4] = {};
            for (int kc = 0; kc < rank; kc += 64) {
                if (i0 == 0 || rank > 64) {    // else B's vectors are those of the last rows
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int a = 0; a < 4; ++a) {
                            const int keep = rank - (kc + 32 * j + 8 * c);
                            w[j][a] = v4u{};
                            if (keep > 0)
                                w[j][a] = *reinterpret_cast<const v4u *>(wrow[a] + wbase + kc + 32 * j);
                        }
                }
                v4f f[U];                      // four ranks of an entry each
#pragma unroll
                for (int e = 0; e < U; ++e) {
                    const int entry = 16 * e + (tid >> 4), k = kc + 4 * (tid & 15);
                    f[e] = v4f{};
                    if (entry < live && k < rank) {
                        const float *src = v + rows.row(i0 + entry, count) * p.R + k;
#pragma unroll 4
                        for (int s = 0; s < chunks; ++s)
                            f[e] += *reinterpret_cast<const v4f *>(src + s * p.M * p.R);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) f[e][q] = k + q < rank ? f[e][q] * scale : 0.0f;
                }
                ring_barrier();                // the parts of the last step have been read
#pragma unroll
                for (int e = 0; e < U; ++e) {
                    const float g[8] = {f[e][0], f[e][1], f[e][2], f[e][3]};
                    v4u part[3];
                    split8(g, part);
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        *reinterpret_cast<uint2 *>(vparts[i] + (16 * e + (tid >> 4)) * kExpandStride +
                                                   8 * (tid & 15)) = make_uint2(part[i][0], part[i][1]);
                }
                ring_barrier();
                if ((rank & 7) && (i0 == 0 || rank > 64)) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int a = 0; a < 4; ++a)
                            w[j][a] = keep_first(w[j][a], rank - (kc + 32 * j + 8 * c));
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (16 * u >= live) continue;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (kc + 32 * j >= rank) continue;
                        v4u vp[3];
#pragma unroll
                        for (int i = 0; i < 3; ++i)
                            vp[i] = *reinterpret_cast<const v4u *>(
                                vparts[i] + (16 * u + r) * kExpandStride + 64 * j + 16 * c);
#pragma unroll
                        for (int a = 0; a < 4; ++a) {
                            v4u wp[kParts<WF>];
                            parts_of<WF>(w[j][a], wp);
                            acc[u][a] = mfma_parts(wp, vp, acc[u][a]);
                        }
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (16 * u + r < live && n < p.N) store16<YF, true>(p, m[u], n, wide, base[u], acc[u]);
        }
    }
    if (blockIdx.z != 0) return;
    if (p.base == p.y) return;
    const int count = rows.take(-1);           // rows without an adapter (every lane takes part)
    if (n >= p.N) return;
    const v4f none[4] = {};
    for (int i = r; i < count; i += 16) {
        const int64_t m = rows.row(i, count);
        Raw16<YF> base;
        load16<YF>(p, m, n, wide, base);
        store16<YF, false>(p, m, n, wide, base, none);
    }
}

// How the rows are dealt to blocks, each of which stands `per` times in the
// grid: windows of rows (a power of two of them, as many as leave `least`
// blocks, so that rows share an adapter's reads), and turns -- blocks of one
// window that take its adapters in turn, for batches of few rows with many
// adapters.
struct Deal {
    int window, turns;
    int64_t windows;
};

// Up to 1024 rows, a batch with many adapters is taken for requests of a few
// rows each, whose windows hold several adapters.
Deal deal_rows(int64_t M, int64_t L, int64_t per, int64_t least, int64_t most) {
    Deal d{kWindow, 1, 0};
    const int64_t adapters = M > 1024 || L < 4 ? 1 : L < 8 ? L / 2 : 4;
    while (d.window > 32 && (M + d.window - 1) / d.window * per * adapters < least) d.window /= 2;
    d.windows = (M + d.window - 1) / d.window;
    int64_t t = most / (d.windows * per);
    const int64_t ids = M < d.window ? M : d.window;
    if (t > ids) t = ids;
    if (t > L) t = L;
    d.turns = t < 1 ? 1 : (int)t;
    return d;
}

// K chunks of the shrink: at least 1024 of K each.
int plan_chunks(int64_t M, int64_t K) {
    const int64_t most = (K + 1023) / 1024 < 16 ? (K + 1023) / 1024 : 16;
    int64_t s = 256 / ((M + 31) / 32);
    if (s > most) s = most;
    return s < 1 ? 1 : (int)s;
}

template <int XF, int WF>
void launch_shrink(const LoraArgs &a, float *v, int64_t chunk, int64_t chunks, hipStream_t stream) {
    const int64_t blocks = (a.R + kShrinkRanks - 1) / kShrinkRanks;
    const Deal d = deal_rows(a.M, a.L, chunks * blocks, 160, 1024);
    const dim3 grid((unsigned)d.windows, (unsigned)chunks, (unsigned)(blocks * d.turns));
    if (a.M > 16)
        hipLaunchKernelGGL((lora_shrink_kernel<XF, WF, 2>), grid, dim3(64 * kShrinkWaves), 0, stream,
                           a, v, chunk, d.window, d.turns);
    else
        hipLaunchKernelGGL((lora_shrink_kernel<XF, WF, 1>), grid, dim3(64 * kShrinkWaves), 0, stream,
                           a, v, chunk, d.window, d.turns);
}

template <int WF, int YF>
void launch_expand(const LoraArgs &a, const float *v, int64_t chunks, hipStream_t stream) {
    const int64_t cols = (a.N + 255) / 256;
    const Deal d = deal_rows(a.M, a.L, cols, 256, 2048);
    hipLaunchKernelGGL((lora_expand_kernel<WF, YF>),
                       dim3((unsigned)d.windows, (unsigned)cols, (unsigned)d.turns), dim3(256), 0,
                       stream, a, v, (int)chunks, d.window, d.turns);
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
    // whole batches of steps for every wave of a block
    const int64_t share = (a.M > 16 ? 64 : 128) * kShrinkWaves;
    const int64_t chunk = (a.K + share * chunks - 1) / (share * chunks) * share;
    chunks = (a.K + chunk - 1) / chunk;
    const bool wb = w_format == kBf16;
    if (x_format == kF32)
        wb ? launch_shrink<kF32, kBf16>(a, work, chunk, chunks, stream)
           : launch_shrink<kF32, kF16>(a, work, chunk, chunks, stream);
    else if (x_format == kBf16)
        wb ? launch_shrink<kBf16, kBf16>(a, work, chunk, chunks, stream)
           : launch_shrink<kBf16, kF16>(a, work, chunk, chunks, stream);
    else
        wb ? launch_shrink<kF16, kBf16>(a, work, chunk, chunks, stream)
           : launch_shrink<kF16, kF16>(a, work, chunk, chunks, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (y_format == kF32)
        wb ? launch_expand<kBf16, kF32>(a, work, chunks, stream)
           : launch_expand<kF16, kF32>(a, work, chunks, stream);
    else
        wb ? launch_expand<kBf16, kBf16>(a, work, chunks, stream)
           : launch_expand<kF16, kBf16>(a, work, chunks, stream);
    return hipGetLastError();
}

}  // namespace pq2
