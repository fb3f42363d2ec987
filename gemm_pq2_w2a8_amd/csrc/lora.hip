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
// into three -- and the parts' products added. Only float32 (x or v) against
// binary16 weights has a pair that is left out: the third part times the second,
// below 2^-22 of the product (parts are cut, not rounded, so it has the product's
// sign). Otherwise v stays float32 this way and the rank dimension costs no
// accuracy.
#include "pq2_device.hpp"
#include "pq2_launch.hpp"

namespace pq2 {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
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

// Sum of the parts' products (a's parts times b's), without the pair of a third
// and a second part (below 2^-22 of the product).
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

    // Row of entry i of the list (the first one past its end), from m0 on.
    __device__ __forceinline__ uint32_t local(int i, int count) const {
        return list[i < count ? i : 0];
    }
    __device__ __forceinline__ int64_t row(int i, int count) const { return m0 + local(i, count); }
};

__device__ __forceinline__ int rank_of(const LoraArgs &p, int id) {
    const int R = (int)p.R;
    return p.ranks ? min(max(p.ranks[id], 0), R) : R;
}

// Shrink: a block sums one K chunk of its rows x 64 ranks, adapter by adapter,
// 16 * TR rows at a time; its eight waves share the chunk's steps and meet in
// LDS, added in wave order. 4096 rows of 5120 bfloat16, rank 64: 28 us (42 MB of
// x, 8.8 us of HBM time); 555 rows of 17408 with 11 adapters: 15 us. A wave's
// steps load, wait and multiply in turn, with nothing in flight from one to the
// next: the block's other waves are what covers a load.
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

// Four consecutive values of a row, as loaded; rows of an odd N are aligned like
// their elements only.
template <int YF>
struct __attribute__((packed, aligned(YF == kF32 ? 4 : 2))) Four {
    uint32_t w[YF == kF32 ? 4 : 2];
};

// A window's rows of base or y: 16 or 8 bytes a lane. Rows are addressed from the
// window's first (128 rows of PQ2_LORA_MAX_N float32 are 2^29 bytes).
// EVEN: every row begins at a multiple of four bytes, and the accesses are buffer
// accesses that a lane without a row, or at the end of a row, makes outside the
// resource: no branches, so requests stay in flight across them. The ends of
// rows (N % 4 columns) go element by element, as all does with other rows.
template <int YF, bool EVEN>
struct RowsOf {
    static constexpr int kSize = YF == kF32 ? 4 : 2;
    char *at;
    int N;
    __amdgpu_buffer_rsrc_t rs;

    __device__ __forceinline__ RowsOf(const void *first, int N_, int64_t m0, int64_t rows)
        : at(const_cast<char *>(static_cast<const char *>(first)) + m0 * N_ * kSize), N(N_),
          rs(make_rsrc(at, rows * N_ * kSize)) {}

    __device__ __forceinline__ void load(uint32_t off, int n, bool live, Four<YF> &o) const {
        if constexpr (EVEN) {
            const int off4 = live && n + 4 <= N ? (int)off : kCopyOob;
            if constexpr (YF == kF32) {
                const v4u u = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rs, off4, 0, 0));
#pragma unroll
                for (int e = 0; e < 4; ++e) o.w[e] = u[e];
            } else {
                const v2u u = __builtin_bit_cast(v2u, __builtin_amdgcn_raw_buffer_load_b64(rs, off4, 0, 0));
                o.w[0] = u[0];
                o.w[1] = u[1];
            }
            if ((N & 3) == 0 || !live || n + 4 <= N) return;
        } else {
            if (!live || n >= N) return;
            if (n + 4 <= N) {
                o = *reinterpret_cast<const Four<YF> *>(at + off);
                return;
            }
            o = Four<YF>{};
        }
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            if (n + e >= N) continue;
            if constexpr (YF == kF32)
                o.w[e] = reinterpret_cast<const uint32_t *>(at + off)[e];
            else
                o.w[e / 2] |= (uint32_t) reinterpret_cast<const uint16_t *>(at + off)[e] << (16 * (e & 1));
        }
    }

    __device__ __forceinline__ void store(uint32_t off, int n, bool live, const Four<YF> &o) const {
        if constexpr (EVEN) {
            const int off4 = live && n + 4 <= N ? (int)off : kCopyOob;
            if constexpr (YF == kF32)
                __builtin_amdgcn_raw_buffer_store_b128(v4u{o.w[0], o.w[1], o.w[2], o.w[3]}, rs, off4, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b64(v2u{o.w[0], o.w[1]}, rs, off4, 0, 0);
            if ((N & 3) == 0 || !live || n + 4 <= N) return;
        } else {
            if (!live || n >= N) return;
            if (n + 4 <= N) {
                *reinterpret_cast<Four<YF> *>(at + off) = o;
                return;
            }
        }
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            if (n + e >= N) continue;
            if constexpr (YF == kF32)
                reinterpret_cast<uint32_t *>(at + off)[e] = o.w[e];
            else
                reinterpret_cast<uint16_t *>(at + off)[e] = (uint16_t)(o.w[e / 2] >> (16 * (e & 1)));
        }
    }
};

// base + d, rounded once.
template <int YF>
__device__ __forceinline__ Four<YF> add4(Four<YF> base, const float (&d)[4]) {
    if constexpr (YF == kF32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t u = base.w[e];
            base.w[e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, u) + d[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t u = base.w[e];
            // v_cvt_pk_bf16_f32: to nearest even, two at once
            const v2bf o = {(__bf16)(__builtin_bit_cast(float, u << 16) + d[2 * e]),
                            (__bf16)(__builtin_bit_cast(float, u & 0xffff0000u) + d[2 * e + 1])};
            base.w[e] = __builtin_bit_cast(uint32_t, o);
        }
    }
    return base;
}

// Expand: a block forms its rows x 256 columns of y, adapter by adapter, in stages
// of 16 rows and 64 ranks: the block's threads add the K chunks' sums of v,
// apply the adapter's scale and leave v's three bfloat16 parts in LDS, then each
// wave multiplies them by B's rows of its 64 columns. Operand A is the rows' v,
// operand B is B's rows (columns of y): column r of MFMA tile a is column
// 4 r + a, so that the four tiles leave a lane with four consecutive columns of
// the rows 4 c + i, and 16 neighbouring lanes read and write 64 consecutive
// columns of one row.
// PIPE (R <= 64): B's vectors stay in registers over an adapter's stages, and a
// stage's v and base are requested while the one before is computed (and waited
// for at its end, where they change registers).
// Memory-bound for many rows (4096 x 17408 bfloat16, rank 64: 74 us, 3.9 TB/s of
// base, y and v), a chain of four dependent reads for a few.
constexpr int kExpandRows = 16;
constexpr int kExpandStride = 144;             // LDS bytes of a row's 64 ranks (128 + pad)

template <int WF, int YF, bool EVEN, bool PIPE>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs p, const float *__restrict__ v,
                                                          int chunks, int window, int turns) {
    __shared__ uint8_t lists[4][kWindow];
    __shared__ __attribute__((aligned(16))) uint8_t vparts[2][3][kExpandRows * kExpandStride];
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1), wave = tid / kWave;
    const int r = lane & 15, c = lane >> 4;
    const int N = (int)p.N, R = (int)p.R;
    const int n = ((int)blockIdx.y * 4 + wave) * 64 + 4 * r;   // this lane's columns
    const int64_t m0 = (int64_t)blockIdx.x * window;
    const int64_t in = p.M - m0 < window ? p.M - m0 : window;  // rows of the window
    const RowsOf<YF, EVEN> base(p.base, N, m0, in), y(p.y, N, m0, in);
    const int entry = tid >> 4, k = 4 * (tid & 15);            // this thread's part of a stage's v
    Rows rows(p, m0, window, lists[wave]);
    int stage = 0;
    for (int at = 0; rows.any(); ++at) {
        const int id = rows.next();
        if (at % turns != (int)blockIdx.z) continue;
        const int count = rows.take(id);
        const int rank = rank_of(p, id);
        const float scale = p.scale ? p.scale[id] : 1.0f;
        // B's rows of the lane's columns, a resource for each of the four tiles
        // that begins a columns on and ends with B: columns past N lie outside
        // by the lane's own offset and read zeros. (Scalar registers only; four
        // offsets a lane cost a wave of occupancy, 16 rows of 16 adapters
        // 25.5 -> 26.7 us.)
        const uint16_t *const bl = static_cast<const uint16_t *>(p.b) + (int64_t)id * N * R;
        __amdgpu_buffer_rsrc_t rs_b[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) rs_b[a] = make_rsrc(bl + a * R, max(2 * (N - a) * R, 0));
        v4u w[2][4];
        auto load_w = [&](int kc) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int a = 0; a < 4; ++a)
                    w[j][a] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(
                        rs_b[a],
                        rank > kc + 32 * j + 8 * c ? 2 * (n * R + kc + 32 * j + 8 * c) : kCopyOob, 0, 0));
        };
        auto mask_w = [&](int kc) __attribute__((always_inline)) {
            if ((rank & 7) == 0) return;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int a = 0; a < 4; ++a) w[j][a] = keep_first(w[j][a], rank - (kc + 32 * j + 8 * c));
        };
        // v of a stage: four ranks of an entry, from kc on, chunk s (ranks past
        // R and entries past the list read zeros)
        auto load_v = [&](int i0, int kc, int s) __attribute__((always_inline)) -> v4f {
            const __amdgpu_buffer_rsrc_t rs_v = make_rsrc(v + (s * p.M + m0) * R, in * R * 4);
            const int off = i0 + entry < count && kc + k < R
                                ? 4 * ((int)rows.local(i0 + entry, count) * R + kc + k) : kCopyOob;
            return __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rs_v, off, 0, 0));
        };
        // A stage's first two chunks of v and its base, requested a stage ahead.
        // The stage's products cover them and nothing more does: the copy of nxt
        // to cur waits for v, then the base (not for the stores issued behind).
        struct Stage {
            v4f v[2];
            uint32_t at[4];
            Four<YF> b[4];
        } cur, nxt;
        auto request = [&](int i0, Stage &o) __attribute__((always_inline)) {
            if constexpr (PIPE) {
                o.v[0] = load_v(i0, 0, 0);
                o.v[1] = chunks > 1 ? load_v(i0, 0, 1) : v4f{};
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = i0 + 4 * c + i;
                o.at[i] = (rows.local(e, count) * (uint32_t)N + (uint32_t)n) * RowsOf<YF, EVEN>::kSize;
                base.load(o.at[i], n, e < count, o.b[i]);
            }
        };
        if constexpr (PIPE) {
            load_w(0);
            request(0, cur);
            mask_w(0);
            wait_vmem<0>();                    // B's vectors stay: no later wait is for them
        }
        for (int i0 = 0; i0 < count; i0 += kExpandRows) {
            if constexpr (!PIPE) request(i0, cur);
            v4f acc[4] = {};
            const int steps = PIPE ? 1 : rank;
            for (int kc = 0; kc < steps; kc += 64, stage ^= 1) {
                v4f f;
                int s = 0;
                if constexpr (!PIPE) {
                    load_w(kc);
                    f = v4f{};
                } else {
                    f = cur.v[0] + cur.v[1];
                    s = 2;
                }
#pragma unroll 4
                for (; s < chunks; ++s) f += load_v(i0, kc, s);
                float g[8] = {};
#pragma unroll
                for (int q = 0; q < 4; ++q) g[q] = kc + k + q < rank ? f[q] * scale : 0.0f;
                v4u part[3];
                split8(g, part);
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    *reinterpret_cast<uint2 *>(vparts[stage][i] + entry * kExpandStride + 2 * k) =
                        make_uint2(part[i][0], part[i][1]);
                // one barrier a step: the other buffer's readers are past it
                ring_barrier();
                if constexpr (PIPE) {
                    if (i0 + kExpandRows < count) request(i0 + kExpandRows, nxt);
                } else {
                    mask_w(kc);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (kc + 32 * j >= rank) continue;
                    v4u vp[3];
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        vp[i] = *reinterpret_cast<const v4u *>(
                            vparts[stage][i] + r * kExpandStride + 64 * j + 16 * c);
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        v4u wp[kParts<WF>];
                        parts_of<WF>(w[j][a], wp);
                        acc[a] = mfma_parts(vp, wp, acc[a]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float d[4] = {acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
                y.store(cur.at[i], n, i0 + 4 * c + i < count, add4<YF>(cur.b[i], d));
            }
            if constexpr (PIPE) cur = nxt;
        }
    }
    if (blockIdx.z != 0 || p.base == p.y) return;
    const int count = rows.take(-1);           // rows without an adapter (every lane takes part)
    for (int i = 0; i < count; i += 4) {
        const uint32_t off = (rows.local(i + c, count) * (uint32_t)N + (uint32_t)n) *
                             RowsOf<YF, EVEN>::kSize;
        Four<YF> o;
        base.load(off, n, i + c < count, o);
        y.store(off, n, i + c < count, o);
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
// rows each, whose windows hold several adapters. The host knows how many are
// loaded, not how many the rows use: a prompt of one adapter among many gets
// their windows and turns, most of which end at once. The limits here and in
// shrink_pairs rest on 1, 16, 555 and 4096 rows; nothing between was timed.
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

// Whether the shrink takes 32 rows at once: prompts, or few adapters.
bool shrink_pairs(int64_t M, int64_t L) {
    return M > 1024 || (M < kWindow ? M : kWindow) > 16 * L;
}

template <int XF, int WF>
void launch_shrink(const LoraArgs &a, float *v, int64_t chunk, int64_t chunks, hipStream_t stream) {
    const int64_t blocks = (a.R + kShrinkRanks - 1) / kShrinkRanks;
    const Deal d = deal_rows(a.M, a.L, chunks * blocks, 160, 1024);
    const dim3 grid((unsigned)d.windows, (unsigned)chunks, (unsigned)(blocks * d.turns));
    if (shrink_pairs(a.M, a.L))
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
    const dim3 grid((unsigned)d.windows, (unsigned)cols, (unsigned)d.turns);
    const bool even = YF == kF32 || (a.N % 2 == 0 && (((uintptr_t)a.base | (uintptr_t)a.y) & 3) == 0);
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a, v, (int)chunks, d.window, d.turns);
    };
    // many 16-row stages of one adapter (4096 rows of 17408 columns, rank 64: 74 us
    // pipelined, 101 not; 16 rows of 16 adapters: 19.6 against 15.1)
    if (a.R <= 64 && a.M > 1024)
        even ? launch(lora_expand_kernel<WF, YF, true, true>)
             : launch(lora_expand_kernel<WF, YF, false, true>);
    else
        even ? launch(lora_expand_kernel<WF, YF, true, false>)
             : launch(lora_expand_kernel<WF, YF, false, false>);
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
    const int64_t share = 32 * (shrink_pairs(a.M, a.L) ? kSteps<2> : kSteps<1>) * kShrinkWaves;
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
