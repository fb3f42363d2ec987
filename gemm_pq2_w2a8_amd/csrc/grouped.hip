// grouped.hip -- PQ2_0 products grouped by expert with ragged sizes.
//
// Slot i of the T slots belongs to expert e with offsets[e] <= i <
// offsets[e + 1] and multiplies activation row rows[i] by the expert's weights:
//   y[i][n] = row_scale[i] * sum_g s[row][g] ws[e][n][g] D(q[row], codes[e][n], g).
// The offsets are only known on the device, so the grid covers the largest
// number of row tiles any offsets can give and every wave finds its own tile
// (TileScan); blocks past the last tile end at once.
//
// Kernels: the stream kernel below for a mean of up to four slots an expert, the
// prefill tiles of prefill_mfma.hip over gathered slots above that, and a plain
// kernel for arrays beyond 31-bit offsets.
#include "pq2_device.hpp"
#include "pq2_grouped.hpp"
#include "pq2_launch.hpp"

namespace pq2 {

namespace {

// 16 slots x 64 columns, one wave per 16 columns, both operands from global
// memory. Operand A of v_mfma_i32_16x16x64_i8 is the activations (slots =
// rows), operand B the code planes (weight rows = columns): lane (r, c) holds
// code words 4 (c & 1) .. + 3 of column r, MFMA a takes their plane
// 2 a + (c >> 1) against the activation bytes 64 a + 16 c .. + 15 of slot r,
// which plane order keeps together.
__global__ __launch_bounds__(256) void grouped_small_kernel(GroupedArgs p) {
    RowTile tile;
    if (!TileScan(p.offsets, (int)p.E, (int)p.T, 16).find(blockIdx.x, tile)) return;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int r = lane & 15, c = lane >> 4;
    const int64_t n0 = ((int64_t)blockIdx.y * 4 + wave) * 16;
    if (n0 >= p.N) return;
    const int G = (int)(p.K / kGroup);
    const int64_t KB = p.K / 4;
    const int64_t row_a = source_row(p, tile, r);
    int64_t row_d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) row_d[i] = source_row(p, tile, 4 * c + i);
    const int64_t n = n0 + r < p.N ? n0 + r : p.N - 1;
    const uint8_t *codes = p.codes + (tile.e * p.N + n) * KB + 16 * (c & 1);
    const uint16_t *ws = p.ws + (tile.e * p.N + n) * G;
    const int8_t *q = p.q + (row_a < 0 ? 0 : row_a) * p.K + 16 * c;
    const int sh0 = 2 * (c >> 1);
    float acc[4] = {};
    for (int g = 0; g < G; ++g) {
        const v4i w = *reinterpret_cast<const v4i *>(codes + 32 * g);
        v4i a0 = {}, a1 = {};
        if (row_a >= 0) {
            a0 = *reinterpret_cast<const v4i *>(q + kGroup * g);
            a1 = *reinterpret_cast<const v4i *>(q + kGroup * g + 64);
        }
        v4i d;
        float sv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[i] = row_d[i] < 0 ? 0 : -p.t[row_d[i] * G + g];
            sv[i] = row_d[i] < 0 ? 0.0f : p.s[row_d[i] * G + g];
        }
        v4i b0, b1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t sh = (uint32_t)w[k] >> sh0;
            b0[k] = (int)(sh & kPlaneMask);
            b1[k] = (int)((sh >> 4) & kPlaneMask);
        }
        d = mfma16x16x64(a0, b0, d);
        d = mfma16x16x64(a1, b1, d);
        const float wv = half_bits_to_float(ws[g]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf((float)d[i], sv[i] * wv, acc[i]);
    }
    if (n0 + r >= p.N) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (4 * c + i >= tile.count) continue;
        const int64_t slot = tile.first + 4 * c + i;
        store_y(p.y, p.y16, slot * p.N + n0 + r, SlotScale(p, slot)(acc[i]));
    }
}

// ---------------------------------------------------------------- few slots per expert
//
// Streams an expert's codes for tiles of up to four slots. Operand A's 16 rows
// are 4 groups x 4 slots, block-diagonal -- row 4 c + i holds slot i's
// activations of group 4 run + c in the k-range that lane group c supplies and
// zeros elsewhere -- so one chain of MFMAs forms the exact dots of four groups,
// and lane (r, c) ends with the dots of column r, group 4 run + c for its four
// slots. Against 16 slot rows of one group that is a quarter of the epilogue,
// each lane reads 32 consecutive code bytes (one whole group of its column) and
// 128 bytes of a column are read together; the MFMA count per group is the same.
// A wave takes 32 columns (two tiles, sharing A) and every waves-th run of four
// groups; the block's waves meet in LDS and are added in wave order.
// Codes and scales are requested two runs ahead into registers, a run's
// activations into the wave's own LDS (buffer -> LDS copies; 16-byte pieces
// permuted so that the four slots of a read fall in different banks). As
// compiled they do not stay in flight that long: the requests are conditional,
// so where their paths meet the first of two runs waits for all of them
// (vmcnt(0) before t) and the second run's 16-bit scales are copied, and so
// waited for, where they are requested: a pair of runs shows about one memory
// latency. Rows that do not exist and groups past the last have lane offsets
// outside the resources, which read zeros and move no memory; the lanes outside
// A's blocks read one zero piece.
// Planes 1 and 3 of a code word are masked in place (4 * code) into an
// accumulator of their own: 4 D = 4 d0 + d1, the factor taken out of the weight
// scale, 5 bit operations per word instead of 7.
// 64 experts of 2048 x 5120 with a slot each 45 us, 3.9 TB/s; 8 of them 9.9 us: a
// chain of dependent reads (offsets, then the codes, then three reads of rows[]
// one after the other behind them, then the activations).
constexpr int kStreamCols = 32;
constexpr int kStreamSlots = 4;
constexpr int kStreamMaxWaves = 4;
constexpr int kStreamRunBytes = kStreamSlots * 4 * kGroup;   // one run's activations
constexpr int kStreamWaveBytes = 2 * kStreamRunBytes + 32;   // two runs and the zero piece
constexpr int kStreamLoads = 10;                             // per run: 2 copies, 8 loads

__global__ __launch_bounds__(64 * kStreamMaxWaves) void grouped_stream_kernel(GroupedArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    RowTile tile;
    if (!TileScan(p.offsets, (int)p.E, (int)p.T, kStreamSlots).find(blockIdx.x, tile)) return;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int waves = blockDim.x / kWave;
    const int r = lane & 15, c = lane >> 4;
    const int G = (int)(p.K / kGroup), KB = (int)(p.K / 4);
    const int runs = (G + 3) / 4;
    const int64_t n0 = (int64_t)blockIdx.y * kStreamCols;
    const int cols = p.N - n0 < kStreamCols ? (int)(p.N - n0) : kStreamCols;
    const int64_t row0 = tile.e * p.N + n0;
    uint8_t *const own = smem + wave * kStreamWaveBytes;
    const __amdgpu_buffer_rsrc_t rs_codes = make_rsrc(p.codes + row0 * KB, (int64_t)cols * KB);
    const __amdgpu_buffer_rsrc_t rs_ws = make_rsrc(p.ws + row0 * G, (int64_t)cols * G * 2);
    const __amdgpu_buffer_rsrc_t rs_q = make_rsrc(p.q, p.R * p.K);
    const __amdgpu_buffer_rsrc_t rs_s = make_rsrc(p.s, p.R * G * 4);
    const __amdgpu_buffer_rsrc_t rs_t = make_rsrc(p.t, p.R * G * 4);

    // what a run needs in registers: the codes and scales of column r of both
    // tiles (group c of the run), s and t of slot r % 4, group c
    struct Run {
        v4i w[2][2];
        uint16_t ws[2];
        float s;
        int t;
    };
    auto load_codes = [&](int run, Run &o) __attribute__((always_inline)) {
        const bool live = 4 * run + c < G;      // groups past the last (G % 4 != 0)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                o.w[b][h] = __builtin_amdgcn_raw_buffer_load_b128(
                    rs_codes, live ? (16 * b + r) * KB + 32 * c + 16 * h : kCopyOob, 128 * run, 0);
            o.ws[b] = __builtin_amdgcn_raw_buffer_load_b16(
                rs_ws, live ? 2 * ((16 * b + r) * G + c) : kCopyOob, 8 * run, 0);
        }
    };
    // copy i of a run: lane l brings piece l % 32 of slot 2 i + l / 32, stored
    // with its plane (bits 1, 2 of the piece) exchanged by the slot
    int coff[2], cgroup, soff;
    auto load_acts = [&](int run, int slot, Run &o) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            copy16_to_lds_at(rs_q, own + slot * kStreamRunBytes + 1024 * i,
                             4 * run + cgroup < G ? coff[i] : kCopyOob, 4 * kGroup * run);
        const int so = 4 * run + c < G ? soff : kCopyOob;
        o.s = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs_s, so, 16 * run, 0));
        o.t = (int)__builtin_amdgcn_raw_buffer_load_b32(rs_t, so, 16 * run, 0);
    };

    Run run0, run1;
    const int second = wave + waves;
    load_codes(wave, run0);                     // waves <= runs
    if (second < runs) load_codes(second, run1);
    __builtin_amdgcn_sched_barrier(0);
    {
        const int piece = lane & 31;
        cgroup = piece >> 3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int slot = 2 * i + (lane >> 5);
            const int row = (int)source_row(p, tile, slot);
            coff[i] = row >= 0 ? row * (int)p.K + 16 * (piece ^ (2 * slot)) : kCopyOob;
        }
        const int row = (int)source_row(p, tile, r & 3);
        soff = row >= 0 ? 4 * (row * G + c) : kCopyOob;
    }
    // A's pieces of plane pl at aoff[pl] + 16 h
    const int zero = 2 * kStreamRunBytes;
    if (lane < 8) reinterpret_cast<uint32_t *>(own + zero)[lane] = 0;
    int aoff[4];
#pragma unroll
    for (int pl = 0; pl < 4; ++pl)
        aoff[pl] = (r >> 2) == c ? 512 * (r & 3) + kGroup * c + 32 * (pl ^ (r & 3)) : -1;
    load_acts(wave, 0, run0);
    if (second < runs) load_acts(second, 1, run1);
    // both runs' codes went out before the first run's activations: the first
    // run is there once only the second's activations are in flight
    if (second < runs)
        wait_vmem<4>();
    else
        wait_vmem<0>();

    float acc[2][4] = {};
    auto compute = [&](const Run &o, int slot) __attribute__((always_inline)) {
        const int ti = o.t, si = __builtin_bit_cast(int, o.s);
        const v4i seed = {-dpp_quad_bcast<0>(ti), -dpp_quad_bcast<1>(ti), -dpp_quad_bcast<2>(ti),
                          -dpp_quad_bcast<3>(ti)};
        v4i d0[2] = {seed, seed}, d1[2] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v4i a[4];
#pragma unroll
            for (int pl = 0; pl < 4; ++pl)
                a[pl] = *reinterpret_cast<const v4i *>(
                    own + (aoff[pl] < 0 ? zero : aoff[pl] + slot * kStreamRunBytes) + 16 * h);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                v4i b0, b1, b2, b3;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t lo = (uint32_t)o.w[b][h][k], hi = lo >> 4;
                    b0[k] = (int)(lo & kPlaneMask);
                    b1[k] = (int)(lo & kPlaneMaskX4);
                    b2[k] = (int)(hi & kPlaneMask);
                    b3[k] = (int)(hi & kPlaneMaskX4);
                }
                d0[b] = mfma16x16x64(a[0], b0, d0[b]);
                d1[b] = mfma16x16x64(a[1], b1, d1[b]);
                d0[b] = mfma16x16x64(a[2], b2, d0[b]);
                d1[b] = mfma16x16x64(a[3], b3, d1[b]);
            }
            __builtin_amdgcn_sched_barrier(0);  // holds A's halves one at a time (126 VGPRs, not 138)
        }
        const int sv[4] = {dpp_quad_bcast<0>(si), dpp_quad_bcast<1>(si), dpp_quad_bcast<2>(si),
                           dpp_quad_bcast<3>(si)};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float wv = 0.25f * half_bits_to_float(o.ws[b]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[b][i] = fmaf((float)(4 * d0[b][i] + d1[b][i]),
                                 __builtin_bit_cast(float, sv[i]) * wv, acc[b][i]);
        }
    };
    // one run: its loads are done once only the next run's are in flight (the
    // least wait that is right; the compiler's own are longer); its LDS is read
    // before the run after that is copied over it
    auto step = [&](int run, Run &o, int slot) __attribute__((always_inline)) {
        if (run + waves < runs)
            wait_vmem<kStreamLoads>();
        else
            wait_vmem<0>();
        compute(o, slot);
        __builtin_amdgcn_s_waitcnt(0xC07F);     // lgkmcnt(0)
        asm volatile("" ::: "memory");
        if (run + 2 * waves < runs) {
            load_codes(run + 2 * waves, o);
            load_acts(run + 2 * waves, slot, o);
        }
    };
    for (int run = wave; run < runs; run += 2 * waves) {
        step(run, run0, 0);
        if (run + waves < runs) step(run + waves, run1, 1);
    }

    // sums over the lane groups (groups 4 run + c); lane (r, c) keeps slot c,
    // the waves' sums meet in LDS
    __syncthreads();
    float *const red = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = acc[b][i];
            v[i] += __shfl_xor(v[i], 16, kWave);
            v[i] += __shfl_xor(v[i], 32, kWave);
        }
        const float mine = c == 0 ? v[0] : c == 1 ? v[1] : c == 2 ? v[2] : v[3];
        red[(wave * kStreamSlots + c) * kStreamCols + 16 * b + r] = mine;
    }
    __syncthreads();
    for (int o = threadIdx.x; o < tile.count * kStreamCols; o += blockDim.x) {
        const int slot = o / kStreamCols, col = o % kStreamCols;
        if (col >= cols) continue;
        float v = red[o];
        for (int w = 1; w < waves; ++w) v += red[w * kStreamSlots * kStreamCols + o];
        const int64_t i = tile.first + slot;
        store_y(p.y, p.y16, i * p.N + n0 + col, SlotScale(p, i)(v));
    }
}

// Waves that share a column tile's runs: one where the tiles fill the GPU
// (64 experts 2048 x 5120, one slot each: 45.1 us against 46.9 with two waves
// and 54.5 with four), four below that (8 experts: 10.2 us against 13.2 with
// one).
hipError_t launch_stream(const GroupedArgs &a, hipStream_t stream) {
    const int64_t slots = max_tiles(a.T, a.E, kStreamSlots);
    const int64_t cols = (a.N + kStreamCols - 1) / kStreamCols;
    const int64_t runs = (a.K / kGroup + 3) / 4;
    int64_t waves = slots * cols >= 1024 ? 1 : kStreamMaxWaves;
    if (waves > runs) waves = runs;
    hipLaunchKernelGGL(grouped_stream_kernel, dim3((unsigned)slots, (unsigned)cols),
                       dim3(64 * (unsigned)waves), (size_t)waves * kStreamWaveBytes, stream, a);
    return hipGetLastError();
}

// Tiles by the mean slots of the experts that can have any: the host knows no
// more than T and E, so slots that gather on a few experts get the kernel of the
// mean (up to a mean of four the stream kernel, which reads an expert's codes
// once for every four of its slots). MI355X, us, 64 experts with shares falling
// off as rank^-0.4, 2048 x 5120 and 5120 x 1024:
//   mean        2        6        8       16       32       64      128      256
//   stream  50 / 31  73 / 45  86 / 55
//   128x16  54 / 30  62 / 33  62 / 34  74 / 43 101 / 68 158/113  281/209  510/386
//   256x32  52 / 32  51 / 37  57 / 37  74 / 43  81 / 55 122/ 87  192/148  346/269
//   256x128 63 / 39  64 / 41  66 / 42  82 / 51 126 / 71 162/106  219/160  328/275
// With equal shares the steps lie at multiples of the tile. Few tiles leave
// CUs idle, and then the smaller one is faster: 8 experts of 2048 x 5120 with
// a mean of 8 slots 16 us on 64 x 16, 20 on 128 x 16, 31 on 256 x 32; of 48,
// 25 on 128 x 16, 39 on 256 x 32.
GroupedTile grouped_tile_of(const GroupedArgs &a) {
    const int64_t some = a.T < a.E ? a.T : a.E;
    const bool ring = (a.K / kGroup) % 8 == 0 && a.K <= 65536;   // scale chunks of 8 groups
    if (!ring) return a.T <= 20 * some ? kGroupedStaged32 : kGroupedStaged64;
    // blocks of a tile, the experts' last tiles taken as half full
    auto blocks = [&](int64_t bm, int64_t bn) {
        return (a.T / bm + (some + 1) / 2) * ((a.N + bn - 1) / bn);
    };
    if (a.T > 160 * some && blocks(128, 256) >= 512) return kGroupedWide128;
    if (a.T > 14 * some && blocks(32, 256) >= 256) return kGroupedWide32;
    return blocks(16, 128) >= 512 || a.T > 14 * some ? kGroupedRing128 : kGroupedRing64;
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs &a, hipStream_t stream) {
    const int64_t G = a.K / kGroup, some = a.T < a.E ? a.T : a.E;
    // gathered rows, and the widest tile's weight rows, by 31-bit lane offsets
    const bool near = a.R * a.K < kCopyOob && 4 * a.R * G < kCopyOob && 256 * (a.K / 4) < kCopyOob;
    // blocks of the smallest tile (32 x 16, one dimension) a grid can have
    if (!near || grouped_blocks(a, 16, 32) >= (int64_t(1) << 24)) {
        const dim3 grid((unsigned)max_tiles(a.T, a.E, 16), (unsigned)((a.N + 63) / 64));
        hipLaunchKernelGGL(grouped_small_kernel, grid, dim3(256), 0, stream, a);
        return hipGetLastError();
    }
    if (a.T <= 4 * some) return launch_stream(a, stream);
    return launch_grouped_tiles(a, grouped_tile_of(a), stream);
}

}  // namespace pq2
