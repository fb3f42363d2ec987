// mx4_plan.hpp -- which tiles a block of an MX4 product computes, and how the
// tiles of a launch are dealt to blocks.
#pragma once

#include "mx4_device.hpp"
#include "pq2_launch.hpp"

namespace pq2 {

// Tiles of a launch: the first `full` are computed whole, the sum of each of the
// others (its `runs`, the steps that a sum is dealt by) is shared by `ways`
// blocks, whose float32 sums lie in part [tiles - full][ways][tile] in the lanes'
// own order until a second launch adds them in order.
struct MxPlan {
    int tiles_n, tiles_m, full, ways, runs;
    float *part;
};

// Tile t: runs of four tiles down, so that what an XCD's contiguous run of tiles
// reads at a time is about as high as wide.
__device__ __forceinline__ void tile_at(const MxPlan &p, int t, int &tn, int &tm) {
    constexpr int kDown = 4;
    const int group = t / (kDown * p.tiles_n), in = t % (kDown * p.tiles_n);
    const int left = p.tiles_m - group * kDown;
    const int high = left < kDown ? left : kDown;
    // (divisions leave uniform results in vector registers)
    tm = __builtin_amdgcn_readfirstlane(group * kDown + in % high);
    tn = __builtin_amdgcn_readfirstlane(in / high);
}

struct MxShare {
    bool live, split;
    int item;                         // of a split tile: its share's place in part
    int tn, tm;
    int q0, q1;                       // runs of this block
};

// Whole tiles come first; each XCD takes a contiguous run of either kind, of shares
// in the order of the runs, so that its tiles at a time are multiplied over the same
// columns.
__device__ __forceinline__ MxShare share_of(const MxPlan &p) {
    MxShare s;
    const int whole = (p.full + 7) / 8 * 8;
    s.split = (int)blockIdx.x >= whole;
    const int b = s.split ? blockIdx.x - whole : blockIdx.x;
    const int count = s.split ? (p.tiles_n * p.tiles_m - p.full) * p.ways : p.full;
    const int at = (b & 7) * ((count + 7) / 8) + (b >> 3);
    s.live = at < count;
    if (!s.live) return s;
    const int ways = s.split ? p.ways : 1, tiles = count / ways, way = at / tiles, t = at - way * tiles;
    s.item = t * ways + way;
    tile_at(p, s.split ? p.full + t : t, s.tn, s.tm);
    s.q0 = __builtin_amdgcn_readfirstlane((int)((uint32_t)p.runs * way / ways));
    s.q1 = __builtin_amdgcn_readfirstlane((int)((uint32_t)p.runs * (way + 1) / ways));
    return s;
}

// A share's sums, acc[I][J] of a block of T threads, as far as j < live.
template <int I, int J, int T>
__device__ __forceinline__ void store_share(const MxPlan &p, int item, int tid, int live, const v4f32 (&acc)[I][J]) {
    float *const to = p.part + (int64_t)item * (I * J * T * 4) + 4 * tid;
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (j < live) *reinterpret_cast<v4f32 *>(to + (i * J + j) * (4 * T)) = acc[i][j];
}

// acc[i0 .. i0 + NI - 1][j0 .. j0 + NJ - 1] of split tile `index`, its shares
// added in order, four requested at a time.
template <int I, int J, int T, int NI, int NJ>
__device__ __forceinline__ void sum_shares(const MxPlan &p, int index, int i0, int j0, int tid, v4f32 (&acc)[NI][NJ]) {
    const float *const from = p.part + (int64_t)index * p.ways * (I * J * T * 4) + 4 * tid;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float *const at = from + ((i0 + i) * J + j0 + j) * (4 * T);
            v4f32 sum = *reinterpret_cast<const v4f32 *>(at);
            for (int way = 1; way < p.ways; way += 4) {
                v4f32 v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (way + u < p.ways)
                        v[u] = *reinterpret_cast<const v4f32 *>(at + (int64_t)(way + u) * (I * J * T * 4));
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (way + u < p.ways) sum += v[u];
            }
            acc[i][j] = sum;
        }
}

// The plan of a tile L for `rows` x M results. Tiles left over after whole rounds
// of the compute units (each holds L::kBlocks) are split where that is faster by
// this count in nanoseconds: a block takes L::kRun for a run alone on the card and
// L::kMore longer with all places taken, L::kEnds for its start and end; a split
// tile's sums are written and read again at about 4 TB/s in a second launch. times:
// how often a run is gone through.
struct MxCost {
    MxPlan plan;
    int64_t ns;
};

template <class L>
MxCost plan_tiles(int64_t M, int64_t rows, int64_t runs, size_t bytes, int64_t times = 1) {
    MxCost c;
    MxPlan &p = c.plan;
    p.tiles_n = (int)((rows + L::BN - 1) / L::BN);
    p.tiles_m = (int)((M + L::BM - 1) / L::BM);
    p.part = nullptr;
    p.ways = 1;
    p.runs = (int)runs;
    const int64_t cus = device_cus() > 0 ? device_cus() : 256, slots = cus * L::kBlocks;
    const int64_t tiles = (int64_t)p.tiles_n * p.tiles_m, rest = tiles % slots;
    p.full = (int)tiles;
    auto rounds = [&](int64_t blocks, int64_t each) {
        const int64_t full = blocks / slots, left = blocks % slots;
        return full * (each * times * (L::kRun + L::kMore) + L::kEnds) +
               (left ? each * times * (L::kRun + L::kMore * left / slots) + L::kEnds : 0);
    };
    const int64_t whole = rounds(tiles - rest, runs);
    c.ns = rounds(tiles, runs);
    const int64_t part = (int64_t)L::BN * L::BM * sizeof(float);
    const int64_t most = M < L::BM ? (M + 15) / 16 * 16 : L::BM;    // tokens whose sums are kept
    for (int w = 2; w <= 16 && w <= runs; ++w) {
        if ((size_t)(rest * w * part) > bytes) break;
        const int64_t sums = rest * w * (part * most / L::BM) * 2 / 4000 + 3000;
        const int64_t ns = whole + rounds(rest * w, (runs + w - 1) / w) + sums;
        if (rest && ns < c.ns) {
            c.ns = ns;
            p.ways = w;
            p.full = (int)(tiles - rest);
        }
    }
    return c;
}

template <class L>
size_t part_bytes(const MxPlan &p) {
    return p.ways > 1 ? (size_t)((int64_t)p.tiles_n * p.tiles_m - p.full) * p.ways * (L::BN * L::BM) * sizeof(float) : 0;
}

inline unsigned plan_blocks(const MxPlan &p) {
    const int rest = p.tiles_n * p.tiles_m - p.full;
    return (unsigned)((p.full + 7) / 8 * 8 + (rest * p.ways + 7) / 8 * 8);
}

}  // namespace pq2
