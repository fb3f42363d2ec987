// pq2_grouped.hpp -- finding a block's tile among experts whose sizes are only
// known on the device; shared by the grouped kernels.
#pragma once

#include "pq2_device.hpp"
#include "pq2_launch.hpp"

namespace pq2 {

// Row tile of a block: slots [first, first + count) of expert e.
struct RowTile {
    int e, first, count;
};

// The experts' tiles of bm slots, counted over the wave: lane l holds a run of
// experts, their tiles and the tiles before them. Offsets are clamped into
// [0, T] and each expert's end to its start, so no slot outside [0, T) is ever
// named; a lane's count is capped (2^24, above any count that valid offsets
// give), so the scan of any contents stays in 32 bits.
struct TileScan {
    const int32_t *offsets;
    int E, T, bm, e0, per;
    int before, mine, total;   // tiles of earlier lanes, of this lane, of all

    __device__ __forceinline__ void range(int e, int &lo, int &hi) const {
        lo = min(max(offsets[e], 0), T);
        hi = min(max(offsets[e + 1], lo), T);
    }

    __device__ __forceinline__ TileScan(const int32_t *offsets_, int E_, int T_, int bm_)
        : offsets(offsets_), E(E_), T(T_), bm(bm_) {
        const int lane = threadIdx.x & (kWave - 1);
        per = (E + kWave - 1) / kWave;
        e0 = lane * per;
        mine = 0;
        for (int k = 0; k < per; ++k) {
            if (e0 + k >= E) break;
            int lo, hi;
            range(e0 + k, lo, hi);
            mine = min(mine + (hi - lo + bm - 1) / bm, 1 << 24);
        }
        int incl = mine;
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const int v = __shfl_up(incl, d, kWave);
            if (lane >= d) incl += v;
        }
        before = incl - mine;
        total = __builtin_amdgcn_readlane(incl, kWave - 1);
    }

    // The b-th tile in expert order; false past the last.
    __device__ __forceinline__ bool find(int b, RowTile &tile) const {
        int rest = b - before;
        const uint64_t here = __ballot(rest >= 0 && rest < mine);
        if (here == 0) return false;
        const int src = __builtin_ctzll(here);
        RowTile t{0, 0, 0};
        if ((int)(threadIdx.x & (kWave - 1)) == src) {
            for (int k = 0; k < per; ++k) {
                if (e0 + k >= E) break;
                int lo, hi;
                range(e0 + k, lo, hi);
                const int tiles = (hi - lo + bm - 1) / bm;
                if (rest < tiles) {
                    t.e = e0 + k;
                    t.first = lo + rest * bm;
                    t.count = min(hi - t.first, bm);
                    break;
                }
                rest -= tiles;
            }
        }
        tile.e = __builtin_amdgcn_readlane(t.e, src);
        tile.first = __builtin_amdgcn_readlane(t.first, src);
        tile.count = __builtin_amdgcn_readlane(t.count, src);
        return tile.count > 0;
    }
};

// Activation row of slot `slot` of a tile, or -1: past the tile, or no row.
__device__ __forceinline__ int64_t source_row(const GroupedArgs &p, const RowTile &tile, int slot) {
    if (slot >= tile.count) return -1;
    const int64_t i = tile.first + slot;
    const int64_t row = p.rows ? (int64_t)p.rows[i] : i;
    return row >= 0 && row < p.R ? row : -1;
}

// What a slot's float32 sums become: y = live ? scale * sum : 0 (a slot without
// activations is zero whatever its row scale holds).
struct SlotScale {
    float scale;
    bool live;

    __device__ __forceinline__ SlotScale(const GroupedArgs &p, int64_t i) : scale(1.0f), live(true) {
        if (p.row_scale) scale = p.row_scale[i];
        if (p.rows) {
            const int64_t row = p.rows[i];
            live = row >= 0 && row < p.R;
        }
    }
    __device__ __forceinline__ float operator()(float sum) const { return live ? scale * sum : 0.0f; }
};

// Dispatch slot b of nb to tile: slot b runs on XCD b % 8, and XCD x receives
// the x-th contiguous run of tile numbers.
constexpr int kNumXcd = 8;

__device__ __forceinline__ int64_t xcd_tile(int64_t b, int64_t nb) {
    const int64_t xcd = b % kNumXcd, idx = b / kNumXcd;
    const int64_t per = nb / kNumXcd, rem = nb % kNumXcd;
    return xcd < rem ? xcd * (per + 1) + idx : rem * (per + 1) + (xcd - rem) * per + idx;
}

// The block's tile of BM slots x BN columns (columns fastest, numbered over the
// XCDs by the number of tiles there really are): its slots and first column.
// False: a block past the last tile.
template <int BM, int BN>
__device__ __forceinline__ bool grouped_tile(const GroupedArgs &p, RowTile &slots, int64_t &n0) {
    const TileScan scan(p.offsets, (int)p.E, (int)p.T, BM);
    const int64_t tiles_n = (p.N + BN - 1) / BN;
    const int64_t blocks = scan.total * tiles_n;
    if ((int64_t)blockIdx.x >= blocks) return false;
    const int64_t tile = xcd_tile(blockIdx.x, blocks);
    if (!scan.find((int)(tile / tiles_n), slots)) return false;
    n0 = tile % tiles_n * BN;
    return true;
}

// Tiles of bm slots that T slots of E experts can form at most: every expert
// with slots has one partly filled tile, the others are full.
inline int64_t max_tiles(int64_t T, int64_t E, int64_t bm) {
    const int64_t some = T < E ? T : E;
    return some + (T - some) / bm;
}

inline int64_t grouped_blocks(const GroupedArgs &a, int64_t bm, int64_t bn) {
    return max_tiles(a.T, a.E, bm) * ((a.N + bn - 1) / bn);
}

}  // namespace pq2
