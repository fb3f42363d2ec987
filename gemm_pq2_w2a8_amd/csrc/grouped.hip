// grouped.hip -- PQ2_0 products grouped by expert with ragged sizes.
//
// Slot i of the T slots belongs to expert e with offsets[e] <= i <
// offsets[e + 1] and multiplies activation row rows[i] by the expert's weights:
//   y[i][n] = row_scale[i] * sum_g s[row][g] ws[e][n][g] D(q[row], codes[e][n], g).
// The offsets are only known on the device, so the grid covers the largest
// number of row tiles any offsets can give and every wave finds its own tile
// (find_tile); blocks past the last tile end at once.
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
        const float v = p.row_scale ? p.row_scale[slot] * acc[i] : acc[i];
        store_y(p.y, p.y16, slot * p.N + n0 + r, v);
    }
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs &a, hipStream_t stream) {
    if (grouped_wide_fits(a)) return launch_grouped_wide(a, stream);
    const dim3 grid((unsigned)max_tiles(a.T, a.E, 16), (unsigned)((a.N + 63) / 64));
    hipLaunchKernelGGL(grouped_small_kernel, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace pq2
