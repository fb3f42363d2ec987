// mx4_launch.hpp -- host-side launchers of the MX4 kernels. Arguments are
// validated by the C ABI layer before any launcher runs; no size is zero.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pq2 {

hipError_t launch_mx4_quantize(const void *x, int format, uint8_t *codes, uint8_t *scales,
                               int64_t M, int64_t K, hipStream_t stream);
hipError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, void *x, int format,
                                 int64_t M, int64_t K, hipStream_t stream);

// pq2_mx4_gemm and pq2_mx4_gated: N is the product's columns, for the gated
// block its width F (the weights then have 2 F rows).
struct Mx4Args {
    const uint8_t *a, *as;       // [M][K / 2], [M][K / 32]
    const uint8_t *w, *ws;       // [N or 2 F][...]
    void *y;                     // [M][N] (the gated block's h, or nullptr)
    int y_format;                // of y and gu
    int act;                     // of the gated block
    uint8_t *hq, *hs;            // [M][F / 2], [M][F / 32] or nullptr
    void *gu;                    // [M][2 F] or nullptr
    int64_t M, N, K;
};
hipError_t launch_mx4_gemm(const Mx4Args &a, bool gated, void *work, size_t work_bytes,
                           hipStream_t stream);
size_t mx4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, bool gated);

// dx = dy W: dy [M][N], W [N][K]. With gu, the gated block's backward pass: dy
// is then dh [M][F] with N = 2 F, and dgu [M][N] (given, or in the workspace)
// what multiplies W.
struct Mx4GradArgs {
    const void *dy;
    const uint8_t *w, *ws;
    void *dx;
    int format;                  // of all of dy, gu, dgu and dx
    const void *gu;
    void *dgu;
    int act;
    int64_t M, N, K;
};
hipError_t launch_mx4_grad(const Mx4GradArgs &a, void *work, size_t work_bytes,
                           hipStream_t stream);
// Least and most bytes of workspace: what the call cannot do without, and what
// its fastest plan takes.
size_t mx4_grad_least_bytes(int64_t M, int64_t N, int format, bool gated, bool keeps_dgu);
size_t mx4_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int format, bool gated,
                                bool keeps_dgu);

}  // namespace pq2
