// mx4_quantize.hip -- values to microscaled 4-bit floating point and back.
//
// A block of 32 values v becomes codes c and one byte b with v ~ value(c) *
// 2^(b - 127), value(c) one of +-{0, .5, 1, 1.5, 2, 3, 4, 6}: b - 127 is the
// exponent of the largest |v| less two, so that value lands in [4, 8) (above 6
// it becomes 6). Rows are dense and their length a multiple of 32, so no block
// crosses a row and both kernels run over the whole array as one run of pieces
// of eight values: 16 bytes of a 16-bit type, 4 bytes of codes, the widest
// accesses that keep every load and store of a wave contiguous. The four lanes
// of a block exchange their largest value in the VALU (quad permutes). The
// largest is taken over bit patterns, whose order as integers is that of the
// magnitudes with infinities and NaN on top, so that one compare finds both.
// Bound by HBM: 4096 x 17408 bfloat16 42 us (4.3 TB/s), back 27 (from the caches, what
// was just written). One row of 5120: 1.6 us each, a launch.
#include "mx4_device.hpp"
#include "mx4_launch.hpp"

namespace pq2 {
namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 4;            // pieces of eight values a thread has in flight
constexpr int kRun = kThreads * kPieces;

template <int FMT>
struct Piece {                        // eight values as they lie in memory
    v4u w[FMT == kF32 ? 2 : 1];
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (FMT == kF32) {
            return as_float(w[i >> 2][i & 3]);
        } else {
            const uint32_t two = w[0][i >> 1];
            return widen<FMT>((uint16_t)(i & 1 ? two >> 16 : two & 0xffffu));
        }
    }
};

// n: pieces, a multiple of four, so a block's lanes are in range together.
template <int FMT>
__global__ __launch_bounds__(kThreads) void mx4_quantize_kernel(const void *__restrict__ x,
                                                                uint32_t *__restrict__ codes,
                                                                uint8_t *__restrict__ scales,
                                                                int64_t n) {
    for (int64_t first = (int64_t)blockIdx.x * kRun + threadIdx.x; first < n;
         first += (int64_t)gridDim.x * kRun) {
        Piece<FMT> v[kPieces];
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int64_t i = first + p * kThreads;
            if (i < n) v[p] = static_cast<const Piece<FMT> *>(x)[i];
        }
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int64_t i = first + p * kThreads;
            if (i >= n) continue;
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = max(top, bits_of(v[p][j]) & 0x7fffffffu);
            top = max(top, (uint32_t)dpp_xor1((int)top));
            top = max(top, (uint32_t)dpp_xor2((int)top));
            const uint32_t byte = mx_scale_byte(top);
            const float scale = mx_scale(byte);
            uint32_t c = 0;
            c = mx_encode2<0>(c, v[p][0], v[p][1], scale);
            c = mx_encode2<1>(c, v[p][2], v[p][3], scale);
            c = mx_encode2<2>(c, v[p][4], v[p][5], scale);
            c = mx_encode2<3>(c, v[p][6], v[p][7], scale);
            codes[i] = byte == 255u ? 0u : c;
            if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
        }
    }
}

// Every value is exact in bfloat16 and float32 but for those beyond the type's
// range; float16 is rounded to nearest even from the float32 value.
template <int FMT>
__global__ __launch_bounds__(kThreads) void mx4_dequantize_kernel(
    const uint32_t *__restrict__ codes, const uint8_t *__restrict__ scales, void *__restrict__ x,
    int64_t n) {
    for (int64_t first = (int64_t)blockIdx.x * kRun + threadIdx.x; first < n;
         first += (int64_t)gridDim.x * kRun) {
        uint32_t c[kPieces], b[kPieces];
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int64_t i = first + p * kThreads;
            if (i < n) {
                c[p] = codes[i];
                b[p] = scales[i >> 2];
            }
        }
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int64_t i = first + p * kThreads;
            if (i >= n) continue;
            const float scale = mx_scale(b[p]);
            Piece<FMT> out;
            auto two = [&](int byte, v2f v) __attribute__((always_inline)) {
                if constexpr (FMT == kF32) {
                    out.w[byte >> 1][2 * (byte & 1)] = bits_of(v.x);
                    out.w[byte >> 1][2 * (byte & 1) + 1] = bits_of(v.y);
                } else {
                    out.w[0][byte] = pack16(FMT, v.x, v.y);
                }
            };
            two(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[p], scale, 0));
            two(1, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[p], scale, 1));
            two(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[p], scale, 2));
            two(3, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[p], scale, 3));
            static_cast<Piece<FMT> *>(x)[i] = out;
        }
    }
}

// A launch holds fewer than 2^32 threads: longer arrays go round again.
unsigned grid(int64_t n) {
    const int64_t blocks = (n + kRun - 1) / kRun;
    return (unsigned)(blocks < (1 << 22) ? blocks : 1 << 22);
}

}  // namespace

hipError_t launch_mx4_quantize(const void *x, int format, uint8_t *codes, uint8_t *scales,
                               int64_t M, int64_t K, hipStream_t stream) {
    const int64_t n = M * K / 8;
    uint32_t *c = reinterpret_cast<uint32_t *>(codes);
    const auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(grid(n)), dim3(kThreads), 0, stream, x, c, scales, n);
        return hipGetLastError();
    };
    return format == kF32 ? run(mx4_quantize_kernel<kF32>)
         : format == kBf16 ? run(mx4_quantize_kernel<kBf16>)
                           : run(mx4_quantize_kernel<kF16>);
}

hipError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, void *x, int format,
                                 int64_t M, int64_t K, hipStream_t stream) {
    const int64_t n = M * K / 8;
    const uint32_t *c = reinterpret_cast<const uint32_t *>(codes);
    const auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(grid(n)), dim3(kThreads), 0, stream, c, scales, x, n);
        return hipGetLastError();
    };
    return format == kF32 ? run(mx4_dequantize_kernel<kF32>)
         : format == kBf16 ? run(mx4_dequantize_kernel<kBf16>)
                           : run(mx4_dequantize_kernel<kF16>);
}

}  // namespace pq2
