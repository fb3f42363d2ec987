// mx4_device.hpp -- device-side helpers of the microscaled 4-bit (MX4) kernels
// (gfx950): formats, activations, the scaled matrix instruction.
#pragma once

#include "pq2_device.hpp"

#include <hip/hip_fp16.h>

namespace pq2 {

constexpr int kMxBlock = 32;          // values per scale

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f32 __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));

// By value: a bit cast of a vector's element in place reads the vector's first.
__device__ __forceinline__ uint32_t bits_of(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ float as_float(uint32_t v) { return __builtin_bit_cast(float, v); }

// Types of unquantised values (PQ2_ACT_*).
constexpr int kF32 = 0, kBf16 = 1, kF16 = 2;

template <int FMT> struct MxType;
template <> struct MxType<kF32> { typedef float T; };
template <> struct MxType<kBf16> { typedef uint16_t T; };
template <> struct MxType<kF16> { typedef uint16_t T; };

template <int FMT>
__device__ __forceinline__ float widen(typename MxType<FMT>::T v) {
    if constexpr (FMT == kF32)
        return v;
    else if constexpr (FMT == kBf16)
        return as_float((uint32_t)v << 16);
    else
        return half_bits_to_float(v);
}

// float32 -> the format, to nearest even (NaN stays NaN).
template <int FMT>
__device__ __forceinline__ typename MxType<FMT>::T narrow(float v) {
    if constexpr (FMT == kF32)
        return v;
    else if constexpr (FMT == kBf16)
        return bf16_rne(v);
    else
        return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// The float32 power of two a scale byte stands for, as the conversions take it:
// they read its exponent field alone, so byte 0 (2^-127) is the zero pattern
// and byte 255 (not a number) infinity's.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
    return as_float(byte << 23);
}

// Scale byte of a block whose largest |x| has these float32 bits: the largest
// value's exponent less two (the format's largest value is 1.5 * 2^2), at least
// 2^-127; 255 where a value is not finite.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? 255u : e < 2u ? 0u : e - 2u;
}

// Two values as the codes of a byte (the first in the low half), rounded to
// nearest, ties to the even code, beyond 6 to 6: byte BYTE of the word, the
// others kept.
template <int BYTE>
__device__ __forceinline__ uint32_t mx_encode2(uint32_t word, float a, float b, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, a, b, scale, BYTE);
}

// a b^T over 128 values: lane l holds 32 consecutive values of row l % 16,
// block l / 16, and their scale in byte BYTE of its word; result i is that of
// a's row 4 (l / 16) + i and b's row l % 16.
template <int BYTE = 0>
__device__ __forceinline__ v4f32 mfma_mx4(v4i a, v4i b, v4f32 c, uint32_t sa, uint32_t sb) {
    const v8i wa = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
    const v8i wb = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, wb, c, 4, 4, BYTE, (int)sa, BYTE,
                                                           (int)sb);
}

// Activations of the gated block (PQ2_GATE_*).
constexpr int kSilu = 0, kGelu = 1, kGeluTanh = 2;

// 1 / (1 + e^-z); 0 and 1 in the far ends.
__device__ __forceinline__ float logistic(float z) { return 1.0f / (1.0f + expf(-z)); }

// The inner term of the tanh form, doubled: (1 + tanh z) / 2 is the logistic
// function of 2 z, which keeps its relative error where tanh nears -1.
__device__ __forceinline__ float gelu_inner(float g) {
    return 1.5957691216057308f * (g + 0.044715f * g * g * g);   // 2 sqrt(2 / pi)
}

// a(g). The exact form's normal distribution function is written with erfc for
// the same reason.
template <int ACT>
__device__ __forceinline__ float gate_act(float g) {
    if constexpr (ACT == kSilu)
        return g * logistic(g);
    else if constexpr (ACT == kGelu)
        return 0.5f * g * erfcf(-0.70710678118654752f * g);
    else
        return g * logistic(gelu_inner(g));
}

// a(g) and a'(g).
template <int ACT>
__device__ __forceinline__ void gate_act_slope(float g, float &a, float &d) {
    if constexpr (ACT == kSilu) {
        const float s = logistic(g);
        a = g * s;
        d = s + a * (1.0f - s);
    } else if constexpr (ACT == kGelu) {
        const float c = 0.5f * erfcf(-0.70710678118654752f * g);
        a = g * c;
        d = c + g * (0.3989422804014327f * expf(-0.5f * g * g));
    } else {
        const float s = logistic(gelu_inner(g));
        a = g * s;
        // from 20 on s is 0 or 1 and the second term 0; g's square would make it NaN
        // once infinite (max and min drop a NaN of g, which s has)
        const float c = fminf(fmaxf(g, -20.0f), 20.0f);
        d = s + c * s * (1.0f - s) * (1.5957691216057308f * (1.0f + 0.134145f * c * c));
    }
}

// One value into an array of a format known at run time.
__device__ __forceinline__ void store_fmt(void *y, int fmt, int64_t i, float v) {
    if (fmt == kF32)
        static_cast<float *>(y)[i] = v;
    else
        static_cast<uint16_t *>(y)[i] = fmt == kBf16 ? narrow<kBf16>(v) : narrow<kF16>(v);
}

__device__ __forceinline__ uint32_t pack16(int fmt, float a, float b) {
    const uint32_t lo = fmt == kBf16 ? narrow<kBf16>(a) : narrow<kF16>(a);
    const uint32_t hi = fmt == kBf16 ? narrow<kBf16>(b) : narrow<kF16>(b);
    return lo | (hi << 16);
}

}  // namespace pq2
