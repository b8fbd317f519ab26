// cache.hpp -- caches in 8 or 4 bits: their formats, and their values.
//
// A group of 32 channels is held as a scale byte s (2^(s - 127); 255: the
// group is NaN) and a code for each channel.  The scale is a power of two, so
// that a value is the product of two exact factors, and gfx950's conversions
// take it with the code in one instruction; every byte of scales 0 .. 255 and
// of codes converts as the definition says (checked for all of them, to
// binary32, binary16 and bfloat16).
#pragma once

#include "dtype.hpp"
#include "tokens.hpp"

namespace mp3d {

constexpr int kPlain = 0, kE4M3 = 1, kE2M1 = 2;   // enum mp3d_cache_format
constexpr int kGroup = 32;                        // channels that share a scale

// bytes of D codes
template <int FMT>
__host__ __device__ constexpr int code_bytes(int D) { return FMT == kE4M3 ? D : (D + 1) / 2; }

__device__ __forceinline__ float scale_of(uint32_t byte)
{
    return __builtin_bit_cast(float, byte << 23);  // (the conversions read the exponent's bits alone)
}

// Two codes of a word, as two elements in a word (16-bit types) or as two
// floats: the codes of bytes 2 I, 2 I + 1 (e4m3, I = 0, 1) or those of byte I
// (e2m1, I = 0 .. 3).
template <typename T, int FMT, int I>
__device__ __forceinline__ auto widen2(uint32_t w, float scale)
{
    if constexpr (FMT == kE4M3) {
        if constexpr (T::code == F32::code) return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, I);
        else if constexpr (T::code == F16::code)
            return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, I));
        else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, I));
    } else {
        if constexpr (T::code == F32::code) return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, I);
        else if constexpr (T::code == F16::code)
            return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, I));
        else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, I));
    }
}

// 8 codes (two words, of e2m1 one) to 8 elements.
template <typename T, int FMT>
__device__ __forceinline__ void widen8(uint32_t w0, uint32_t w1, float scale, u32x4 *out)
{
    if constexpr (T::code == F32::code) {
        float f[8];
        auto put = [&](int i, auto v) {
            f[2 * i] = v[0];
            f[2 * i + 1] = v[1];
        };
        if constexpr (FMT == kE4M3) {
            put(0, widen2<T, FMT, 0>(w0, scale));
            put(1, widen2<T, FMT, 1>(w0, scale));
            put(2, widen2<T, FMT, 0>(w1, scale));
            put(3, widen2<T, FMT, 1>(w1, scale));
        } else {
            put(0, widen2<T, FMT, 0>(w0, scale));
            put(1, widen2<T, FMT, 1>(w0, scale));
            put(2, widen2<T, FMT, 2>(w0, scale));
            put(3, widen2<T, FMT, 3>(w0, scale));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            out[i] = u32x4{__builtin_bit_cast(uint32_t, f[4 * i]),
                           __builtin_bit_cast(uint32_t, f[4 * i + 1]),
                           __builtin_bit_cast(uint32_t, f[4 * i + 2]),
                           __builtin_bit_cast(uint32_t, f[4 * i + 3])};
    } else if constexpr (FMT == kE4M3) {
        out[0] = u32x4{widen2<T, FMT, 0>(w0, scale), widen2<T, FMT, 1>(w0, scale),
                       widen2<T, FMT, 0>(w1, scale), widen2<T, FMT, 1>(w1, scale)};
    } else {
        out[0] = u32x4{widen2<T, FMT, 0>(w0, scale), widen2<T, FMT, 1>(w0, scale),
                       widen2<T, FMT, 2>(w0, scale), widen2<T, FMT, 3>(w0, scale)};
    }
}

// One element of a row: channel d.
template <typename T, int FMT>
__device__ __forceinline__ float value_at(const uint8_t *codes, const uint8_t *scales, int d)
{
    const uint32_t w = FMT == kE4M3 ? codes[d] : codes[d >> 1] >> (4 * (d & 1));
    const auto v = widen2<T, FMT, 0>(w, scale_of(scales[d / kGroup]));
    if constexpr (T::code == F32::code) return v[0];
    else return T::widen((typename T::raw)(v & 0xffffu));
}

}  // namespace mp3d
