// Blocks of 128 numbers in 8-bit floating point (e4m3) with one 32-bit scale: what the kernels that make and read
// them share.
//
// The scale that is made here is the smallest power of two, 2^-126 at least, that brings the largest finite magnitude of
// the block to 448 (e4m3's largest) or below; 1 for a block of zeros.  A power of two costs e4m3 nothing but the last
// part of one binade at its lower end, dividing by it is exact, and so a block in 8 bits is the same on any path:
// one rounding, to nearest, of each number.  What is not finite becomes NaN.  Scales that are read may be any number.
#pragma once

#include <cuda_fp8.h>

#include "groups.h"

namespace sg {

constexpr int kBlock8 = 128;   // numbers that share a scale
constexpr int kPiece = 8;      // consecutive numbers of a lane: 16 lanes hold a block

inline int64_t blocks8(int64_t n) { return ceil_div(n, kBlock8); }

// A piece of a row in 32 bits, zeros past its end.  `whole`: rows start on 16 bytes.
template <typename T>
__device__ __forceinline__ void load_piece(const T* __restrict__ row, int64_t c, int64_t cols, bool whole, float (&v)[kPiece]) {
  if (whole && c + kPiece <= cols) {
    constexpr int kWords = sizeof(T) * kPiece / 16;
    uint4 w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(row + c)[i];
#pragma unroll
    for (int e = 0; e < kPiece; ++e) v[e] = to_f32(reinterpret_cast<const T*>(w)[e]);
  } else {
#pragma unroll
    for (int e = 0; e < kPiece; ++e) v[e] = c + e < cols ? to_f32(row[c + e]) : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void store_piece(T* __restrict__ row, int64_t c, int64_t cols, bool whole, const float (&v)[kPiece]) {
  if (whole && c + kPiece <= cols) {
    constexpr int kWords = sizeof(T) * kPiece / 16;
    uint4 w[kWords];
#pragma unroll
    for (int e = 0; e < kPiece; ++e) reinterpret_cast<T*>(w)[e] = from_f32<T>(v[e]);
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4*>(row + c)[i] = w[i];
  } else {
#pragma unroll
    for (int e = 0; e < kPiece; ++e)
      if (c + e < cols) row[c + e] = from_f32<T>(v[e]);
  }
}
// the same in 8 bits (rows start on 16 bytes); nothing past the row's end is touched
__device__ __forceinline__ uint2 load_piece8(const uint8_t* __restrict__ row, int64_t c, int64_t cols) {
  if (c + kPiece <= cols) return *reinterpret_cast<const uint2*>(row + c);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < kPiece; ++e)
    if (c + e < cols) w[e / 4] |= static_cast<uint32_t>(row[c + e]) << (e % 4 * 8);
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_piece8(uint8_t* __restrict__ row, int64_t c, int64_t cols, uint2 q) {
  if (c + kPiece <= cols) {
    *reinterpret_cast<uint2*>(row + c) = q;
  } else {
#pragma unroll
    for (int e = 0; e < kPiece; ++e)
      if (c + e < cols) row[c + e] = static_cast<uint8_t>((e < 4 ? q.x : q.y) >> (e % 4 * 8));
  }
}

// The bits of the largest magnitude of a piece (integers order magnitudes as the floats do, what is not finite above them)
__device__ __forceinline__ uint32_t most_of(const float (&v)[kPiece]) {
  uint32_t most = 0;
#pragma unroll
  for (int e = 0; e < kPiece; ++e) most = max(most, __float_as_uint(v[e]) & 0x7fffffffu);
  return most;
}
// ... and the largest finite one, for blocks that hold others too
__device__ __forceinline__ uint32_t most_finite_of(const float (&v)[kPiece]) {
  uint32_t most = 0;
#pragma unroll
  for (int e = 0; e < kPiece; ++e) {
    const uint32_t m = __float_as_uint(v[e]) & 0x7fffffffu;
    most = max(most, m < 0x7f800000u ? m : 0u);
  }
  return most;
}
__device__ __forceinline__ bool all_finite(uint32_t most) { return most < 0x7f800000u; }
// the largest of the 16 lanes of a block
__device__ __forceinline__ uint32_t most_of_block(uint32_t most) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
  return most;
}

struct Scale8 {
  float scale, inverse;
};
// 448 = 1.75 * 2^8: the exponent of the largest magnitude less 8, one more where its mantissa is above 1.75
__device__ __forceinline__ Scale8 scale_of(uint32_t most) {
  if (most == 0) return {1.0f, 1.0f};
  const int e = max(static_cast<int>((most + 0x1fffffu) >> 23) - 8, 1);
  return {__uint_as_float(static_cast<uint32_t>(e) << 23), __uint_as_float(static_cast<uint32_t>(254 - e) << 23)};
}

__device__ __forceinline__ uint2 quantise_piece(const float (&v)[kPiece], float inverse) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * inverse, v[4 * i + 1] * inverse), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * inverse, v[4 * i + 3] * inverse), __NV_SATFINITE, __NV_E4M3);
    w[i] = __byte_perm(lo, hi, 0x5410);
  }
  return make_uint2(w[0], w[1]);
}
// A piece of a block whose largest magnitude is `most`: its scale and its 8 bits.  The conversion saturates: infinities
// are made NaN before it.  All lanes of the block call it.
__device__ __forceinline__ uint2 quantise_block(const float (&v)[kPiece], uint32_t most, Scale8* s) {
  if (__all_sync(0xffffffffu, all_finite(most))) {
    *s = scale_of(most);
    return quantise_piece(v, s->inverse);
  }
  *s = scale_of(most_of_block(most_finite_of(v)));
  float w[kPiece];
#pragma unroll
  for (int e = 0; e < kPiece; ++e) w[e] = fabsf(v[e]) < INFINITY ? v[e] : NAN;
  return quantise_piece(w, s->inverse);
}
__device__ __forceinline__ void dequantise_piece(uint2 q, float scale, float (&v)[kPiece]) {
#pragma unroll
  for (int e = 0; e < kPiece; e += 2) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>((e < 4 ? q.x : q.y) >> (e % 4 * 8) & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[e] = f.x * scale;
    v[e + 1] = f.y * scale;
  }
}

// To 16 bits, without the infinity that f16's largest numbers would become when their 8 bits were rounded up.
template <typename T>
__device__ __forceinline__ float held(float v) { return v; }
template <>
__device__ __forceinline__ float held<__half>(float v) { return fabsf(v) > 65504.0f ? copysignf(65504.0f, v) : v; }

// 1 / (1 + exp(-g)).  SHORT: the short exponential and division, for results that are rounded to 16 bits and |g| up to kShortGate:
// relative error below 2^-17 there (the exponent -g log2(e) is rounded to 2^-18 at most and its factor to 2^-26 of 126, times
// ln 2; the approximations themselves a few units).  The short division gives 0 where its divisor passes 2^126 (g below -87.3).
constexpr float kShortGate = 87.0f;
template <bool SHORT>
__device__ __forceinline__ float sigmoid(float g) {
  return SHORT ? __fdividef(1.0f, 1.0f + __expf(-g)) : 1.0f / (1.0f + expf(-g));
}

}  // namespace sg
