// Device helpers of the activation operators (zs_act.hip, zs_wgrad.hip): 16-byte accesses at
// any element alignment, element conversions, and the 8-bit codes with power-of-two scales.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zs_act.h"
#include "zs_internal.h"

namespace zs {
namespace act {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
// The same vectors at the alignment of their elements: matrices may start anywhere and have
// any row stride, and gfx950 takes 16-byte global accesses at any address, in one
// instruction (a misaligned one touches one cache line more).
typedef v4u v4u_a2 __attribute__((aligned(2)));
typedef v4u v4u_a4 __attribute__((aligned(4)));

__device__ __forceinline__ float bits_f(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t f_bits(float f) { return __float_as_uint(f); }

// ------------------------------------------------------------------ 2-byte elements

template <int DT>
__device__ __forceinline__ float lo_f(uint32_t w) {  // the low half of a word
  if constexpr (DT == ZS_BF16) return bits_f(w << 16);
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w)));
}
template <int DT>
__device__ __forceinline__ float hi_f(uint32_t w) {
  if constexpr (DT == ZS_BF16) return bits_f(w & 0xFFFF0000u);
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w >> 16)));
}
// fp32 -> 2 bytes, round to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t half_bits(float f) {
  if constexpr (DT == ZS_BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
  return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
}
template <int DT>
__device__ __forceinline__ uint32_t pair_bits(float a, float b) {
  return half_bits<DT>(a) | (half_bits<DT>(b) << 16);
}

template <int DT>
__device__ __forceinline__ void widen8(const v4u& w, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = lo_f<DT>(w[j]);
    f[2 * j + 1] = hi_f<DT>(w[j]);
  }
}
template <int DT>
__device__ __forceinline__ v4u narrow8(const float (&f)[8]) {
  v4u w;
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = pair_bits<DT>(f[2 * j], f[2 * j + 1]);
  return w;
}

// The first cnt (0 .. 8) of eight consecutive 2-byte elements; the others read as zero and
// their memory is not touched.
__device__ __forceinline__ v4u load8h(const uint16_t* p, int cnt) {
  if (cnt >= 8) return *reinterpret_cast<const v4u_a2*>(p);
  v4u w = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < cnt) w[j >> 1] |= static_cast<uint32_t>(p[j]) << ((j & 1) * 16);
  return w;
}
__device__ __forceinline__ v4u load8h_nt(const uint16_t* p, int cnt) {
  if (cnt >= 8) return __builtin_nontemporal_load(reinterpret_cast<const v4u_a2*>(p));
  return load8h(p, cnt);
}
__device__ __forceinline__ void store8h(uint16_t* p, const v4u& w, int cnt) {
  if (cnt >= 8) {
    __builtin_nontemporal_store(w, reinterpret_cast<v4u_a2*>(p));
    return;
  }
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < cnt) p[j] = static_cast<uint16_t>(w[j >> 1] >> ((j & 1) * 16));
}

// ------------------------------------------------------------------ 8-bit codes

constexpr int kActGroup = 32;

// Scale byte of a group from the bits of its largest magnitude (as integers the bits of
// non-negative floats are in the floats' order, infinities and NaN above all others).
// 448 = 1.75 * 2^8 and 127 = 1.984375 * 2^6: an amax of 1.M * 2^(E-127) fits under
// qmax * 2^(E - 127 - 8 or 6) exactly if its mantissa does, otherwise one step more.
template <int CODE>
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255;
  const int e = static_cast<int>(amax_bits >> 23);
  const uint32_t m = amax_bits & 0x7FFFFFu;
  const int b = CODE == ZS_E4M3 ? e - 8 + (m > 0x600000u) : e - 6 + (m > 0x7E0000u);
  return b > 0 ? b : 0;
}
// 2^(b - 127) and its reciprocal (b <= 249 for codes written here), NaN for b = 255.
__device__ __forceinline__ float scale_value(int b) {
  return bits_f(b == 255 ? 0x7FC00000u : b == 0 ? 0x00400000u : static_cast<uint32_t>(b) << 23);
}
__device__ __forceinline__ float scale_inverse(int b) { return bits_f(static_cast<uint32_t>(254 - b) << 23); }

// Codes of eight values under scale byte b: x / s is exact (a power of two), the rounding to
// the code is the only one.  gfx950 divides and rounds a pair to e4m3 in one instruction, which
// takes the scale from the exponent field alone.  For int8 the sum with 1.5 * 2^23 rounds to an
// integer, to nearest even, whose low byte is the code.
template <int CODE>
__device__ __forceinline__ v2u encode8(const float (&f)[8], int b) {
  if (b == 255) return v2u{0u, 0u};
  v2u c;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float* q = f + 4 * j;
    if constexpr (CODE == ZS_E4M3) {
      typedef short v2s __attribute__((ext_vector_type(2)));
      const float s = bits_f(static_cast<uint32_t>(b) << 23);
      v2s w = {0, 0};
      w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, q[0], q[1], s, false);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, q[2], q[3], s, true);
      c[j] = __builtin_bit_cast(uint32_t, w);
    } else {
      constexpr float kRound = 12582912.0f;
      const float inv = scale_inverse(b);
      const uint32_t i0 = f_bits(q[0] * inv + kRound), i1 = f_bits(q[1] * inv + kRound);
      const uint32_t i2 = f_bits(q[2] * inv + kRound), i3 = f_bits(q[3] * inv + kRound);
      c[j] = (i0 & 0xFFu) | ((i1 & 0xFFu) << 8) | ((i2 & 0xFFu) << 16) | (i3 << 24);
    }
  }
  return c;
}

// Values of four codes.
template <int CODE>
__device__ __forceinline__ void decode4(uint32_t c, float s, float* f) {
  if constexpr (CODE == ZS_E4M3) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c), false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c), true);
    f[0] = a[0] * s;
    f[1] = a[1] * s;
    f[2] = b[0] * s;
    f[3] = b[1] * s;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = static_cast<float>(static_cast<int8_t>(c >> (8 * j))) * s;
  }
}
template <int CODE>
__device__ __forceinline__ void decode8(const v2u& c, float s, float (&f)[8]) {
  decode4<CODE>(c[0], s, f);
  decode4<CODE>(c[1], s, f + 4);
}

// A value for an fp16 destination: code * s may lie up to one code step past the largest
// fp16 number although the source did not, and comes back as that number; NaN stays.
__device__ __forceinline__ float to_fp16_range(float v) { return fabsf(v) > 65504.0f ? copysignf(65504.0f, v) : v; }
template <int DT>
__device__ __forceinline__ void clamp8(float (&f)[8]) {
  if constexpr (DT == ZS_FP16) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = to_fp16_range(f[j]);
  }
}

// Bits of the largest magnitude of eight values (a NaN among them wins), then over the four
// neighbouring lanes that hold a group of 32 (two quad permutes).
__device__ __forceinline__ uint32_t group_amax(const float (&f)[8]) {
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; j += 2)
    top = __builtin_elementwise_maximum(__builtin_elementwise_maximum(top, fabsf(f[j])), fabsf(f[j + 1]));
  uint32_t m = f_bits(top) & 0x7FFFFFFFu;
  uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0xB1, 0xF, 0xF, true));
  m = o > m ? o : m;
  o = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x4E, 0xF, 0xF, true));
  return o > m ? o : m;
}

// Encode a lane's eight values (lanes 4i .. 4i+3 hold one group) and store codes and scale
// at chunk index `at` (in units of eight codes) of the checkpoint.
template <int CODE>
__device__ __forceinline__ void encode_store(const float (&f)[8], uint8_t* codes, uint8_t* scales, int64_t at) {
  const int b = scale_byte<CODE>(group_amax(f));
  const v2u c = encode8<CODE>(f, b);
  __builtin_nontemporal_store(c, reinterpret_cast<v2u*>(codes) + at);
  if ((threadIdx.x & 3) == 0) scales[at >> 2] = static_cast<uint8_t>(b);
}

}  // namespace act
}  // namespace zs
