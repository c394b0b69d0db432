// Codes of the moments in fewer bits (include/zds.h describes the formats):
// encoding and decoding of quads, the exponent byte of a block of 32, and the
// random bits of a wave's quads. Shared by the conversions and the step.
//
// Both 8-bit formats are the top bits of an fp32 number after a scaling by a
// power of two that puts the block's largest magnitude at the format's largest
// exponent field and the format's linear range at fp32's subnormals. So one
// shift of the fp32 bits is the conversion, with whatever was added below as
// its rounding, in every range of the format and without a special case.
#pragma once

#include "zds_device.h"
#include "zds_random.h"

namespace zds {

template <int F>
struct StateFormat;
template <>
struct StateFormat<ZDS_STATE_E4M3> {
  static constexpr int top = 15;       // exponent field of the block's largest binade
  static constexpr uint32_t least = 0; // least exponent byte
  static constexpr uint32_t mask = 0x7fu;
};
template <>
struct StateFormat<ZDS_STATE_UE5M3> {
  static constexpr int top = 31;
  static constexpr uint32_t least = 11;  // the least code, 2^(s - 160), stays an fp32 number
  static constexpr uint32_t mask = 0xffu;
};

// Magnitude bits of a value. The order of the bits is the order of the
// magnitudes, with infinity and NaN at the top.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The largest magnitude over the 8 lanes (32 elements) of a block, on each of
// them: exchanges inside pairs, inside quads, and of the half row's quads.
__device__ __forceinline__ uint32_t block_max(uint32_t a) {
  const auto over = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
  a = over(a, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(a), 0xB1, 0xf, 0xf, false)));
  a = over(a, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(a), 0x4E, 0xf, 0xf, false)));
  a = over(a, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(a), 0x141, 0xf, 0xf, false)));
  return a;
}

// Exponent byte of a block whose largest magnitude has these bits: its
// exponent field, one more over 1.75.
template <int F>
__device__ __forceinline__ uint32_t exponent_byte(uint32_t amax) {
  const uint32_t s = (amax + 0x1fffffu) >> 23;
  const uint32_t t = s < 255u ? s : 255u;
  return t > StateFormat<F>::least ? t : StateFormat<F>::least;
}

// One code. r: 16 random bits, used as they come (RANDOM only).
template <int F, bool RANDOM>
__device__ __forceinline__ uint32_t encode1(float x, uint32_t s, uint32_t r) {
  const uint32_t bits = __float_as_uint(x), mag = bits & 0x7fffffffu;
  const uint32_t z = __float_as_uint(ldexpf(__uint_as_float(mag), StateFormat<F>::top - static_cast<int>(s)));
  const uint32_t up = RANDOM ? (r << 4) + 8u : 0x7ffffu + ((z >> 20) & 1u);
  uint32_t c = (z + up) >> 20;
  if (F == ZDS_STATE_UE5M3) {
    c = mag != 0u && c == 0u ? 1u : c;
    c = mag >= 0x7f800000u || (bits != mag && mag != 0u) ? 0xffu : c;
    return c;
  }
  c = mag >= 0x7f800000u ? 0x7fu : c;
  return c | ((bits >> 24) & 0x80u);
}

template <int F>
__device__ __forceinline__ float decode1(uint32_t code, uint32_t s) {
  const uint32_t mag = code & StateFormat<F>::mask;
  float x = ldexpf(__uint_as_float(mag << 20), static_cast<int>(s) - StateFormat<F>::top);
  x = mag == StateFormat<F>::mask ? __uint_as_float(0x7fc00000u) : x;
  return F == ZDS_STATE_E4M3 && code > 0x7fu ? -x : x;
}

// The 16-bit format: the value's top bits.
template <bool RANDOM>
__device__ __forceinline__ uint32_t encode_bf16(float x, uint32_t r) {
  const uint32_t bits = __float_as_uint(x), mag = bits & 0x7fffffffu;
  const uint32_t up = RANDOM ? r : 0x7fffu + ((mag >> 16) & 1u);
  uint32_t c = (mag + up) >> 16;
  c = mag != 0u && c == 0u ? 1u : c;
  if (mag >= 0x7f800000u) c = (mag >> 16) | (mag > 0x7f800000u ? 0x40u : 0u);
  return c | ((bits >> 16) & 0x8000u);
}

// The two bytes of each 16-bit half exchanged.
__device__ __forceinline__ uint32_t swap_bytes(uint32_t w) { return __builtin_amdgcn_perm(0u, w, 0x02030001u); }

// Random bits of the two quads that a lane holds of a wave's unit of 512
// elements: row 0's quad `lane` and row 1's (256 elements further), two words
// each (four 16-bit halves in element order). A call of the generator covers 8
// elements, the quads of an even lane and the odd one after it: the even lane
// makes row 0's call and the odd one row 1's, and they exchange the half that
// is the other's. call0: the call of the unit's first element.
struct QuadBits {
  uint32_t r0[2], r1[2];
};
__device__ __forceinline__ QuadBits unit_random_bits(uint64_t seed, uint64_t call0, uint32_t steps_seen, int lane) {
  const bool odd = lane & 1;
  const RandomWords q = random_words(seed, call0 + static_cast<uint64_t>((lane >> 1) + (odd ? 32 : 0)), steps_seen,
                                     kStreamRounding);
  const int g0 = static_cast<int>(odd ? q.w[0] : q.w[2]), g1 = static_cast<int>(odd ? q.w[1] : q.w[3]);
  const uint32_t t0 = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, g0, 0xB1, 0xf, 0xf, false));
  const uint32_t t1 = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, g1, 0xB1, 0xf, 0xf, false));
  return odd ? QuadBits{{t0, t1}, {q.w[2], q.w[3]}} : QuadBits{{q.w[0], q.w[1]}, {t0, t1}};
}

// Four codes of a quad in a word. w: its 8 random bytes.
template <int F, bool RANDOM>
__device__ __forceinline__ uint32_t encode_quad(const float (&x)[4], uint32_t s, const uint32_t (&w)[2]) {
  const uint32_t a = F == ZDS_STATE_E4M3 ? w[0] : swap_bytes(w[0]), b = F == ZDS_STATE_E4M3 ? w[1] : swap_bytes(w[1]);
  return encode1<F, RANDOM>(x[0], s, a & 0xffffu) | (encode1<F, RANDOM>(x[1], s, a >> 16) << 8) |
         (encode1<F, RANDOM>(x[2], s, b & 0xffffu) << 16) | (encode1<F, RANDOM>(x[3], s, b >> 16) << 24);
}
template <bool RANDOM>
__device__ __forceinline__ u32x2 encode_quad_bf16(const float (&x)[4], const uint32_t (&w)[2]) {
  const uint32_t a = swap_bytes(w[0]), b = swap_bytes(w[1]);
  return u32x2{encode_bf16<RANDOM>(x[0], a & 0xffffu) | (encode_bf16<RANDOM>(x[1], a >> 16) << 16),
               encode_bf16<RANDOM>(x[2], b & 0xffffu) | (encode_bf16<RANDOM>(x[3], b >> 16) << 16)};
}
template <int F>
__device__ __forceinline__ void decode_quad(uint32_t w, uint32_t s, float (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = decode1<F>((w >> (8 * i)) & 0xffu, s);
}

// Elements a wave takes at once, and the largest n of a call.
constexpr int kStateUnit = 512;
constexpr int64_t kStateMost = int64_t(1) << 40;

}  // namespace zds
