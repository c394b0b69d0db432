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

// The same over the 32 lanes of a block that has one element on each.
__device__ __forceinline__ uint32_t block_max_lanes(uint32_t a) {
  const auto over = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
  a = block_max(a);
  a = over(a, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(a), 0x128, 0xf, 0xf, false)));  // row_ror:8
  return over(a, static_cast<uint32_t>(__builtin_amdgcn_ds_swizzle(static_cast<int>(a), 0x401f)));  // lane ^ 16
}

// Exponent byte of a block whose largest magnitude has these bits: its
// exponent field, one more over 1.75.
template <int F>
__device__ __forceinline__ uint32_t exponent_byte(uint32_t amax) {
  const uint32_t s = (amax + 0x1fffffu) >> 23;
  const uint32_t t = s < 255u ? s : 255u;
  return t > StateFormat<F>::least ? t : StateFormat<F>::least;
}

// One code of any value. r: 16 random bits, used as they come (RANDOM only).
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

// The value of one code.
template <int F>
__device__ __forceinline__ float decode1(uint32_t code, uint32_t s) {
  const uint32_t mag = code & StateFormat<F>::mask;
  const float x = ldexpf(__uint_as_float(mag << 20), static_cast<int>(s) - StateFormat<F>::top);
  if (mag == StateFormat<F>::mask) return __uint_as_float(0x7fc00000u);
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

// The 16 random bits of the element with flat index f.
__device__ __forceinline__ uint32_t element_random_bits(uint64_t seed, uint64_t f, uint32_t steps_seen) {
  const RandomWords q = random_words(seed, f >> 3, steps_seen, kStreamRounding);
  const uint32_t lo = (f & 2) ? q.w[1] : q.w[0], hi = (f & 2) ? q.w[3] : q.w[2];
  const uint32_t w = (f & 4) ? hi : lo;
  return (f & 1) ? w >> 16 : w & 0xffffu;
}

// Four codes of a quad in a word. amax: the block's largest magnitude; w: the
// quad's 8 random bytes. (z + 16 r + 8) >> 20 is ((z + 8) >> 4) + r, shifted by
// 16, so that each random half is added as it lies; the code is then the upper
// half's low byte (the sign stays four bits above it: a magnitude's sum never
// reaches it), and byte permutations gather the four. What the formats say of
// special values is left to a branch that a wave takes only where it holds one:
// infinities and NaN are known from amax, a UE5M3 code 0 from the least sum, a
// negative value (where NONNEGATIVE does not rule them out) from the largest.
template <int F, bool RANDOM, bool NONNEGATIVE = false>
__device__ __forceinline__ uint32_t encode_quad(const float (&x)[4], uint32_t s, uint32_t amax, const uint32_t (&w)[2]) {
  const uint32_t a = F == ZDS_STATE_E4M3 ? w[0] : swap_bytes(w[0]), b = F == ZDS_STATE_E4M3 ? w[1] : swap_bytes(w[1]);
  const uint32_t r[4] = {a & 0xffffu, a >> 16, b & 0xffffu, b >> 16};
  const int k = StateFormat<F>::top - static_cast<int>(s);
  uint32_t t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t z = __float_as_uint(ldexpf(x[i], k));
    t[i] = RANDOM ? ((z + 8u) >> 4) + r[i] : (z + 0x7ffffu + ((z >> 20) & 1u)) >> 4;
  }
  // (selectors 0-3 name bytes of the second operand, 4-7 of the first)
  uint32_t p = __builtin_amdgcn_perm(t[1], t[0], 0x07060302u), q = __builtin_amdgcn_perm(t[3], t[2], 0x07060302u);
  if (F == ZDS_STATE_E4M3) {
    p |= (p >> 4) & 0x00800080u;
    q |= (q >> 4) & 0x00800080u;
  }
  uint32_t c = __builtin_amdgcn_perm(q, p, 0x06040200u);
  bool special = amax >= 0x7f800000u;
  if (F == ZDS_STATE_UE5M3) {
    uint32_t least = t[0];
    uint32_t most = t[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      least = t[i] < least ? t[i] : least;
      most = t[i] > most ? t[i] : most;
    }
    special = special || least < 0x10000u || (!NONNEGATIVE && most >= 0x8000000u);
  }
  if (special)
    c = encode1<F, RANDOM>(x[0], s, r[0]) | (encode1<F, RANDOM>(x[1], s, r[1]) << 8) |
        (encode1<F, RANDOM>(x[2], s, r[2]) << 16) | (encode1<F, RANDOM>(x[3], s, r[3]) << 24);
  return c;
}
template <bool RANDOM>
__device__ __forceinline__ u32x2 encode_quad_bf16(const float (&x)[4], const uint32_t (&w)[2]) {
  const uint32_t a = swap_bytes(w[0]), b = swap_bytes(w[1]);
  return u32x2{encode_bf16<RANDOM>(x[0], a & 0xffffu) | (encode_bf16<RANDOM>(x[1], a >> 16) << 16),
               encode_bf16<RANDOM>(x[2], b & 0xffffu) | (encode_bf16<RANDOM>(x[3], b >> 16) << 16)};
}
// E4M3 codes are the 8-bit floats that the hardware converts (two at a time,
// NaN included); of UE5M3 codes the top one is looked for in the whole word
// (a zero byte of its complement).
template <int F>
__device__ __forceinline__ void decode_quad(uint32_t w, uint32_t s, float (&x)[4]) {
  if constexpr (F == ZDS_STATE_E4M3) {
    const int k = static_cast<int>(s) - 127 - 8;  // 448 = 1.75 * 2^8 is the largest code's value
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    x[0] = ldexpf(lo[0], k);
    x[1] = ldexpf(lo[1], k);
    x[2] = ldexpf(hi[0], k);
    x[3] = ldexpf(hi[1], k);
  } else {
    const int k = static_cast<int>(s) - StateFormat<F>::top;
    x[0] = ldexpf(__uint_as_float((w << 20) & 0x0ff00000u), k);
    x[1] = ldexpf(__uint_as_float((w << 12) & 0x0ff00000u), k);
    x[2] = ldexpf(__uint_as_float((w << 4) & 0x0ff00000u), k);
    x[3] = ldexpf(__uint_as_float((w >> 4) & 0x0ff00000u), k);
    if ((~w - 0x01010101u) & w & 0x80808080u) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (((w >> (8 * i)) & 0xffu) == 0xffu) x[i] = __uint_as_float(0x7fc00000u);
    }
  }
}

// Elements a wave takes at once, and the largest n of a call.
constexpr int kStateUnit = 512;
constexpr int64_t kStateMost = int64_t(1) << 40;

}  // namespace zds
