// Weights of logits as whole numbers, for engram_sample_tokens.
//
//   a = min((m - l) c, 64),  n = a rounded, f = a - n,  w = floor(2^38 P(f) 2^-n)
//
// Every float operation rounds by itself (no fused multiply-add), so the same
// weights come out of any program that does the same operations.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "f32x2.cuh"

namespace engram {
namespace sample {

// P(f) = 2^-f on [-1/2, 1/2] to 1.0e-7 of the value with the roundings: a
// weighted least-squares fit of (2^-f - 1) / f, reweighted until the error is level.
constexpr float kP1 = -0.6931472f, kP2 = 0.24022648f, kP3 = -0.055503324f, kP4 = 0.009618437f, kP5 = -0.0013398875f,
                kP6 = 0.00015353362f;
constexpr float kFar = 64.f;              // powers of two below the largest: weight 0
constexpr float kRound = 12582912.f;      // 1.5 2^23: adding it rounds to whole numbers, in the low bits

// A row's constants.
struct Scale {
  float top;      // largest logit
  float c;        // log2(e) / temperature
  bool odd;       // top or c infinite: only logits equal to top have weight
};

__device__ __forceinline__ Scale make_scale(float top, float temperature) {
  Scale s;
  s.top = top;
  s.c = __fdiv_rn(1.4426950408889634f, temperature);
  s.odd = isinf(s.c) || isinf(top);
  return s;
}

// a of two logits.  Of NaN: the minimum with it is 64.
__device__ __forceinline__ float2 exponents(const Scale& s, float x0, float x1) {
  if (s.odd) return make_float2(x0 == s.top ? 0.f : kFar, x1 == s.top ? 0.f : kFar);
  const float2 a = unpack2(mul2(add2(pack2(s.top, s.top), pack2(-x0, -x1)), pack2(s.c, s.c)));
  return make_float2(fminf(a.x, kFar), fminf(a.y, kFar));
}

// 2^38 P(f) 2^-n of two exponents, as floats.
__device__ __forceinline__ float2 weights38(float2 a) {
  const F2 a2 = pack2(a.x, a.y);
  const F2 r = add2(a2, pack2(kRound, kRound));
  const F2 n = add2(r, pack2(-kRound, -kRound));
  const float2 nn = unpack2(n);
  const F2 f = add2(a2, pack2(-nn.x, -nn.y));
  F2 y = mul2(pack2(kP6, kP6), f);
  y = mul2(add2(y, pack2(kP5, kP5)), f);
  y = mul2(add2(y, pack2(kP4, kP4)), f);
  y = mul2(add2(y, pack2(kP3, kP3)), f);
  y = mul2(add2(y, pack2(kP2, kP2)), f);
  y = mul2(add2(y, pack2(kP1, kP1)), f);
  const float2 p = unpack2(add2(y, pack2(1.f, 1.f))), k = unpack2(r);
  // the low bits of a + kRound are n: off the exponent it goes
  return make_float2(__uint_as_float(__float_as_uint(p.x) + (38u << 23) - (__float_as_uint(k.x) << 23)),
                     __uint_as_float(__float_as_uint(p.y) + (38u << 23) - (__float_as_uint(k.y) << 23)));
}

// From a = 6.5 on a weight is below 2^32, from 39 on it is 0 (P(-1/2) 2^-1 < 1).
constexpr float kSmall = 6.5f;
constexpr float kNone = 39.f;

// floor of 0 <= x <= 2^38, and of x < 2^32, from the fields of the number: the
// significand stands at bit 38 (31) and goes right by what the exponent is below
// that.  The conversion instructions have a quarter of the rate and less.
__device__ __forceinline__ uint64_t whole(float x) {
  const uint32_t b = __float_as_uint(x), shift = 165u - (b >> 23);
  const uint64_t m = static_cast<uint64_t>((b & 0x7FFFFFu) | 0x800000u) << 15;
  return shift > 63u ? 0ull : m >> shift;
}
__device__ __forceinline__ uint32_t whole_small(float x) {
  const uint32_t b = __float_as_uint(x);
  uint32_t r;
  asm("shr.u32 %0, %1, %2;" : "=r"(r) : "r"((b << 8) | 0x80000000u), "r"(158u - (b >> 23)));   // 0 from a shift of 32
  return r;
}

// Order of logits as unsigned numbers: NaN as -inf, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(fmaxf(x, -INFINITY) + 0.f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

}  // namespace sample
}  // namespace engram
