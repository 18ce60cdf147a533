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
  float c;        // -log2(e) / temperature
  bool odd;       // top or c infinite: only logits equal to top have weight
};

__device__ __forceinline__ Scale make_scale(float top, float temperature) {
  Scale s;
  s.top = top;
  s.c = -__fdiv_rn(1.4426950408889634f, temperature);
  s.odd = isinf(s.c) || isinf(top);
  return s;
}

// a of two logits, as (l - m) times -c: the same roundings.  Of NaN: the minimum with it is 64.
__device__ __forceinline__ float2 finite_exponents(const Scale& s, float x0, float x1) {
  const float2 a = unpack2(mul2(add2(pack2(x0, x1), pack2(-s.top, -s.top)), pack2(s.c, s.c)));
  return make_float2(fminf(a.x, kFar), fminf(a.y, kFar));
}
__device__ __forceinline__ float2 exponents(const Scale& s, float x0, float x1) {
  if (s.odd) return make_float2(x0 == s.top ? 0.f : kFar, x1 == s.top ? 0.f : kFar);
  return finite_exponents(s, x0, x1);
}

// Two weights 2^38 p 2^-n as the numbers p (0.7 to 1.42) and n + kRound.
struct Pair {
  float2 p, k;
};

__device__ __forceinline__ Pair powers(float2 a) {
  const F2 a2 = pack2(a.x, a.y);
  const F2 r = add2(a2, pack2(kRound, kRound));
  const F2 f = add2(a2, fma2(r, pack2(-1.f, -1.f), pack2(kRound, kRound)));      // a - n: both steps are exact
  F2 y = mul2(pack2(kP6, kP6), f);
  y = mul2(add2(y, pack2(kP5, kP5)), f);
  y = mul2(add2(y, pack2(kP4, kP4)), f);
  y = mul2(add2(y, pack2(kP3, kP3)), f);
  y = mul2(add2(y, pack2(kP2, kP2)), f);
  y = mul2(add2(y, pack2(kP1, kP1)), f);
  return {unpack2(add2(y, pack2(1.f, 1.f))), unpack2(r)};
}

// From a = 8.5 on a weight is below 3/4 2^30, from 39 on it is 0 (P(-1/2) 2^-1 < 1).
constexpr float kSmall = 8.5f;
constexpr float kNone = 39.f;

// floor(2^38 p 2^-n) from the fields of p (its significand's first bit stands for 1 or 1/2) and the low
// bits of n + kRound (0x4B400000 + n), by shifts: the conversion instructions have a quarter of the rate
// and less.  whole_small: of weights below 2^31.
__device__ __forceinline__ uint64_t whole(float p, float k) {
  const uint32_t b = __float_as_uint(p), shift = __float_as_uint(k) + (127u - 0x4B400000u) - (b >> 23);
  const uint64_t m = static_cast<uint64_t>((b & 0x7FFFFFu) | 0x800000u) << 15;
  return shift > 63u ? 0ull : m >> shift;
}
__device__ __forceinline__ uint32_t whole_small(float p, float k) {
  const uint32_t b = __float_as_uint(p);
  uint32_t r;
  asm("shr.u32 %0, %1, %2;"        // 0 from a shift of 32
      : "=r"(r)
      : "r"((b << 8) | 0x80000000u), "r"(__float_as_uint(k) + (120u - 0x4B400000u) - (b >> 23)));
  return r;
}

// The weight of one logit.
__device__ __forceinline__ uint64_t weight_of(const Scale& s, float x) {
  const Pair y = powers(exponents(s, x, x));
  return whole(y.p.x, y.k.x);
}

// Order of logits as unsigned numbers: NaN as -inf, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(fmaxf(x, -INFINITY) + 0.f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// How many of the largest logits each of `blocks` blocks names, so that together they have the first top_k of
// V.  top_k is any number: from V on (2^31 - 1 among them) it is off, and not added to.
__host__ __device__ __forceinline__ int top_k_share(int top_k, int V, int blocks) {
  const int kept = top_k < 0 ? 0 : (top_k < V ? top_k : V);
  return (kept + blocks - 1) / blocks;
}

}  // namespace sample
}  // namespace engram
