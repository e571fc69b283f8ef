// Angles of the position rotation.
//
// A pair's frequency is held as phase = f / (2 pi) in units of 2^-64 turns, so
// the angle of position p is the wrapped 64-bit product p * phase: exact range
// reduction by integer arithmetic, for any int32 position.  (A float32 product
// p * f is off by up to 0.06 rad at a million tokens; float64 arithmetic is slow
// on this GPU.)
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace mlalb {

constexpr double kTwoPi = 6.283185307179586476925286766559;

// (cos, sin) of position `pos`, float32 accurate: the angle's upper 32 bits are off by
// 2^-33 turns (7e-10 rad), and as a float32 of half turns by up to 2^-25 of them
// (9.4e-8 rad).
__device__ __forceinline__ float2 rope_sincos(int pos, uint64_t phase) {
  const uint64_t p = (uint64_t)(long long)pos * phase + 0x80000000ull;
  float s, c;
  sincospif((float)(int)(p >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

// cos and sin of the 256 angles k / 256 turns, each as a float32 and its
// remainder.  Taylor series in float64 at compile time (|x| <= pi / 2: the
// terms alternate and shrink, and 13 of each series leave less than 1e-17).
struct TurnTable {
  float v[256][4];  // cos high, cos low, sin high, sin low
  constexpr TurnTable() : v() {
    for (int k = 0; k < 256; ++k) {
      const double x = (k % 64) * (kTwoPi / 256);
      double c = 0, s = 0, tc = 1, ts = x;
      for (int j = 0; j < 13; ++j) {
        c += tc;
        s += ts;
        tc *= -x * x / ((2 * j + 1) * (2 * j + 2));
        ts *= -x * x / ((2 * j + 2) * (2 * j + 3));
      }
      if (k % 64 == 0) {
        c = 1;
        s = 0;
      }
      // quadrant k / 64: (c, s) turned by that many quarter turns
      const int q = k / 64;
      const double cq = q == 0 ? c : q == 1 ? -s : q == 2 ? -c : s;
      const double sq = q == 0 ? s : q == 1 ? c : q == 2 ? -s : -c;
      v[k][0] = (float)cq;
      v[k][1] = (float)(cq - (double)v[k][0]);
      v[k][2] = (float)sq;
      v[k][3] = (float)(sq - (double)v[k][2]);
    }
  }
};
static __device__ constexpr TurnTable kTurns{};

// Two float32 operations in one instruction (each rounded to nearest)
__device__ __forceinline__ uint64_t as_u64(float2 f) {
  return (uint64_t)__float_as_uint(f.x) | ((uint64_t)__float_as_uint(f.y) << 32);
}
__device__ __forceinline__ float2 as_f2(uint64_t u) {
  return make_float2(__uint_as_float((uint32_t)u), __uint_as_float((uint32_t)(u >> 32)));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
  return as_f2(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(d);
}

// A value as an unevaluated sum of two float32.
struct Two {
  float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {  // exact
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return Two{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ Two two_prod(float a, float b) {  // exact
  const float p = __fmul_rn(a, b);
  return Two{p, __fmaf_rn(a, b, -p)};
}

// cos and sin of position `pos` to about 2^-36: the nearest of 256 tabulated
// angles, turned by the remainder r (|r| <= pi / 256) with r, and the product
// that it leads, in two floats.
__device__ __forceinline__ void rope_sincos_two(int pos, uint64_t phase, Two& c, Two& s) {
  constexpr double kUnit = kTwoPi * 0x1p-40;  // rad
  constexpr float kUnitH = (float)kUnit, kUnitL = (float)(kUnit - (double)kUnitH);
  const uint64_t p = (uint64_t)(long long)pos * phase;
  const uint64_t near = (p + (1ull << 55)) >> 56;
  const int units = (int)((long long)(p - (near << 56)) >> 24);
  const float uf = (float)units;
  const float ur = (float)(units - __float2int_rn(uf));  // (saturating: off by a unit where uf is 2^31)
  Two r = two_prod(uf, kUnitH);
  r.l += fmaf(uf, kUnitL, ur * kUnitH);
  const float4 t = *reinterpret_cast<const float4*>(kTurns.v[near & 255]);
  const float r2 = r.h * r.h;
  // sin r = r.h + sl, cos r = 1 - vr
  const float sl = fmaf(r.h * r2, fmaf(r2, 1.f / 120.f, -1.f / 6.f), r.l);
  const float vr = r2 * fmaf(r2, -1.f / 24.f, 0.5f);
  // cos = C - (S sin r + C vr), sin = S + (C sin r - S vr)
  const Two ps = two_prod(t.z, r.h), pc = two_prod(t.x, r.h);
  c = two_sum(t.x, -ps.h);
  c.l += t.y - (ps.l + fmaf(t.z, sl, fmaf(t.w, r.h, t.x * vr)));
  s = two_sum(t.z, pc.h);
  s.l += t.w + (pc.l + fmaf(t.x, sl, fmaf(t.y, r.h, -(t.z * vr))));
}

// The float32 nearest to h + l, and with it the bf16 nearest to the sum: where
// the float32 lies exactly between two bf16 values the rest decides the side.
__device__ __forceinline__ __nv_bfloat16 round_bf16(float h, float l) {
  const float f = __fadd_rn(h, l), rest = __fsub_rn(l, __fsub_rn(f, h));
  uint32_t u = __float_as_uint(f);
  if ((u & 0xFFFFu) == 0x8000u && rest != 0.f) u += (rest > 0.f) == (f > 0.f) ? 1u : ~0u;
  return __float2bfloat16_rn(__uint_as_float(u));
}

}  // namespace mlalb
