// The cache append from a projection's output (mla_lowbit_norm_rope_write):
// norm of the latent, rotation of the key, quantisation, and the stores of the
// writer, in one pass over each token.
//
//   ckv = bf16(latent * w * r),  r = 1 / sqrt(mean(latent^2) + eps)
//   krope = bf16(m (a cos - b sin)), bf16(m (a sin + b cos))
//   code = clamp(rne((x - m16) / s16)) per 64-channel group (mla_lowbit_write)
//
// A code flips when its value crosses a rounding border, so the values have to
// be the ones of exact arithmetic, not of some order of float32 sums.  Float32
// arithmetic decides nearly all of them: it gives a value and a bound on its
// error, and where both ends of that interval round to the same bf16 value, that
// is the one.  A token with a value for which they do not (about one in six) is
// redone in two-float arithmetic, to 2^-36 and better.  In the same way two products,
// 2^-20 to either side, enclose a code's quotient, and where they round to different
// codes it is redone by true division.
//
// A warp takes a token: lane l holds content channels 16l .. 16l + 15 (a quarter
// of a group, so a group's minimum is two shuffles and a token's codes are one
// coalesced store) and one pair of the key.  Large calls run as many warps as
// fit, each loading its next token while it works on one.
//
// 30,011 tokens in a graph, in brackets what their bytes take at the measured copy
// rate, without and with both bf16 outputs: INT4 pages 27.6 us (6.9) and 28.4 (12.0),
// rotated 33.1 and 34.0, INT2 29.0 (6.3) and 29.8, rotated 34.2 and 35.5, bf16 pages,
// without the quantiser, 18.1 (10.4) and 21.2 (15.6).  It is bound by instructions and
// latency together: about 640 warp instructions a token (150 the codes, 140 the norm,
// 70 the rotation, 40 the share of tokens whose norm is redone) keep the issue slots
// 65 % busy with 28 % of the warps that an SM can hold, each in a token's chain of
// about 25 dependent rounds of shuffles.  All tokens in two-float arithmetic and by
// true division took 39 us.
#include <algorithm>
#include <cmath>

#include "rope.cuh"

namespace mlalb {
namespace {

struct AppendArgs {
  const uint16_t* kv;  // rows of 576 bf16
  long long kv_stride;
  const uint32_t* w;  // [512] bf16 pairs or null
  const uint64_t* phase;
  const int32_t* seq_idx;
  const int32_t* pos;
  const int32_t* lens_after;
  const int32_t* block_table;
  uint8_t* pool;
  uint32_t* sink;
  uint32_t* recent;
  uint32_t* ckv_out;
  uint32_t* krope_out;
  int32_t* err;
  long long num_pages;
  float eps, mscale;
  int n_tokens, num_seqs, max_pages, interleaved;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float bf16_of(uint32_t w, int e) { return e & 1 ? bf16hi_to_f32(w) : bf16lo_to_f32(w); }

// Codes of 2 P values of one group with scale sf and min mf, packed in
// kBits-wide fields from bit 0: the float32 definition's clamp(rne((x - mf) /
// sf)), 0 when sf is 0.  [mn, mx]: the group's range.
template <int P, int kBits>
__device__ __forceinline__ uint32_t codes_of(const float2 (&x)[P], float mn, float mx, float sf, float mf) {
  constexpr int kLevels = (1 << kBits) - 1;
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number, ties to even
  if (sf == 0.f) return 0;
  // The reciprocal is within 2^-22 of 1 / sf, the quotient's own rounding is 2^-24:
  // with 2^-20 taken off and added the two products enclose the quotient, and where
  // they round to the same whole number that is the code.  (They are in order, so
  // that their differences add up, but for quotients below 0, which the range shows.)
  const float inv = __fdividef(1.f, sf), lo = inv * (1.f - 0x1p-20f), hi = inv * (1.f + 0x1p-20f);
  const float2 m2 = make_float2(-mf, -mf), lo2 = make_float2(lo, lo), hi2 = make_float2(hi, hi);
  const float2 k2 = make_float2(kRound, kRound), minus = make_float2(-1.f, -1.f);
  float2 differ = make_float2(0.f, 0.f);
  uint32_t out = 0, ones = 0;
#pragma unroll
  for (int k = 0; k < P; ++k) {
    const float2 d = add2(x[k], m2), t = fma2(d, lo2, k2);
    differ = add2(differ, fma2(t, minus, fma2(d, hi2, k2)));
    // the sum's bits are 0x4B400000 + the whole number: fields by multiplication
    out += (__float_as_uint(t.x) << (2 * k * kBits)) + (__float_as_uint(t.y) << ((2 * k + 1) * kBits));
    ones += (0x4B400000u << (2 * k * kBits)) + (0x4B400000u << ((2 * k + 1) * kBits));
  }
  out -= ones;
  // (the range's ends say whether a code could need the clamp)
  const bool clamps = (mn - mf) * inv < -0.499f || (mx - mf) * inv > kLevels + 0.499f;
  if (!(differ.x + differ.y == 0.f) || clamps) {  // (NaN, also the difference of infinities: so)
    out = 0;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int c0 = __float2int_rn(__fdiv_rn(__fsub_rn(x[k].x, mf), sf));
      const int c1 = __float2int_rn(__fdiv_rn(__fsub_rn(x[k].y, mf), sf));
      out |= (uint32_t)min(max(c0, 0), kLevels) << (2 * k * kBits);
      out |= (uint32_t)min(max(c1, 0), kLevels) << ((2 * k + 1) * kBits);
    }
  }
  return out;
}

template <int kLevels>
__device__ __forceinline__ void scale_min(float mn, float mx, uint32_t& meta, float& sf, float& mf) {
  mn = __fadd_rn(mn, 0.f);  // a zero minimum is stored as +0
  // (mx - mn) / levels, correctly rounded: the product with the reciprocal and
  // one correction by the exact remainder.  (The quotient by 15 or 3 is a float32
  // midpoint or at least 2^-29 from one, the corrected value within 2^-45 of it;
  // below the normal range, where the remainder is not exact, the fp16 scale is 0.)
  const float range = __fsub_rn(mx, mn), inv = 1.f / kLevels, q = __fmul_rn(range, inv);
  const float s32 = __fmaf_rn(__fmaf_rn(-(float)kLevels, q, range), inv, q);
  const __half s16 = __float2half_rn(fminf(s32, 65504.f));
  const __half m16 = __float2half_rn(fminf(fmaxf(mn, -65504.f), 65504.f));
  meta = (uint32_t)__half_as_ushort(s16) | ((uint32_t)__half_as_ushort(m16) << 16);
  sf = __half2float(s16);
  mf = __half2float(m16);
}

__device__ __forceinline__ float2 pair_of(uint32_t w) { return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w)); }

// r = 1 / sqrt(sum of squares / 512 + eps) of a row (lane: 16 values) in two
// floats: squares of bf16 values are exact, their sum is kept to 2^-45, and a
// Newton step r (1 - m r^2) / 2 with its residual in exact products follows the
// float32 root.  All 32 lanes must call it.
__device__ __noinline__ Two root_two(const uint4 x0, const uint4 x1, float eps) {
  const uint32_t x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  auto plus = [](Two u, Two v) {
    const Two t = two_sum(u.h, v.h);
    return Two{t.h, (u.l + v.l) + t.l};
  };
  Two ss{0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 v = pair_of(x[k]);
    ss = plus(ss, two_sum(__fmul_rn(v.x, v.x), __fmul_rn(v.y, v.y)));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    ss = plus(ss, Two{__shfl_xor_sync(0xffffffffu, ss.h, o), __shfl_xor_sync(0xffffffffu, ss.l, o)});
  Two m = two_sum(ss.h * (1.f / kLatent), eps);
  m.l += ss.l * (1.f / kLatent);
  Two r{__frsqrt_rn(m.h), 0.f};
  const Two t = two_prod(r.h, r.h), q = two_prod(m.h, t.h);
  r.l = 0.5f * r.h * ((1.f - q.h) - (q.l + (m.h * t.l + m.l * t.h)));
  if (!isfinite(r.l)) r.l = 0.f;  // m = 0 and eps = 0: r is infinite
  return r;
}

// The 16 normed channels of a lane, rounded once (pairs).  All 32 lanes call it.
__device__ __forceinline__ void normed(const uint32_t (&x)[8], const float2 (&w)[8], float eps, uint32_t (&y)[8]) {
  float2 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = pair_of(x[k]);
  float2 s[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) s[k] = fma2(v[2 * k], v[2 * k], mul2(v[2 * k + 1], v[2 * k + 1]));
  const float2 t = add2(add2(s[0], s[1]), add2(s[2], s[3]));
  float ss = __fadd_rn(t.x, t.y);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
  // With u = 2^-24: the sum of exact squares is a balanced tree of 9 roundings, eps
  // one more, halved by the root: 5 u; the root after a Newton step is within 1 u
  // and a little; the products below round once (x w is exact) and so do the
  // interval's ends: below 9 u in all.
  const float m = fmaf(ss, 1.f / kLatent, eps);
  float r = rsqrtf(m);
  const float better = fmaf(0.5f * r, fmaf(-(m * r), r, 1.f), r);
  r = isfinite(better) ? better : r;  // m = 0 and eps = 0: r is infinite
  const float lo = r * (1.f - 9 * 0x1p-24f), hi = r * (1.f + 10 * 0x1p-24f);
  const float2 lo2 = make_float2(lo, lo), hi2 = make_float2(hi, hi);
  uint32_t differ = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 xw = mul2(v[k], w[k]), f = mul2(xw, lo2), g = mul2(xw, hi2);
    y[k] = pack_bf16(f.x, f.y);
    differ |= y[k] ^ pack_bf16(g.x, g.y);
  }
  if (__any_sync(0xffffffffu, differ != 0)) {
    const Two r = root_two(make_uint4(x[0], x[1], x[2], x[3]), make_uint4(x[4], x[5], x[6], x[7]), eps);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 xw = mul2(pair_of(x[k]), w[k]), g = mul2(xw, hi2);
      if (y[k] == pack_bf16(g.x, g.y)) continue;
      const Two p = two_prod(xw.x, r.h), q = two_prod(xw.y, r.h);
      y[k] = (uint32_t)__bfloat16_as_ushort(round_bf16(p.h, fmaf(xw.x, r.l, p.l))) |
             ((uint32_t)__bfloat16_as_ushort(round_bf16(q.h, fmaf(xw.y, r.l, q.l))) << 16);
    }
  }
}

// A pair of the key turned by the angle of position p, each rounded once (a, b).
__device__ __noinline__ uint32_t turned_two(float fa, float fb, int p, uint64_t phase, float mscale) {
  Two c, sn;
  rope_sincos_two(p, phase, c, sn);
  auto sum_of = [&](float u, Two cu, float v, Two cv) {  // u cu + v cv, times mscale
    const Two pu = two_prod(u, cu.h), pv = two_prod(v, cv.h), sum = two_sum(pu.h, pv.h);
    const float low = sum.l + ((pu.l + pv.l) + fmaf(u, cu.l, v * cv.l));
    const Two sc = two_prod(sum.h, mscale);
    if (!isfinite(sc.l)) return pack_bf16((u * cu.h + v * cv.h) * mscale, 0.f) & 0xFFFFu;  // infinite or NaN
    return (uint32_t)__bfloat16_as_ushort(round_bf16(sc.h, fmaf(low, mscale, sc.l)));
  };
  return sum_of(fa, c, -fb, sn) | (sum_of(fa, sn, fb, c) << 16);
}
__device__ __forceinline__ uint32_t turned(float fa, float fb, int p, uint64_t phase, float mscale) {
  const float2 cs = rope_sincos(p, phase);
  // With u = 2^-24: the angle is off by pi 2^-25 rad (its float32) and 2^-33 turns,
  // 2 u; cos and sin by a step more, 2 u; each product, the sum and mscale round
  // once: below 8 u of |a| + |b| times mscale in all, the ends' rounding included.
  const float e = 10 * 0x1p-24f * (fabsf(fa) + fabsf(fb)) * fabsf(mscale);
  const float ra = fmaf(fa, cs.x, -(fb * cs.y)) * mscale, rb = fmaf(fa, cs.y, fb * cs.x) * mscale;
  const uint32_t lo = pack_bf16(ra - e, rb - e);
  if (lo == pack_bf16(ra + e, rb + e)) return lo;
  return turned_two(fa, fb, p, phase, mscale);
}

__device__ __forceinline__ uint32_t min_bf16(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_bf16(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

constexpr int kMaxWarps = 4;

constexpr int kBlocksPerSm = 5;

template <int CB, bool kRot, bool kVec>
__global__ void __launch_bounds__(kMaxWarps * 32, kBlocksPerSm) append_kernel(AppendArgs a) {
  wait_for_stream();
  constexpr PageGeom G = page_geom(CB);
  const int lane = threadIdx.x & 31;
  const int warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int warps = gridDim.x * (blockDim.x >> 5);
  const int ka = a.interleaved ? 2 * lane : lane, kb = a.interleaved ? 2 * lane + 1 : lane + 32;

  // a token's row, sequence and position, loaded one token ahead
  uint32_t next[8];
  uint32_t next_a = 0, next_b = 0;
  int next_s = -1, next_p = 0;
  auto fetch = [&](int i) {
    if (i >= a.n_tokens) return;
    const uint16_t* row_in = a.kv + i * a.kv_stride;
    if (kVec) {
      const uint4 t0 = reinterpret_cast<const uint4*>(row_in)[2 * lane];
      const uint4 t1 = reinterpret_cast<const uint4*>(row_in)[2 * lane + 1];
      next[0] = t0.x; next[1] = t0.y; next[2] = t0.z; next[3] = t0.w;
      next[4] = t1.x; next[5] = t1.y; next[6] = t1.z; next[7] = t1.w;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        next[k] = (uint32_t)row_in[16 * lane + 2 * k] | ((uint32_t)row_in[16 * lane + 2 * k + 1] << 16);
    }
    next_a = row_in[kLatent + ka];
    next_b = row_in[kLatent + kb];
    next_s = a.seq_idx ? a.seq_idx[i] : i;
    next_p = a.pos[i];
  };
  fetch(warp);
  float2 w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = pair_of(a.w ? a.w[8 * lane + k] : 0x3F803F80u);
  const uint64_t phase = a.phase[lane];

  for (int i = warp; i < a.n_tokens; i += warps) {
    // ---- where the token goes (its page's id travels while the norm is computed)
    uint32_t x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = next[k];
    const float fa = __uint_as_float(next_a << 16), fb = __uint_as_float(next_b << 16);
    const int s = next_s, p = next_p;
    const bool in_range = s >= 0 && s < a.num_seqs && p >= 0 && p < a.max_pages * kPageTokens;
    const long long page = in_range ? a.block_table[(long long)s * a.max_pages + p / kPageTokens] : -1;
    const int len_after = in_range && a.lens_after ? a.lens_after[s] : p + 1;
    fetch(i + warps);

    uint32_t y[8];
    normed(x, w, a.eps, y);

    // ---- rotation of the lane's pair, then (halves) into pairs of neighbours
    uint32_t kr = turned(fa, fb, p, phase, a.mscale);
    if (!a.interleaved) {  // lane l has channels l and l + 32, and takes 2l and 2l + 1
      const int src = (2 * lane) & 31;
      const uint32_t e = __shfl_sync(0xffffffffu, kr, src), o = __shfl_sync(0xffffffffu, kr, src + 1);
      kr = lane < 16 ? (e & 0xFFFFu) | (o << 16) : (e >> 16) | (o & 0xFFFF0000u);
    }
    if (page < 0 || page >= a.num_pages) {  // padding (s < 0) is no error
      if (lane == 0 && s >= 0)
        set_error(a.err, s >= a.num_seqs ? MLA_LOWBIT_DEV_BAD_SEQ
                         : !in_range     ? MLA_LOWBIT_DEV_BAD_POS
                                         : MLA_LOWBIT_DEV_BAD_PAGE);
      continue;
    }
    if (a.ckv_out) {
      uint4* o = reinterpret_cast<uint4*>(a.ckv_out + (long long)i * (kLatent / 2) + 8 * lane);
      o[0] = make_uint4(y[0], y[1], y[2], y[3]);
      o[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
    if (a.krope_out) a.krope_out[(long long)i * (kRope / 2) + lane] = kr;

    if (kRot) {
      // R = H_64 / 8 on the group (four lanes): stages 1..8 in the lane, 16
      // and 32 across lanes, in the layout's order
      float f[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] = bf16_of(y[e >> 1], e);
#pragma unroll
      for (int h = 1; h < 16; h <<= 1)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (!(e & h)) {
            const float u = f[e], v = f[e + h];
            f[e] = __fadd_rn(u, v);
            f[e + h] = __fsub_rn(u, v);
          }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float v = __shfl_xor_sync(0xffffffffu, f[e], o);
          f[e] = lane & o ? __fsub_rn(v, f[e]) : __fadd_rn(f[e], v);
        }
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = pack_bf16(f[2 * k] * 0.125f, f[2 * k + 1] * 0.125f);
    }

    // ---- stores
    const int row = p % kPageTokens;
    uint8_t* base = a.pool + page * G.page_bytes;
    auto store_row = [&](uint32_t* dst) {  // 576 bf16 (16-byte aligned rows)
      uint4* o = reinterpret_cast<uint4*>(dst + 8 * lane);
      o[0] = make_uint4(y[0], y[1], y[2], y[3]);
      o[1] = make_uint4(y[4], y[5], y[6], y[7]);
      dst[kLatent / 2 + lane] = kr;
    };
    if constexpr (CB == 16) {
      store_row(reinterpret_cast<uint32_t*>(base + row * G.content_row));
    } else {
      if (p < kSink) store_row(a.sink + ((long long)s * kSink + p) * (kDim / 2));
      if (p >= len_after - kLocal) store_row(a.recent + ((long long)s * kLocal + p % kLocal) * (kDim / 2));

      // the group's range, as bf16 pairs
      uint32_t lo2 = y[0], hi2 = y[0];
#pragma unroll
      for (int k = 1; k < 8; ++k) {
        lo2 = min_bf16(lo2, y[k]);
        hi2 = max_bf16(hi2, y[k]);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        lo2 = min_bf16(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
        hi2 = max_bf16(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
      }
      const float mn = fminf(bf16lo_to_f32(lo2), bf16hi_to_f32(lo2));
      const float mx = fmaxf(bf16lo_to_f32(hi2), bf16hi_to_f32(hi2));
      uint32_t meta;
      float sf, mf;
      scale_min<(1 << CB) - 1>(mn, mx, meta, sf, mf);
      float2 f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = pair_of(y[k]);
      uint8_t* content = base + G.content_off + row * G.content_row;
      if constexpr (CB == 4) {
        const float2 f0[4] = {f[0], f[1], f[2], f[3]}, f1[4] = {f[4], f[5], f[6], f[7]};
        reinterpret_cast<uint2*>(content)[lane] =
            make_uint2(codes_of<4, 4>(f0, mn, mx, sf, mf), codes_of<4, 4>(f1, mn, mx, sf, mf));
      } else {
        reinterpret_cast<uint32_t*>(content)[lane] = codes_of<8, 2>(f, mn, mx, sf, mf);
      }
      uint32_t* mrow = reinterpret_cast<uint32_t*>(base + G.meta_off + row * G.meta_row);
      if ((lane & 3) == 0) mrow[lane >> 2] = meta;

      // the key: one group over the whole warp
      uint32_t klo = kr, khi = kr;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        klo = min_bf16(klo, __shfl_xor_sync(0xffffffffu, klo, o));
        khi = max_bf16(khi, __shfl_xor_sync(0xffffffffu, khi, o));
      }
      const float kmn = fminf(bf16lo_to_f32(klo), bf16hi_to_f32(klo));
      const float kmx = fmaxf(bf16lo_to_f32(khi), bf16hi_to_f32(khi));
      scale_min<15>(kmn, kmx, meta, sf, mf);
      const float2 kf[1] = {pair_of(kr)};
      uint32_t v = codes_of<1, 4>(kf, kmn, kmx, sf, mf);
      v |= __shfl_down_sync(0xffffffffu, v, 1) << 8;
      v |= __shfl_down_sync(0xffffffffu, v, 2) << 16;
      if ((lane & 3) == 0) reinterpret_cast<uint32_t*>(base + G.rope_off + row * G.rope_row)[lane >> 2] = v;
      if (lane == 0) mrow[8] = meta;
    }
  }
}

}  // namespace
}  // namespace mlalb

using namespace mlalb;

extern "C" int mla_lowbit_norm_rope_write(
    const mla_lowbit_layout* layout, int n_tokens, const void* kv, int64_t kv_stride, const void* weight, float eps,
    int interleaved, const uint64_t* phase, float mscale, const int32_t* seq_idx, const int32_t* pos,
    const int32_t* seq_lens_after, int num_seqs, const int32_t* block_table, int max_pages, void* page_pool,
    int64_t num_pages, void* sink_buf, void* recent_buf, void* ckv_out, void* krope_out, int32_t* err_word,
    void* stream) {
  const int st = check_layout(layout);
  if (st != MLA_LOWBIT_OK) return st;
  if (n_tokens < 0 || num_seqs < 0 || max_pages < 0 || num_pages < 0) return MLA_LOWBIT_ESIZE;
  if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(mscale)) return MLA_LOWBIT_EINVAL;
  if (n_tokens == 0) return MLA_LOWBIT_OK;
  if (num_seqs == 0 || max_pages == 0 || num_pages == 0) return MLA_LOWBIT_ESIZE;
  if ((long long)max_pages * kPageTokens > INT32_MAX) return MLA_LOWBIT_ESIZE;
  if (kv_stride < kDim) return MLA_LOWBIT_EINVAL;
  const bool packed = layout->content_bits != 16;
  if (!kv || !phase || !pos || !block_table || !page_pool || !err_word) return MLA_LOWBIT_ENULL;
  if (packed && (!sink_buf || !recent_buf)) return MLA_LOWBIT_ENULL;
  if (!seq_idx && n_tokens > num_seqs) return MLA_LOWBIT_EINVAL;
  if (reinterpret_cast<uintptr_t>(kv) % 2 || !aligned16(weight) || !aligned16(phase) || !aligned16(page_pool) ||
      !aligned16(ckv_out) || !aligned16(krope_out) || (packed && (!aligned16(sink_buf) || !aligned16(recent_buf))))
    return MLA_LOWBIT_EALIGN;
  AppendArgs a;
  a.kv = static_cast<const uint16_t*>(kv);
  a.kv_stride = kv_stride;
  a.w = static_cast<const uint32_t*>(weight);
  a.phase = phase;
  a.seq_idx = seq_idx;
  a.pos = pos;
  a.lens_after = seq_lens_after;
  a.block_table = block_table;
  a.pool = static_cast<uint8_t*>(page_pool);
  a.sink = static_cast<uint32_t*>(sink_buf);
  a.recent = static_cast<uint32_t*>(recent_buf);
  a.ckv_out = static_cast<uint32_t*>(ckv_out);
  a.krope_out = static_cast<uint32_t*>(krope_out);
  a.err = err_word;
  a.num_pages = num_pages;
  a.eps = eps;
  a.mscale = mscale;
  a.n_tokens = n_tokens;
  a.num_seqs = num_seqs;
  a.max_pages = max_pages;
  a.interleaved = interleaved != 0;
  const bool vec = aligned16(kv) && kv_stride % 8 == 0;
  void (*kern)(AppendArgs);
  switch (layout->content_bits) {
    case 4:
      kern = layout->rotate ? (vec ? append_kernel<4, true, true> : append_kernel<4, true, false>)
                            : (vec ? append_kernel<4, false, true> : append_kernel<4, false, false>);
      break;
    case 2:
      kern = layout->rotate ? (vec ? append_kernel<2, true, true> : append_kernel<2, true, false>)
                            : (vec ? append_kernel<2, false, true> : append_kernel<2, false, false>);
      break;
    default: kern = vec ? append_kernel<16, false, true> : append_kernel<16, false, false>;
  }
  const int sms = device_sm_count();
  if (sms <= 0) return MLA_LOWBIT_ECUDA;
  // a warp a block while that spreads the tokens over more SMs; then as many
  // warps as run at once, each taking a token after the other
  const int warps = n_tokens <= 16 * sms ? 1 : kMaxWarps;
  const int blocks = (n_tokens + warps - 1) / warps, most = warps == 1 ? blocks : kBlocksPerSm * sms;
  return launch_in_chain(kern, dim3(std::min(blocks, most)), dim3(32 * warps), 0, static_cast<cudaStream_t>(stream), 1,
                         a) == cudaSuccess
             ? MLA_LOWBIT_OK
             : MLA_LOWBIT_ECUDA;
}
