// RMS norm of heads and rotation of a part of their channels in one pass
// (mla_lowbit_norm_rope), and the host side of the rotation's frequencies.
//
//   v = x * w / sqrt(mean(x^2) + eps),  (a, b) -> m (a cos - b sin, a sin + b cos)
//
// Every element is read once and written once and costs a handful of
// instructions: the bound is HBM bandwidth for large calls and the launch for
// small ones.  So a row (one head of one token) stays in the registers of 8, 16
// or 32 lanes as 16-byte chunks, its sum of squares is a few shuffles, and the
// sines of a block's tokens are computed once, by the block together, while its
// loads are in flight.  What it took to be bound by bandwidth, 4,096 tokens x 128
// heads x 192 bf16 channels (403 MB; a device copy of them takes 62 us): one
// round of rows a block 91 us; several rounds with the next one's loads in flight,
// the weights in registers and paired float32 arithmetic 70 us; at most 72
// registers, so that seven blocks fit an SM, 62.5 us.
// Rows on any boundary (131 bf16 channels: 116 us for 275 MB, 2.4 TB/s; element by
// element 193 us) pay for the shifting: about twice the instructions.
#include <algorithm>
#include <cmath>

#include <cuda_fp16.h>

#include "rope.cuh"

namespace mlalb {
namespace {

struct NormRopeArgs {
  const void* x;
  void* y;
  const void* w;
  const uint64_t* phase;
  const int32_t* pos;
  long long x_tok, x_head, y_tok, y_head;  // strides in elements
  float eps, mscale, inv_dim;
  int rows, heads, dim, half, offset, interleaved;  // half = rot / 2
  int lanes, iters, partner, cs_entries;  // of the chunked kernel
  const void* x_end;                      // behind x's last element
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32(__half v) {
  return __half2float(v);
}
template <>
__device__ __forceinline__ float to_f32(float v) {
  return v;
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ float from_f32(float v) {
  return v;
}

// 16 bytes of T as float pairs, and back
template <typename T>
struct Pairs {
  static constexpr int N = 8 / sizeof(T);
  float2 v[N];
};
__device__ __forceinline__ float2 pair_of(uint32_t w, __nv_bfloat16) {
  return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w));
}
__device__ __forceinline__ float2 pair_of(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t word_of(float2 f, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t word_of(float2 f, __half) { return pack_half2(f.x, f.y); }
template <typename T>
__device__ __forceinline__ Pairs<T> unpack(uint4 u) {
  Pairs<T> p;
  if constexpr (sizeof(T) == 4) {
    p.v[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    p.v[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  } else {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) p.v[i] = pair_of(w[i], T());
  }
  return p;
}
template <typename T>
__device__ __forceinline__ uint4 pack(const Pairs<T>& p) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(p.v[0].x), __float_as_uint(p.v[0].y), __float_as_uint(p.v[1].x),
                      __float_as_uint(p.v[1].y));
  } else {
    return make_uint4(word_of(p.v[0], T()), word_of(p.v[1], T()), word_of(p.v[2], T()), word_of(p.v[3], T()));
  }
}

// Rows that do not start on a 16-byte boundary are loaded and stored as the
// aligned 16-byte words that they touch.  16 bytes from byte `shift` (< 16, a
// multiple of 2) of the 32 bytes (lo, hi):
__device__ __forceinline__ uint4 bytes_from(uint4 lo, uint4 hi, int shift) {
  const bool two = shift & 8, one = shift & 4;
  const uint32_t a0 = two ? lo.z : lo.x, a1 = two ? lo.w : lo.y, a2 = two ? hi.x : lo.z, a3 = two ? hi.y : lo.w,
                 a4 = two ? hi.z : hi.x, a5 = two ? hi.w : hi.y;
  const uint32_t b0 = one ? a1 : a0, b1 = one ? a2 : a1, b2 = one ? a3 : a2, b3 = one ? a4 : a3, b4 = one ? a5 : a4;
  const int bits = (shift & 2) * 8;
  return make_uint4(__funnelshift_r(b0, b1, bits), __funnelshift_r(b1, b2, bits), __funnelshift_r(b2, b3, bits),
                    __funnelshift_r(b3, b4, bits));
}
// 16 bytes up to byte `shift` from the end of the 32 bytes (lo, hi)
__device__ __forceinline__ uint4 bytes_before(uint4 lo, uint4 hi, int shift) {
  return shift == 0 ? hi : bytes_from(lo, hi, 16 - shift);
}
__device__ __forceinline__ uint4 shfl(uint4 v, int src, int width) {
  return make_uint4(__shfl_sync(0xffffffffu, v.x, src, width), __shfl_sync(0xffffffffu, v.y, src, width),
                    __shfl_sync(0xffffffffu, v.z, src, width), __shfl_sync(0xffffffffu, v.w, src, width));
}
// Elements e0 .. e0 + 16 / sizeof(T) - 1 of a row, at p (16-byte aligned): those in [0, dim)
template <typename T>
__device__ __noinline__ uint4 load_some(const T* p, int e0, int dim) {
  constexpr int E = 16 / sizeof(T);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if (e0 + i < 0 || e0 + i >= dim) continue;
    if constexpr (sizeof(T) == 4)
      w[i] = __float_as_uint(p[i]);
    else
      w[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, uint4 v, int e0, int dim) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  auto in = [&](int e) { return e >= 0 && e < dim; };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t* q = reinterpret_cast<uint32_t*>(p) + i;
    if constexpr (sizeof(T) == 4) {
      if (in(e0 + i)) *q = w[i];
    } else {
      const bool a = in(e0 + 2 * i), b = in(e0 + 2 * i + 1);
      if (a && b)
        *q = w[i];
      else if (a)
        reinterpret_cast<uint16_t*>(q)[0] = (uint16_t)w[i];
      else if (b)
        reinterpret_cast<uint16_t*>(q)[1] = (uint16_t)(w[i] >> 16);
    }
  }
}

constexpr int kThreads = 128;
constexpr int kMaxRounds = 8;
constexpr int kMaxRows = INT32_MAX - kMaxRounds * kThreads;  // a block's rows stay within int
constexpr int kMaxSines = 16384;  // bytes of a block's sines beyond which it takes fewer rounds

// Rows of 16-byte chunks: lane l of a row's `lanes` lanes holds chunks l +
// lanes * k, k < K.  A block takes a.iters rounds of kThreads / lanes consecutive
// rows, the next round's chunks loaded while one is computed; its weights stay in
// registers.  The rotated part (the caller chooses):
//   kPairs:  whole chunks of neighbouring pairs, turned where they are;
//   kHalves: a chunk's partner is the same chunk of lane l ^ a.partner;
//   kShared: any other offset and size: its chunks go through the row's floats in
//            shared memory, where the row's lanes turn a pair each;
//   kShifted: the same for rows of any size, alignment and strides: they come and
//            go as the aligned chunks that they touch, and shuffles shift them to
//            where the row begins.
enum Part { kPairs, kHalves, kShared, kShifted };
constexpr int kRowPad = 8;  // floats between two rows' copies (banks)
template <typename T, int K, bool kNorm, Part kPart>
__global__ void __launch_bounds__(kThreads, K == 4 && sizeof(T) == 2 ? (kPart == kShifted ? 6 : 5) : 7)
    norm_rope_kernel(NormRopeArgs a) {
  constexpr int P = Pairs<T>::N, E = 2 * P;
  constexpr bool kRow = kPart == kShared || kPart == kShifted;
  // shifted rows take their weights from shared memory (139 -> 116 us where they had
  // spilled registers; chunks in place 29 us from registers, 35 from shared memory)
  constexpr bool kSharedW = kNorm && kPart == kShifted;
  wait_for_stream();
  extern __shared__ float2 s_cs[];  // [tokens of the block][half] (cos, sin) * mscale
  const int lanes = a.lanes, lane = threadIdx.x & (lanes - 1);
  const int per_round = kThreads / lanes;
  const int row0 = blockIdx.x * per_round * a.iters, end = min(a.rows, row0 + per_round * a.iters);
  const int tok0 = row0 / a.heads, chunks = kPart == kShifted ? (a.dim + E - 1) / E : a.dim / E;
  int row = row0 + threadIdx.x / lanes;
  int tok = row / a.heads, head = row - tok * a.heads;
  const T* xbase = static_cast<const T*>(a.x);
  auto at = [&](const T* p, long long ts, long long hs) { return p + tok * ts + head * hs; };
  uint4 next[K];
  int x_shift = 0;  // of the row in next: its elements before the first one of its chunk
  auto shift_of = [](const T* p) { return (int)(reinterpret_cast<uintptr_t>(p) / sizeof(T) & (E - 1)); };
  auto fetch = [&] {
    const T* x = at(xbase, a.x_tok, a.x_head);
    if (kPart == kShifted) {
      x_shift = shift_of(x);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int e0 = (lane + lanes * k) * E - x_shift;
        if (row >= end || e0 >= a.dim) continue;
        const T* p = x + e0;
        if (p >= xbase && p + E <= static_cast<const T*>(a.x_end))
          next[k] = __ldcs(reinterpret_cast<const uint4*>(p));
        else
          next[k] = load_some(p, e0, a.dim);
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = lane + lanes * k;
      if (row < end && c < chunks) next[k] = __ldcs(reinterpret_cast<const uint4*>(x + c * E));
    }
  };
#pragma unroll
  for (int k = 0; k < K; ++k) next[k] = make_uint4(0, 0, 0, 0);
  fetch();
  Pairs<T> w[kSharedW ? 1 : K];
  float* s_rows = reinterpret_cast<float*>(s_cs + a.cs_entries);
  float* s_w = s_rows + (a.half ? per_round * (chunks * E + kRowPad) : 0);
  if (kSharedW) {
    for (int e = threadIdx.x; e < chunks * E; e += kThreads)
      s_w[e] = a.w && e < a.dim ? to_f32(static_cast<const T*>(a.w)[e]) : 1.f;
  }
  if (kNorm && !kSharedW) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = lane + lanes * k;
#pragma unroll
      for (int i = 0; i < P; ++i) w[k].v[i] = make_float2(1.f, 1.f);
      if (a.w && c < chunks) w[k] = unpack<T>(reinterpret_cast<const uint4*>(static_cast<const T*>(a.w) + c * E)[0]);
    }
  }
  if (a.half) {
    const int n = ((end - 1) / a.heads - tok0 + 1) * a.half;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int t = i / a.half;
      const float2 cs = rope_sincos(a.pos[tok0 + t], a.phase[i - t * a.half]);
      s_cs[i] = make_float2(cs.x * a.mscale, cs.y * a.mscale);
    }
  }
  if (a.half || kSharedW) __syncthreads();
  for (int it = 0; it < a.iters; ++it) {
    const bool live = row < end;
    T* y = static_cast<T*>(a.y) + tok * a.y_tok + head * a.y_head;
    const float2* cs = s_cs + (tok - tok0) * a.half;
    Pairs<T> v[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (kPart == kShifted) {  // chunk c of the row: from chunks c and c + 1 of what it touches
        const uint4 after = k + 1 < K ? next[k + 1 < K ? k + 1 : k] : make_uint4(0, 0, 0, 0);
        const uint4 hi = shfl(lane == 0 ? after : next[k], lane + 1, lanes);
        v[k] = unpack<T>(bytes_from(next[k], hi, x_shift * (int)sizeof(T)));
        const int e0 = (lane + lanes * k) * E;
        if (e0 + E > a.dim) {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            if (e0 + 2 * i >= a.dim) v[k].v[i].x = 0.f;
            if (e0 + 2 * i + 1 >= a.dim) v[k].v[i].y = 0.f;
          }
        }
      } else {
        v[k] = unpack<T>(next[k]);
      }
    }
    // the next round's row (a row of a later token only where rows are left)
    row += per_round;
    head += per_round;
    if (head >= a.heads) {
      const int t = a.heads >= per_round ? 1 : head / a.heads;
      tok += t;
      head -= t * a.heads;
    }
    if (it + 1 < a.iters) fetch();
    float2 r2 = make_float2(1.f, 1.f);
    float* s_row = nullptr;
    if (kRow) s_row = s_rows + (threadIdx.x / lanes) * (chunks * E + kRowPad);
    if (kNorm) {
      float2 ss = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) ss = fma2(v[k].v[i], v[k].v[i], ss);
      float sum = ss.x + ss.y;
      for (int o = lanes >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float r = rsqrtf(fmaf(sum, a.inv_dim, a.eps));
      r2 = make_float2(r, r);
    }
    auto normed = [&](int k) {
      if (kSharedW) {
        const int c = lane + lanes * k;
        if (c >= chunks) return;
#pragma unroll
        for (int i = 0; i < P; i += 2) {
          const float4 f = *reinterpret_cast<const float4*>(s_w + c * E + 2 * i);
          v[k].v[i] = mul2(v[k].v[i], mul2(r2, make_float2(f.x, f.y)));
          v[k].v[i + 1] = mul2(v[k].v[i + 1], mul2(r2, make_float2(f.z, f.w)));
        }
        return;
      }
#pragma unroll
      for (int i = 0; i < P; ++i) v[k].v[i] = mul2(v[k].v[i], mul2(r2, w[k].v[i]));
    };
    if (kNorm && kRow) {
#pragma unroll
      for (int k = 0; k < K; ++k) normed(k);
    }
    if (kRow && a.half) {
      auto in_part = [&](int c) { return c < chunks && c * E < a.offset + 2 * a.half && c * E + E > a.offset; };
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = lane + lanes * k;
        if (!in_part(c)) continue;
#pragma unroll
        for (int i = 0; i < P; i += 2)
          *reinterpret_cast<float4*>(s_row + c * E + 2 * i) =
              make_float4(v[k].v[i].x, v[k].v[i].y, v[k].v[i + 1].x, v[k].v[i + 1].y);
      }
      __syncwarp();
      const int step = a.interleaved ? 1 : a.half;
      for (int p = lane; p < a.half; p += lanes) {
        float* u = s_row + a.offset + (a.interleaved ? 2 * p : p);
        const float2 z = cs[p];
        const float f = u[0], g = u[step];
        u[0] = f * z.x - g * z.y;
        u[step] = f * z.y + g * z.x;
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = lane + lanes * k;
        if (!in_part(c)) continue;
#pragma unroll
        for (int i = 0; i < P; i += 2) {
          const float4 f = *reinterpret_cast<const float4*>(s_row + c * E + 2 * i);
          v[k].v[i] = make_float2(f.x, f.y);
          v[k].v[i + 1] = make_float2(f.z, f.w);
        }
      }
      __syncwarp();  // (before the next round's rows)
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = lane + lanes * k, e0 = c * E - a.offset;
      const bool turned = c < chunks && e0 >= 0 && e0 < 2 * a.half;
      Pairs<T>& f = v[k];
      if (kNorm && !kRow) normed(k);
      if (kPart == kPairs) {
        if (turned) {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const float2 z = cs[(e0 >> 1) + i], p = f.v[i];
            f.v[i] = make_float2(p.x * z.x - p.y * z.y, p.x * z.y + p.y * z.x);
          }
        }
      } else if (kPart == kHalves && __any_sync(0xffffffffu, turned)) {
        const bool low = e0 < a.half;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 p = f.v[i];
          const float2 q = make_float2(__shfl_xor_sync(0xffffffffu, p.x, a.partner),
                                       __shfl_xor_sync(0xffffffffu, p.y, a.partner));
          if (turned) {
            const int j = (low ? e0 : e0 - a.half) + 2 * i;
            const float2 z0 = cs[j], z1 = cs[j + 1];
            f.v[i] = low ? make_float2(p.x * z0.x - q.x * z0.y, p.y * z1.x - q.y * z1.y)
                         : make_float2(q.x * z0.y + p.x * z0.x, q.y * z1.y + p.y * z1.x);
          }
        }
      }
      if (kPart == kShifted || !live || c >= chunks) continue;
      __stcs(reinterpret_cast<uint4*>(y + c * E), pack<T>(f));
    }
    if (kPart == kShifted) {  // chunk c of what y's row touches: from chunks c - 1 and c of the row
      const int y_shift = shift_of(y);
      uint4 before = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const uint4 mine = pack<T>(v[k]);
        const uint4 lo = shfl(lane == lanes - 1 ? before : mine, lane + lanes - 1, lanes);
        before = mine;
        const uint4 u = bytes_before(lo, mine, y_shift * (int)sizeof(T));
        const int e0 = (lane + lanes * k) * E - y_shift;
        if (!live || e0 >= a.dim) continue;
        if (e0 >= 0 && e0 + E <= a.dim)
          __stcs(reinterpret_cast<uint4*>(y + e0), u);
        else
          store_some(y + e0, u, e0, a.dim);
      }
    }
  }
}

// Rows too long for the registers of a warp: a warp a row, element by element, its
// floats in shared memory.  Norm of rows of 1,536 channels (in brackets what their
// bytes take at the measured copy rate): bf16 1 row 3.8 us, 128 4.0, 8,192 17.4 (7.5),
// 65,536 104 (60); float32 3.7, 4.0, 21.6 (15.1) and 140 (121).  It is bound by the
// element-wise loads, stores and passes through shared memory: 65,536 rows of 1,024
// bf16 channels, in registers, take 43.6 us (40.2).
constexpr int kLongWarps = 4;
template <typename T, bool kNorm>
__global__ void __launch_bounds__(kLongWarps * 32) norm_rope_long_kernel(NormRopeArgs a) {
  wait_for_stream();
  extern __shared__ float s_any[];  // [kLongWarps][dim], then (cos, sin) * mscale of [tokens][half]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x * kLongWarps, row = row0 + warp, end = min(a.rows, row0 + kLongWarps);
  const bool live = row < end;
  const int tok0 = row0 / a.heads;
  const int tok = live ? row / a.heads : tok0, head = live ? row - tok * a.heads : 0;
  const T* x = static_cast<const T*>(a.x) + tok * a.x_tok + head * a.x_head;
  T* y = static_cast<T*>(a.y) + tok * a.y_tok + head * a.y_head;
  const T* w = static_cast<const T*>(a.w);
  float* v = s_any + warp * a.dim;
  float* s_cs = s_any + kLongWarps * a.dim;
  float ss = 0.f;
  if (live) {
    for (int e = lane; e < a.dim; e += 32) {
      const float f = to_f32(x[e]);
      v[e] = f;
      ss = fmaf(f, f, ss);
    }
  }
  if (a.half) {
    const int n = ((end - 1) / a.heads - tok0 + 1) * a.half;
    for (int i = threadIdx.x; i < n; i += kLongWarps * 32) {
      const int t = i / a.half;
      const float2 cs = rope_sincos(a.pos[tok0 + t], a.phase[i - t * a.half]);
      s_cs[2 * i] = cs.x * a.mscale;
      s_cs[2 * i + 1] = cs.y * a.mscale;
    }
    __syncthreads();
  }
  if (!live) return;  // (whole warps; no block barrier below)
  if (kNorm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(fmaf(ss, a.inv_dim, a.eps));
    for (int e = lane; e < a.dim; e += 32) v[e] *= w ? r * to_f32(w[e]) : r;
  }
  __syncwarp();
  if (a.half) {
    const float* cs = s_cs + 2 * (tok - tok0) * a.half;
    const int step = a.interleaved ? 1 : a.half;
    for (int p = lane; p < a.half; p += 32) {
      float* u = v + a.offset + (a.interleaved ? 2 * p : p);
      const float f = u[0], g = u[step], c = cs[2 * p], s = cs[2 * p + 1];
      u[0] = f * c - g * s;
      u[step] = f * s + g * c;
    }
    __syncwarp();
  }
  for (int e = lane; e < a.dim; e += 32) y[e] = from_f32<T>(v[e]);
}

template <typename T, bool kNorm, Part kPart>
void (*chunk_kernel(int K))(NormRopeArgs) {
  return K == 1   ? norm_rope_kernel<T, 1, kNorm, kPart>
         : K == 2 ? norm_rope_kernel<T, 2, kNorm, kPart>
         : K == 3 ? norm_rope_kernel<T, 3, kNorm, kPart>
                  : norm_rope_kernel<T, 4, kNorm, kPart>;
}

template <typename T, bool kNorm>
cudaError_t launch_norm_rope(NormRopeArgs a, bool vec, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(T);
  const int chunks = (a.dim + E - 1) / E + (vec ? 0 : 1);  // (shifted rows touch one more)
  if (chunks <= 4 * 32) {
    // the fewest lanes (at least 8) that hold the row in four chunks each
    a.lanes = chunks <= 32 ? 8 : chunks <= 64 ? 16 : 32;
    Part part = vec ? kPairs : kShifted;
    if (vec && a.half && !a.interleaved) {
      // halves: their distance in chunks a power of two, the rotated part on a
      // multiple of twice that, and as many lanes as both halves have chunks
      const int p = a.half / E;
      const bool fits = a.half % E == 0 && p > 0 && (p & (p - 1)) == 0 && p <= 16 && a.offset % (2 * a.half) == 0;
      part = fits ? kHalves : kShared;
      if (fits) a.lanes = std::max(a.lanes, 2 * p);
      a.partner = p;
    } else if (vec && a.half && (a.offset % E || 2 * a.half % E)) {
      part = kShared;
    }
    const int K = (chunks + a.lanes - 1) / a.lanes;
    const int per_round = kThreads / a.lanes;
    const int rounds = (a.rows + per_round - 1) / per_round;
    // one round a block while the rounds do not fill the GPU twice over, then up
    // to kMaxRounds (weights, sines and the first loads' latency are shared)
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorUnknown;
    a.iters = std::min(kMaxRounds, std::max(1, rounds / (sms * 16)));
    auto tokens = [&] { return std::min(per_round * a.iters, (per_round * a.iters - 1) / a.heads + 2); };
    while (a.iters > 1 && tokens() * a.half * (int)sizeof(float2) > kMaxSines) --a.iters;
    a.cs_entries = (tokens() * a.half + 1) / 2 * 2;  // (the rows' floats behind them are 16-byte words)
    const int smem = a.cs_entries * (int)sizeof(float2) +
                     (part >= kShared && a.half ? per_round * (chunks * E + kRowPad) * (int)sizeof(float) : 0) +
                     (part == kShifted && kNorm ? chunks * E * (int)sizeof(float) : 0);
    auto kern = part == kPairs    ? chunk_kernel<T, kNorm, kPairs>(K)
                : part == kHalves ? chunk_kernel<T, kNorm, kHalves>(K)
                : part == kShared ? chunk_kernel<T, kNorm, kShared>(K)
                                  : chunk_kernel<T, kNorm, kShifted>(K);
    const cudaError_t e = smem <= 48 * 1024 ? cudaSuccess : ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    return launch_in_chain(kern, dim3((rounds + a.iters - 1) / a.iters), dim3(kThreads), smem, stream, 1, a);
  } else {
    const int tokens = std::min(kLongWarps, (kLongWarps - 1) / a.heads + 2);
    const int smem = (kLongWarps * a.dim + 2 * tokens * a.half) * (int)sizeof(float);
    auto kern = norm_rope_long_kernel<T, kNorm>;
    const cudaError_t e = smem <= 48 * 1024 ? cudaSuccess : ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    return launch_in_chain(kern, dim3((a.rows + kLongWarps - 1) / kLongWarps), dim3(kLongWarps * 32), smem, stream, 1, a);
  }
}

// Whether two rows of the strided array can share an element: rows of `dim`
// contiguous elements, n of them `tok` apart, h of them `head` apart.
bool rows_overlap(long long n, long long tok, long long h, long long head, long long dim) {
  if (n > 1 && h > 1) {
    const bool tok_outer = tok >= (h - 1) * head + dim && head >= dim;
    const bool head_outer = head >= (n - 1) * tok + dim && tok >= dim;
    return !tok_outer && !head_outer;
  }
  if (n > 1) return tok < dim;
  return h > 1 && head < dim;
}

}  // namespace
}  // namespace mlalb

using namespace mlalb;

extern "C" {

int mla_lowbit_rope_table(int rot, double theta, int scaling, double factor, int original_len,
                          double beta_fast, double beta_slow, uint64_t* phase_host,
                          float* mscale_host) {
  if (rot < 2 || rot > 2048 || rot % 2) return MLA_LOWBIT_ESIZE;
  if (!phase_host || !mscale_host) return MLA_LOWBIT_ENULL;
  if (!(theta > 1.0) || !std::isfinite(theta) || scaling < MLA_LOWBIT_ROPE_NONE || scaling > MLA_LOWBIT_ROPE_YARN)
    return MLA_LOWBIT_EINVAL;
  if (scaling != MLA_LOWBIT_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return MLA_LOWBIT_EINVAL;
  double low = 0, high = 0;
  if (scaling == MLA_LOWBIT_ROPE_YARN) {
    if (original_len < 1 || !(beta_slow > 0) || !(beta_fast >= beta_slow) || !std::isfinite(beta_fast))
      return MLA_LOWBIT_EINVAL;
    auto pair_of = [&](double beta) { return rot * std::log(original_len / (kTwoPi * beta)) / (2 * std::log(theta)); };
    low = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
    high = std::fmin(std::ceil(pair_of(beta_slow)), rot - 1.0);
  }
  const double base =
      scaling == MLA_LOWBIT_ROPE_NTK && rot > 2 ? theta * std::pow(factor, rot / (rot - 2.0)) : theta;
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == MLA_LOWBIT_ROPE_LINEAR) f /= factor;
    if (scaling == MLA_LOWBIT_ROPE_YARN) {
      const double r = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
      f = f * (1 - r) + f / factor * r;
    }
    phase_host[i] = (uint64_t)std::round(std::ldexp(f / kTwoPi, 64));  // f <= 1: less than a turn
  }
  *mscale_host = scaling == MLA_LOWBIT_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return MLA_LOWBIT_OK;
}

int mla_lowbit_norm_rope(int dtype, int n_tokens, int heads, int dim, const void* x,
                         int64_t x_token_stride, int64_t x_head_stride, void* y,
                         int64_t y_token_stride, int64_t y_head_stride, int norm,
                         const void* weight, float eps, int rot, int offset, int interleaved,
                         const uint64_t* phase, float mscale, const int32_t* pos, void* stream) {
  if (dtype < MLA_LOWBIT_BF16 || dtype > MLA_LOWBIT_FP32) return MLA_LOWBIT_EINVAL;
  if (n_tokens < 0 || heads < 1 || dim < 1 || dim > 2048 || (long long)n_tokens * heads > kMaxRows)
    return MLA_LOWBIT_ESIZE;
  if (rot < 0 || rot % 2 || offset < 0 || (long long)offset + rot > dim) return MLA_LOWBIT_ESIZE;
  if (!norm && !rot) return MLA_LOWBIT_EINVAL;
  if (norm && (!(eps >= 0.f) || !std::isfinite(eps))) return MLA_LOWBIT_EINVAL;
  if (rot && !std::isfinite(mscale)) return MLA_LOWBIT_EINVAL;
  if (x_token_stride < 0 || x_head_stride < 0 || y_token_stride < 0 || y_head_stride < 0) return MLA_LOWBIT_EINVAL;
  if (n_tokens == 0) return MLA_LOWBIT_OK;
  if (!x || !y || (rot && (!phase || !pos))) return MLA_LOWBIT_ENULL;
  const int es = dtype == MLA_LOWBIT_FP32 ? 4 : 2;
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x), ya = reinterpret_cast<uintptr_t>(y),
                  wa = reinterpret_cast<uintptr_t>(weight);
  if (xa % es || ya % es || wa % es || reinterpret_cast<uintptr_t>(phase) % 8) return MLA_LOWBIT_EALIGN;
  if (rows_overlap(n_tokens, y_token_stride, heads, y_head_stride, dim)) return MLA_LOWBIT_EINVAL;
  // x and y: the same rows, or apart, or other columns of the same rows
  const long long x_span = (n_tokens - 1) * x_token_stride + (heads - 1) * x_head_stride + dim;
  const long long y_span = (n_tokens - 1) * y_token_stride + (heads - 1) * y_head_stride + dim;
  const bool meet = xa < ya + y_span * es && ya < xa + x_span * es;
  const bool same_strides = (n_tokens == 1 || x_token_stride == y_token_stride) &&
                            (heads == 1 || x_head_stride == y_head_stride);
  if (meet && !(same_strides && xa == ya)) {
    // columns: no row of x reaches a row of y, wherever in the array it is
    const long long d = (long long)(ya > xa ? ya - xa : xa - ya);
    const long long inner = heads > 1 ? (n_tokens > 1 ? (x_head_stride < x_token_stride ? x_head_stride : x_token_stride)
                                                      : x_head_stride)
                                      : x_token_stride;
    const bool columns = same_strides && d % es == 0 && d / es >= dim && d / es + dim <= inner &&
                         !rows_overlap(n_tokens, x_token_stride, heads, x_head_stride, d / es + dim);
    // or all heads of a token beside the other array's (all tokens of a head): of every
    // `outer` elements x has the first ex and y others
    const long long apart = ya > xa ? d / es : -(d / es);
    auto beside = [&](long long outer, long long ex, long long ey) {
      if (outer <= 0 || d % es) return false;
      const long long r = (apart % outer + outer) % outer;
      return r >= ex && r + ey <= outer;
    };
    const bool tokens = n_tokens > 1 && x_token_stride == y_token_stride &&
                        beside(x_token_stride, (heads - 1) * x_head_stride + dim, (heads - 1) * y_head_stride + dim);
    const bool by_head = heads > 1 && x_head_stride == y_head_stride &&
                         beside(x_head_stride, (n_tokens - 1) * x_token_stride + dim, (n_tokens - 1) * y_token_stride + dim);
    if (!columns && !tokens && !by_head) return MLA_LOWBIT_EINVAL;
  }
  NormRopeArgs a;
  a.x = x;
  a.y = y;
  a.w = norm ? weight : nullptr;
  a.phase = phase;
  a.pos = pos;
  a.x_tok = x_token_stride;
  a.x_head = x_head_stride;
  a.y_tok = y_token_stride;
  a.y_head = y_head_stride;
  a.eps = eps;
  a.mscale = mscale;
  a.rows = n_tokens * heads;
  a.heads = heads;
  a.dim = dim;
  a.x_end = static_cast<const char*>(x) + x_span * es;
  a.half = rot / 2;
  a.offset = offset;
  a.interleaved = interleaved != 0;
  a.lanes = a.iters = a.partner = a.cs_entries = 0;
  a.inv_dim = 1.f / (float)dim;
  auto chunked = [&](long long elements) { return elements * es % 16 == 0; };
  // a single token or head has no stride
  if (n_tokens == 1) a.x_tok = a.y_tok = 0;
  if (heads == 1) a.x_head = a.y_head = 0;
  const bool vec = xa % 16 == 0 && ya % 16 == 0 && wa % 16 == 0 && chunked(dim) && chunked(a.x_tok) &&
                   chunked(a.x_head) && chunked(a.y_tok) && chunked(a.y_head);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (dtype) {
    case MLA_LOWBIT_BF16:
      e = norm ? launch_norm_rope<__nv_bfloat16, true>(a, vec, s) : launch_norm_rope<__nv_bfloat16, false>(a, vec, s);
      break;
    case MLA_LOWBIT_FP16:
      e = norm ? launch_norm_rope<__half, true>(a, vec, s) : launch_norm_rope<__half, false>(a, vec, s);
      break;
    default:
      e = norm ? launch_norm_rope<float, true>(a, vec, s) : launch_norm_rope<float, false>(a, vec, s);
  }
  return e == cudaSuccess ? MLA_LOWBIT_OK : MLA_LOWBIT_ECUDA;
}

}  // extern "C"
