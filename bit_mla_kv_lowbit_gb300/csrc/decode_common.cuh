// Device helpers shared by the decode kernels: the channel pairing of the
// nibble/crumb unpack, the unpack itself, hi/lo splitting and the split lookup.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace mlalb {

constexpr int kHC = 16;  // heads per CTA

// ---------------------------------------------------------------- pairing
// The unpack of one thread's 16 channels (16j..16j+15 of a group) yields 8
// fp16 pairs P_0..P_7.  INT4 ("type A"): P_i = (8(i>>2) + (i&3), +4).  INT2
// ("type B"): P_i = (i, i+8).  mma k-step s takes b0 = P_2s, b1 = P_2s+1.

__device__ __forceinline__ int phys_of_logical(int k, bool typeB) {
  const int s = k >> 4, h = (k >> 3) & 1, j = (k >> 1) & 3, e = k & 1;
  const int i = 2 * s + h;
  return typeB ? 16 * j + i + 8 * e : 16 * j + 8 * (i >> 2) + (i & 3) + 4 * e;
}

// Inverse of phys_of_logical.
__device__ __forceinline__ int logical_of_phys(int p, bool typeB) {
  const int j = p >> 4, rem = p & 15;
  int i, e;
  if (typeB) {
    e = rem >> 3;
    i = rem & 7;
  } else {
    e = (rem >> 2) & 1;
    i = 4 * (rem >> 3) + (rem & 3);
  }
  return 16 * (i >> 1) + 8 * (i & 1) + 2 * j + e;
}

// Physical channel of PV output column n (0..7) of tile chunk c (0..7).
__device__ __forceinline__ int phys_of_chunk(int c, int n, bool typeB) {
  const int jj = c >> 1, wd = c & 1, r = n >> 1, e = n & 1, i = 4 * wd + r;
  return typeB ? 16 * jj + i + 8 * e : 16 * jj + 8 * wd + r + 4 * e;
}

__device__ __forceinline__ uint32_t h2fma(uint32_t x, uint32_t m, uint32_t a) {
  __half2 r = __hfma2(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&m),
                      *reinterpret_cast<__half2*>(&a));
  return *reinterpret_cast<uint32_t*>(&r);
}

constexpr uint32_t kMagic = 0x64006400u;  // fp16 1024 in both halves

// Codes are centred before they reach the tensor cores (INT4: c - 8 in
// [-8, 7]; INT2: c - 2 in [-2, 1]) and the min is moved by the same amount
// (m' = m + 8s or m + 2s).  The products stay exact; the point is that the MMA
// sums over thousands of tokens then have mixed signs, so the fp32 tensor-core
// accumulation, whose adds are not round-to-nearest, does not drift.
constexpr int kCentre4 = 8;
constexpr int kCentre2 = 2;

// 8 nibbles (channels 0..7 of the word) -> (c0,c4) (c1,c5) (c2,c6) (c3,c7), minus 8.
__device__ __forceinline__ void unpack_int4(uint32_t w, uint32_t* p) {
  const uint32_t w8 = w >> 8;
  p[0] = h2fma((w & 0x000F000Fu) | kMagic, 0x3C003C00u, 0xE408E408u);   // x*1 - 1032
  p[1] = h2fma((w & 0x00F000F0u) | kMagic, 0x2C002C00u, 0xD480D480u);   // x/16 - 72
  p[2] = h2fma((w8 & 0x000F000Fu) | kMagic, 0x3C003C00u, 0xE408E408u);
  p[3] = h2fma((w8 & 0x00F000F0u) | kMagic, 0x2C002C00u, 0xD480D480u);
}

// 16 crumbs (channels 0..15) -> (c0,c8) (c1,c9) ... (c7,c15), minus 2.
__device__ __forceinline__ void unpack_int2(uint32_t w, uint32_t* p) {
  const uint32_t w8 = w >> 8;
  p[0] = h2fma((w & 0x00030003u) | kMagic, 0x3C003C00u, 0xE402E402u);   // x - 1026
  p[1] = h2fma((w & 0x000C000Cu) | kMagic, 0x34003400u, 0xDC08DC08u);   // x/4 - 258
  p[2] = h2fma((w & 0x00300030u) | kMagic, 0x2C002C00u, 0xD420D420u);   // x/16 - 66
  p[3] = h2fma((w & 0x00C000C0u) | kMagic, 0x24002400u, 0xCC80CC80u);   // x/64 - 18
  p[4] = h2fma((w8 & 0x00030003u) | kMagic, 0x3C003C00u, 0xE402E402u);
  p[5] = h2fma((w8 & 0x000C000Cu) | kMagic, 0x34003400u, 0xDC08DC08u);
  p[6] = h2fma((w8 & 0x00300030u) | kMagic, 0x2C002C00u, 0xD420D420u);
  p[7] = h2fma((w8 & 0x00C000C0u) | kMagic, 0x24002400u, 0xCC80CC80u);
}

// 16 bf16 values (v[k] = channels 2k, 2k+1) -> fp16 pairs in the given pairing.
template <bool kB>
__device__ __forceinline__ void pairs_from_bf16(const uint32_t* v, uint32_t* p) {
  float f[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    f[2 * k] = bf16lo_to_f32(v[k]);
    f[2 * k + 1] = bf16hi_to_f32(v[k]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int a = kB ? i : 8 * (i >> 2) + (i & 3);
    const int b = kB ? i + 8 : a + 4;
    p[i] = pack_half2(f[a], f[b]);
  }
}

__device__ __forceinline__ void split_hi_lo(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 hf = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_half2(a - hf.x, b - hf.y);
}

// ---------------------------------------------------------------- split work
// Units [split * chunk, (split + 1) * chunk) of a sequence of length L: packed
// pages page_begin .. page_begin + n_pages - 1, then bf16 tiles bf_begin ..
// bf_begin + n_bf - 1 (the tiles whose first unit falls in the range); bf16
// tile k holds protected tokens 64k .. 64k + 63 of the list (sink tokens
// 0 .. n_sink - 1, then recent tokens from rec_start), n_tok in all, in
// bf_total tiles.  has_last: the split holds the last protected token.
struct SplitWork {
  int page_begin, n_pages, bf_begin, n_bf, n_sink, rec_start, n_tok, bf_total;
  bool has_last;
  int nA, bB;  // window: list index of a page -> page (page_at)
};
__device__ __forceinline__ SplitWork split_work(int L, int split, int chunk, bool packed) {
  SplitWork w;
  const int pages = packed_pages_of(L, packed);
  const int u0 = split * chunk, u1 = min(units_of(L, packed), u0 + chunk);
  w.page_begin = u0;
  w.nA = w.bB = 0;
  w.n_pages = max(0, min(u1, pages) - u0);
  w.bf_total = bf16_tiles_of(L, packed);
  // first unit of tile k is pages + kBf16TileUnits * k
  const int k0 = max(0, (u0 - pages + kBf16TileUnits - 1) / kBf16TileUnits);
  const int k1 = min(w.bf_total, max(0, (u1 - pages + kBf16TileUnits - 1) / kBf16TileUnits));
  w.bf_begin = min(k0, w.bf_total);
  w.n_bf = max(0, k1 - w.bf_begin);
  w.n_sink = packed ? min(L, kSink) : 0;
  w.rec_start = max(kSink, L - kLocal);
  w.n_tok = bf16_tokens_of(L, packed);
  w.has_last = w.n_bf > 0 && w.bf_begin + w.n_bf == w.bf_total;
  return w;
}

// ---------------------------------------------------------------- window work
// The tokens that some of a sequence's n_q queries may see through a window of
// W tokens and K first tokens: t < K, or t >= lo = L - n_q - W + 1 (the oldest
// token of the first query's window).
//
// Its pages are nA pages from the sequence's first (the K tokens) and then pages
// from bB on (the window), without a repetition; page_at names the i-th.  The
// protected list is cut the same way.  All counts are of tokens that exist; W
// and K are at most max_pages * 64.
struct WinPages {
  int nA, bB, pages, n_sink, rec_start, n_tok;
};
__host__ __device__ inline WinPages win_pages(int L, int n_q, int W, int K, bool packed) {
  WinPages w{0, 0, 0, 0, 0, 0};
  if (L <= 0) return w;
  const int lo = L - n_q - W + 1 > 0 ? L - n_q - W + 1 : 0;
  const int end = packed ? L - kLocal : L;  // pages serve tokens [first, end)
  const int first = packed ? kSink : 0;
  if (end > first) {
    const int k_end = K < end ? K : end;
    w.nA = k_end > first ? (k_end - 1) / kPageTokens + 1 : 0;
    const int from = lo > first ? lo : first;
    w.bB = from / kPageTokens;
    if (w.bB < w.nA) w.bB = w.nA;
    const int last = (end - 1) / kPageTokens;
    w.pages = w.nA + (from < end && last >= w.bB ? last - w.bB + 1 : 0);
  }
  if (packed) {
    const int sinks = L < kSink ? L : kSink;
    w.n_sink = lo < kSink || K >= sinks ? sinks : K;
    const int ring = L - kLocal > kSink ? L - kLocal : kSink;  // oldest token of the recent buffer's part
    w.rec_start = K > ring || lo <= ring ? ring : lo;
    w.n_tok = w.n_sink + (L > w.rec_start ? L - w.rec_start : 0);
  }
  return w;
}
// A unit is a page or a tile of 64 protected tokens, which costs about as much here.
__host__ __device__ inline int win_units(const WinPages& w) {
  return w.pages + (w.n_tok + kPageTokens - 1) / kPageTokens;
}
// At most this many units for a sequence of any length up to `most`.
inline long long win_units_bound(int most, int n_q, int W, int K, bool packed) {
  const long long span = (long long)W + n_q - 1;  // tokens of all the queries' windows
  const long long paged = (span < most ? span : most) - (packed ? kLocal : 0);
  // a run of n tokens touches at most (n + 62) / 64 + 1 pages
  const long long pages = (K > 0 ? (K - 1) / kPageTokens + 1 : 0) + (paged > 0 ? (paged + 62) / kPageTokens + 1 : 0);
  const long long all = (most - 1) / kPageTokens + 1;
  // more than four first tokens can reach into the recent buffer's part
  const long long kept = !packed ? 0 : K > kSink ? kProtected : (kSink + span < kProtected ? kSink + span : kProtected);
  return (pages < all ? pages : all) + (kept + kPageTokens - 1) / kPageTokens;
}
__device__ __forceinline__ bool win_sees(int t, int p, int W, int K) { return t <= p && (t < K || t > p - W); }

// Units of each chunk but a sequence's last.
__device__ __forceinline__ int win_chunk(const WinCut& c, int units) {
  return max(1, (int)(((long long)units * c.num + c.den - 1) / c.den));
}
// Splits of a sequence that hold units.
__device__ __forceinline__ int win_splits_used(const WinCut& c, int units) {
  const int chunk = win_chunk(c, units);
  return min(c.splits, (units + chunk - 1) / chunk);
}
// One split's work; n_units is 0 behind a sequence's last split.
__device__ __forceinline__ SplitWork window_work(int L, int split, const WinCut& cut, int n_q, int W, int K, bool packed,
                                                 int& n_units) {
  const WinPages p = win_pages(L, n_q, W, K, packed);
  const int units = win_units(p), chunk = win_chunk(cut, units);
  const int u0 = min((long long)units, (long long)split * chunk);
  const int u1 = split == cut.splits - 1 ? units : min(units, u0 + chunk);
  n_units = u1 - u0;
  SplitWork w;
  w.page_begin = u0;
  w.nA = p.nA;
  w.bB = p.bB;
  w.n_pages = max(0, min(u1, p.pages) - u0);
  w.n_sink = p.n_sink;
  w.rec_start = p.rec_start;
  w.n_tok = p.n_tok;
  w.bf_total = (p.n_tok + kPageTokens - 1) / kPageTokens;
  w.bf_begin = min(max(0, u0 - p.pages), w.bf_total);
  w.n_bf = max(0, u1 - p.pages - w.bf_begin);
  w.has_last = false;
  return w;
}
// The result of a sequence that is one split (DecodeArgs.win_out).
__device__ __forceinline__ float lse_of(float m, float l) {
  return l <= 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;  // (of a NaN: NaN)
}
__device__ __forceinline__ void store_result(const DecodeArgs& a, long long at, float4 v) {
  if (a.win_bf16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.win_out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(a.win_out) + at) = v;
  }
}
// Zeros, lse -inf, for rows row0 .. row0 + rows - 1 and the 256 channels from 256 half
// on, by kThreads threads from thread t0 on.
template <int kThreads>
__device__ __forceinline__ void store_nothing(const DecodeArgs& a, long long row0, int rows, int half, int t0 = 0) {
  const int t = threadIdx.x - t0;
  for (int k = t; k < rows * 64; k += kThreads)
    store_result(a, (row0 + (k >> 6)) * kLatent + 256 * half + 4 * (k & 63), make_float4(0.f, 0.f, 0.f, 0.f));
  if (half == 0 && a.win_lse)
    for (int k = t; k < rows; k += kThreads) a.win_lse[row0 + k] = -INFINITY;
}
// Page of the sequence at index i of its page list.
__device__ __forceinline__ int page_at(const SplitWork& w, int i) { return i < w.nA ? i : w.bB + (i - w.nA); }

// Position of entry idx of the protected-token list.
__device__ __forceinline__ int bf16_pos(const SplitWork& w, int idx) {
  return idx < w.n_sink ? idx : w.rec_start + (idx - w.n_sink);
}

// ---------------------------------------------------------------- plan lookup
// Every CTA recomputes the per-sequence split counts (same integer formula as
// the host) and finds which (sequence, split) its blockIdx.x names.
// `target` is the split's global index (blockIdx.x by default).
template <int kThreads>
__device__ void find_split(const DecodeArgs& a, bool packed, int* scan, int& b_out,
                           int& split_out, int& nsplit_out, int target_index = -1) {
  constexpr int kCtaWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  const int max_tok = a.max_pages * kPageTokens;
  int local = 0;
  for (int b = b0; b < b1; ++b) {
    int L = a.seq_lens[b];
    if (L < 0 || L > max_tok) L = 0;
    local += splits_of(L, packed, a.chunk_pages);
  }
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) scan[warp] = incl;
  if (tid == 0) scan[kCtaWarps] = -1;
  __syncthreads();
  if (tid == 0) {
    int acc = 0;
    for (int w = 0; w < kCtaWarps; ++w) {
      const int t = scan[w];
      scan[w] = acc;
      acc += t;
    }
    scan[kCtaWarps + 1] = acc;  // device-side total
  }
  __syncthreads();
  const int excl = scan[warp] + incl - local;
  const int target = target_index >= 0 ? target_index : (int)blockIdx.x;
  if (target >= excl && target < excl + local) {
    int acc = excl;
    for (int b = b0; b < b1; ++b) {
      int L = a.seq_lens[b];
      if (L < 0 || L > max_tok) L = 0;
      const int n = splits_of(L, packed, a.chunk_pages);
      if (target < acc + n) {
        scan[kCtaWarps + 2] = b;
        scan[kCtaWarps + 3] = target - acc;
        scan[kCtaWarps + 4] = n;
        scan[kCtaWarps] = 1;
        break;
      }
      acc += n;
    }
  }
  __syncthreads();
  if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) {
    if (scan[kCtaWarps + 1] != a.total_splits) set_error(a.err, MLA_LOWBIT_DEV_PLAN);
    for (int b = 0; b < a.B; ++b) {
      const int L = a.seq_lens[b];
      if (L < 0 || L > max_tok) set_error(a.err, MLA_LOWBIT_DEV_BAD_LEN);
    }
  }
  if (scan[kCtaWarps] == 1) {
    b_out = scan[kCtaWarps + 2];
    split_out = scan[kCtaWarps + 3];
    nsplit_out = scan[kCtaWarps + 4];
  } else {
    b_out = -1;
  }
}

}  // namespace mlalb
