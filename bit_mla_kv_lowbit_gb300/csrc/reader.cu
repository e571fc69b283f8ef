// Cached tokens back as values (mla_lowbit_read): the gather of chunked prefill
// and migration, key = s16 * code + m16 or the bf16 copy of a protected token.
//
// A token is 196 to 1,152 bytes in and 1,152 (bf16) or 2,304 (float32) out: the
// bound is HBM bandwidth, mostly of the stores.  For a token lane l holds content
// channels 8l .. 8l + 7 and 256 + 8l .. 256 + 8l + 7 (two 16-byte stores, each of
// them 512 contiguous bytes over the warp; with 16 channels in a row, and so half
// sectors a store, 200,003 tokens of bf16 pages took 76.6 us instead of 71.8) and
// one pair of the key.
//
// The way to a token's bytes is three dependent loads (index, block table, row),
// and one token's row is little to have in flight: a warp of a large call takes
// kBatch tokens, looks their pages up in kBatch lanes at once, and loads kDeep
// rows before it works on the first; its stores are marked as streaming (more than
// L2 holds goes by).  200,003 tokens of INT2 pages: 65.5 us with a token a warp,
// 49 with the batch, 45 with streaming stores (6.0 TB/s).
// 30,008 tokens in a graph, to bf16 and to float32 (in brackets what their bytes take
// at the measured copy rate): INT4 8.2 (6.7) and 17.3 us (11.8), INT2 7.9 (6.1) and
// 17.1 (11.3), bf16 pages 13.2 (10.4) and 23.6 (15.6); rotated INT4 14.2 and 17.6, INT2
// 14.7 and 17.6 (the butterflies' shuffles).
#include "rope.cuh"

namespace mlalb {
namespace {

struct ReadArgs {
  const int32_t* seq_idx;
  const int32_t* pos;
  const int32_t* seq_lens;  // null: packed copies
  const int32_t* block_table;
  const uint8_t* pool;
  const uint32_t* sink;
  const uint32_t* recent;
  void* out;
  int32_t* err;
  long long num_pages;
  int n_tokens, num_seqs, max_pages;
  bool clear;  // the rows of skipped tokens are zeros, not left as they were
};

constexpr int kWarps = 4;
constexpr int kBatch = 8;
constexpr int kDeep = 4;

// Bytes j of e and o as float32 whole numbers, exact (8388608 + code, minus it).
__device__ __forceinline__ float2 code_pair(uint32_t e, uint32_t o, int j) {
  const float2 f = make_float2(__uint_as_float(__byte_perm(e, 0x4B000000u, 0x7440 + j)),
                               __uint_as_float(__byte_perm(o, 0x4B000000u, 0x7440 + j)));
  return add2(f, make_float2(-8388608.f, -8388608.f));
}

template <bool kStream, typename T>
__device__ __forceinline__ void store(T* p, T v) {
  if constexpr (kStream)
    __stcs(p, v);
  else
    *p = v;
}

// kF32: float32 values, else bf16
template <int CB, bool kRot, bool kF32, int kTokens>
__global__ void __launch_bounds__(kWarps * 32) read_kernel(ReadArgs a) {
  wait_for_stream();
  constexpr PageGeom G = page_geom(CB);
  constexpr int kRows = kTokens < kDeep ? kTokens : kDeep;
  const int lane = threadIdx.x & 31;
  const int i0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kTokens;
  if (i0 >= a.n_tokens) return;

  // ---- lane t: where token i0 + t is.  A row of bf16 values (kind 1), or row
  // `row` of a packed page (kind 2); kind 0: skipped
  const uint8_t* at = nullptr;
  int kind_row = 0;
  if (lane < kTokens && i0 + lane < a.n_tokens) {
    const int i = i0 + lane, s = a.seq_idx[i], p = a.pos[i];
    if (s >= a.num_seqs) {
      set_error(a.err, MLA_LOWBIT_DEV_BAD_SEQ);
    } else if (s >= 0) {  // below 0: padding
      const int len = a.seq_lens ? a.seq_lens[s] : 0, row = p % kPageTokens;
      if (p < 0 || p >= a.max_pages * kPageTokens || (a.seq_lens && p >= len)) {
        set_error(a.err, MLA_LOWBIT_DEV_BAD_POS);
      } else if (CB != 16 && a.seq_lens && (p < kSink || p >= len - kLocal)) {
        at = reinterpret_cast<const uint8_t*>(p < kSink ? a.sink + ((long long)s * kSink + p) * (kDim / 2)
                                                        : a.recent + ((long long)s * kLocal + p % kLocal) * (kDim / 2));
        kind_row = 1;
      } else {
        const long long page = a.block_table[(long long)s * a.max_pages + p / kPageTokens];
        if (page < 0 || page >= a.num_pages) {
          set_error(a.err, MLA_LOWBIT_DEV_BAD_PAGE);
        } else if (CB == 16) {
          at = a.pool + page * G.page_bytes + row * G.content_row;
          kind_row = 1;
        } else {
          at = a.pool + page * G.page_bytes;
          kind_row = 2 | (row << 2);
        }
      }
    }
  }
  const unsigned long long at_bits = reinterpret_cast<unsigned long long>(at);

#pragma unroll 1
  for (int t0 = 0; t0 < kTokens; t0 += kRows) {
    uint4 u0[kRows], u1[kRows];
    uint32_t key[kRows];
    int kr[kRows];
#pragma unroll
    for (int t = 0; t < kRows; ++t) {
      kr[t] = __shfl_sync(0xffffffffu, kind_row, t0 + t);
      const uint8_t* base = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, at_bits, t0 + t));
      const int kind = kr[t] & 3, row = kr[t] >> 2;
      if (kind == 1) {
        u0[t] = reinterpret_cast<const uint4*>(base)[lane];
        u1[t] = reinterpret_cast<const uint4*>(base)[32 + lane];
        key[t] = reinterpret_cast<const uint32_t*>(base)[kLatent / 2 + lane];
      } else if (CB != 16 && kind == 2) {
        const uint8_t* content = base + G.content_off + row * G.content_row;
        const uint32_t* mrow = reinterpret_cast<const uint32_t*>(base + G.meta_off + row * G.meta_row);
        if constexpr (CB == 4) {
          u0[t].x = reinterpret_cast<const uint32_t*>(content)[lane];
          u0[t].y = reinterpret_cast<const uint32_t*>(content)[32 + lane];
        } else {
          u0[t].x = reinterpret_cast<const uint16_t*>(content)[lane];
          u0[t].y = reinterpret_cast<const uint16_t*>(content)[32 + lane];
        }
        u0[t].z = mrow[lane >> 3];
        u1[t].x = mrow[4 + (lane >> 3)];
        u0[t].w = mrow[8];
        key[t] = (base + G.rope_off + row * G.rope_row)[lane];
      }
    }
#pragma unroll
    for (int t = 0; t < kRows; ++t) {
      const int kind = kr[t] & 3;
      if (kind == 0) {
        if (!a.clear || i0 + t0 + t >= a.n_tokens) continue;
        constexpr int kWords = kDim * (kF32 ? 4 : 2) / 16;
        uint4* o = static_cast<uint4*>(a.out) + (long long)(i0 + t0 + t) * kWords;
        for (int c = lane; c < kWords; c += 32) store<kTokens != 1>(o + c, make_uint4(0, 0, 0, 0));
        continue;
      }
      float2 f[8], k;
      if (CB == 16 || kind == 1) {
        const uint32_t w[8] = {u0[t].x, u0[t].y, u0[t].z, u0[t].w, u1[t].x, u1[t].y, u1[t].z, u1[t].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = make_float2(bf16lo_to_f32(w[j]), bf16hi_to_f32(w[j]));
        k = make_float2(bf16lo_to_f32(key[t]), bf16hi_to_f32(key[t]));
      } else {
        const float2 sk = __half22float2(*reinterpret_cast<const __half2*>(&u0[t].w));
        // (scale * code is exact: 11 + 4 bits; one rounding in the sum)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w = h ? u0[t].y : u0[t].x, mt = h ? u1[t].x : u0[t].z;
          const float2 sm = __half22float2(*reinterpret_cast<const __half2*>(&mt));
          const float2 s2 = make_float2(sm.x, sm.x), m2 = make_float2(sm.y, sm.y);
          if constexpr (CB == 4) {
            const uint32_t e = w & 0x0F0F0F0Fu, o = (w >> 4) & 0x0F0F0F0Fu;
#pragma unroll
            for (int j = 0; j < 4; ++j) f[4 * h + j] = fma2(code_pair(e, o, j), s2, m2);
          } else {
            // byte j: codes 4j .. 4j + 3
            const uint32_t c0 = w & 0x0303u, c1 = (w >> 2) & 0x0303u, c2 = (w >> 4) & 0x0303u, c3 = (w >> 6) & 0x0303u;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              f[4 * h + 2 * j] = fma2(code_pair(c0, c1, j), s2, m2);
              f[4 * h + 2 * j + 1] = fma2(code_pair(c2, c3, j), s2, m2);
            }
          }
        }
        k = fma2(code_pair(key[t] & 15u, key[t] >> 4, 0), make_float2(sk.x, sk.x), make_float2(sk.y, sk.y));
      }
      if (kRot) {
        // back by R = R^T = H_64 / 8 over the group's eight lanes (both halves of
        // the lane alike): stage 1 in a pair, 2 and 4 between the lane's pairs, 8 to
        // 32 across lanes
        const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = make_float2(__fadd_rn(f[j].x, f[j].y), __fsub_rn(f[j].x, f[j].y));
#pragma unroll
        for (int h = 1; h < 4; h <<= 1)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (!(j & h)) {
              const float2 u = f[j], v = f[j + h];
              f[j] = add2(u, v);
              f[j + h] = fma2(v, minus, u);
            }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 v = make_float2(__shfl_xor_sync(0xffffffffu, f[j].x, o), __shfl_xor_sync(0xffffffffu, f[j].y, o));
            f[j] = lane & o ? fma2(f[j], minus, v) : add2(f[j], v);
          }
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = mul2(f[j], make_float2(0.125f, 0.125f));
      }
      const long long i = i0 + t0 + t;
      if (kF32) {
        float* o = static_cast<float*>(a.out) + i * kDim;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          store<kTokens != 1>(reinterpret_cast<float4*>(o + 256 * (j >> 1) + 8 * lane) + (j & 1),
                              make_float4(f[2 * j].x, f[2 * j].y, f[2 * j + 1].x, f[2 * j + 1].y));
        store<kTokens != 1>(reinterpret_cast<float2*>(o + kLatent) + lane, k);
      } else {
        uint32_t* o = static_cast<uint32_t*>(a.out) + i * (kDim / 2);
        uint32_t y[9];
#pragma unroll
        for (int j = 0; j < 9; ++j) {
          const __nv_bfloat162 v = j < 8 ? __floats2bfloat162_rn(f[j].x, f[j].y) : __floats2bfloat162_rn(k.x, k.y);
          y[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
        store<kTokens != 1>(reinterpret_cast<uint4*>(o) + lane, make_uint4(y[0], y[1], y[2], y[3]));
        store<kTokens != 1>(reinterpret_cast<uint4*>(o) + 32 + lane, make_uint4(y[4], y[5], y[6], y[7]));
        store<kTokens != 1>(o + kLatent / 2 + lane, y[8]);
      }
    }
  }
}

template <bool kF32, int kTokens>
cudaError_t launch_read(int cbits, int rotate, const ReadArgs& a, cudaStream_t stream) {
  void (*kern)(ReadArgs) =
      cbits == 4   ? (rotate ? read_kernel<4, true, kF32, kTokens> : read_kernel<4, false, kF32, kTokens>)
      : cbits == 2 ? (rotate ? read_kernel<2, true, kF32, kTokens> : read_kernel<2, false, kF32, kTokens>)
                   : read_kernel<16, false, kF32, kTokens>;
  constexpr int kPerBlock = kWarps * kTokens;
  return launch_in_chain(kern, dim3((a.n_tokens + kPerBlock - 1) / kPerBlock), dim3(kWarps * 32), 0, stream, 1, a);
}

}  // namespace
}  // namespace mlalb

using namespace mlalb;

extern "C" int mla_lowbit_read(const mla_lowbit_layout* layout, int n_tokens, const int32_t* seq_idx,
                               const int32_t* pos, int num_seqs, const int32_t* seq_lens, const int32_t* block_table,
                               int max_pages, const void* page_pool, int64_t num_pages, const void* sink_buf,
                               const void* recent_buf, int out_dtype, void* out, int32_t* err_word, void* stream) {
  const int st = check_layout(layout);
  if (st != MLA_LOWBIT_OK) return st;
  if (n_tokens < 0 || num_seqs < 0 || max_pages < 0 || num_pages < 0) return MLA_LOWBIT_ESIZE;
  const bool clear = (out_dtype & MLA_LOWBIT_CLEAR_SKIPPED) != 0;
  out_dtype &= ~MLA_LOWBIT_CLEAR_SKIPPED;
  if (out_dtype != MLA_LOWBIT_BF16 && out_dtype != MLA_LOWBIT_FP32) return MLA_LOWBIT_EINVAL;
  if (n_tokens == 0) return MLA_LOWBIT_OK;
  if (num_seqs == 0 || max_pages == 0 || num_pages == 0) return MLA_LOWBIT_ESIZE;
  if ((long long)max_pages * kPageTokens > INT32_MAX) return MLA_LOWBIT_ESIZE;
  if (!seq_idx || !pos || !block_table || !page_pool || !out || !err_word) return MLA_LOWBIT_ENULL;
  const bool copies = layout->content_bits != 16 && seq_lens;
  if (copies && (!sink_buf || !recent_buf)) return MLA_LOWBIT_ENULL;
  if (!aligned16(page_pool) || !aligned16(out) || (copies && (!aligned16(sink_buf) || !aligned16(recent_buf))))
    return MLA_LOWBIT_EALIGN;
  ReadArgs a;
  a.seq_idx = seq_idx;
  a.pos = pos;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.pool = static_cast<const uint8_t*>(page_pool);
  a.sink = static_cast<const uint32_t*>(sink_buf);
  a.recent = static_cast<const uint32_t*>(recent_buf);
  a.out = out;
  a.err = err_word;
  a.num_pages = num_pages;
  a.n_tokens = n_tokens;
  a.num_seqs = num_seqs;
  a.max_pages = max_pages;
  a.clear = clear;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = device_sm_count();
  if (sms <= 0) return MLA_LOWBIT_ECUDA;
  // a token a warp while the warps all run at once
  const bool many = n_tokens > 64 * sms;
  const int cb = layout->content_bits, rot = layout->rotate;
  const cudaError_t e = out_dtype == MLA_LOWBIT_FP32
                            ? (many ? launch_read<true, kBatch>(cb, rot, a, s) : launch_read<true, 1>(cb, rot, a, s))
                            : (many ? launch_read<false, kBatch>(cb, rot, a, s) : launch_read<false, 1>(cb, rot, a, s));
  return e == cudaSuccess ? MLA_LOWBIT_OK : MLA_LOWBIT_ECUDA;
}
