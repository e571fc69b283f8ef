// Block tables and slot maps of a step (mla_lowbit_assign).
//
// Three prefix sums over the sequences (new tokens, new pages, released pages)
// say where each one's tokens and pages go; the rest is copying.  Nothing here
// is bound by bytes (16 a slot): a call is a launch and a few rounds of dependent
// loads.  So it is one launch: every CTA computes the same sums over all
// sequences for itself and keeps them in shared memory, and released pages, new
// pages and slots are flat lists whose entries find their sequence by bisection,
// one round of loads for each list however the pages are spread over sequences.
//
// Where one CTA is not enough the launch is one cluster of kClusterCtas, whose
// barrier stands between the phase that reads the old state (lengths, released
// rows, count) and the one that overwrites it (so the state may be updated in
// place) or reads the pages that other CTAs pushed.  Many slots are filled by a
// second kernel over all SMs, from the new state (48 prompts: 32,768 slots 7.9 us in
// one kernel, 8.2 in two; 65,536 10.3 and 8.5; 262,144 23 and 9.2).
#include <algorithm>

#include "common.cuh"
#include "tc_util.cuh"

namespace mlalb {
namespace {

constexpr int kThreads = 1024;  // at most
constexpr int kBatch = 4;       // released pages of a thread in flight
constexpr int kClusterCtas = 8;  // the portable cluster size
constexpr int kFillFrom = 32768;  // slots beyond which they get a kernel of their own
constexpr int kMaxSeqs = 8192;   // four ints a sequence in shared memory

struct AssignArgs {
  const int32_t* new_lens;
  const int32_t* release;
  const int32_t* seq_lens;
  const int32_t* free_count;
  int32_t* table;
  int32_t* stack;
  int32_t* lens_after;
  int32_t* count_after;
  int32_t* token_start;
  int32_t* seq_idx;
  int32_t* pos;
  long long* slots;
  int32_t* err;
  int num_seqs, max_pages, num_pages, max_tokens;
  bool fill;  // the slots too
};

__device__ __forceinline__ int pages_for(int tokens) { return (tokens + kPageTokens - 1) / kPageTokens; }

// Exclusive sums over the block's threads of (tokens, pages, released pages);
// the totals come back too.
struct Sums {
  long long tok;
  int need, back;
};
__device__ __forceinline__ Sums warp_scan(Sums v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, v.tok, o);
    const int n = __shfl_up_sync(0xffffffffu, v.need, o);
    const int b = __shfl_up_sync(0xffffffffu, v.back, o);
    if (lane >= o) {
      v.tok += t;
      v.need += n;
      v.back += b;
    }
  }
  return v;
}
__device__ __forceinline__ Sums shfl(Sums v, int src) {
  return Sums{__shfl_sync(0xffffffffu, v.tok, src), __shfl_sync(0xffffffffu, v.need, src),
              __shfl_sync(0xffffffffu, v.back, src)};
}
__device__ Sums block_scan(Sums mine, Sums* warp_sums, Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const Sums incl = warp_scan(mine);
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  const Sums all = warp_scan(lane < warps ? warp_sums[lane] : Sums{0, 0, 0});
  total = shfl(all, 31);
  Sums before = shfl(all, max(0, warp - 1));
  if (warp == 0) before = Sums{0, 0, 0};
  return Sums{before.tok + incl.tok - mine.tok, before.need + incl.need - mine.need,
              before.back + incl.back - mine.back};
}

// The last s in [0, S) with start[s] <= t (start ascending, start[0] <= t).
__device__ __forceinline__ int find(const int* start, int S, int t) {
  int s = 0;
  while (S - s > 1) {
    const int mid = (s + S) >> 1;
    if (start[mid] <= t)
      s = mid;
    else
      S = mid;
  }
  return s;
}

// Four consecutive slots from t0 on (a multiple of four), as far as there are any.
__device__ __forceinline__ void store_slots(const AssignArgs& a, long long t0, const int (&idx)[4], const int (&pos)[4],
                                            const long long (&slot)[4]) {
  if (t0 + 4 <= a.max_tokens) {
    *reinterpret_cast<int4*>(a.seq_idx + t0) = make_int4(idx[0], idx[1], idx[2], idx[3]);
    *reinterpret_cast<int4*>(a.pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    if (a.slots) {
      *reinterpret_cast<longlong2*>(a.slots + t0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<longlong2*>(a.slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (t0 + k >= a.max_tokens) break;
      a.seq_idx[t0 + k] = idx[k];
      a.pos[t0 + k] = pos[k];
      if (a.slots) a.slots[t0 + k] = slot[k];
    }
  }
}

template <bool kCluster>
__global__ void __launch_bounds__(kThreads, 1) assign_kernel(AssignArgs a) {
  wait_for_stream();
  extern __shared__ int s_dyn[];
  const int S = a.num_seqs;
  int* s_start = s_dyn;              // [S + 1] first token
  int* s_nth = s_start + S + 1;      // [S + 1] new pages of the sequences before
  int* s_back = s_nth + S + 1;       // [S + 1] released pages of the sequences before
  int* s_kept = s_back + S + 1;      // [S] tokens that stay
  __shared__ Sums warp_sums[kThreads / 32];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int rank = kCluster ? (int)tc::cluster_rank() : 0, ctas = kCluster ? kClusterCtas : 1;
  const int lead = rank * threads + tid, stride = ctas * threads;  // of the flat lists
  const long long most = (long long)a.max_pages * kPageTokens;
  const int count = *a.free_count;

  // ---- the sums (the same in every CTA)
  const int per = (S + threads - 1) / threads, first = min(S, tid * per), last = min(S, first + per);
  Sums mine{0, 0, 0};
  bool bad = false;
  for (int s = first; s < last; ++s) {
    const int len = a.seq_lens[s], add = a.new_lens[s];
    const bool ends = a.release && a.release[s] != 0;
    const long long kept = ends ? 0 : len;
    if (len < 0 || len > most || add < 0 || kept + add > most) {
      bad = true;
      continue;
    }
    mine.tok += add;
    mine.need += pages_for((int)kept + add) - pages_for((int)kept);
    mine.back += ends ? pages_for(len) : 0;
  }
  const bool any_bad = __syncthreads_or(bad) != 0;
  Sums total;
  Sums at = block_scan(mine, warp_sums, total);
  const bool no_room = count < 0 || (long long)count + total.back > a.num_pages ||
                       total.need > (long long)count + total.back || total.tok > a.max_tokens;
  const bool ok = !any_bad && !no_room;
  if (ok) {
    for (int s = first; s < last; ++s) {
      const int len = a.seq_lens[s], add = a.new_lens[s];
      const bool ends = a.release && a.release[s] != 0;
      const int kept = ends ? 0 : len;
      s_start[s] = (int)at.tok;
      s_nth[s] = at.need;
      s_back[s] = at.back;
      s_kept[s] = kept;
      at.tok += add;
      at.need += pages_for(kept + add) - pages_for(kept);
      at.back += ends ? pages_for(len) : 0;
    }
    if (tid == 0) {
      s_start[S] = (int)total.tok;
      s_nth[S] = total.need;
      s_back[S] = total.back;
    }
  }
  if (rank == 0 && tid == 0 && !ok)
    set_error(a.err, (any_bad ? MLA_LOWBIT_DEV_BAD_LEN : 0) | (no_room && !any_bad ? MLA_LOWBIT_DEV_NO_ROOM : 0));
  __syncthreads();

  // ---- released pages onto the stack (kBatch loads in flight: a round trip to
  // L2 costs about 1,100 cycles, more than anything else here)
  if (ok) {
    for (unsigned i0 = lead; i0 < (unsigned)total.back; i0 += kBatch * stride) {
      int page[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const unsigned i = i0 + k * stride;
        if (i < (unsigned)total.back) {
          const int s = find(s_back, S, i);
          page[k] = a.table[(long long)s * a.max_pages + (i - s_back[s])];
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const unsigned i = i0 + k * stride;
        if (i < (unsigned)total.back) {
          if (page[k] < 0 || page[k] >= a.num_pages) set_error(a.err, MLA_LOWBIT_DEV_BAD_PAGE);
          a.stack[count + i] = page[k];
        }
      }
    }
  }
  if (kCluster)
    tc::cluster_sync();
  else
    __syncthreads();

  // ---- the new state
  const int top = count + total.back;
  if (rank == 0) {
    for (int s = tid; s < S; s += threads) {
      a.lens_after[s] = ok ? s_kept[s] + (s_start[s + 1] - s_start[s]) : a.seq_lens[s];
      if (a.token_start) a.token_start[s] = ok ? s_start[s] : 0;
    }
    if (tid == 0) {
      a.count_after[0] = ok ? top - total.need : count;
      if (a.token_start) a.token_start[S] = ok ? (int)total.tok : 0;
    }
  }
  if (ok) {
    for (unsigned i = lead; i < (unsigned)total.need; i += stride) {
      const int s = find(s_nth, S, i);
      const int page = __ldcg(a.stack + top - 1 - i);
      if (page < 0 || page >= a.num_pages) set_error(a.err, MLA_LOWBIT_DEV_BAD_PAGE);
      a.table[(long long)s * a.max_pages + pages_for(s_kept[s]) + (i - s_nth[s])] = page;
    }
  }
  if (!a.fill) return;
  // slots: four consecutive tokens a thread, the sequence of the first by
  // bisection.  A page from before the step is in the table, a new one still
  // on the stack (the table's new entries are being written by other warps).
  // Threads count from the last one: in small calls other warps than the new
  // pages' take the slots, and the two lists' round trips overlap.
  for (long long t0 = 4LL * (stride - 1 - lead); t0 < a.max_tokens; t0 += 4LL * stride) {
    int idx[4], pos[4], page[4];
    const int* from[4];
    int s = ok && t0 < total.tok ? find(s_start, S, (int)t0) : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const long long t = t0 + k;
      const bool live = ok && t < total.tok;
      if (live)
        while (t >= s_start[s + 1]) ++s;  // sequences without new tokens are passed over
      idx[k] = live ? s : -1;
      pos[k] = live ? s_kept[s] + (int)(t - s_start[s]) : -1;
      const int j = pos[k] / kPageTokens, have = live ? pages_for(s_kept[s]) : 0;
      from[k] = !live || !a.slots ? nullptr
                : j < have        ? a.table + (long long)s * a.max_pages + j
                                  : a.stack + top - 1 - s_nth[s] - (j - have);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = from[k] ? __ldcg(from[k]) : -1;
    long long slot[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      slot[k] = page[k] >= 0 && page[k] < a.num_pages ? (long long)page[k] * kPageTokens + pos[k] % kPageTokens : -1;
    store_slots(a, t0, idx, pos, slot);
  }
}

// The slots from the new state: lengths, first tokens and block tables.  A block
// takes kFillSlots consecutive slots, four a thread; the sequences' first tokens
// are in shared memory for the bisection.
constexpr int kFillThreads = 512;
constexpr int kFillSlots = 4 * kFillThreads;
__global__ void __launch_bounds__(kFillThreads) fill_slots_kernel(AssignArgs a) {
  extern __shared__ int s_dyn[];
  wait_for_stream();
  const int S = a.num_seqs;
  for (int i = threadIdx.x; i <= S; i += kFillThreads) s_dyn[i] = __ldcg(a.token_start + i);
  __syncthreads();
  const int total = s_dyn[S];
  const long long t0 = (long long)blockIdx.x * kFillSlots + 4 * threadIdx.x;
  if (t0 >= a.max_tokens) return;
  int idx[4], pos[4], page[4];
  int s = t0 < total ? find(s_dyn, S, (int)t0) : 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const long long t = t0 + k;
    idx[k] = pos[k] = page[k] = -1;
    if (t >= total) continue;
    while (t >= s_dyn[s + 1]) ++s;
    idx[k] = s;
    pos[k] = __ldcg(a.lens_after + s) - (s_dyn[s + 1] - (int)t);
  }
  if (a.slots) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (idx[k] >= 0) page[k] = __ldcg(a.table + (long long)idx[k] * a.max_pages + pos[k] / kPageTokens);
  }
  long long slot[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    slot[k] = page[k] >= 0 && page[k] < a.num_pages ? (long long)page[k] * kPageTokens + pos[k] % kPageTokens : -1;
  store_slots(a, t0, idx, pos, slot);
}

}  // namespace
}  // namespace mlalb

using namespace mlalb;

extern "C" int mla_lowbit_assign(int num_seqs, int max_pages, int num_pages, int max_tokens,
                                 const int32_t* new_lens, const int32_t* release,
                                 const int32_t* seq_lens, const int32_t* free_count,
                                 int32_t* block_table, int32_t* free_pages, int32_t* seq_lens_after,
                                 int32_t* free_count_after, int32_t* token_start, int32_t* seq_idx,
                                 int32_t* pos, int64_t* slots, int32_t* err_word, void* stream) {
  if (num_seqs <= 0 || num_seqs > kMaxSeqs || max_pages <= 0 || num_pages < 0 || max_tokens < 0)
    return MLA_LOWBIT_ESIZE;
  if ((long long)max_pages * kPageTokens > INT32_MAX || (long long)num_seqs * max_pages > INT32_MAX)
    return MLA_LOWBIT_ESIZE;
  if (!new_lens || !seq_lens || !free_count || !block_table || !seq_lens_after || !free_count_after || !err_word)
    return MLA_LOWBIT_ENULL;
  if (num_pages > 0 && !free_pages) return MLA_LOWBIT_ENULL;
  if (max_tokens > 0 && (!seq_idx || !pos)) return MLA_LOWBIT_ENULL;
  auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!aligned(seq_idx) || !aligned(pos) || !aligned(slots)) return MLA_LOWBIT_EALIGN;
  AssignArgs a;
  a.new_lens = new_lens;
  a.release = release;
  a.seq_lens = seq_lens;
  a.free_count = free_count;
  a.table = block_table;
  a.stack = free_pages;
  a.lens_after = seq_lens_after;
  a.count_after = free_count_after;
  a.token_start = token_start;
  a.seq_idx = seq_idx;
  a.pos = pos;
  a.slots = reinterpret_cast<long long*>(slots);
  a.err = err_word;
  a.num_seqs = num_seqs;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.max_tokens = max_tokens;
  // one CTA while its threads have a sequence and one round of slots each (8,192
  // slots: 9.0 us on one, 7.3 on the cluster); beyond that a cluster.  Few threads
  // where nothing is released (they cost barrier time), all where any number of
  // pages may be.
  const bool cluster = max_tokens > 4 * kThreads || num_seqs > kThreads;
  const int want = std::max(num_seqs, max_tokens / 8);
  const int threads = cluster || release ? kThreads : std::min(kThreads, std::max(256, (want + 31) / 32 * 32));
  auto kern = cluster ? assign_kernel<true> : assign_kernel<false>;
  const int smem = (4 * num_seqs + 3) * (int)sizeof(int);
  constexpr int kNoLimitNeeded = 48 * 1024 - 1024;  // (the kernel's static arrays are below 1 KB)
  if (smem > kNoLimitNeeded && ensure_smem_limit(reinterpret_cast<const void*>(kern), smem) != cudaSuccess)
    return MLA_LOWBIT_ECUDA;
  // the second kernel needs the first tokens of the sequences from the first
  a.fill = !(token_start && max_tokens > kFillFrom);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_in_chain(kern, dim3(cluster ? kClusterCtas : 1), dim3(threads), smem, st,
                                  cluster ? kClusterCtas : 1, a);
  if (e == cudaSuccess && !a.fill)
    e = launch_in_chain(fill_slots_kernel, dim3((max_tokens + kFillSlots - 1) / kFillSlots), dim3(kFillThreads),
                        (num_seqs + 1) * sizeof(int), st, 1, a);  // at most 32 KB
  return e == cudaSuccess ? MLA_LOWBIT_OK : MLA_LOWBIT_ECUDA;
}
