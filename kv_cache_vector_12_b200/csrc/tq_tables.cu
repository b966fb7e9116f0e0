// Tables of one engine step, built on the GPU from request lengths, sm_100a.
//
// Sequence s holds c_s cached tokens and gets w_s new ones.  With blocks of B
// tokens it needs t_s = ceil((c_s + w_s) / B) - ceil(c_s / B) new blocks, so
// with the exclusive sums W_s = sum_{r < s} w_r and T_s = sum_{r < s} t_r
//   row W_s + i of the packed new tokens is position c_s + i of sequence s,
//   new block i of sequence s is entry start + T_s + i of the free list.
// Everything is a function of the two length arrays (existing table entries
// are only read), so every CTA scans the lengths on its own into shared
// memory (two sums of at most kMaxTableSeqs values) and then writes its share
// of the tokens and of the table: one launch, no second pass over the output
// and no workspace.  What bounds it: the launch and two dependent memory
// round trips for a decode step, the 16 bytes written per token for prompts.
#include <cuda_runtime.h>

#include <atomic>
#include <climits>

#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabWarps = kTabThreads / 32;

struct TablesArgs {
  unsigned *err;
  int32_t *table;           // [n_seqs][per_seq] or null (contiguous layout)
  int n_seqs, capacity, block_size, n_blocks, per_seq;
  const int32_t *cached, *fresh;
  const int32_t *free_list;
  int n_free;
  const int32_t *free_start;
  int32_t *free_end;
  const int32_t *cu_group, *prefix;
  int n_groups;
  int n_tok;
  int32_t *seq_idx, *pos;
  int64_t *slots;           // or null
  int32_t *cu_new, *seq_lens;
  uint32_t div_mul;         // x / block_size = umulhi(x, div_mul) >> div_shift
  int div_shift;
};

// Division by the block size without the divide's code: a launch starts with
// cold instruction caches, and a run of a few microseconds pays for every line.
__device__ __forceinline__ int block_of(const TablesArgs &a, int x) {
  return (int)(a.div_mul ? __umulhi((unsigned)x, a.div_mul) >> a.div_shift : (unsigned)x >> a.div_shift);
}
// Blocks that x tokens fill or begin.
__device__ __forceinline__ int blocks_of(const TablesArgs &a, int x) {
  return x > 0 ? block_of(a, x - 1) + 1 : 0;
}

// Sums of lengths that may pass 2^31 saturate there: any such total is past
// the outputs' end anyway.  (Both terms are in [0, INT_MAX].)
__device__ __forceinline__ int sat_add(int a, int b) { return (int)min((unsigned)a + (unsigned)b, (unsigned)INT_MAX); }

__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = sat_add(v, u);
  }
  return v;
}

// The last index i in [0, n) with cu[i] <= x (cu non-decreasing, cu[0] <= x).
__device__ __forceinline__ int last_at_most(const int *cu, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The lengths of sequence s as the call uses them: a sequence whose lengths
// are negative or pass the capacity gets no tokens and length 0.
__device__ __forceinline__ bool lengths_of(const TablesArgs &a, int s, int &c, int &w) {
  c = a.cached[s];
  w = a.fresh[s];
  if (c >= 0 && w >= 0 && c <= a.capacity && w <= a.capacity - c) return true;
  c = w = 0;
  return false;
}

// Entry `i` of the free list's unused part, or -1 (flagged) when the list is
// exhausted or names no block.
__device__ __forceinline__ int take_block(const TablesArgs &a, int start, int i) {
  const long at = (long)start + i;
  const int b = at < a.n_free ? a.free_list[at] : -1;
  if (b >= 0 && b < a.n_blocks) return b;
  atomicOr(a.err, kErrTokenRange);
  return -1;
}

template <bool VEC>
__global__ void __launch_bounds__(kTabThreads) build_tables_kernel(const TablesArgs a) {
  // [n_seqs + 1] W, [n_seqs + 1] T, [n_seqs] c, [n_groups + 1] group bounds
  extern __shared__ int s_dyn[];
  int *s_tok = s_dyn, *s_blk = s_tok + a.n_seqs + 1, *s_c = s_blk + a.n_seqs + 1, *s_g = s_c + a.n_seqs;
  __shared__ int s_sum[2][kTabWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool paged = a.table != nullptr;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  bool bad = false;
  for (int s = tid; s < a.n_seqs; s += kTabThreads) {
    int c, w;
    bad |= !lengths_of(a, s, c, w);
    s_c[s] = c;
    s_tok[s] = w;
    s_blk[s] = paged ? blocks_of(a, c + w) - blocks_of(a, c) : 0;
    if (blockIdx.x == 0) a.seq_lens[s] = c + w;
  }
  bool ordered = true;  // (groups that overlap would copy entries that others are writing)
  for (int g = tid; g <= a.n_groups; g += kTabThreads)
    if (a.n_groups) {
      s_g[g] = a.cu_group[g];
      ordered &= g == a.n_groups || s_g[g] <= a.cu_group[g + 1];
    }
  int start = 0;
  if (paged) {
    start = *a.free_start;
    if (start < 0 || start > a.n_free) start = a.n_free;
  }
  if ((bad || !ordered) && blockIdx.x == 0) atomicOr(a.err, kErrSeqLen);
  const bool groups = __syncthreads_and(ordered) && a.n_groups > 0;

  // ---- the two exclusive sums, side by side: half of the threads takes the
  // tokens, half the blocks, every thread a run of consecutive sequences
  {
    constexpr int kHalf = kTabThreads / 2, kHalfWarps = kTabWarps / 2;
    const int half = tid / kHalf, t = tid % kHalf, hw = t >> 5;
    int *v = half ? s_blk : s_tok;
    const int run = (a.n_seqs + kHalf - 1) / kHalf;
    const int s0 = min(t * run, a.n_seqs), s1 = min(s0 + run, a.n_seqs);
    int sum = 0;
    for (int s = s0; s < s1; ++s) sum = sat_add(sum, v[s]);
    const int inc = warp_inclusive(sum, lane);
    if (lane == 31) s_sum[half][hw] = inc;
    int excl = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 0) excl = 0;
    __syncthreads();
    for (int w = 0; w < hw; ++w) excl = sat_add(excl, s_sum[half][w]);
    for (int s = s0; s < s1; ++s) {
      const int x = v[s];
      v[s] = excl;
      if (half == 0 && blockIdx.x == 0) a.cu_new[s] = excl;
      excl = sat_add(excl, x);
    }
    if (t == kHalf - 1) v[a.n_seqs] = excl;  // (runs past the end are empty: the total)
  }
  __syncthreads();
  const int total_tok = s_tok[a.n_seqs], total_blk = s_blk[a.n_seqs];
  if (tid == 0 && blockIdx.x == 0) {
    a.cu_new[a.n_seqs] = total_tok;
    if (paged) *a.free_end = (int)min((long)start + total_blk, (long)a.n_free);
    if (total_tok > a.n_tok) atomicOr(a.err, kErrTokenRange);
  }

  // ---- per-token maps: a row per thread, or (VEC) four, in one 16-byte store
  // per map (two for the slots) where they lie in one sequence, and paged in one
  // block of it
  constexpr int kTokVec = VEC ? 4 : 1;
  const int rows = min(total_tok, a.n_tok);
  const unsigned stride = gridDim.x * kTabThreads;  // (unsigned: an index past 2^31 - 1 ends its loop)
  auto slot_of = [&](int s, int c, int p) -> long {
    if (!paged) return (long)s * a.capacity + p;
    const int j = block_of(a, p), first = blocks_of(a, c);
    // a block of this call, or the one that the cached tokens end in
    const int b = j >= first ? take_block(a, start, s_blk[s] + (j - first)) : a.table[(long)s * a.per_seq + j];
    if (b >= 0 && b < a.n_blocks) return (long)b * a.block_size + (p - j * a.block_size);
    atomicOr(a.err, kErrTokenRange);
    return -1;
  };
#pragma unroll 1
  for (unsigned at = kTokVec * (blockIdx.x * kTabThreads + tid); at < (unsigned)rows; at += kTokVec * stride) {
    const int r0 = (int)at;
    int s = last_at_most(s_tok, a.n_seqs, r0);
    const int c = s_c[s], p = c + (r0 - s_tok[s]);
    if (VEC && min(rows, s_tok[s + 1]) - r0 >= kTokVec &&
        (!paged || block_of(a, p) == block_of(a, p + kTokVec - 1))) {
      *reinterpret_cast<int4 *>(a.seq_idx + r0) = make_int4(s, s, s, s);
      *reinterpret_cast<int4 *>(a.pos + r0) = make_int4(p, p + 1, p + 2, p + 3);
      if (a.slots) {
        const long x = slot_of(s, c, p), d = x < 0 ? 0 : 1;
        *reinterpret_cast<longlong2 *>(a.slots + r0) = make_longlong2(x, x + d);
        *reinterpret_cast<longlong2 *>(a.slots + r0 + 2) = make_longlong2(x + 2 * d, x + 3 * d);
      }
    } else {
#pragma unroll 1
      for (int r = r0; r < r0 + min(kTokVec, rows - r0); ++r) {
        while (r >= s_tok[s + 1]) ++s;  // the next sequence with tokens
        const int q = s_c[s] + (r - s_tok[s]);
        a.seq_idx[r] = s;
        a.pos[r] = q;
        if (a.slots) a.slots[r] = slot_of(s, s_c[s], q);
      }
    }
  }
  if (!paged) return;

  // ---- new table entries, one per thread
  for (unsigned at = blockIdx.x * kTabThreads + tid; at < (unsigned)total_blk; at += stride) {
    const int i = (int)at, s = last_at_most(s_blk, a.n_seqs, i);
    a.table[(long)s * a.per_seq + blocks_of(a, s_c[s]) + (i - s_blk[s])] = take_block(a, start, i);
  }

  // ---- shared prefixes: every member but the first takes the first one's
  // entries, a warp per sequence.  An entry that the first member gets in this
  // call is taken from the free list again, so nothing waits for its store.
  if (!groups) return;
  for (int s = blockIdx.x * kTabWarps + warp; s < a.n_seqs; s += gridDim.x * kTabWarps) {
    if (s < s_g[0]) continue;
    const int g = last_at_most(s_g, a.n_groups, s);
    const int lead = s_g[g];
    if (s >= s_g[g + 1] || s == lead) continue;
    if (s_c[s] == 0 && s_tok[s + 1] == s_tok[s]) continue;  // no tokens: takes no part (a padded batch)
    const int prefix = a.prefix[g];
    // (lengths out of bounds count as 0 here, and were flagged above)
    const int cl = lead >= 0 ? s_c[lead] : 0;
    const int tl = lead >= 0 ? cl + (s_tok[lead + 1] - s_tok[lead]) : 0;
    if (prefix < 0 || block_of(a, prefix) * a.block_size != prefix || prefix > s_c[s] || prefix > tl) {
      if (lane == 0) atomicOr(a.err, kErrSeqLen);
      continue;
    }
    const int held = blocks_of(a, cl);
    const int n = block_of(a, prefix);
    const int32_t *src = a.table + (long)lead * a.per_seq;
    int32_t *dst = a.table + (long)s * a.per_seq;
    constexpr int kBatch = 8;  // loads of a lane in flight ahead of its stores
    for (int j0 = lane; j0 < n; j0 += 32 * kBatch) {
      int b[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int j = j0 + 32 * e;
        if (j < min(n, held)) b[e] = src[j];
        else if (j < n) b[e] = take_block(a, start, s_blk[lead] + (j - held));
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
        if (j0 + 32 * e < n) dst[j0 + 32 * e] = b[e];
    }
  }
}

}  // namespace

// A thread per token, and with groups a warp per sequence, up to the CTAs that
// are resident at once (four per SM): a decode step of up to 512 tokens without
// groups is a single CTA.  More tokens than resident threads (prompts, whose rows
// run on in one block) are taken four to a thread: 1.05 M tokens 8.6 us, and 9.7
// with one to a thread (contiguous, 1.13 M tokens 7.3 us); a step of 32 sequences
// 3.6 us with four, 2.4 with one.
int launch_tables(const DeviceParams &p, const tq_cache &c, int32_t *block_table, const int32_t *cached,
                  const int32_t *fresh, const int32_t *free_list, int n_free, const int32_t *free_start,
                  int32_t *free_end, const int32_t *cu_group, const int32_t *prefix, int n_groups, int n_tok,
                  int32_t *seq_idx, int32_t *pos, int64_t *slots, int32_t *cu_new, int32_t *seq_lens, void *stream) {
  TablesArgs a{};
  a.err = p.err;
  a.table = block_table;
  a.n_seqs = c.n_seqs;
  a.capacity = c.capacity;
  a.block_size = block_table ? c.block_size : 1;
  a.n_blocks = c.n_blocks;
  a.per_seq = block_table ? c.capacity / c.block_size : 0;
  a.cached = cached;
  a.fresh = fresh;
  a.free_list = free_list;
  a.n_free = n_free;
  a.free_start = free_start;
  a.free_end = free_end;
  a.cu_group = cu_group;
  a.prefix = prefix;
  a.n_groups = block_table ? n_groups : 0;
  a.n_tok = n_tok;
  a.seq_idx = seq_idx;
  a.pos = pos;
  a.slots = slots;
  a.cu_new = cu_new;
  a.seq_lens = seq_lens;
  // floor(x / d) for 0 <= x < 2^31: a shift for powers of two, else with s the
  // bits of d - 1 and m = ceil(2^(31 + s) / d) < 2^32 it is m x >> (31 + s), as
  // m d - 2^(31 + s) < d <= 2^s
  const unsigned d = (unsigned)a.block_size;
  int bits = 0;
  while ((1u << bits) < d) ++bits;
  if ((1u << bits) == d) {
    a.div_mul = 0;
    a.div_shift = bits;
  } else {
    a.div_mul = (uint32_t)(((1ull << (31 + bits)) + d - 1) / d);
    a.div_shift = bits - 1;
  }
  const long sms = sm_count();
  const bool vec =
      n_tok > 4 * sms * kTabThreads && (((uintptr_t)seq_idx | (uintptr_t)pos | (uintptr_t)slots) & 15u) == 0;
  const long per_cta = (vec ? 4 : 1) * kTabThreads;
  long ctas = ((long)n_tok + per_cta - 1) / per_cta;
  if (a.n_groups > 0) {
    const long by_seq = ((long)c.n_seqs + kTabWarps - 1) / kTabWarps;
    ctas = ctas > by_seq ? ctas : by_seq;
  }
  ctas = ctas < 1 ? 1 : ctas > 4 * sms ? 4 * sms : ctas;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kTabThreads);
  const size_t words = 3 * (size_t)c.n_seqs + 2 + (size_t)a.n_groups + 1;
  const auto kernel = vec ? build_tables_kernel<true> : build_tables_kernel<false>;
  static std::atomic<bool> configured[kMaxDevices][2];
  std::atomic<bool> &done = configured[current_device()][vec];
  if (!done.load(std::memory_order_acquire)) {  // more than 48 KB from about 3000 sequences in groups on
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)((4 * (size_t)kMaxTableSeqs + 3) * sizeof(int)));
    if (e != cudaSuccess) return (int)e;
    done.store(true, std::memory_order_release);
  }
  cfg.dynamicSmemBytes = words * sizeof(int);
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace tq
