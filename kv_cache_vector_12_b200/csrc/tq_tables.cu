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
constexpr int kTokVec = 4;  // consecutive tokens of one thread: 16-byte stores

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
  bool vec;                 // every per-token output is 16-byte aligned
};

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

__device__ __forceinline__ int blocks_of(int tokens, int bs) { return tokens / bs + (tokens % bs != 0); }

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
    if (blockIdx.x == 0) a.seq_lens[s] = c + w;
  }
  for (int g = tid; g <= a.n_groups; g += kTabThreads)
    if (a.n_groups) s_g[g] = a.cu_group[g];
  int start = 0;
  if (paged) {
    start = *a.free_start;
    if (start < 0 || start > a.n_free) start = a.n_free;
  }
  __syncthreads();

  // ---- the two exclusive sums; thread t takes a run of consecutive sequences
  const int run = (a.n_seqs + kTabThreads - 1) / kTabThreads;
  const int s0 = min(tid * run, a.n_seqs), s1 = min(s0 + run, a.n_seqs);
  int tok = 0, blk = 0;
  for (int s = s0; s < s1; ++s) {
    const int c = s_c[s], w = s_tok[s];
    s_blk[s] = paged ? blocks_of(c + w, a.block_size) - blocks_of(c, a.block_size) : 0;
    tok = sat_add(tok, w);
    blk = sat_add(blk, s_blk[s]);
  }
  if (bad && blockIdx.x == 0) atomicOr(a.err, kErrSeqLen);
  const int itok = warp_inclusive(tok, lane), iblk = warp_inclusive(blk, lane);
  if (lane == 31) {
    s_sum[0][warp] = itok;
    s_sum[1][warp] = iblk;
  }
  __syncthreads();
  if (warp == 0) {
    const int v0 = lane < kTabWarps ? s_sum[0][lane] : 0, v1 = lane < kTabWarps ? s_sum[1][lane] : 0;
    const int i0 = warp_inclusive(v0, lane), i1 = warp_inclusive(v1, lane);
    if (lane < kTabWarps) {
      s_sum[0][lane] = i0;
      s_sum[1][lane] = i1;
    }
  }
  __syncthreads();
  int btok = warp ? s_sum[0][warp - 1] : 0, bblk = warp ? s_sum[1][warp - 1] : 0;
  {
    const int utok = __shfl_up_sync(0xffffffffu, itok, 1), ublk = __shfl_up_sync(0xffffffffu, iblk, 1);
    if (lane) {
      btok = sat_add(btok, utok);
      bblk = sat_add(bblk, ublk);
    }
  }
  for (int s = s0; s < s1; ++s) {
    const int w = s_tok[s], t = s_blk[s];
    s_tok[s] = btok;
    s_blk[s] = bblk;
    if (blockIdx.x == 0) a.cu_new[s] = btok;
    btok = sat_add(btok, w);
    bblk = sat_add(bblk, t);
  }
  const int total_tok = s_sum[0][kTabWarps - 1], total_blk = s_sum[1][kTabWarps - 1];
  if (tid == 0) {
    s_tok[a.n_seqs] = total_tok;
    s_blk[a.n_seqs] = total_blk;
    if (blockIdx.x == 0) {
      a.cu_new[a.n_seqs] = total_tok;
      if (paged) *a.free_end = (int)min((long)start + total_blk, (long)a.n_free);
      if (total_tok > a.n_tok) atomicOr(a.err, kErrTokenRange);
    }
  }
  __syncthreads();

  // ---- per-token maps: kTokVec consecutive rows per thread
  const int rows = min(total_tok, a.n_tok);
  const int stride = gridDim.x * kTabThreads;
  const int n_vec = (rows + kTokVec - 1) / kTokVec;
  for (int v = blockIdx.x * kTabThreads + tid; v < n_vec; v += stride) {
    const int r0 = v * kTokVec;
    int s = last_at_most(s_tok, a.n_seqs, r0);
    int c = s_c[s], j = -1, b = -1;  // j: the logical block that b is for
    int sq[kTokVec], ps[kTokVec];
    long sl[kTokVec];
#pragma unroll
    for (int e = 0; e < kTokVec; ++e) {
      const int r = min(r0 + e, rows - 1);
      while (r >= s_tok[s + 1]) {  // the next sequence with tokens
        c = s_c[++s];
        j = -1;
      }
      const int p = c + (r - s_tok[s]);
      sq[e] = s;
      ps[e] = p;
      if (!paged) {
        sl[e] = (long)s * a.capacity + p;
      } else if (a.slots) {
        const int jp = p / a.block_size;
        if (jp != j) {
          j = jp;
          const int first = blocks_of(c, a.block_size);
          if (j >= first) {
            b = take_block(a, start, s_blk[s] + (j - first));
          } else {  // the block that the cached tokens end in
            b = a.table[(long)s * a.per_seq + j];
            if (b < 0 || b >= a.n_blocks) {
              atomicOr(a.err, kErrTokenRange);
              b = -1;
            }
          }
        }
        sl[e] = b < 0 ? -1 : (long)b * a.block_size + (p - j * a.block_size);
      } else {
        sl[e] = -1;
      }
    }
    if (a.vec && r0 + kTokVec <= rows) {
      *reinterpret_cast<int4 *>(a.seq_idx + r0) = make_int4(sq[0], sq[1], sq[2], sq[3]);
      *reinterpret_cast<int4 *>(a.pos + r0) = make_int4(ps[0], ps[1], ps[2], ps[3]);
      if (a.slots) {
        *reinterpret_cast<longlong2 *>(a.slots + r0) = make_longlong2(sl[0], sl[1]);
        *reinterpret_cast<longlong2 *>(a.slots + r0 + 2) = make_longlong2(sl[2], sl[3]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kTokVec; ++e) {
        if (r0 + e < rows) {
          a.seq_idx[r0 + e] = sq[e];
          a.pos[r0 + e] = ps[e];
          if (a.slots) a.slots[r0 + e] = sl[e];
        }
      }
    }
  }
  if (!paged) return;

  // ---- new table entries, one per thread
  for (int i = blockIdx.x * kTabThreads + tid; i < total_blk; i += stride) {
    const int s = last_at_most(s_blk, a.n_seqs, i);
    a.table[(long)s * a.per_seq + blocks_of(s_c[s], a.block_size) + (i - s_blk[s])] = take_block(a, start, i);
  }

  // ---- shared prefixes: every member but the first takes the first one's
  // entries, a warp per sequence.  An entry that the first member gets in this
  // call is taken from the free list again, so nothing waits for its store.
  if (a.n_groups == 0) return;
  for (int s = blockIdx.x * kTabWarps + warp; s < a.n_seqs; s += gridDim.x * kTabWarps) {
    if (s < s_g[0]) continue;
    const int g = last_at_most(s_g, a.n_groups, s);
    const int lead = s_g[g];
    if (s >= s_g[g + 1] || s == lead) continue;
    const int prefix = a.prefix[g];
    // (lengths out of bounds count as 0 here, and were flagged above)
    const int cl = lead >= 0 ? s_c[lead] : 0;
    const int tl = lead >= 0 ? cl + (s_tok[lead + 1] - s_tok[lead]) : 0;
    if (prefix < 0 || prefix % a.block_size != 0 || prefix > s_c[s] || prefix > tl) {
      if (lane == 0) atomicOr(a.err, kErrSeqLen);
      continue;
    }
    const int held = blocks_of(cl, a.block_size);
    const int n = prefix / a.block_size;
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

// One CTA per 2048 tokens (a thread's four), and with groups one per 16
// sequences (a warp's one), at most four per SM (what its threads allow): a
// decode step of a few sequences is a single CTA, a million prompt tokens are
// in flight at once.  Measured for 1.05 M tokens of 32 prompts: one CTA per SM
// 9.9 us, four 6.0.
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
  a.vec = (((uintptr_t)seq_idx | (uintptr_t)pos | (uintptr_t)slots) & 15u) == 0;
  long ctas = ((long)n_tok + kTabThreads * kTokVec - 1) / (kTabThreads * kTokVec);
  if (a.n_groups > 0) {
    const long by_seq = ((long)c.n_seqs + kTabWarps - 1) / kTabWarps;
    ctas = ctas > by_seq ? ctas : by_seq;
  }
  const long sms = sm_count();
  ctas = ctas < 1 ? 1 : ctas > 4 * sms ? 4 * sms : ctas;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kTabThreads);
  const size_t words = 3 * (size_t)c.n_seqs + 2 + (size_t)a.n_groups + 1;
  static std::atomic<bool> configured[kMaxDevices];
  std::atomic<bool> &done = configured[current_device()];
  if (!done.load(std::memory_order_acquire)) {  // more than 48 KB from about 3000 sequences in groups on
    const cudaError_t e = cudaFuncSetAttribute(build_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)((4 * (size_t)kMaxTableSeqs + 3) * sizeof(int)));
    if (e != cudaSuccess) return (int)e;
    done.store(true, std::memory_order_release);
  }
  cfg.dynamicSmemBytes = words * sizeof(int);
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, build_tables_kernel, a);
}

}  // namespace tq
