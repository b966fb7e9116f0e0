// Groups of sequences that share a prefix (device side): sequences
// cu_group[g] .. cu_group[g + 1] - 1 begin with the same prefix[g] tokens, held
// by the first of them.  Every function is called by whole warps and returns
// the same in every lane; nothing is assumed of the arrays' contents but that
// cu_group should be non-decreasing (what is not is reported or left out, and
// every index returned is in bounds).
#pragma once

#include "tq_internal.h"

namespace tq {
namespace {

// Members first .. first + count - 1 of group `group`, whose first sequence is
// `lead`: unit z of the groups cut into runs of at most `members` sequences.
struct SharedUnit {
  int group, lead, first, count;
};

__device__ __forceinline__ SharedUnit find_members(const int32_t *cu, int n_groups, int max_group, int members,
                                                   int n_seqs, int z, int lane) {
  SharedUnit u = {0, 0, 0, 0};
  int done = 0;  // units of the groups before g0
  for (int g0 = 0; g0 < n_groups; g0 += 32) {
    const int g = g0 + lane;
    int b = 0, e = 0;
    if (g < n_groups) {
      b = cu[g];
      e = cu[g + 1];
      if (b < 0 || e < b || e > n_seqs || e - b > max_group) b = e = 0;
    }
    int inc = (e - b + members - 1) / members;
    const int own = inc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, done + inc > z);
    if (past) {
      const int l = __ffs(past) - 1;
      const int k = z - done - (__shfl_sync(0xffffffffu, inc, l) - __shfl_sync(0xffffffffu, own, l));
      const int bb = __shfl_sync(0xffffffffu, b, l), ee = __shfl_sync(0xffffffffu, e, l);
      u.group = g0 + l;
      u.lead = bb;
      u.first = bb + k * members;
      u.count = min(members, ee - u.first);
      return u;
    }
    done += __shfl_sync(0xffffffffu, inc, 31);
  }
  return u;
}

// Whether a member of the unit takes part.  A unit of finished sequences has no
// work, and its table rows may hold anything.
__device__ __forceinline__ bool any_member(const int32_t *seq_lens, const SharedUnit &u, int lane) {
  bool any = false;
  for (int i = lane; i < u.count; i += 32) any |= seq_lens[u.first + i] > 0;
  return __any_sync(0xffffffffu, any);
}

// The pass behind the prefixes runs beside the prefix pass, before that grid has
// completed, and reads what the kernels in front of the call wrote.  Those are
// visible to the prefix pass, which waited for them; its first thread hands them
// on by a store-release of the call's token, and every CTA of the other pass
// acquires it: causality order takes the writes along.  (The prefix grid lets the
// next one start after that store, so the token is there at the first look;
// should it not be, the wait for the whole prefix grid serves as well.)  The
// merge clears the word, so that a replayed call does not meet its own token.
__device__ __forceinline__ void hand_on(unsigned long long *word, unsigned long long token) {
  asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(word), "l"(token) : "memory");
}
__device__ __forceinline__ void take_over(const unsigned long long *word, unsigned long long token) {
  for (int i = 0; i < 64; ++i) {
    unsigned long long x;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(x) : "l"(word) : "memory");
    if (x == token) return;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// That word: the two floats of the first partial that hold nothing (a partial is
// m, l, two unused, the outputs).
__device__ __forceinline__ unsigned long long *token_word(float *partials) {
  return reinterpret_cast<unsigned long long *>(partials + 2);
}

// What sequence s attends over: its group's prefix [0, prefix) and its own
// [prefix, len).  Length 0: no part.  bad: outside every group, or its group or
// lengths outside the call's bounds, or cu decreasing somewhere (groups would
// overlap); its len and prefix are then 0.  Every group that is not bad here is
// one that find_members cuts into units.
struct SeqRange {
  int group, prefix, len;
  bool bad;
};

__device__ __forceinline__ SeqRange sequence_range(const int32_t *cu, const int32_t *prefix, int n_groups,
                                                   const int32_t *seq_lens, int max_group, int max_prefix,
                                                   int max_suffix, int capacity, int n_seqs, int s, int lane) {
  SeqRange r = {0, 0, 0, true};
  const int len = seq_lens[s];
  // the last group that begins at or before s: groups are counted by the warp
  int count = 0;
  bool ordered = true;
  for (int g = lane; g < n_groups; g += 32) {
    const int b = cu[g];
    count += b <= s;
    ordered &= b <= cu[g + 1];
  }
  count = (int)__reduce_add_sync(0xffffffffu, (unsigned)count);
  if (!__all_sync(0xffffffffu, ordered) || count == 0) return r;
  const int g = count - 1;
  const int p = prefix[g], b = cu[g], e = cu[g + 1];
  if (s >= e || b < 0 || e > n_seqs || e - b > max_group) return r;
  if (len == 0) {
    r.group = g;
    r.bad = false;
    return r;
  }
  if (p < 0 || p > max_prefix || len < p || len > capacity || len - p > max_suffix) return r;
  return {g, p, len, false};
}

}  // namespace
}  // namespace tq
