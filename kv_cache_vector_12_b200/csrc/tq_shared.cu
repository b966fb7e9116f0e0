// Decode attention over the packed cache for groups of sequences that share a
// prefix, sm_100a.
//
// The members of a group attend over the same prefix [0, P) and each over its
// own positions [P, n_s).  Attention over a union of key sets is the merge of
// the attentions over each,
//   o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,   m = max_i m_i
// with (m_i, l_i, o_i) the running maximum (log2 units), sum and unnormalised
// output of part i.  So the prefix is streamed and expanded once for the rows
// (member, query head) of a whole group, split along its length, and only the
// positions behind it sequence by sequence; the merge joins both passes'
// partials, rotates back (Pi^T) and rounds to the output's type once.
//
// The passes are the decode attention kernel in its SHARED build
// (tq_decode_kernel.cuh), up to 16 rows per CTA; groups of more rows at d = 128
// without QJL take the prefix pass of tq_shared_tc.cu, up to 128 rows per CTA.
#include <atomic>
#include <chrono>
#include <cmath>

#include "tq_decode_kernel.cuh"
#include "tq_merge.cuh"
#include "tq_shared_tc.h"

namespace tq {
namespace {

// Rows of a group above which the tcgen05 prefix pass runs.  One group, 8 KV
// heads, 3/3 bits, the whole call, tcgen05 / 16-row tiles: 16 rows, 8192 shared
// positions 25 / 27 us, 65536 71 / 56; 20 rows 25 / 28 and 72 / 83; 64 rows 31 / 42
// and 75 / 145; 128 rows 38 / 58 and 84 / 277.
constexpr int kTcMinRows = 16;
constexpr int kTcFixed = 4;      // a tcgen05 CTA's prologue and partial, in tile times (8 us; a tile takes 2)
constexpr int kMaxPrefixSplits = 128, kMaxSuffixSplits = 64;
constexpr int kSuffixFixed = 1;  // a CTA's prologue in the 16-row passes, in stages of 128 positions

struct MergeArgs {
  DeviceParams p;
  const int32_t *seq_lens, *cu_group, *prefix;
  int n_groups, max_group, max_prefix, max_suffix, capacity, n_seqs, n_q_heads;
  int p_chunk, p_splits, s_chunk, s_splits;
  float *partials;
  void *out;
  bool out_f32;
  float *lse;
};

// kMergeRows (sequence, query head) rows per CTA: a warp joins the split partials
// of one row, then every thread takes output coordinate `tid` of all of them, so
// that a row of Pi^T is loaded once for kMergeRows rows.  One row per CTA, as the merge of
// tq_decode_attention has it, reads Pi^T (32 KB) for every row: 21 us for 1024
// rows of 25 partials, where this takes 11.5 for 1024 rows of 19.  At d = 256 a row
// of Pi^T (512 bytes) is too long for a thread: 8 warps take 32 coordinates each,
// a coordinate's row over the lanes (16 rows 43 us with two rows read by a thread).
constexpr int kMergeRows = 4;
constexpr int merge_threads(int dh) { return dh == 256 ? 256 : 128; }

template <int DH>
__global__ void __launch_bounds__(merge_threads(DH)) shared_merge_kernel(const MergeArgs a, int n_rows) {
  constexpr int PF = DH + 4, PL = DH / 32;
  __shared__ __align__(16) float s_ot[kMergeRows][DH];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row0 = blockIdx.x * kMergeRows, row = row0 + warp;
  Bf16Row<DH> pw;  // (DH = 256: unused)
  if (DH < 256 && tid < DH) pw.load(a.p.pivt + tid * DH);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0 && tid == 0 && a.p_splits) *token_word(a.partials) = 0;
  if (warp < kMergeRows && row < n_rows) {
    const int s = row / a.n_q_heads;
    const SeqRange g = sequence_range(a.cu_group, a.prefix, a.n_groups, a.seq_lens, a.max_group, a.max_prefix,
                                      a.max_suffix, a.capacity, a.n_seqs, s, lane);
    // the slots in use: the splits that hold positions, of either pass
    const int n_p = g.len > 0 && a.p_splits ? (g.prefix + a.p_chunk - 1) / a.p_chunk : 0;
    const int n_s = g.len > g.prefix ? (g.len - (g.prefix & ~63) + a.s_chunk - 1) / a.s_chunk : 0;
    const int used = n_p + n_s;
    const float *src = a.partials + (long)row * (a.p_splits + a.s_splits) * PF;
    auto slot = [&](int i) { return src + (long)(i < n_p ? i : a.p_splits + i - n_p) * PF; };
    float mm = -INFINITY, ll = 0.f, acc[PL];
#pragma unroll
    for (int c = 0; c < PL; ++c) acc[c] = 0.f;
    for (int i0 = 0; i0 < used; i0 += 32) {  // 32 slots at a time: lane i holds (m, l) of slot i0 + i
      float2 ml = make_float2(-INFINITY, 0.f);
      if (i0 + lane < used) ml = *reinterpret_cast<const float2 *>(slot(i0 + lane));
      float mx = ml.x;
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float nm = fmaxf(mm, mx), old = mm == -INFINITY ? 0.f : exp2f(mm - nm);
      const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - nm);
      mm = nm;
      float lw = w * ml.y;
#pragma unroll
      for (int o = 16; o; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
      ll = fmaf(ll, old, lw);
#pragma unroll
      for (int c = 0; c < PL; ++c) acc[c] *= old;
      const int n = min(32, used - i0);
#pragma unroll 8
      for (int i = 0; i < n; ++i) {
        float v[PL];
        load_floats<PL>(slot(i0 + i) + 4 + lane * PL, v);
        const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
        for (int c = 0; c < PL; ++c) acc[c] = fmaf(wi, v[c], acc[c]);
      }
    }
    const float il = used > 0 ? 1.f / ll : 0.f;
#pragma unroll
    for (int c = 0; c < PL; ++c) s_ot[warp][lane * PL + c] = acc[c] * il;
    if (a.lse && lane == 0) a.lse[row] = used > 0 ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
  }
  __syncthreads();
  auto store = [&](int e, int i, float x) {
    const long at = (long)(row0 + e) * DH + i;
    if (a.out_f32) static_cast<float *>(a.out)[at] = x;
    else static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(x);
  };
  if constexpr (DH < 256) {
#pragma unroll
    for (int e = 0; e < kMergeRows; ++e) {
      if (row0 + e >= n_rows) break;
      if (tid < DH) store(e, tid, dot_bf16_row<DH>(pw, s_ot[e]));
    }
  } else {
    static_assert(kMergeRows == 4, "the sums below are those of four rows");
    float x[kMergeRows][8];  // entries 8 lane .. 8 lane + 7 of every row
#pragma unroll
    for (int e = 0; e < kMergeRows; ++e) load_floats<8>(s_ot[e] + 8 * lane, x[e]);
    __syncthreads();  // (s_ot takes the outputs)
#pragma unroll 8
    for (int o = 0; o < 32; ++o) {
      const int i = 32 * warp + o;
      const uint4 v = reinterpret_cast<const uint4 *>(a.p.pivt + (size_t)i * DH)[lane];
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      float sum[kMergeRows];
#pragma unroll
      for (int e = 0; e < kMergeRows; ++e) {
        sum[e] = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          sum[e] = fmaf(__uint_as_float(u[c] << 16), x[e][2 * c], sum[e]);
          sum[e] = fmaf(__uint_as_float(u[c] & 0xffff0000u), x[e][2 * c + 1], sum[e]);
        }
      }
      // sums over the lanes, row lane / 8 in every lane: halves change rows first
      const bool b4 = lane & 16, b3 = lane & 8;
      float s0 = b4 ? sum[2] : sum[0], s1 = b4 ? sum[3] : sum[1];
      s0 += __shfl_xor_sync(0xffffffffu, b4 ? sum[0] : sum[2], 16);
      s1 += __shfl_xor_sync(0xffffffffu, b4 ? sum[1] : sum[3], 16);
      float t = b3 ? s1 : s0;
      t += __shfl_xor_sync(0xffffffffu, b3 ? s0 : s1, 8);
#pragma unroll
      for (int m = 4; m; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
      if ((lane & 7) == 0) s_ot[lane >> 3][i] = t;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kMergeRows; ++e)
      if (row0 + e < n_rows) store(e, tid, s_ot[e][tid]);
  }
}

}  // namespace

namespace {

// plan_shared with at most p_most and s_most splits.
SharedPlan plan_splits(int d, int bits_k, int bits_v, int qjl, int n_seqs, int n_q_heads, int n_kv_heads, int n_groups,
                       int max_group, int max_prefix, int max_suffix, long p_most, long s_most) {
  SharedPlan s = {};
  const int per = n_q_heads / n_kv_heads;
  s.tc = d == kHeadDim && !qjl && (long)per * max_group > kTcMinRows;
  s.nt_p = (long)per * max_group > 8 ? 2 : 1;
  s.members = (s.tc ? 128 : 8 * s.nt_p) / per;
  const long by_group = (long)n_groups * ((max_group + s.members - 1) / s.members);
  // sum ceil(c / m) <= sum (c + m - 1) / m over the groups' sizes c
  const long by_seq = ((long)n_seqs + (long)n_groups * (s.members - 1)) / s.members;
  s.units = (int)(by_group < by_seq ? by_group : by_seq);
  if (max_prefix > 0 && s.tc) {
    // splits of whole 128-key tiles, one CTA per SM: the count with the fewest
    // tile times over all waves, kTcFixed of them per CTA for its prologue
    // (q rotation) and its partial
    const long tiles = (max_prefix + 127) / 128, lanes = (long)s.units * n_kv_heads, sms = sm_count();
    long best = -1;
    for (long n = 1; n <= tiles && n <= p_most; ++n) {
      const long per_split = (tiles + n - 1) / n, used = (tiles + per_split - 1) / per_split;
      const long cost = (lanes * used + sms - 1) / sms * (per_split + kTcFixed);
      if (best < 0 || cost < best) {
        best = cost;
        s.p_chunk = (int)(per_split * 128);
        s.p_splits = (int)used;
      }
    }
  } else if (max_prefix > 0) {
    // the count with the fewest stage times over all waves, counted in halves of
    // a stage, and a tenth of one for each split (its CTA's prologue beside
    // others, and the merge).  Whole calls, 3/3 bits, 8 KV heads, 16 rows: 8192
    // shared positions, 18 splits 28 us, 22 26, 26 27, 37 26; 65536, 27 splits 63,
    // 37 57, 46 (two waves) 74; 16 groups of 4096, 1 split 95, 2 69, 3 80.  With
    // QJL the prologue has a second product (128 rows, 16384: 4 splits 164, 8 181).
    const long fixed = qjl ? 3 : kSuffixFixed;
    const long halves = (max_prefix + 63) / 64, lanes = (long)s.units * n_kv_heads;
    const long slots = (long)sm_count() * shared_ctas_per_sm(d, bits_k, bits_v, qjl, s.nt_p);
    long best = -1;
    for (long n = 1; n <= halves && n <= p_most; ++n) {
      const long per_split = (halves + n - 1) / n, used = (halves + per_split - 1) / per_split;
      const long cost = 5 * ((lanes * used + slots - 1) / slots * (per_split + 2 * fixed)) + used;
      if (best < 0 || cost < best) {
        best = cost;
        s.p_chunk = (int)(per_split * 64);
        s.p_splits = (int)used;
      }
    }
  }
  s.nt_s = per > 8 ? 2 : 1;
  // The pass behind the prefix starts up to 63 positions before the prefix's
  // end.  Its units are many and short, so a split has to pay for its CTA's
  // prologue: the count with the fewest stage times over all waves.  32
  // sequences of up to 1500 positions behind 32768 shared ones, 8 KV heads, the
  // whole call: 1 split 78 us, 2 70, 3 (taken) 66, 4 69, 7 73.
  {
    const long stages = (max_suffix + 63 + 127) / 128, units = (long)n_seqs * n_kv_heads;
    const long slots = (long)sm_count() * shared_ctas_per_sm(d, bits_k, bits_v, qjl, s.nt_s);
    long best = -1;
    for (long n = 1; n <= stages && n <= s_most; ++n) {
      const long per_split = (stages + n - 1) / n, used = (stages + per_split - 1) / per_split;
      const long cost = (units * used + slots - 1) / slots * (per_split + kSuffixFixed);
      if (best < 0 || cost < best) {
        best = cost;
        s.s_chunk = (int)(per_split * 128);
        s.s_splits = (int)used;
      }
    }
  }
  const size_t rows = (size_t)n_seqs * n_q_heads;
  s.workspace = rows * (size_t)(s.p_splits + s.s_splits) * (size_t)(d + 4) * sizeof(float);
  return s;
}

}  // namespace

SharedPlan plan_shared(int d, int bits_k, int bits_v, int qjl, int n_seqs, int n_q_heads, int n_kv_heads, int n_groups,
                       int max_group, int max_prefix, int max_suffix, size_t room) {
  const auto plan = [&](long p_most, long s_most) {
    return plan_splits(d, bits_k, bits_v, qjl, n_seqs, n_q_heads, n_kv_heads, n_groups, max_group, max_prefix, max_suffix,
                       p_most, s_most);
  };
  const SharedPlan s = plan(kMaxPrefixSplits, kMaxSuffixSplits);
  if (s.workspace <= room) return s;
  // Fewer slots than the fastest counts take (they follow waves, and a smaller
  // call may want more than a larger one): both passes in proportion, one at least.
  const long slots = (long)(room / ((size_t)n_seqs * n_q_heads * (size_t)(d + 4) * sizeof(float)));
  if (s.p_splits == 0) return plan(0, slots > 1 ? slots : 1);
  const long total = s.p_splits + s.s_splits, p = (slots * s.p_splits + total / 2) / total;
  const long p_most = p < 1 ? 1 : p > slots - 1 && slots > 1 ? slots - 1 : p;
  return plan(p_most, slots - p_most > 1 ? slots - p_most : 1);
}

namespace {

// A number that no earlier call of the process had and that a workspace does not
// hold by chance: a counter from a start of its own, mixed (SplitMix64's step).
unsigned long long next_token() {
  static std::atomic<uint64_t> count{0};
  static const uint64_t start =
      (uint64_t)std::chrono::system_clock::now().time_since_epoch().count() ^ ((uint64_t)(uintptr_t)&count << 20);
  uint64_t z = start + 0x9E3779B97F4A7C15ull * (count.fetch_add(1, std::memory_order_relaxed) + 1);
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  z ^= z >> 31;
  return z ? z : 1;
}

}  // namespace

int launch_shared(const DeviceParams &p, const tq_cache &c, const void *q, int q_dtype, int n_q_heads,
                  const int32_t *seq_lens, const int32_t *cu_group, const int32_t *prefix, int n_groups,
                  int max_group, int max_prefix, int max_suffix, float scale, void *out, bool out_f32, float *lse,
                  char *workspace, const SharedPlan &plan, void *stream) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;

  DecodeArgs args{};
  args.p = p;
  args.c = c;
  args.n_q_heads = n_q_heads;
  args.n_splits = plan.p_splits + plan.s_splits;
  args.seq_lens = seq_lens;
  args.q = q;
  args.q_dtype = q_dtype;
  args.scale = scale;
  args.partials = reinterpret_cast<float *>(workspace);
  args.cu_group = cu_group;
  args.prefix = prefix;
  args.n_groups = n_groups;
  args.max_group = max_group;
  args.max_prefix = max_prefix;
  args.max_suffix = max_suffix;
  args.members = plan.members;
  args.token = next_token();
  cfg.blockDim = dim3(kThreads);
  if (plan.p_splits > 0 && plan.tc) {
    const SharedTcArgs t{p,      c,        n_q_heads, q,          q_dtype,      scale,        seq_lens,      cu_group,
                         prefix, n_groups, max_group, max_prefix, plan.members, plan.p_chunk, args.partials, args.n_splits,
                         args.token};
    cfg.gridDim = dim3(plan.p_splits, c.n_kv_heads, plan.units);
    const int e = launch_shared_prefix_tc(t, cfg);
    if (e != 0) return e;
    cfg.blockDim = dim3(kThreads);
  } else if (plan.p_splits > 0) {
    shared_ctas_per_sm(p.d, p.bits_k, p.bits_v, p.qjl, plan.nt_p);  // sets the kernel's shared memory
    const DecodeVariant v = shared_kernel(p, plan.nt_p);
    args.pass = kPassPrefix;
    args.chunk = plan.p_chunk;
    args.slot0 = 0;
    cfg.gridDim = dim3(plan.p_splits, c.n_kv_heads, plan.units);
    cfg.dynamicSmemBytes = v.smem;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, v.fn, args);
    if (e != cudaSuccess) return (int)e;
  }
  {
    shared_ctas_per_sm(p.d, p.bits_k, p.bits_v, p.qjl, plan.nt_s);
    const DecodeVariant v = shared_kernel(p, plan.nt_s);
    args.pass = kPassSuffix;
    args.chunk = plan.s_chunk;
    args.slot0 = plan.p_splits;
    args.beside = plan.p_splits > 0;
    cfg.gridDim = dim3(plan.s_splits, c.n_kv_heads, c.n_seqs + (args.beside ? 1 : 0));
    cfg.dynamicSmemBytes = v.smem;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, v.fn, args);
    if (e != cudaSuccess) return (int)e;
  }
  const MergeArgs m{p,          seq_lens,   cu_group, prefix,    n_groups,     max_group,     max_prefix,
                    max_suffix, c.capacity, c.n_seqs, n_q_heads, plan.p_chunk, plan.p_splits, plan.s_chunk,
                    plan.s_splits, args.partials, out, out_f32, lse};
  const int n_rows = c.n_seqs * n_q_heads;
  cfg.gridDim = dim3((unsigned)((n_rows + kMergeRows - 1) / kMergeRows));
  cfg.blockDim = dim3(merge_threads(p.d));
  cfg.dynamicSmemBytes = 0;
  const auto merge = p.d == 64 ? shared_merge_kernel<64> : p.d == 256 ? shared_merge_kernel<256> : shared_merge_kernel<128>;
  return (int)cudaLaunchKernelEx(&cfg, merge, m, n_rows);
}

}  // namespace tq
