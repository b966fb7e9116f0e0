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
#include <cmath>

#include "tq_decode_kernel.cuh"
#include "tq_merge.cuh"
#include "tq_shared_tc.h"

namespace tq {
namespace {

constexpr int kTcMinRows = 16;   // rows of a group above which the tcgen05 prefix pass runs
constexpr int kTcFixed = 4;
constexpr int kMaxSlots = 1024;  // split partials of one row, both passes

struct MergeArgs {
  DeviceParams p;
  const int32_t *seq_lens, *cu_group, *prefix;
  int n_groups, max_group, max_prefix, max_suffix, capacity, n_q_heads;
  int p_chunk, p_splits, s_chunk, s_splits;
  const float *partials;
  void *out;
  bool out_f32;
  float *lse;
};

// One CTA of 128 threads per (sequence, query head).
template <int DH>
__global__ void __launch_bounds__(128) shared_merge_kernel(const MergeArgs a) {
  constexpr int PF = DH + 4, PL = DH / 32;
  __shared__ float s_ot[DH];
  __shared__ float s_w[kMaxSlots];
  __shared__ __align__(16) float s_acc[4][DH];
  __shared__ float red[4];
  const int row = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Bf16Row<DH> pw0, pw1;
  if (tid < DH) pw0.load(a.p.pivt + tid * DH);
  if constexpr (DH == 256) pw1.load(a.p.pivt + (tid + 128) * DH);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int s = row / a.n_q_heads;
  const SeqRange g = sequence_range(a.cu_group, a.prefix, a.n_groups, a.seq_lens, a.max_group, a.max_prefix,
                                    a.max_suffix, a.capacity, s, lane);
  // the slots in use: the splits that hold positions, of either pass
  const int n_p = g.len > 0 && a.p_splits ? (g.prefix + a.p_chunk - 1) / a.p_chunk : 0;
  const int n_s = g.len > g.prefix ? (g.len - (g.prefix & ~63) + a.s_chunk - 1) / a.s_chunk : 0;
  const int used = n_p + n_s;
  const float *src = a.partials + (long)row * (a.p_splits + a.s_splits) * PF;
  auto slot = [&](int i) { return src + (long)(i < n_p ? i : a.p_splits + i - n_p) * PF; };
  float mloc = -INFINITY;
  for (int i = tid; i < used; i += 128) mloc = fmaxf(mloc, s_w[i] = slot(i)[0]);
  const float mm = block_max128(mloc, red);
  float lpart = 0.f;
  for (int i = tid; i < used; i += 128) {
    const float w = s_w[i] == -INFINITY ? 0.f : exp2f(s_w[i] - mm);
    s_w[i] = w;
    lpart = fmaf(w, slot(i)[1], lpart);
  }
  __syncthreads();
  float acc[PL];
#pragma unroll
  for (int c = 0; c < PL; ++c) acc[c] = 0.f;
#pragma unroll 4
  for (int i = warp; i < used; i += 4) {
    float v[PL];
    load_floats<PL>(slot(i) + 4 + lane * PL, v);
    const float w = s_w[i];
#pragma unroll
    for (int c = 0; c < PL; ++c) acc[c] = fmaf(w, v[c], acc[c]);
  }
#pragma unroll
  for (int c = 0; c < PL; ++c) s_acc[warp][lane * PL + c] = acc[c];
  for (int o = 16; o; o >>= 1) lpart += __shfl_xor_sync(0xffffffffu, lpart, o);
  if (lane == 0) red[warp] = lpart;
  __syncthreads();
  const float ll = (red[0] + red[1]) + (red[2] + red[3]);
  for (int i = tid; i < DH; i += 128) {
    const float oo = (s_acc[0][i] + s_acc[1][i]) + (s_acc[2][i] + s_acc[3][i]);
    s_ot[i] = used > 0 ? oo / ll : 0.f;
  }
  __syncthreads();
  auto store = [&](int i, float x) {
    if (a.out_f32) static_cast<float *>(a.out)[(long)row * DH + i] = x;
    else static_cast<__nv_bfloat16 *>(a.out)[(long)row * DH + i] = __float2bfloat16_rn(x);
  };
  if (tid < DH) store(tid, dot_bf16_row<DH>(pw0, s_ot));
  if constexpr (DH == 256) store(tid + 128, dot_bf16_row<DH>(pw1, s_ot));
  if (a.lse && tid == 0) a.lse[row] = used > 0 ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

SharedPlan plan_shared(int d, int bits_k, int bits_v, int qjl, int n_seqs, int n_q_heads, int n_kv_heads, int n_groups,
                       int max_group, int max_prefix, int max_suffix) {
  SharedPlan s = {};
  const int per = n_q_heads / n_kv_heads;
  s.tc = d == kHeadDim && !qjl && (long)per * max_group > kTcMinRows;
  s.nt_p = (long)per * max_group > 8 ? 2 : 1;
  s.members = (s.tc ? 128 : 8 * s.nt_p) / per;
  const long by_group = (long)n_groups * ((max_group + s.members - 1) / s.members);
  const long by_seq = (long)n_seqs / s.members + n_groups;
  s.units = (int)(by_group < by_seq ? by_group : by_seq);
  if (max_prefix > 0 && s.tc) {
    // splits of whole 128-key tiles, one CTA per SM: the count with the fewest
    // tile times over all waves, kTcFixed of them per CTA for its prologue
    // (q rotation) and its partial
    const long tiles = (max_prefix + 127) / 128, lanes = (long)s.units * n_kv_heads, sms = sm_count();
    long best = -1;
    for (long n = 1; n <= tiles && n <= 128; ++n) {
      const long per_split = (tiles + n - 1) / n, used = (tiles + per_split - 1) / per_split;
      const long cost = (lanes * used + sms - 1) / sms * (per_split + kTcFixed);
      if (best < 0 || cost < best) {
        best = cost;
        s.p_chunk = (int)(per_split * 128);
        s.p_splits = (int)used;
      }
    }
  } else if (max_prefix > 0) {
    const DecodeSplit sp =
        decode_split(s.units, n_kv_heads, max_prefix, shared_ctas_per_sm(d, bits_k, bits_v, qjl, s.nt_p));
    s.p_chunk = sp.chunk;
    s.p_splits = sp.n_splits;
  }
  s.nt_s = per > 8 ? 2 : 1;
  // (the suffix pass starts up to 63 positions before the prefix's end)
  const DecodeSplit ss =
      decode_split(n_seqs, n_kv_heads, max_suffix + 63, shared_ctas_per_sm(d, bits_k, bits_v, qjl, s.nt_s));
  s.s_chunk = ss.chunk;
  s.s_splits = ss.n_splits;
  const size_t rows = (size_t)n_seqs * n_q_heads;
  s.workspace = (rows * (size_t)(s.p_splits + s.s_splits) * (size_t)(d + 4) * sizeof(float) + 255) / 256 * 256;
  return s;
}

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
  cfg.blockDim = dim3(kThreads);
  if (plan.p_splits > 0 && plan.tc) {
    const SharedTcArgs t{p,         c,        n_q_heads,  q,            q_dtype,      scale,         cu_group, prefix,
                         n_groups, max_group, max_prefix, plan.members, plan.p_chunk, args.partials, args.n_splits};
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
    cfg.gridDim = dim3(plan.s_splits, c.n_kv_heads, c.n_seqs);
    cfg.dynamicSmemBytes = v.smem;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, v.fn, args);
    if (e != cudaSuccess) return (int)e;
  }
  const MergeArgs m{p,          seq_lens,   cu_group,  prefix,       n_groups,      max_group,    max_prefix,
                    max_suffix, c.capacity, n_q_heads, plan.p_chunk, plan.p_splits, plan.s_chunk, plan.s_splits,
                    args.partials, out, out_f32, lse};
  cfg.gridDim = dim3((unsigned)(c.n_seqs * n_q_heads));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  const auto merge = p.d == 64 ? shared_merge_kernel<64> : p.d == 256 ? shared_merge_kernel<256> : shared_merge_kernel<128>;
  return (int)cudaLaunchKernelEx(&cfg, merge, m);
}

}  // namespace tq
