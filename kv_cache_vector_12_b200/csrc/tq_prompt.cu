// Causal attention over whole bf16 prompts packed one behind the other,
// grouped query heads, sm_100a: the exact attention of a prompt's own tokens,
// the step a serving loop runs beside tq_quantize (which packs the same K and
// V for the decode that follows).
//
//   o_i = sum_{j <= i} p_ij v_j / l_i,  p_ij = 2^(c q_i . k_j - r_i),
//   l_i = sum_{j <= i} p_ij,            c = scale log2(e),
//   lse_i = ln 2 (r_i + log2 l_i)
// with r_i a running reference: the row's maximum when it was last moved.
// Keys are taken 64 at a time; r_i moves only when a step's maximum passes it
// by more than kLazy (so p <= 2^kLazy, far below the range of bf16 and fp32),
// which makes rescaling O rare: after the first steps almost no row moves.
//
// A CTA takes NT tiles of 128 query rows of one KV head (a row is one
// (position, query head) pair: with G heads per KV head a tile holds 128 / G
// positions, so K and V are read once for the whole group and a prompt of one
// token still fills G rows) against the keys at or before them:
//   producer  (1 thread)  Q once, then K and V tiles by TMA into a ring of
//             128-byte-swizzled slots;
//   MMA       (1 warp per row tile)  S = Q K^T, then O += P V with P as the A operand in
//             tensor memory and V read from its token-major tile as an
//             MN-major B operand (no transpose anywhere);
//   softmax   (4 warps per row tile, one thread per row)  S from tensor
//             memory, mask on diagonal steps only, exp2, P as bf16 back over
//             the S it came from, and at the end O / l to global memory.
// Every row tile has two S buffers of 64 keys: the scores of step h + 1 are
// there when the softmax of step h ends, so the softmax warps, which bound the
// kernel (one exp2 per score), do not wait for an MMA.  (With one buffer of
// 128 keys a row tile alternated between 2000 cycles of softmax and 2100 of
// hand-over and MMAs.)  Two row tiles per CTA at d = 64 and 128, one at d = 256,
// where O alone takes half of tensor memory; Q has the room that is left there,
// so that the scores' A operand takes no shared-memory reads (32 cycles an MMA
// of N = 64 instead of 50) and the ring has 7 slots instead of 5 (a K tile's load
// no longer waits for the values of the step before): 540 -> 438 us for 5 prompts
// of up to 5000 tokens, 16 over 4 heads, in a loop on one input (whose K and V
// then stay in L2).
// Measured on changing inputs: one prompt of 32768 tokens, 32 over 8 heads, d = 128,
// 7.9 ms (1.11 PFLOP/s, a plain bf16 GEMM sustains 1.40), one of 16384 at 28 over 4
// heads 1.84 ms (1.05); 17 of up to 4001 tokens 1.43 ms (0.86); d = 256, 5 of up to
// 5000, 435 us (0.92).  No pipe is full (tensor 47 %, MUFU 36 %, issue 42 %): a long
// prompt is bound by the hand-overs between the softmax and MMA warps of a row tile,
// many short ones also by each CTA's start and end, which one CTA per SM leaves
// uncovered.
// P is rounded to bf16, V's type (one MMA takes one type for A and B); l is
// summed in fp32 from the unrounded weights.
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "tq_tc.cuh"

namespace tq {
namespace {

// longest prompt up to which the form with one row tile runs.  Measured, 32768
// tokens of prompts of 1 .. n tokens, 8 KV and 32 query heads, one row tile / two:
// d = 64, n = 256 116 / 146 us, 1024 160 / 173, 2048 232 / 231, 4096 455 / 430;
// d = 128, n = 256 144 / 181, 512 181 / 201, 1024 215 / 211, 4096 645 / 456.
constexpr int kSmallLen64 = 2048, kSmallLen128 = 768;
constexpr int kStep = 64;     // keys per step: one S buffer
constexpr int kPoly = 4;      // pairs of every 16 whose exp2 runs on the FMA pipe
constexpr float kLazy = 8.f;  // log2 units a tile's maximum may pass the reference
constexpr float kFloor = -3.0e38f;  // of the reference: a difference to it is never inf - inf

// Two forms.  With two row tiles (d = 64 and 128) a CTA fills an SM and shares
// K and V between them: long prompts.  With one row tile, tiles of 64 keys and
// half of tensor memory two CTAs fit an SM (d = 64 and 128), so that the start
// and the end of one run under the other: short prompts.  At d = 256 O takes
// half of tensor memory for one row tile, and a CTA the SM.
template <int DH, int ROWS>
struct PromptCfg {
  static constexpr int NT = ROWS;                   // row tiles of 128
  static constexpr int KT = NT == 1 ? 64 : 128;     // keys per tile of K or V
  static constexpr int kSteps = KT / kStep;         // steps per tile
  static constexpr int kPerSm = NT == 1 && DH < 256 ? 2 : 1;  // CTAs per SM
  static constexpr int kBoxes = DH / 64;            // 64-column swizzled boxes per operand
  static constexpr int kQBox = 128 * 128;           // bytes of one box of a Q tile
  static constexpr int kKVBox = KT * 128;           // bytes of one box of a K or V tile
  static constexpr int kQTile = kBoxes * kQBox;
  static constexpr int kSlot = kBoxes * kKVBox;
  // Q goes to tensor memory where that has room for it (d = 256): through the
  // ring's first kQItems slots, so that K and V have 7 slots instead of 5
  static constexpr bool kQTmem = DH == 256;
  static constexpr int kQItems = kQTmem ? kQTile / kSlot : 0;
  static constexpr int kSlots = DH == 64 ? (NT == 2 ? 8 : 5) : DH == 128 ? (NT == 1 ? 4 : 5) : 7;  // at least 4
  static constexpr int kSoftWarps = 4 * NT;
  static constexpr int kProdWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
  static constexpr int kThreads = 32 * (kSoftWarps + 1 + NT);  // an MMA warp per row tile
  static constexpr int kQBytes = kQTmem ? 0 : NT * kQTile;
  static constexpr int smem = 1024 + kQBytes + kSlots * kSlot;
  // tensor-memory columns: two S buffers per row tile (P over them), O, and Q at d = 256
  static constexpr uint32_t kCols = NT * (128u + DH) <= 256 ? 256 : 512;
  static constexpr uint32_t s_col(int i, int b) { return 128u * i + 64u * b; }
  static constexpr uint32_t o_col(int i) { return 128u * NT + (uint32_t)DH * i; }
  static constexpr uint32_t q_col = (128u + DH) * NT;
  static_assert(!kQTmem || (NT == 1 && q_col + DH / 2 <= kCols && kQTile % kSlot == 0), "room for Q");
  // instruction descriptors, kind::f16: bf16 A and B, fp32 D, M = 128; S has
  // both operands K-major, O has B MN-major (bit 16)
  static constexpr uint32_t base = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 4) << 24);
  static constexpr uint32_t idesc_s = base | ((uint32_t)(kStep >> 3) << 17);
  static constexpr uint32_t idesc_o = base | (1u << 16) | ((uint32_t)(DH >> 3) << 17);
};

struct PromptArgs {
  unsigned *err;
  const int32_t *cu;
  int n_seqs, n_tok, max_len;
  int n_q_heads, n_kv_heads, per_tile;  // positions per row tile
  float c;                              // scale log2(e)
  void *out;                            // [n_tok][n_q_heads][d], bf16 or fp32
  bool out_f32;
  float *lse;                           // [n_tok][n_q_heads] or null
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float f(uint32_t x) { return __uint_as_float(x); }

// 2^x of two numbers on the FMA pipe: x = n + f with n the nearest integer
// (added and subtracted 1.5 2^23), a polynomial of degree 5 for 2^f on
// [-1/2, 1/2] (minimax of the relative error, fitted by weighted least squares:
// 2.3e-7 in fp32, what ex2.approx has), and n added to the exponent.  Below
// 2^-126 the result is some number under 2^-125 rather than 0.  NaN and +inf are
// lost here: the row's maximum finds them.
__device__ __forceinline__ float2 exp2_fma(float2 x) {
  x.x = fmaxf(x.x, -126.f);
  x.y = fmaxf(x.y, -126.f);
  const float2 big = make_float2(12582912.f, 12582912.f);
  const float2 t = add2(x, big);
  const float2 g = add2(x, mul2(add2(t, make_float2(-big.x, -big.y)), make_float2(-1.f, -1.f)));
  float2 p = make_float2(1.3276471e-3f, 1.3276471e-3f);
  p = fma2(p, g, make_float2(9.6755410e-3f, 9.6755410e-3f));
  p = fma2(p, g, make_float2(5.5507131e-2f, 5.5507131e-2f));
  p = fma2(p, g, make_float2(2.4022120e-1f, 2.4022120e-1f));
  p = fma2(p, g, make_float2(6.9314694e-1f, 6.9314694e-1f));
  p = fma2(p, g, make_float2(1.0000001f, 1.0000001f));
  return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23)));
}

// A bounded wait; false (the error flagged, the producer told to stop) once it
// expires: every role then ends at its own next wait, at most 2 s later.  Only the first test is inlined: the waits are many, and the loop
// and its error path would crowd the instruction cache.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, unsigned *err, int *stop) {
  if (bar_wait(bar, parity)) return true;
  atomicOr(err, kErrWaitExpired);
  *(volatile int *)stop = 1;
  return false;
}
__device__ __forceinline__ bool wait_or_stop(uint64_t *bar, uint32_t parity, unsigned *err, int *stop) {
  const uint32_t b = smem_addr(bar);
  return bar_try(b, parity) || wait_slow(b, parity, err, stop);
}
// The same by a whole warp: every lane leaves with the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, unsigned *err, int *stop) {
  return __all_sync(0xffffffffu, wait_or_stop(bar, parity, err, stop));
}

// The first tests of three waits, in flight together: 1 if all have passed.
__device__ __forceinline__ uint32_t test_three(uint64_t *b0, uint32_t p0, uint64_t *b1, uint32_t p1, uint64_t *b2,
                                               uint32_t p2) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q, r;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 r, [%5], %6;\n"
      " and.pred p, p, q;\n and.pred p, p, r;\n selp.b32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_addr(b0)), "r"(p0), "r"(smem_addr(b1)), "r"(p1), "r"(smem_addr(b2)), "r"(p2)
      : "memory");
  return ok;
}

// Query blocks (of `span` positions) of sequence s; 0 for a sequence outside
// the call's bounds.
__device__ __forceinline__ int blocks_of_seq(const PromptArgs &a, int s, int span, bool &bad) {
  const int b = a.cu[s], e = a.cu[s + 1];
  bad = b < 0 || e < b || e > a.n_tok || e - b > a.max_len;
  return bad ? 0 : (e - b + span - 1) / span;
}

__device__ __forceinline__ int inclusive(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Blocks of the run of sequences that thread t counts for find_block.
template <int kThreads>
__device__ __forceinline__ int count_run(const PromptArgs &a, int span, int t) {
  const int run = (a.n_seqs + kThreads - 1) / kThreads, b = min(t * run, a.n_seqs), e = min(b + run, a.n_seqs);
  int n = 0;
  bool bad, any_bad = false;
#pragma unroll 4
  for (int i = b; i < e; ++i) {
    n += blocks_of_seq(a, i, span, bad);
    any_bad |= bad;
  }
  if (any_bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, kErrSeqLen);
  return n;
}

// The sequence and query block of CTA x, by one warp; s = -1 when there is
// none.  Blocks with more keys come first, so that the last CTAs to start are
// the shortest: within a sequence from its end, and with at most 32 sequences
// (one per lane) across them too.  F(L) = sum_s max(0, blocks_s - L) blocks lie
// at level L or above; the CTA's level is the largest L with F(L) > x.
// With more than 32, part[t] holds the blocks of run t of kThreads equal runs of
// sequences, counted by thread t beforehand.
template <int kThreads>
__device__ __forceinline__ void find_block(const PromptArgs &a, int span, int x, int lane, const int *part, int &s,
                                           int &blk) {
  s = -1;
  blk = 0;
  bool bad = false, any_bad = false;
  if (a.n_seqs <= 32) {
    const int nb = lane < a.n_seqs ? blocks_of_seq(a, lane, span, bad) : 0;
    any_bad = bad;
    const unsigned total = __reduce_add_sync(0xffffffffu, (unsigned)nb);
    if ((unsigned)x < total) {
      int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu, (unsigned)nb);  // F(lo) > x >= F(hi)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__reduce_add_sync(0xffffffffu, (unsigned)max(0, nb - mid)) > (unsigned)x) lo = mid;
        else hi = mid;
      }
      // the blocks above level lo come first; this is the k-th sequence that reaches it
      const int k = x - (int)__reduce_add_sync(0xffffffffu, (unsigned)max(0, nb - lo - 1));
      const unsigned reach = __ballot_sync(0xffffffffu, nb > lo);
      s = __fns(reach, 0, k + 1);
      blk = lo;
    }
  } else {
    // the run that holds block x, then the sequence in it
    const int run = (a.n_seqs + kThreads - 1) / kThreads;
    int done = 0, lo = -1;  // done: blocks of the sequences before lo
    for (int t0 = 0; t0 < kThreads && lo < 0; t0 += 32) {
      const int n = part[t0 + lane], inc = inclusive(n, lane);
      const unsigned past = __ballot_sync(0xffffffffu, done + inc > x);
      const int l = past ? __ffs(past) - 1 : 31;
      done += __shfl_sync(0xffffffffu, past ? inc - n : inc, l);
      if (past) lo = (t0 + l) * run;
    }
    for (int i0 = 0; lo >= 0 && s < 0 && i0 < run; i0 += 32) {
      const int i = lo + i0 + lane;
      const int n = i0 + lane < run && i < a.n_seqs ? blocks_of_seq(a, i, span, bad) : 0, inc = inclusive(n, lane);
      const unsigned past = __ballot_sync(0xffffffffu, done + inc > x);
      const int l = past ? __ffs(past) - 1 : 31, end = done + __shfl_sync(0xffffffffu, inc, l);
      if (past) {
        s = lo + i0 + l;
        blk = end - 1 - x;  // from the sequence's end
      }
      done = end;
    }
  }
  if (any_bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, kErrSeqLen);
}

template <int DH, int ROWS>
__global__ void __launch_bounds__(PromptCfg<DH, ROWS>::kThreads, PromptCfg<DH, ROWS>::kPerSm)
    prompt_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
  using C = PromptCfg<DH, ROWS>;
  constexpr int NT = C::NT, KT = C::KT;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *sm = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  unsigned char *ring = sm + C::kQBytes;
  __shared__ __align__(8) uint64_t q_full, full[C::kSlots], empty[C::kSlots];
  __shared__ __align__(8) uint64_t s_full[2][2], p_full[2][2], pv_done[2], o_full[2], fin[2];  // [row tile][buffer]
  __shared__ uint32_t tmem_slot;
  __shared__ int stop, s_seq, s_blk, s_part[C::kThreads];

  const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31, h_kv = blockIdx.y;
  const int G = a.n_q_heads / a.n_kv_heads, PC = a.per_tile, span = NT * PC;
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_q) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v) : "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (a.n_seqs > 32) {
    s_part[tid] = count_run<C::kThreads>(a, span, tid);
    __syncthreads();
  }
  if (warp == 0) {
    int s, blk;
    find_block<C::kThreads>(a, span, blockIdx.x, lane, s_part, s, blk);
    if (lane == 0) {
      s_seq = s;
      s_blk = blk;
      stop = 0;
    }
  } else if (warp == C::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                 "r"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == C::kProdWarp && lane == 0) {
    bar_init(smem_addr(&q_full), C::kQTmem ? 4 : 1);  // (in tensor memory: by the softmax warps)
    for (int i = 0; i < C::kSlots; ++i) {
      bar_init(smem_addr(&full[i]), 1);
      bar_init(smem_addr(&empty[i]), NT);
    }
    for (int i = 0; i < 2; ++i) {
      for (int b = 0; b < 2; ++b) {
        bar_init(smem_addr(&s_full[i][b]), 1);
        bar_init(smem_addr(&p_full[i][b]), 4);
      }
      bar_init(smem_addr(&pv_done[i]), 1);
      bar_init(smem_addr(&o_full[i]), 1);
      bar_init(smem_addr(&fin[i]), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (with all 512 columns this CTA's, they start at column 0)
  const uint32_t tmem = C::kCols == 512 ? 0u : tmem_slot;
  const int s = s_seq;

  if (s >= 0) {
    const int tok0 = a.cu[s], len = a.cu[s + 1] - tok0;
    const int first = s_blk * span;                    // first query position
    // keys at or before the last query of each row tile, in steps and tiles
    int steps[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int b = first + i * PC, e = min(len, b + PC);
      steps[i] = e > b ? (e + kStep - 1) / kStep : 0;
    }
    const int n_steps = NT == 2 ? max(steps[0], steps[1]) : steps[0];
    const int n_tiles = (n_steps + C::kSteps - 1) / C::kSteps;

    if (warp == C::kProdWarp) {
      // ---------------- producer
      if (lane == 0) {
        const uint32_t box = (uint32_t)(PC * G * 128);
        if (!C::kQTmem) bar_expect_tx(smem_addr(&q_full), (NT == 2 && steps[1] ? 2 : 1) * C::kBoxes * box);
        for (int i = 0; i < C::kQItems; ++i) bar_expect_tx(smem_addr(&full[i]), C::kSlot / C::kQBox * box);
        for (int i = 0; i < NT; ++i)
          if (steps[i])
            for (int b = 0; b < C::kBoxes; ++b)  // (in the ring: a slot after the other)
              tma_load_3d(smem_addr(sm + i * C::kQTile + b * C::kQBox), &map_q, 64 * b, h_kv * G, tok0 + first + i * PC,
                          smem_addr(C::kQTmem ? &full[b * C::kQBox / C::kSlot] : &q_full));
        int issued = C::kQItems;
        int slot = C::kQItems, phase = 1;
        for (int it = C::kQItems; it < C::kQItems + 2 * n_tiles; ++it) {  // K 0, V 0, K 1, V 1, ...
          if (it >= C::kSlots && !wait_or_stop(&empty[slot], phase, a.err, &stop)) break;
          if (*(volatile int *)&stop) break;
          bar_expect_tx(smem_addr(&full[slot]), C::kSlot);
          for (int b = 0; b < C::kBoxes; ++b)
            tma_load_3d(smem_addr(ring + slot * C::kSlot + b * C::kKVBox), (it & 1) ? &map_v : &map_k, 64 * b, h_kv,
                        tok0 + ((it - C::kQItems) >> 1) * KT, smem_addr(&full[slot]));
          issued = it + 1;
          if (++slot == C::kSlots) {
            slot = 0;
            phase ^= 1;
          }
        }
        if (*(volatile int *)&stop) {  // never leave copies in flight
          if (!C::kQTmem) bar_wait(smem_addr(&q_full), 0);
          for (int it = max(0, issued - C::kSlots); it < issued; ++it)
            bar_wait(smem_addr(&full[it % C::kSlots]), (it / C::kSlots) & 1);
        }
      }
    } else if (warp >= C::kMmaWarp) {
      // ---------------- MMA issuer of row tile i (the whole warp; one lane
      // issues).  A warp per row tile: with one for both, the issue (about 55
      // cycles an MMA beside busy softmax warps) and the waits in between took
      // longer than the MMAs.
      const int i = warp - C::kMmaWarp, mine = steps[i];
      // K tile of the step whose scores are next and V tile of the step whose
      // values are next: ring slots and their phases, advanced without division
      int ks = C::kQItems, kp = 0, vs = C::kQItems + 1, vp = 0;
      auto advance = [&](int &slot, int &phase) {
        slot += 2;
        if (slot >= C::kSlots) {
          slot -= C::kSlots;
          phase ^= 1;
        }
      };
      const uint64_t q = sw128_desc(smem_addr(sm + i * C::kQTile));
      const uint64_t k0 = sw128_desc(smem_addr(ring)), v0 = mn_desc(smem_addr(ring), C::kKVBox);
      const uint32_t d_o = tmem + C::o_col(0) + (uint32_t)DH * i, d_s = tmem + 128u * i;
      constexpr int kSlotU = C::kSlot >> 4, kStepU = (kStep * 128) >> 4;  // descriptor units
      // Step h: O += P V, then S of step h + 2 over the P just read (MMAs of one
      // thread run in order); two S go ahead.  A tile's slot is given back after
      // its last step, also by a row tile that needs fewer.
      bool ok = warp_wait(&q_full, 0, a.err, &stop);
      if (lane < C::kQItems && ok) bar_arrive(smem_addr(&empty[lane]));  // (Q's slots, read by the softmax warps)
      const int last = n_tiles * C::kSteps;
#pragma unroll 1
      for (int h = -2; ok && h < last; ++h) {
        const int n = h + 2;
        const bool need_v = h >= 0 && h % C::kSteps == 0, need_k = n < last && n % C::kSteps == 0;
        const bool need_p = h >= 0 && h < mine;
        // (one row tile: usually all three are there, and one test of each is
        // quicker than three waits, 373 us against 438 for 5 prompts of up to
        // 5000 tokens at d = 256 in a loop on one input; with two row tiles P
        // mostly is not, and the tests in front of the wait cost 3 %)
        uint32_t ready = 0;
        if (NT == 1 && need_v && need_k && need_p)
          ready = test_three(&full[vs], vp, &full[ks], kp, &p_full[i][h & 1], (h >> 1) & 1);
        if (NT == 2 || !__all_sync(0xffffffffu, ready)) {
          if (need_v) ok = warp_wait(&full[vs], vp, a.err, &stop);
          if (ok && need_k) ok = warp_wait(&full[ks], kp, a.err, &stop);
          if (ok && need_p) ok = warp_wait(&p_full[i][h & 1], (h >> 1) & 1, a.err, &stop);
          if (!ok) break;
        }
        tc_fence_after();
        const bool v_end = h >= 0 && h % C::kSteps == C::kSteps - 1, k_end = n < last && n % C::kSteps == C::kSteps - 1;
        if (elect_one()) {
          if (h >= 0 && h < mine) {
            const uint64_t v = v0 + (uint64_t)(vs * kSlotU + (h % C::kSteps) * kStepU);
#pragma unroll
            for (int kk = 0; kk < kStep / 16; ++kk)  // 16 tokens: 2048 bytes
              mma_ts(d_o, d_s + 64u * (h & 1) + 8 * kk, v + kk * (2048 >> 4), C::idesc_o, (h > 0 || kk > 0) ? 1u : 0u);
            if (h + 2 == mine) tc_commit(smem_addr(&pv_done[i]));
            if (h + 1 == mine) tc_commit(smem_addr(&o_full[i]));
          }
          if (v_end) tc_commit(smem_addr(&empty[vs]));
          if (n < mine) {
            const uint64_t k = k0 + (uint64_t)(ks * kSlotU + (n % C::kSteps) * kStepU);
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk)
              if (C::kQTmem)
                mma_ts(d_s + 64u * (n & 1), tmem + C::q_col + 8 * kk, k + (((kk >> 2) * C::kKVBox + (kk & 3) * 32) >> 4),
                       C::idesc_s, kk > 0);
              else
                tc_mma_n(d_s + 64u * (n & 1), q + (((kk >> 2) * C::kQBox + (kk & 3) * 32) >> 4),
                         k + (((kk >> 2) * C::kKVBox + (kk & 3) * 32) >> 4), C::idesc_s, kk > 0);
            tc_commit(smem_addr(&s_full[i][n & 1]));
          }
          if (k_end) tc_commit(smem_addr(&empty[ks]));
        }
        __syncwarp();
        if (v_end) advance(vs, vp);
        if (k_end) advance(ks, kp);
      }
      // every MMA issued here has completed before the tensor memory is released
      if (elect_one()) tc_commit(smem_addr(&fin[i]));
      __syncwarp();
      bar_wait(smem_addr(&fin[i]), 0);
    } else {
      // ---------------- softmax: row tile i, one thread per row
      const int i = NT == 2 ? warp >> 2 : 0, row = tid & 127;
      const int n = steps[i], base = first + i * PC;
      const int t = row / G, pos = (row < PC * G && base + t < len) ? base + t : -1;
      const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
      const uint32_t t_o = tmem + C::o_col(i) + lanes;
      const float kNan = __int_as_float(0x7fc00000);
      float ref = 0.f, l = 0.f;
      bool ok = true;
      if constexpr (C::kQTmem) {
        // Q's row from the swizzled boxes into tensor memory, as the scores' A operand
#pragma unroll 1
        for (int b = 0; ok && b < C::kBoxes; ++b) {
          if (b * C::kQBox % C::kSlot == 0) ok = warp_wait(&full[b * C::kQBox / C::kSlot], 0, a.err, &stop);
          if (!ok) break;
          uint32_t x[32];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint4 u = *reinterpret_cast<const uint4 *>(sm + b * C::kQBox + 128 * row + 16 * (e ^ (row & 7)));
            x[4 * e] = u.x;
            x[4 * e + 1] = u.y;
            x[4 * e + 2] = u.z;
            x[4 * e + 3] = u.w;
          }
          tmem_st32(tmem + C::q_col + lanes + 32 * b, x);
        }
        st_wait();
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) bar_arrive(smem_addr(&q_full));
      }
#pragma unroll 1
      for (int h = 0; ok && h < n; ++h) {
        const uint32_t t_s = tmem + C::s_col(i, h & 1) + lanes;
        ok = warp_wait(&s_full[i][h & 1], (h >> 1) & 1, a.err, &stop);
        if (!ok) break;
        tc_fence_after();
        uint32_t v[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(t_s + 32 * c, v[c]);
        ld_wait();
#pragma unroll
        for (int c = 0; c < 2; ++c) pin32(v[c]);
        const int key0 = h * kStep;
        if (key0 + kStep - 1 > base) {  // some row of the tile does not see every key
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (key0 + 32 * c + e > pos) v[c][e] = 0xff800000u;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2) mx = max3_nan(mx, f(v[c][e]), f(v[c][e + 1]));
        mx *= a.c;
        // A row with a score of NaN or +inf is NaN (inf - inf): its sum becomes NaN
        // here, as the maximum tells, since exp2_fma keeps neither.
        if (h == 0) {
          ref = fmaxf(mx, kFloor);
          if (!(mx < INFINITY)) l = kNan;
        } else if (__any_sync(0xffffffffu, pos >= 0 && !(mx <= ref + kLazy))) {  // (rows of no query hold anything)
          // O is rescaled once the values of step h - 1 are in it: the scores of
          // step h + 1 were issued behind them (in front of the last step nothing
          // was, so those have a barrier of their own)
          ok = h + 1 < n ? warp_wait(&s_full[i][(h + 1) & 1], ((h + 1) >> 1) & 1, a.err, &stop)
                         : warp_wait(&pv_done[i], 0, a.err, &stop);
          if (!ok) break;
          tc_fence_after();
          const float nref = fmaxf(ref, mx), al = ex2(ref - nref);
          ref = nref;
          l = mx < INFINITY ? l * al : kNan;
#pragma unroll 1
          for (int c = 0; c < DH / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(t_o + 32 * c, o);
            ld_wait();
            pin32(o);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 w = mul2(make_float2(f(o[e]), f(o[e + 1])), make_float2(al, al));
              o[e] = __float_as_uint(w.x);
              o[e + 1] = __float_as_uint(w.y);
            }
            tmem_st32(t_o + 32 * c, o);
          }
        }
        const float2 c2 = make_float2(a.c, a.c), r2 = make_float2(-ref, -ref);
        float2 sum = make_float2(0.f, 0.f);
        // kPoly of every 16 pairs on the FMA pipe, the others on the MUFU (16 a
        // clock and SM: 64 scores of a warp take it 512 cycles); steps with
        // masked scores, whose weights have to be exactly 0, all on the MUFU
        auto weights = [&](auto mixed) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 x = fma2(make_float2(f(v[c][2 * e]), f(v[c][2 * e + 1])), c2, r2);
              float2 w;
              if (decltype(mixed)::value && e % (16 / kPoly) == 1) w = exp2_fma(x);
              else w = make_float2(ex2(x.x), ex2(x.y));
              sum = add2(sum, w);
              p[e] = pack_bf16(w.x, w.y);
            }
            tmem_st16(t_s + 16 * c, p);
          }
        };
        if (key0 + kStep - 1 > base) weights(std::false_type{});
        else weights(std::true_type{});
        l += sum.x + sum.y;
        if (key0 + kStep > len) {
          // the step's rows behind the sequence's end hold other tokens: zero
          // them, so that a weight of 0 times what they hold stays 0
          const int vs = C::kQItems + 2 * (h / C::kSteps) + 1;
          ok = warp_wait(&full[vs % C::kSlots], (vs / C::kSlots) & 1, a.err, &stop);
          if (!ok) break;
          unsigned char *vt = ring + (vs % C::kSlots) * C::kSlot + (h % C::kSteps) * (kStep * 128);
          for (int x = 128 * (len - key0) + 16 * row; x < kStep * 128; x += 128 * 16)
#pragma unroll
            for (int b = 0; b < C::kBoxes; ++b) *reinterpret_cast<uint4 *>(vt + b * C::kKVBox + x) = make_uint4(0, 0, 0, 0);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&p_full[i][h & 1]));
      }
      if (ok && n > 0) {
        ok = warp_wait(&o_full[i], 0, a.err, &stop);
        if (ok) {
          tc_fence_after();
          // A row whose scores are all -inf (its reference never moved off the
          // floor) has no weights but what the polynomial puts for 2^-inf:
          // o = 0 / 0 and lse = -inf, or NaN where a score was one
          if (!(ref > kFloor)) l *= 0.f;
          const float il = l > 0.f ? 1.f / l : kNan;
          const long orow = pos < 0 ? 0 : (long)(tok0 + pos) * a.n_q_heads + h_kv * G + row % G;
#pragma unroll 1
          for (int c = 0; c < DH / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(t_o + 32 * c, o);
            ld_wait();
            pin32(o);
            if (pos >= 0) {
              if (a.out_f32) {
                float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + orow * DH + 32 * c);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  dst[e] = make_float4(f(o[4 * e]) * il, f(o[4 * e + 1]) * il, f(o[4 * e + 2]) * il, f(o[4 * e + 3]) * il);
              } else {
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + orow * DH + 32 * c);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  dst[e] = make_uint4(pack_bf16(f(o[8 * e]) * il, f(o[8 * e + 1]) * il),
                                      pack_bf16(f(o[8 * e + 2]) * il, f(o[8 * e + 3]) * il),
                                      pack_bf16(f(o[8 * e + 4]) * il, f(o[8 * e + 5]) * il),
                                      pack_bf16(f(o[8 * e + 6]) * il, f(o[8 * e + 7]) * il));
              }
            }
          }
          if (a.lse && pos >= 0) a.lse[orow] = (ref + log2f(l)) * 0.6931471805599453f;
        }
      }
    }
  }
  // release the tensor memory once every MMA and tcgen05 access is finished
  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_slot), "r"(C::kCols) : "memory");
  }
}

// 3-D map over bf16 rows [tokens][heads][DH] with a token stride (elements),
// boxes of 64 columns x box_heads x box_tokens, 128-byte swizzle.
bool make_token_map(CUtensorMap *m, const void *base, int d, int heads, long tokens, long stride, int box_heads,
                    int box_tokens) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  const cuuint32_t estride[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DH, int ROWS>
int launch(PromptArgs args, const void *q, const void *k, const void *v, long qs, long ks, long vs,
           void *stream) {
  using C = PromptCfg<DH, ROWS>;
  const int G = args.n_q_heads / args.n_kv_heads;
  CUtensorMap mq, mk, mv;
  if (!make_token_map(&mq, q, DH, args.n_q_heads, args.n_tok, qs, G, args.per_tile) ||
      !make_token_map(&mk, k, DH, args.n_kv_heads, args.n_tok, ks, 1, C::KT) ||
      !make_token_map(&mv, v, DH, args.n_kv_heads, args.n_tok, vs, 1, C::KT))
    return (int)cudaErrorInvalidValue;
  static std::atomic<bool> configured[kMaxDevices];
  std::atomic<bool> &done = configured[current_device()];
  if (!done.load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(prompt_kernel<DH, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
    if (e != cudaSuccess) return (int)e;
    done.store(true, std::memory_order_release);
  }
  // at most this many query blocks, whatever the lengths
  const long span = (long)C::NT * args.per_tile;
  const long by_tok = (long)args.n_tok / span + args.n_seqs, by_len = (args.max_len + span - 1) / span * args.n_seqs;
  const long ctas = by_tok < by_len ? by_tok : by_len;
  if (ctas > 0x7fffffffl) return (int)cudaErrorInvalidConfiguration;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, args.n_kv_heads);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::smem;
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, prompt_kernel<DH, ROWS>, args, mq, mk, mv);
}

}  // namespace

int launch_prompt(const DeviceParams &p, const void *q, const void *k, const void *v, long q_stride, long k_stride,
                  long v_stride, int n_tok, int n_q_heads, int n_kv_heads, const int32_t *cu, int n_seqs, int max_len,
                  float scale, void *out, bool out_f32, float *lse, void *stream) {
  PromptArgs a{};
  a.err = p.err;
  a.cu = cu;
  a.n_seqs = n_seqs;
  a.n_tok = n_tok;
  a.max_len = max_len;
  a.n_q_heads = n_q_heads;
  a.n_kv_heads = n_kv_heads;
  a.per_tile = 128 / (n_q_heads / n_kv_heads);
  a.c = scale * 1.4426950408889634f;
  a.out = out;
  a.out_f32 = out_f32;
  a.lse = lse;
  const bool small = max_len <= (p.d == 64 ? kSmallLen64 : kSmallLen128);
  if (p.d == 256) return launch<256, 1>(a, q, k, v, q_stride, k_stride, v_stride, stream);
  if (p.d == 64)
    return small ? launch<64, 1>(a, q, k, v, q_stride, k_stride, v_stride, stream)
                 : launch<64, 2>(a, q, k, v, q_stride, k_stride, v_stride, stream);
  return small ? launch<128, 1>(a, q, k, v, q_stride, k_stride, v_stride, stream)
               : launch<128, 2>(a, q, k, v, q_stride, k_stride, v_stride, stream);
}

}  // namespace tq
