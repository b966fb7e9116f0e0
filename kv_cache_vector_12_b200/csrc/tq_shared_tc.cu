// The prefix pass of shared-prefix decode attention on tcgen05, sm_100a:
// 128 rows (member, query head) of one KV head against a split of the packed
// prefix (d = 128, contexts without QJL).
//
// Keys are expanded in tiles of 128 and attended in halves of 64; four roles
// overlap across them:
//   expand   (8 warps, 16 keys of a tile each) K~ and ||v|| V~ from the
//            codes, token by token, as fp16 operands in shared memory, each
//            double-buffered (V~ is an MN-major operand: no transpose);
//   MMA      (1 thread) S = Q^_hi K~^T + Q^_lo K~^T (two-part fp16 q_hat in
//            tensor memory, about 22 bits), O += P (||v|| V~) with P in tensor
//            memory over the S it came from; S is double-buffered;
//   softmax  (4 x 4 warps, one thread per row) the sets take the halves in
//            turn: S from tensor memory, exp2 against the row's reference, P as
//            fp16 back;
//   producer (1 thread) the packed planes by bulk copies.
// A row's reference r is handed from half to half between the sets.  It
// moves, and O is rescaled, only when a half's maximum may pass it by more than
// kLazy log2 units (p <= 2^kLazy stays far inside fp16): the test takes
// max S times the half's largest key norm, a bound, and only when the bound
// fails the exact maximum, so the norms are read once per score.
// Roundings: P to fp16 (2^-11) and ||v|| c to fp16 (2^-11, the centroids times
// kVScale so that small norms stay normal); l is summed in fp32 from the
// unrounded weights.  Each CTA writes (r, l, O) of its rows for its split.
//
// Why 128 rows: a 16-row mma.sync tile re-expands every code once per 16 rows,
// and expansion (byte-permute lookups) is what bounds that path; here a code is
// expanded once for 128 rows.  Why loops that are not unrolled: with every
// loop unrolled (90 KB of code for five kinds of warps) instruction fetch took
// two thirds of the time.
// Measured, 3/3 bits, 8 KV heads: 128 rows behind 32768 positions 50 us (the
// 16-row tiles 130), 32 rows behind 131008 123 us.  No pipe is full (tensor 29 %,
// ALU 41 %, issue 55 %): a tile of 128 keys takes about 3700 cycles through the
// hand-overs between the roles.
#include <atomic>
#include <cmath>

#include "tq_expand.cuh"
#include "tq_f32x2.cuh"
#include "tq_groups.cuh"
#include "tq_shared_tc.h"
#include "tq_tmem.cuh"

namespace tq {
namespace {

constexpr float kLazy = 8.f;
constexpr float kVScale = 4.f;
constexpr int kHalf = 64, kBufs = 4;  // keys per S buffer, S buffers
// warps: four softmax sets, expansion, the producer and the MMA issuer; 26 warps
// leave 72 registers a thread
constexpr int kSets = 4, kSoftWarps = 4 * kSets, kExpWarps = 8;
constexpr int kExpWarp0 = kSoftWarps, kProdWarp = kExpWarp0 + kExpWarps, kMmaWarp = kProdWarp + 1;
constexpr int kTcThreads = 32 * (kMmaWarp + 1);
constexpr int kStagesTc = 4, kNormBufs = 4;
// tensor-memory columns: S buffers (P' over them), O, q_hat hi and lo
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384;

template <int BK, int BV>
struct SharedTc {
  static constexpr int kt = 0, vt = 2 * kOpBytes, ring = 4 * kOpBytes;
  static constexpr int stage = Stage<BK, BV, false, kTcKeys>::bytes;
  static constexpr int norms = ring + kStagesTc * stage;  // key norms, [buffer][key] fp32
  static constexpr int bytes = 1024 + norms + kNormBufs * kTcKeys * 4;
};

// kind::f16, fp32 accumulator, M = N = 128, A and B K-major: fp16 inputs
// (scores, values) and bf16 (the q rotation).
constexpr uint32_t kDescS = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kDescO = kDescS | (1u << 16);  // (V~ by tokens: B is MN-major)
constexpr uint32_t kDescQ = kDescS | (1u << 7) | (1u << 10);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
               "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
               : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ float f(uint32_t x) { return __uint_as_float(x); }

// A bounded wait; false (the error flagged, the kernel told to stop) once it
// expires.  Only the first test is inlined: the waits are many, and the loop
// and its error path would crowd the instruction cache.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, unsigned *err, int *stop) {
  if (mbar_wait(bar, parity)) return true;
  atomicOr(err, kErrWaitExpired);
  *(volatile int *)stop = 1;
  return false;
}
__device__ __forceinline__ bool wait_or_stop(uint64_t *bar, uint32_t parity, unsigned *err, int *stop) {
  const uint32_t b = smem_u32(bar);
  return mbar_try_wait(b, parity) || wait_slow(b, parity, err, stop);
}
// The same by a whole warp: every lane leaves with the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, unsigned *err, int *stop) {
  return __all_sync(0xffffffffu, wait_or_stop(bar, parity, err, stop));
}

template <int BK, int BV>
__global__ void __launch_bounds__(kTcThreads, 1) shared_prefix_tc_kernel(const SharedTcArgs a) {
  using L = SharedTc<BK, BV>;
  using St = Stage<BK, BV, false, kTcKeys>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *sm = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t full[kStagesTc], empty[kStagesTc];
  __shared__ __align__(8) uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2];
  __shared__ __align__(8) uint64_t p_full[kBufs], pv_done[kBufs], n_full[kNormBufs];
  __shared__ __align__(8) uint64_t checked[4][kSets], q_mma, q_ready, fin;
  __shared__ float s_ref[128], s_fq[128], s_l[kSets][128], s_lref[kSets][128];
  __shared__ float s_kmax[kNormBufs][kExpWarps];  // largest key norm of each warp's 16 keys
  __shared__ uint32_t tmem_slot;
  __shared__ int stop;

  const int split = blockIdx.x, h = blockIdx.y;
  const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
  const int per = a.n_q_heads / a.c.n_kv_heads;
  // Pi's rows in the K fragment order, the B operand of q_hat = Pi q, into
  // V~ of tile 1 (parameters: read before the kernels in front have ended)
  for (int i = tid; i < 128 * 16; i += kTcThreads) {
    const int row = i >> 4, c = 8 * (i & 15);
    *reinterpret_cast<uint4 *>(sm + L::vt + kOpBytes + sw_off(row, c)) =
        *reinterpret_cast<const uint4 *>(a.p.pi + (size_t)a.p.kperm[row] * D + c);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (the pass behind the prefix may start: it takes over what the kernels in
  // front of the call wrote, and the merge waits for both)
  if (tid == 0) {
    if (blockIdx.x + blockIdx.y + blockIdx.z == 0) hand_on(token_word(a.partials), a.token);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  const SharedUnit u = find_members(a.cu_group, a.n_groups, a.max_group, a.members, a.c.n_seqs, blockIdx.z, lane);
  if (u.count == 0) return;
  const int prefix = a.prefix[u.group];
  if (!any_member(a.seq_lens, u, lane)) return;
  // (a prefix outside its bounds is flagged by the pass behind it)
  if (prefix <= 0 || prefix > a.max_prefix || prefix > a.c.capacity) return;
  const int t0 = split * a.chunk;
  if (t0 >= prefix) return;
  const int t1 = min(prefix, t0 + a.chunk);
  const int n_tiles = (t1 - t0 + kTcKeys - 1) / kTcKeys, n_half = (t1 - t0 + kHalf - 1) / kHalf;
  const int rows = u.count * per;
  unsigned *err = a.p.err;

  if (tid == 0) {
    for (int i = 0; i < kStagesTc; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), kExpWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&k_full[b]), kExpWarps);
      mbar_init(smem_u32(&v_full[b]), kExpWarps);
      mbar_init(smem_u32(&k_empty[b]), 1);
      mbar_init(smem_u32(&v_empty[b]), 1);
      mbar_init(smem_u32(&s_full[b]), 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(smem_u32(&p_full[b]), 4);
      mbar_init(smem_u32(&pv_done[b]), 1);
    }
    for (int b = 0; b < kNormBufs; ++b) mbar_init(smem_u32(&n_full[b]), kExpWarps);
    for (int b = 0; b < kSets; ++b)
      for (int w = 0; w < 4; ++w) mbar_init(smem_u32(&checked[w][b]), 1);
    mbar_init(smem_u32(&q_mma), 1);
    mbar_init(smem_u32(&q_ready), 4);
    mbar_init(smem_u32(&fin), 1);
    stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // q's rows (bf16; fp32 q as hi + lo) into K~ of tile 1 (lo: of tile 0); zero
  // for members that take no part, whatever theirs hold: a moving reference
  // rescales a warp's rows together
  const bool f32 = a.q_dtype == TQ_F32;
  for (int i = tid; i < 128 * 16; i += kTcThreads) {
    const int row = i >> 4, c = 8 * (i & 15);
    uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
    if (row < rows && a.seq_lens[u.first + row / per] > 0) {
      const long at = ((long)(u.first + row / per) * a.n_q_heads + h * per + row % per) * D + c;
      if (f32) {
        const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + at);
        const float4 x = src[0], y = src[1];
        split_bf16x2(x.x, x.y, hi.x, lo.x);
        split_bf16x2(x.z, x.w, hi.y, lo.y);
        split_bf16x2(y.x, y.y, hi.z, lo.z);
        split_bf16x2(y.z, y.w, hi.w, lo.w);
      } else {
        hi = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + at);
      }
    }
    *reinterpret_cast<uint4 *>(sm + L::kt + kOpBytes + sw_off(row, c)) = hi;
    if (f32) *reinterpret_cast<uint4 *>(sm + L::kt + sw_off(row, c)) = lo;
  }
  fence_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // all 512 columns are this CTA's: the base is column 0 of lane 0
  constexpr uint32_t tmem = 0;

  if (warp < kSoftWarps) {
    // ---------------- softmax: set w takes halves w, w + 4, ...
    const int w = warp >> 2, quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const bool idle = 32 * quarter >= rows;  // no row of this warp is in use
    bool ok = true;
    if (w == 0) {
      // q_hat from tensor memory: a power of two puts the row's largest entry
      // in [2^13, 2^14), then hi + lo in fp16 for the scores' A operand
      ok = warp_wait(&q_mma, 0, err, &stop);
      if (ok && !idle) {
        tc_fence_after();
        float m = 0.f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld32(tmem + kColS + lanes + 32 * c, v);
          ld_wait();
          pin32(v);
#pragma unroll
          for (int e = 0; e < 32; e += 2) m = max3(m, fabsf(f(v[e])), fabsf(f(v[e + 1])));
        }
        int ex = 0;
        if (m > 0.f) frexpf(m, &ex);
        const float sc = m > 0.f ? ldexpf(1.f, 14 - ex) : 1.f;
        s_fq[row] = a.scale * kLog2e / sc;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32], hi[16], lo[16];
          tmem_ld32(tmem + kColS + lanes + 32 * c, v);
          ld_wait();
          pin32(v);
#pragma unroll
          for (int e = 0; e < 16; ++e) split_f16x2(f(v[2 * e]) * sc, f(v[2 * e + 1]) * sc, hi[e], lo[e]);
          tmem_st16(tmem + kColQ + lanes + 16 * c, hi);
          tmem_st16(tmem + kColQ + 64 + lanes + 16 * c, lo);
        }
        st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&q_ready));
    }
    ok = ok && warp_wait(&q_ready, 0, err, &stop);
    const float fq = ok && !idle ? s_fq[row] : 0.f;
    float l = 0.f, mine = 0.f;  // the sum, and the reference it is relative to
    for (int i = w; ok && i < n_half; i += kSets) {
      const int t = i >> 1, buf = i & (kBufs - 1);
      const uint32_t t_s = tmem + kColS + kHalf * buf + lanes;
      // the half's key norms and S.  (The norms have barriers of their own:
      // K~ of tile t + 2 may be complete before this set looks for tile t, and
      // a wait on k_full would then be a phase behind.)
      ok = warp_wait(&n_full[t % kNormBufs], (t / kNormBufs) & 1, err, &stop) &&
           warp_wait(&s_full[t & 1], (t >> 1) & 1, err, &stop);
      if (!ok || *(volatile int *)&stop) {
        ok = false;
        break;
      }
      if (!idle) {
        tc_fence_after();
        const float4 *kn = reinterpret_cast<const float4 *>(sm + L::norms) + (t % kNormBufs) * (kTcKeys / 4) + 16 * (i & 1);
        const int left = t1 - t0 - i * kHalf;  // keys of this half in the split
        // S is read from tensor memory again wherever it is used: 32 columns at a
        // time fit the registers that 26 warps leave
        auto load = [&](int c, uint32_t (&v)[32]) {
          tmem_ld32(t_s + 32 * c, v);
          ld_wait();
          pin32(v);
          if (left < kHalf) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e >= left) v[e] = 0xff800000u;
          }
        };
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t v[32];
          load(c, v);
#pragma unroll
          for (int e = 0; e < 32; e += 2) mx = max3(mx, f(v[e]), f(v[e + 1]));
        }
        const float *km = s_kmax[t % kNormBufs] + 4 * (i & 1);
        const float bound = fmaxf(mx, 0.f) * fmaxf(fmaxf(km[0], km[1]), fmaxf(km[2], km[3])) * fq;
        // the reference, handed over by the check of half i - 1
        float ref = -INFINITY;
        if (i > 0) {
          ok = warp_wait(&checked[quarter][(i - 1) % kSets], ((i - 1) / kSets) & 1, err, &stop);
          if (!ok) break;
          ref = s_ref[row];
        }
        // (a NaN bound takes the exact path too)
        if (__any_sync(0xffffffffu, !(bound <= ref + kLazy))) {
          mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t v[32];
            load(c, v);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 k4 = kn[8 * c + e / 4];
              const float2 x = mul2(make_float2(f(v[e]), f(v[e + 1])), make_float2(k4.x, k4.y));
              const float2 y = mul2(make_float2(f(v[e + 2]), f(v[e + 3])), make_float2(k4.z, k4.w));
              mx = max3(mx, x.x, x.y);
              mx = max3(mx, y.x, y.y);
            }
          }
          mx *= fq;
          if (i == 0) {
            ref = fmaxf(mx, -3.0e38f);
            s_ref[row] = ref;
          } else if (__any_sync(0xffffffffu, mx > ref + kLazy)) {
            // O is rescaled once the values of half i - 1 are in it
            ok = warp_wait(&pv_done[(i - 1) & (kBufs - 1)], ((i - 1) / kBufs) & 1, err, &stop);
            if (!ok) break;
            tc_fence_after();
            const float nref = fmaxf(ref, mx), al = fast_exp2(ref - nref);
            ref = nref;
            s_ref[row] = ref;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tmem_ld16w(tmem + kColO + lanes + 16 * c, o);
              ld_wait();
              pin16(o);
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const float2 z = mul2(make_float2(f(o[e]), f(o[e + 1])), make_float2(al, al));
                o[e] = __float_as_uint(z.x);
                o[e + 1] = __float_as_uint(z.y);
              }
              tmem_st16(tmem + kColO + lanes + 16 * c, o);
            }
            st_wait();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&checked[quarter][w]));
        if (i == w) mine = ref;  // this set's first half: its sum is empty
        l *= fast_exp2(mine - ref);
        mine = ref;
        const float2 f2 = make_float2(fq, fq), r2 = make_float2(-ref, -ref);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t v[32], p[16];
          load(c, v);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 k4 = kn[8 * c + e / 4];
            const float2 x = fma2(mul2(make_float2(f(v[e]), f(v[e + 1])), make_float2(k4.x, k4.y)), f2, r2);
            const float2 y = fma2(mul2(make_float2(f(v[e + 2]), f(v[e + 3])), make_float2(k4.z, k4.w)), f2, r2);
            const float2 px = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            const float2 py = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            sum = add2(sum, add2(px, py));
            p[e / 2] = pack_half2(px.x, px.y);
            p[e / 2 + 1] = pack_half2(py.x, py.y);
          }
          // P of chunk c lies over columns 16 c .. 16 c + 15 of S, which are read
          tmem_st16(t_s + 16 * c, p);
        }
        l += sum.x + sum.y;
        st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&p_full[buf]));
    }
    // ---------------- the split's partial: r, l and O of every row in use
    // (a barrier of its own: this set may be two phases of v_empty behind)
    ok = ok && warp_wait(&fin, 0, err, &stop);
    s_l[w][row] = l;
    s_lref[w][row] = mine;
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftWarps) : "memory");
    // O leaves in the V fragment order, through shared memory (every MMA has
    // completed and the copies are consumed: the operands' place is free)
    float *so = reinterpret_cast<float *>(sm);  // [128][kPad]
    constexpr int kPad = D + 1;
    if (ok && !idle) {
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t o[16];
        tmem_ld16w(tmem + kColO + lanes + 32 * w + 16 * c, o);
        ld_wait();
        pin16(o);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          so[row * kPad + a.p.kvperm[32 * w + 16 * c + e]] = f(o[e]) * (1.f / kVScale);
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftWarps) : "memory");
    if (ok) {
      for (int i = warp; i < rows; i += kSoftWarps) {  // a warp per row
        const long out_row = (long)(u.first + i / per) * a.n_q_heads + h * per + i % per;
        float *dst = a.partials + (out_row * a.n_slots + split) * (D + 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) dst[4 + 32 * c + lane] = so[i * kPad + 32 * c + lane];
        if (lane == 0) {
          const float ref = s_ref[i];
          dst[0] = ref;
          float l_all = 0.f;
          for (int e = 0; e < min(kSets, n_half); ++e) l_all = fmaf(s_l[e][i], fast_exp2(s_lref[e][i] - ref), l_all);
          dst[1] = l_all;
        }
      }
    }
  } else if (warp < kProdWarp) {
    // ---------------- expansion: keys 16 ew .. 16 ew + 15 of every tile, K~ one
    // tile ahead of V~ (the scores of a tile are needed that much sooner)
    const int ew = warp - kExpWarp0, r = lane >> 2, q = lane & 3;
    const Lut lk = fp16_lut<BK>(a.p.cb), lv = fp16_lut<BV>(a.p.cb + 2 * kMaxLevels, kVScale);
    bool ok = true;
    for (int j = 0; ok && j <= n_tiles; ++j) {
      if (j < n_tiles) {
        const int b = j & 1;
        ok = warp_wait(&full[j % kStagesTc], (j / kStagesTc) & 1, err, &stop);
        // the q rotation's operands: lo in K~ 0 (fp32 q), hi and Pi in the buffers of tile 1
        if (ok && ((j == 0 && f32) || j == 1)) ok = warp_wait(&q_mma, 0, err, &stop);
        if (ok && j >= 2) ok = warp_wait(&k_empty[b], ((j >> 1) - 1) & 1, err, &stop);
        if (!ok || *(volatile int *)&stop) break;
        const unsigned char *st = sm + L::ring + (j % kStagesTc) * L::stage;
        // the key norms; past the split's end 1, so that a masked score stays -inf
        const int key = 16 * ew + (lane & 15);
        float n = __half2float(reinterpret_cast<const __half *>(st + St::kn)[key]);
        if (key >= t1 - t0 - j * kTcKeys) n = 1.f;
        if (lane < 16) reinterpret_cast<float *>(sm + L::norms)[(j % kNormBufs) * kTcKeys + key] = n;
        expand_rows16<BK>(st + St::kc, sm + L::kt + b * kOpBytes, lk, 16 * ew, r, q);
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&k_full[b]));
#pragma unroll
        for (int o = 8; o; o >>= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
        if (lane == 0) s_kmax[j % kNormBufs][ew] = n;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&n_full[j % kNormBufs]));
      }
      if (j >= 1) {
        const int t = j - 1, b = t & 1;
        if (t >= 2) ok = warp_wait(&v_empty[b], ((t >> 1) - 1) & 1, err, &stop);
        if (!ok) break;
        const unsigned char *st = sm + L::ring + (t % kStagesTc) * L::stage;
        expand_rows16<BV, true>(st + St::vc, sm + L::vt + b * kOpBytes, lv, 16 * ew, r, q,
                                reinterpret_cast<const __half *>(st + St::vn), t1 - t0 - t * kTcKeys);
        fence_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&v_full[b]));
          mbar_arrive(smem_u32(&empty[t % kStagesTc]));
        }
      }
    }
  } else {
    if (warp == kProdWarp && lane == 0) {
      // ---------------- producer
      int issued = 0;
      for (int j = 0; j < n_tiles; ++j) {
        const int slot = j % kStagesTc;
        if (j >= kStagesTc && !wait_or_stop(&empty[slot], ((j / kStagesTc) - 1) & 1, err, &stop)) break;
        if (*(volatile int *)&stop) break;
        unsigned char *st = sm + L::ring + slot * L::stage;
        const uint32_t bar = smem_u32(&full[slot]);
        const int first = t0 + j * kTcKeys;
        // up to the split's end rounded up to 64 positions (the capacity is a multiple of 64)
        const uint32_t n = (uint32_t)min(kTcKeys, (t1 - first + 63) & ~63);
        mbar_arrive_expect_tx(bar, n * (D * BK / 8 + D * BV / 8 + 4));
        for (uint32_t done = 0; done < n;) {
          long tok;
          uint32_t run = n - done;
          if (a.c.block_table) {
            const int p = first + (int)done, jb = p / a.c.block_size, off = p - jb * a.c.block_size;
            run = min(run, (uint32_t)(a.c.block_size - off));
            int bl = a.c.block_table[(long)u.lead * (a.c.capacity / a.c.block_size) + jb];
            if (bl < 0 || bl >= a.c.n_blocks) {  // flagged; a valid block is read in its place
              atomicOr(err, kErrTokenRange);
              bl = 0;
            }
            tok = ((long)bl * a.c.n_kv_heads + h) * a.c.block_size + off;
          } else {
            tok = ((long)u.lead * a.c.n_kv_heads + h) * a.c.capacity + first + done;
          }
          bulk_g2s(smem_u32(st + St::kc + done * (D * BK / 8)), a.c.codes_k + tok * (D * BK / 8), run * (D * BK / 8), bar);
          bulk_g2s(smem_u32(st + St::vc + done * (D * BV / 8)), a.c.codes_v + tok * (D * BV / 8), run * (D * BV / 8), bar);
          bulk_g2s(smem_u32(st + St::kn + done * 2), a.c.norm_k + tok, run * 2, bar);
          bulk_g2s(smem_u32(st + St::vn + done * 2), a.c.norm_v + tok, run * 2, bar);
          done += run;
        }
        issued = j + 1;
      }
      if (*(volatile int *)&stop) {  // never leave copies in flight
        for (int j = max(0, issued - kStagesTc); j < issued; ++j)
          mbar_wait(smem_u32(&full[j % kStagesTc]), (j / kStagesTc) & 1);
      }
    } else if (warp == kMmaWarp) {
      // ---------------- MMA issuer (the whole warp; one lane issues)
      if (elect_one()) {
        const uint32_t hi = smem_u32(sm + L::kt + kOpBytes), lo = smem_u32(sm + L::kt);
        const uint32_t pi = smem_u32(sm + L::vt + kOpBytes);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * kOpBox + (kk & 3) * 32;
          mma_ss(tmem + kColS, sw128_desc(hi + off), sw128_desc(pi + off), kDescQ, kk > 0);
          if (f32) mma_ss(tmem + kColS, sw128_desc(lo + off), sw128_desc(pi + off), kDescQ, 1);
        }
        tc_commit(smem_u32(&q_mma));
      }
      bool ok = warp_wait(&q_ready, 0, err, &stop);
      // O += P V of the two halves of tile t, then S of tile t + 2 over the P
      // just read (MMAs of one thread run in order); the first two S go ahead.
      // (S in halves of 64 keys is no cheaper: with A in tensor memory an MMA
      // takes about 75 cycles at N = 64 and at N = 128.)
      for (int t = -2; ok && t < n_tiles; ++t) {
        for (int i = 2 * t; t >= 0 && i < min(2 * t + 2, n_half); ++i) {
          const int buf = i & (kBufs - 1);
          ok = warp_wait(&v_full[t & 1], (t >> 1) & 1, err, &stop) &&
               warp_wait(&p_full[buf], (i / kBufs) & 1, err, &stop);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t v = mn_desc(smem_u32(sm + L::vt + (t & 1) * kOpBytes + (i & 1) * (kHalf * 128)), kOpBox);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // (16 keys: 2048 bytes)
              mma_ts(tmem + kColO, tmem + kColS + kHalf * buf + 8 * kk, v + kk * (2048 >> 4), kDescO,
                     (i > 0 || kk > 0) ? 1u : 0u);
            tc_commit(smem_u32(&pv_done[buf]));
            if ((i & 1) || i + 1 == n_half) tc_commit(smem_u32(&v_empty[t & 1]));
          }
          __syncwarp();
        }
        const int n = t + 2;
        if (ok && n < n_tiles) {
          ok = warp_wait(&k_full[n & 1], (n >> 1) & 1, err, &stop);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t k = sw128_desc(smem_u32(sm + L::kt + (n & 1) * kOpBytes));
            const uint32_t d = tmem + kColS + 128 * (n & 1);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = ((kk >> 2) * kOpBox + (kk & 3) * 32) >> 4;
              mma_ts(d, tmem + kColQ + 8 * kk, k + off, kDescS, kk > 0);
              mma_ts(d, tmem + kColQ + 64 + 8 * kk, k + off, kDescS, 1);
            }
            tc_commit(smem_u32(&s_full[n & 1]));
            tc_commit(smem_u32(&k_empty[n & 1]));
          }
          __syncwarp();
        }
        if (__shfl_sync(0xffffffffu, *(volatile int *)&stop, 0)) break;
      }
      // every MMA issued here has completed before the tensor memory is released
      if (elect_one()) tc_commit(smem_u32(&fin));
      __syncwarp();
      mbar_wait(smem_u32(&fin), 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_slot), "r"(512u) : "memory");
  }
}

using Fn = void (*)(const SharedTcArgs);

template <int BK, int BV>
int configure_and_launch(const SharedTcArgs &a, cudaLaunchConfig_t &cfg) {
  static std::atomic<bool> configured[kMaxDevices];
  std::atomic<bool> &done = configured[current_device()];
  if (!done.load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(shared_prefix_tc_kernel<BK, BV>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, SharedTc<BK, BV>::bytes);
    if (e != cudaSuccess) return (int)e;
    done.store(true, std::memory_order_release);
  }
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = SharedTc<BK, BV>::bytes;
  return (int)cudaLaunchKernelEx(&cfg, shared_prefix_tc_kernel<BK, BV>, a);
}

template <int BK>
int launch_v(const SharedTcArgs &a, cudaLaunchConfig_t &cfg) {
  return a.p.bits_v == 2   ? configure_and_launch<BK, 2>(a, cfg)
         : a.p.bits_v == 3 ? configure_and_launch<BK, 3>(a, cfg)
                           : configure_and_launch<BK, 4>(a, cfg);
}

}  // namespace

int launch_shared_prefix_tc(const SharedTcArgs &a, cudaLaunchConfig_t &cfg) {
  return a.p.bits_k == 2 ? launch_v<2>(a, cfg) : a.p.bits_k == 3 ? launch_v<3>(a, cfg) : launch_v<4>(a, cfg);
}

}  // namespace tq
