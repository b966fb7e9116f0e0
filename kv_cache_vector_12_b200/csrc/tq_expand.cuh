// Expansion of packed codes into the shared-memory operands of the tcgen05
// attention kernels (prefill over the packed cache, shared prefixes), d = 128:
// 128-byte-swizzled K-major 128 x 128 fp16 tiles.  Internal to the library.
#pragma once

#include "tq_stream.cuh"

namespace tq {
namespace {

constexpr int kTcKeys = 128;                  // keys per tile
constexpr int kOpBytes = 128 * kHeadDim * 2;  // one 128 x 128 16-bit operand: two 128 x 64 swizzled boxes
constexpr int kOpBox = kOpBytes / 2;

// Byte offset of element (row, col) of a 128 x 128 16-bit operand stored as
// two boxes of 128 rows x 64 columns, 128-byte rows, 16-byte chunks swizzled
// by the row within each 8-row (1024-byte) atom.
__device__ __forceinline__ uint32_t sw_off(int row, int col) {
  const int box = col >> 6, cc = col & 63;
  return (uint32_t)(box * kOpBox + row * 128 + ((((cc >> 3) ^ (row & 7)) & 7) << 4) + ((cc & 7) << 1));
}

// fp16 pairs (codes 0, 1) and (codes 2, 3) of one lookup's low and high bytes.
__device__ __forceinline__ void f16_pairs(uint32_t lo, uint32_t hi, uint32_t &p01, uint32_t &p23) {
  p01 = prmt(lo, hi, 0x5140u);
  p23 = prmt(lo, hi, 0x7362u);
}

// X~[key][kappa] of keys kb .. kb + 15 of a tile (the table's entries of B-bit
// codes, rows of D B / 8 bytes from `codes`, K fragment order) into xt, by one
// warp (r = lane / 4, q = lane % 4).  SCALED: times the keys' norms, rounded to
// fp16 once; keys at or past `left` become 0, whatever their norms hold.
template <int B, bool SCALED = false>
__device__ __forceinline__ void expand_rows16(const unsigned char *codes, unsigned char *xt, const Lut &lut, int kb,
                                              int r, int q, const __half *norms = nullptr, int left = kTcKeys) {
  // rows 0 2 4 6 1 3 5 7 by r: the four rows of a half-warp's 8-byte stores then
  // fall on different pairs of swizzled 16-byte chunks (in natural order two
  // and two share a pair, which halves the store rate)
  const int k0 = kb + (((r << 1) & 6) | (r >> 2)), k1 = k0 + 8;
  uint32_t wk0[B], wk1[B];
  const unsigned char *kr0 = codes + k0 * (D * B / 8) + q * 4 * B;
  const unsigned char *kr1 = codes + k1 * (D * B / 8) + q * 4 * B;
#pragma unroll
  for (int i = 0; i < B; ++i) {
    wk0[i] = reinterpret_cast<const uint32_t *>(kr0)[i];
    wk1[i] = reinterpret_cast<const uint32_t *>(kr1)[i];
  }
  __half2 n0, n1;
  if constexpr (SCALED) {
    const __half z = __ushort_as_half(0);
    n0 = __half2half2(k0 < left ? norms[k0] : z);
    n1 = __half2half2(k1 < left ? norms[k1] : z);
  }
  auto put = [&](int key, int kap, uint32_t sel, __half2 n) {
    uint32_t lo, hi, p01, p23;
    lookup<B>(lut, sel, lo, hi);
    f16_pairs(lo, hi, p01, p23);
    if constexpr (SCALED) {
      auto times = [&](uint32_t x) {
        const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&x), n);
        return *reinterpret_cast<const uint32_t *>(&y);
      };
      p01 = times(p01), p23 = times(p23);
    }
    *reinterpret_cast<uint2 *>(xt + sw_off(key, kap)) = make_uint2(p01, p23);
  };
#pragma unroll
  for (int sg = 0; sg < 8; ++sg) {
    const int kap = 32 * (sg >> 1) + 16 * (sg & 1) + 4 * q;
    put(k0, kap, k_selector<B>(wk0, sg), n0);
    put(k1, kap, k_selector<B>(wk1, sg), n1);
  }
}

// V~^T[kappa_v][key] of keys kb .. kb + 15 (fp16 V centroids, V fragment
// order) into vt.
template <int BK, int BV>
__device__ __forceinline__ void expand_values16(const unsigned char *st, unsigned char *vt, const Lut &lv, int kb,
                                                int r, int q) {
  using St = Stage<BK, BV, false, kTcKeys>;
  // V~^T: rows in the V fragment order, keys as columns (decode's A
  // fragments: a0 = row 16 mt + r, keys 2q, 2q+1; a1 = row + 8; a2, a3:
  // keys + 8)
  constexpr int VB = D * BV / 8;
  const unsigned char *vc = st + St::vc + (kb + 2 * q) * VB;
  auto put = [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
    *reinterpret_cast<uint32_t *>(vt + sw_off(16 * mt + r, kb + 2 * q)) = a0;
    *reinterpret_cast<uint32_t *>(vt + sw_off(16 * mt + r + 8, kb + 2 * q)) = a1;
    *reinterpret_cast<uint32_t *>(vt + sw_off(16 * mt + r, kb + 8 + 2 * q)) = a2;
    *reinterpret_cast<uint32_t *>(vt + sw_off(16 * mt + r + 8, kb + 8 + 2 * q)) = a3;
  };
  if constexpr (BV == 3) {
    const int gofs = 12 * (r >> 1);
    const uint32_t gs = (r & 1) ? 0x7362u : 0x5140u;
    uint32_t ya[3], yb[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      ya[k] = prmt(reinterpret_cast<const uint32_t *>(vc + gofs)[k],
                   reinterpret_cast<const uint32_t *>(vc + VB + gofs)[k], gs);
      yb[k] = prmt(reinterpret_cast<const uint32_t *>(vc + 8 * VB + gofs)[k],
                   reinterpret_cast<const uint32_t *>(vc + 9 * VB + gofs)[k], gs);
    }
    const uint32_t spa = spare3(ya[0], ya[1], ya[2]), spb = spare3(yb[0], yb[1], yb[2]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t za = k < 3 ? (ya[k < 3 ? k : 0] & 0x77777777u) : spa;
      const uint32_t zb = k < 3 ? (yb[k < 3 ? k : 0] & 0x77777777u) : spb;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t a0, a1, a2, a3;
        v_pairs<3>(lv, hh ? za >> 16 : za, a0, a1);
        v_pairs<3>(lv, hh ? zb >> 16 : zb, a2, a3);
        put(2 * k + hh, a0, a1, a2, a3);
      }
    }
  } else if constexpr (BV == 2) {
    const uint32_t A0 = reinterpret_cast<const uint32_t *>(vc)[r];
    const uint32_t B0 = reinterpret_cast<const uint32_t *>(vc + VB)[r];
    const uint32_t A1 = reinterpret_cast<const uint32_t *>(vc + 8 * VB)[r];
    const uint32_t B1 = reinterpret_cast<const uint32_t *>(vc + 9 * VB)[r];
#pragma unroll
    for (int yh = 0; yh < 2; ++yh) {
      const uint32_t gs = yh ? 0x7362u : 0x5140u;
      const uint32_t ya = prmt(A0, B0, gs), yb = prmt(A1, B1, gs);
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        const uint32_t za = (ya >> (2 * par)) & 0x33333333u, zb = (yb >> (2 * par)) & 0x33333333u;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t a0, a1, a2, a3;
          v_pairs<2>(lv, hh ? za >> 16 : za, a0, a1);
          v_pairs<2>(lv, hh ? zb >> 16 : zb, a2, a3);
          put(4 * yh + 2 * par + hh, a0, a1, a2, a3);
        }
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t A0 = reinterpret_cast<const uint32_t *>(vc)[2 * r + u];
      const uint32_t B0 = reinterpret_cast<const uint32_t *>(vc + VB)[2 * r + u];
      const uint32_t A1 = reinterpret_cast<const uint32_t *>(vc + 8 * VB)[2 * r + u];
      const uint32_t B1 = reinterpret_cast<const uint32_t *>(vc + 9 * VB)[2 * r + u];
#pragma unroll
      for (int yh = 0; yh < 2; ++yh) {
        const uint32_t gs = yh ? 0x7362u : 0x5140u;
        const uint32_t ya = prmt(A0, B0, gs), yb = prmt(A1, B1, gs);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t a0, a1, a2, a3;
          v_pairs<4>(lv, hh ? ya >> 16 : ya, a0, a1);
          v_pairs<4>(lv, hh ? yb >> 16 : yb, a2, a3);
          put(4 * u + 2 * yh + hh, a0, a1, a2, a3);
        }
      }
    }
  }
}

// K~ and V~^T of the 32 keys of warp ew (0-3).
template <int BK, int BV>
__device__ __forceinline__ void expand_keys(const unsigned char *st, unsigned char *kt, const Lut &lkf, int ew, int r,
                                            int q) {
#pragma unroll
  for (int rb = 0; rb < 2; ++rb)
    expand_rows16<BK>(st + Stage<BK, BV, false, kTcKeys>::kc, kt, lkf, 32 * ew + 16 * rb, r, q);
}
template <int BK, int BV>
__device__ __forceinline__ void expand_values(const unsigned char *st, unsigned char *vt, const Lut &lv, int ew, int r,
                                              int q) {
#pragma unroll
  for (int rb = 0; rb < 2; ++rb) expand_values16<BK, BV>(st, vt, lv, 32 * ew + 16 * rb, r, q);
}

// 2^BITS centroids times `scale` as fp16 byte tables (exact for a power of two
// that stays in range: the centroids are fp16 values).
template <int BITS>
__device__ __forceinline__ Lut fp16_lut(const float *cb, float scale = 1.f) {
  Lut t;
#pragma unroll
  for (int i = 0; i < 4; ++i) t.lo[i] = t.hi[i] = 0u;
#pragma unroll
  for (int e = 0; e < (1 << BITS); ++e) {
    const uint16_t hb = __half_as_ushort(__float2half_rn(cb[e] * scale));
    t.lo[e / 4] |= (uint32_t)(hb & 0xff) << (8 * (e % 4));
    t.hi[e / 4] |= (uint32_t)(hb >> 8) << (8 * (e % 4));
  }
  return t;
}

}  // namespace
}  // namespace tq
