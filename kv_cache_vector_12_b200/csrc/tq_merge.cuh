// Pieces of the split merges (device side): the maximum over a block of 128
// threads, a bf16 row of Pi^T times a vector in shared memory, and vector
// loads of the split partials.  Internal to the library.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace tq {
namespace {

__device__ __forceinline__ float block_max128(float v, float *red) {
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const float r = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  __syncthreads();
  return r;
}

// A bf16 row of DH entries (16-byte aligned): held in registers as
// independent 16-byte loads (DH <= 128, loaded ahead of use) or read on the
// fly (DH = 256).
template <int DH>
struct Bf16Row {
  static constexpr int kHeld = DH <= 128 ? DH / 8 : 1;
  uint4 w[kHeld];
  const uint16_t *row;
  __device__ __forceinline__ void load(const uint16_t *r) {
    row = r;
    if constexpr (DH <= 128) {
#pragma unroll
      for (int c = 0; c < DH / 8; ++c) w[c] = reinterpret_cast<const uint4 *>(r)[c];
    }
  }
  __device__ __forceinline__ uint4 get(int c) const {
    if constexpr (DH <= 128) return w[c];
    else return reinterpret_cast<const uint4 *>(row)[c];
  }
};

// Dot product of a bf16 row with a vector in shared memory, four partial sums.
template <int DH>
__device__ __forceinline__ float dot_bf16_row(const Bf16Row<DH> &w, const float *x) {
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < DH / 8; ++c) {
    const uint4 v = w.get(c);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = 8 * c + 2 * e;
      acc[e] = fmaf(__uint_as_float(u[e] << 16), x[j], acc[e]);
      acc[e] = fmaf(__uint_as_float(u[e] & 0xffff0000u), x[j + 1], acc[e]);
    }
  }
  return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// PL consecutive floats (PL * 4-byte aligned) as vector loads.
template <int PL>
__device__ __forceinline__ void load_floats(const float *src, float (&v)[PL]) {
  if constexpr (PL == 2) {
    const float2 x = *reinterpret_cast<const float2 *>(src);
    v[0] = x.x, v[1] = x.y;
  } else {
#pragma unroll
    for (int c = 0; c < PL / 4; ++c) {
      const float4 x = reinterpret_cast<const float4 *>(src)[c];
      v[4 * c] = x.x, v[4 * c + 1] = x.y, v[4 * c + 2] = x.z, v[4 * c + 3] = x.w;
    }
  }
}

}  // namespace
}  // namespace tq
