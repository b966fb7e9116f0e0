// The tcgen05 prefix pass of shared-prefix decode attention (tq_shared_tc.cu).
#pragma once

#include <cuda_runtime.h>

#include "tq_internal.h"

namespace tq {

struct SharedTcArgs {
  DeviceParams p;
  tq_cache c;
  int n_q_heads;
  const void *q;  // [n_seqs][n_q_heads][d], fp32 or bf16 (q_dtype)
  int q_dtype;
  float scale;
  const int32_t *seq_lens, *cu_group, *prefix;
  int n_groups, max_group, max_prefix;
  int members;       // sequences per CTA: 128 / (query heads per KV head)
  int chunk;         // positions per split, a multiple of 128
  float *partials;   // [rows][n_slots][d + 4], this pass's splits first
  int n_slots;
  unsigned long long token;  // of the call, for the pass beside this one (tq_groups.cuh)
};

// Launches on cfg's stream and grid; returns a cudaError_t as int.
int launch_shared_prefix_tc(const SharedTcArgs &a, cudaLaunchConfig_t &cfg);

}  // namespace tq
