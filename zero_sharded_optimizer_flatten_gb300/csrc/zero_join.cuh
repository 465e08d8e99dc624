// What the block join's translation units share: the arguments of a launch
// and the launchers.
#pragma once

#include "zero_rows.cuh"

namespace zero {

// Column sums of the backward pass (gradients of the parameters).
enum JoinSum { kSumWPre = 0, kSumBiasPre, kSumWPost, kSumBiasPost, kSumGate, kJoinSums };

struct JoinArgs {
  zero_join_desc d;
  zero_join_inputs in;
  void* o;
  void* n;
  const void* d_o;
  const void* d_n;
  float4* stats;       // per row: mean and 1/deviation of b, then of o
  void* dx;
  void* db;
  void* dgate;         // row and full gates (a channel gate's goes through sums)
  float* partial;      // [workers][n_sums][hidden]
  int32_t slot[kJoinSums];  // place among the partials, -1: not wanted
  int32_t n_sums;
  int32_t layer;       // mean subtracted
  float eps, scale, inv_h;
};

// The parameter gradients from the workers' partials.
struct JoinSumArgs {
  const float* partial;
  int64_t hidden;
  int32_t workers, n_sums;
  void* out[kJoinSums];     // by slot
  int32_t type[kJoinSums];  // by slot
};

int launch_join(const JoinArgs& a, cudaStream_t s);
// workers: CTAs that leave partials (join_workers of the same arguments).
int launch_join_backward(const JoinArgs& a, int workers, cudaStream_t s);
int join_workers(const JoinArgs& a);

}  // namespace zero
