// What the block join's translation units share: the arguments of a launch
// and the launchers.
#pragma once

#include "zero_rows.cuh"

namespace zero {

// Column sums of the backward pass over its rows (see zero_join_rows.cuh):
// sum dn oh, sum dn, sum y go v, sum y go.
enum JoinSum { kSumP = 0, kSumQ, kSumS, kSumB, kJoinSums };

constexpr int kJoinRowMost = 8192;         // channels of the kernels that hold rows in registers, at most
constexpr int kJoinNarrow = 4096;          // rows above it: 16 columns a thread, rms
constexpr int kJoinNarrowLayer = 2047;     // and layer norms forward
constexpr int kJoinThreadsForward = 1024;  // threads of an SM's CTAs there
constexpr int kJoinThreadsBackward = 768;

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
  void* dgate;         // row and full gates (a channel gate's comes from the sums)
  float* partial;      // [workers][n_sums][hidden]
  int32_t slot[kJoinSums];  // place among the partials, -1: not wanted
  int32_t n_sums;
  int32_t layer;       // mean subtracted
  float eps, scale, inv_h;
};

// The parameter gradients from the workers' partials.
struct JoinSumArgs {
  JoinArgs a;
  int32_t workers;
  void *dw_pre, *dbias_pre, *dw_post, *dbias_post, *dgate;  // dgate: channel gates only
};

// Kernels for rows of up to kJoinRowMost channels; -1: the rows are longer, or
// do not fit into shared memory.
// *workers: CTAs launched, each leaving its partials.
template <class A, class R>
int launch_join_rows(const JoinArgs& a, bool backward, int* workers, cudaStream_t s);

}  // namespace zero
