// The router of sparse experts: probabilities, choices, counts and the losses
// that keep the experts in balance, and the gradient. Argument checks, kernels,
// launches.
//
//   p = softmax(z) over the experts, lse = log sum exp z
//   choices: the topk largest z of a token, of equal ones the lowest expert
//     first; -inf is never chosen (id -1, weight 0)
//   weights: p of the choices, or those divided by their sum (normalize)
//   counts_e: how often expert e was chosen; n: tokens with any z above -inf
//   balance = E / (topk n^2) sum_e counts_e sum_t p_te,  zloss = sum_t lse_t^2 / n
//   dz_te = p_te (a_te - sum_f p_tf a_tf) + 2 d_zloss / n lse_t p_te (+ what the
//     normalised weights add), a_te = d_balance E counts_e / (topk n^2), plus
//     dweights of the choices
//
// A warp has a token, each lane VPT neighbouring experts in registers; the
// choices come one after the other as the warp's largest value. What bounds
// large calls is issue slots (see k_route). Each CTA leaves its counts and sums
// of p in the workspace, added up in order by k_route_finish, so the same call
// gives the same bits; a call that one CTA does has no second launch.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <inttypes.h>

#include <algorithm>
#include <cfloat>

#include "zero_capi_util.h"
#include "zero_rows.cuh"
#include "zero_tensor_core.cuh"

namespace cg = cooperative_groups;

namespace zero {
namespace {

constexpr int kExpertsMost = 1024, kTopkMost = 32;
constexpr int kThreads = 1024;
constexpr int kCtasMost = kSMs;
constexpr int kFinishCtas = 8;  // of the finishing cluster
// Warps of a CTA: 16 experts a lane and more take more registers.
constexpr int warps_of(int vpt) { return vpt <= 8 ? 32 : 16; }
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct RouteArgs {
  const void* z;
  int64_t tokens, stride;
  int32_t experts, topk, normalize, vec;
  int32_t* ids;
  float* weights;
  int32_t* counts;
  float* losses;
  float* stats;      // [tokens + 1]: lse, n
  // [CTAs][experts] each, then [CTAs][2]: n and the sum of lse^2
  int32_t* part_counts;
  float* part_sums;
  float* part_ends;
  int32_t ctas;
  // gradient
  const float *d_weights, *d_losses;
  void* dz;
};

// Of sums of at least 1: within one place in the last; the logarithm within 2^-22
// of itself (absolutely only below 2), up to 1.7e-6 of 1024 experts' lse, where
// it goes into lse and the z loss alone. (logf: 43.1 us in place of 41.1 for 65536 x
// 256.)
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// exp(z - top), 0 for -inf.  The difference comes first: top * log2(e) rounded
// beforehand would leave up to 2^-24 of its size in every exponent, all of p for
// rows around -1e9, and infinities for rows at the type's end.  In pairs it costs
// what one multiplication and addition of single values did.
__device__ __forceinline__ float exp_from(float z, float top) { return tc::exp2_of((z - top) * kLog2e); }
template <int VPT>
__device__ __forceinline__ void exp_from(float (&z)[VPT], float top) {
  if constexpr (VPT == 1) {
    z[0] = exp_from(z[0], top);
  } else {
    const F2 minus = f2(-top), by = f2(kLog2e);
#pragma unroll
    for (int j = 0; j < VPT; j += 2) {
      f2_out(mul2(add2(f2(z[j], z[j + 1]), minus), by), z[j], z[j + 1]);
      z[j] = tc::exp2_of(z[j]), z[j + 1] = tc::exp2_of(z[j + 1]);
    }
  }
}
__device__ __forceinline__ float log2_of(float v) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Two sums over the warp, side by side.
__device__ __forceinline__ void sum_both(float& a, float& b) {
  F2 v = f2(a, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    f2_out(v, a, b);
    v = add2(v, f2(__shfl_xor_sync(kFull, a, o), __shfl_xor_sync(kFull, b, o)));
  }
  f2_out(v, a, b);
}

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// A lane's VPT values of a row, `fill` past its end.
template <class T, int VPT>
__device__ __forceinline__ void load_row(const T* row, int lane, int experts, bool vec, float fill, float (&v)[VPT]) {
  if constexpr (VPT * sizeof(T) >= 32) {
    if (vec) {  // 32 bytes a load: by 16 a warp touches every line twice
      constexpr int kLoads = VPT * sizeof(T) / 32, kEach = 32 / sizeof(T);
      uint32_t w[kLoads][8];
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3]), "=r"(w[i][4]), "=r"(w[i][5]),
                       "=r"(w[i][6]), "=r"(w[i][7])
                     : "l"(row + lane * VPT + i * kEach));
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if constexpr (sizeof(T) == 4)
            v[i * kEach + j] = __uint_as_float(w[i][j]);
          else
            Elem<T>::unpack(w[i][j], v[i * kEach + 2 * j], v[i * kEach + 2 * j + 1]);
      return;
    }
  } else if constexpr (VPT * sizeof(T) == 16) {
    if (vec) {
      constexpr int kWords = VPT * sizeof(T) / 16, kEach = 16 / sizeof(T);
      uint4 w[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(row + lane * VPT)[i];
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if constexpr (sizeof(T) == 4)
            v[i * kEach + j] = __uint_as_float(x[j]);
          else
            Elem<T>::unpack(x[j], v[i * kEach + 2 * j], v[i * kEach + 2 * j + 1]);
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    v[j] = lane * VPT + j < experts ? Elem<T>::widen(row[lane * VPT + j]) : fill;
}

// The results that need all tokens, from the experts' counts and sums of p (of
// thread e, up to the CTA's size at a time) and the tokens' n and sum of lse^2.
struct Totals {
  float product = 0.f;
  __device__ __forceinline__ void expert(const RouteArgs& a, int e, int count, float sum) {
    a.counts[e] = count;
    product = fmaf(static_cast<float>(count), sum, product);
  }
  // every thread of the CTA; part: a float a warp
  __device__ __forceinline__ void finish(const RouteArgs& a, float n, float squares, float* part) {
    const float s = warp_all_sum(product);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      float all = 0.f;
      for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) all += part[w];
      const float by = fmaxf(n, 1.f);
      a.losses[0] = all * (static_cast<float>(a.experts) / static_cast<float>(a.topk)) / by / by;
      a.losses[1] = squares / by;
      a.stats[a.tokens] = n;
    }
  }
};

// A token's choices. The K-th largest different lane maximum is a bound that at
// least K values reach (a redux a round); the few that do are put side by side,
// a lane each, and every one finds its rank by comparing itself with all of
// them. Where more than a warp of them reach it (many equal values), they are
// taken one after the other instead: the warp's largest value, the first lane
// that holds it and there the first place. NaN counts as +inf.
//
// Measured, 65536 tokens, 8 of 256 fp32 (67 MB): 38-40 us (498
// instructions a token); one after the other always 53, by integer keys 74.
template <class T, int VPT>
__global__ void __launch_bounds__(32 * warps_of(VPT), 1) k_route(const RouteArgs a) {
  constexpr int kWarps = warps_of(VPT);
  extern __shared__ int smem[];  // [experts] counts, [kWarps][experts] sums of p
  __shared__ float ends[kWarps][2], part[kWarps];
  __shared__ __align__(16) float2 candidates[kWarps][32];
  let_next_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.experts, K = a.topk;
  float* sums = reinterpret_cast<float*>(smem + E);
  for (int e = threadIdx.x; e < E; e += 32 * kWarps) smem[e] = 0;
  __syncthreads();
  float total[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) total[j] = 0.f;
  float n = 0.f, squares = 0.f;
  const T* z = static_cast<const T*>(a.z);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.tokens; t += step) {
    float v[VPT];
    load_row<T, VPT>(z + t * a.stride, lane, E, a.vec, -INFINITY, v);
    float most = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      v[j] = fminf(v[j], INFINITY);  // NaN to +inf
      most = fmaxf(most, v[j]);
    }
    float bound = warp_max(most), x = most;
    const bool any = bound > -INFINITY;
    const float top = any ? bound : 0.f;
#pragma unroll 4
    for (int k = 1; k < K; ++k) {
      x = x == bound ? -INFINITY : x;
      bound = warp_max(x);
    }
    // choice `slot` of the token, of this lane
    float chosen_z = -INFINITY;
    int chosen = -1, slot = lane;
    unsigned reach[VPT];
    int count = 0;
    bound = fmaxf(bound, -FLT_MAX);  // -inf is not a choice
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      reach[j] = __ballot_sync(kFull, v[j] >= bound);
      count += __popc(reach[j]);
    }
    if (count <= 32) {
      int at = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (reach[j] >> lane & 1)
          candidates[warp][at + __popc(reach[j] & ((1u << lane) - 1))] = make_float2(v[j], __int_as_float(lane * VPT + j));
        at += __popc(reach[j]);
      }
      // up to a whole four of them, -inf after the last
      if (lane >= count && lane < (count + 3) / 4 * 4) candidates[warp][lane] = make_float2(-INFINITY, 0.f);
      __syncwarp();
      const float2 own = candidates[warp][lane];
      const int e = __float_as_int(own.y);
      int rank = 0;
      for (int c = 0; c < count; c += 4) {
        const float4 p = *reinterpret_cast<const float4*>(&candidates[warp][c]);
        const float4 q = *reinterpret_cast<const float4*>(&candidates[warp][c + 2]);
        rank += p.x > own.x || (p.x == own.x && __float_as_int(p.y) < e);
        rank += p.z > own.x || (p.z == own.x && __float_as_int(p.w) < e);
        rank += q.x > own.x || (q.x == own.x && __float_as_int(q.y) < e);
        rank += q.z > own.x || (q.z == own.x && __float_as_int(q.w) < e);
      }
      __syncwarp();
      const bool takes = lane < count && rank < K;
      if (takes) chosen = e, chosen_z = own.x, slot = rank;
      if (count < K && lane >= count) {
        // fewer experts left than choices: the slots after them stay empty
      } else if (!takes) {
        slot = K;
      }
    } else {
      float w[VPT];  // what is not chosen yet
      int where = 0;
#pragma unroll
      for (int j = VPT - 1; j >= 0; --j) w[j] = v[j], where = v[j] == most ? j : where;
      for (int k = 0; k < K; ++k) {
        const float best = warp_max(most);
        if (best == -INFINITY) break;  // the same for all lanes
        const int owner = __ffs(__ballot_sync(kFull, most == best)) - 1;
        const int e = __shfl_sync(kFull, lane * VPT + where, owner);
        if (lane == k) chosen = e, chosen_z = best;
        if (lane == owner) {
          most = -INFINITY;
#pragma unroll
          for (int j = 0; j < VPT; ++j) {
            w[j] = j == where ? -INFINITY : w[j];
            most = fmaxf(most, w[j]);
          }
#pragma unroll
          for (int j = VPT - 1; j >= 0; --j) where = w[j] == most ? j : where;
        }
      }
    }
    exp_from(v, top);
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) s += v[j];
    s = warp_all_sum(s);
    const float inv = any ? reciprocal(s) : 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) total[j] = fmaf(v[j], inv, total[j]);
    const float lse = any ? top + log2_of(s) * kLn2 : 0.f;
    if (any) n += 1.f, squares = fmaf(lse, lse, squares);
    float weight = exp_from(chosen_z, top);  // 0 without a choice
    if (a.normalize) {
      const float all = warp_all_sum(weight);
      weight = any ? weight * reciprocal(all) : 0.f;
    } else {
      weight *= inv;
    }
    if (slot < K) {
      a.ids[t * K + slot] = chosen;
      a.weights[t * K + slot] = weight;
      if (chosen >= 0) atomicAdd(smem + chosen, 1);
    }
    if (lane == 0) a.stats[t] = lse;
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    if (lane * VPT + j < E) sums[warp * E + lane * VPT + j] = total[j];
  if (lane == 0) ends[warp][0] = n, ends[warp][1] = squares;
  __syncthreads();
  n = squares = 0.f;
  for (int w = 0; w < kWarps; ++w) n += ends[w][0], squares += ends[w][1];
  Totals totals;
  for (int e = threadIdx.x; e < E; e += 32 * kWarps) {
    float s = 0.f;
    for (int w = 0; w < kWarps; ++w) s += sums[w * E + e];
    const int64_t at = static_cast<int64_t>(blockIdx.x) * E + e;
    if (gridDim.x == 1)
      totals.expert(a, e, smem[e], s);
    else
      a.part_counts[at] = smem[e], a.part_sums[at] = s;
  }
  if (gridDim.x == 1)
    totals.finish(a, n, squares, part);
  else if (threadIdx.x == 0)
    a.part_ends[blockIdx.x * 2] = n, a.part_ends[blockIdx.x * 2 + 1] = squares;
}

// The CTAs' counts and sums added up, in order: a cluster, whose groups of
// threads take a share of the CTAs each, then the groups, then the cluster's
// CTAs. (One CTA: 12 us for 152 CTAs of 256 experts.)
__global__ void __cluster_dims__(kFinishCtas, 1, 1) __launch_bounds__(kThreads) k_route_finish(const RouteArgs a) {
  __shared__ int counts[kThreads];
  __shared__ float sums[kThreads], ends[2], part[32];
  wait_for_previous();
  cg::cluster_group cluster = cg::this_cluster();
  const int me = static_cast<int>(cluster.block_rank());
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.experts;
  if (me == 0 && warp < 2) {  // n and the sum of squares
    float s = 0.f;
    for (int c = lane; c < a.ctas; c += 32) s += a.part_ends[c * 2 + warp];
    s = warp_all_sum(s);
    if (lane == 0) ends[warp] = s;
  }
  const int here = kThreads / E, groups = here * kFinishCtas;  // here: at least one
  const int g = threadIdx.x / E, e = threadIdx.x - g * E;
  const int each = (a.ctas + groups - 1) / groups;
  int count = 0;
  float sum = 0.f;
  if (g < here) {
    const int c0 = (me * here + g) * each, c1 = min(a.ctas, c0 + each);
    for (int c = c0; c < c1; c += 4) {
      int n[4];
      float s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = static_cast<int64_t>(min(c + i, c1 - 1)) * E + e;
        n[i] = a.part_counts[at], s[i] = a.part_sums[at];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < c1) count += n[i], sum += s[i];
    }
  }
  counts[threadIdx.x] = count, sums[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x < E) {
    for (int k = 1; k < here; ++k) count += counts[k * E + e], sum += sums[k * E + e];
    counts[e] = count, sums[e] = sum;
  }
  cluster.sync();
  if (me == 0) {
    Totals totals;
    if (threadIdx.x < E) {
      int n[kFinishCtas];
      float s[kFinishCtas];
#pragma unroll
      for (int c = 0; c < kFinishCtas; ++c)
        n[c] = cluster.map_shared_rank(counts, c)[e], s[c] = cluster.map_shared_rank(sums, c)[e];
      count = 0, sum = 0.f;
#pragma unroll
      for (int c = 0; c < kFinishCtas; ++c) count += n[c], sum += s[c];
      totals.expert(a, e, count, sum);
    }
    totals.finish(a, ends[0], ends[1], part);
  }
  cluster.sync();  // no CTA leaves while the first one reads its sums
}

// CTAs an SM: one fewer at 8 experts a lane (70 registers in place of 64) took
// 30.6 us in place of 26.7 (65536 x 256 fp32).
constexpr int backward_ctas(int vpt) { return vpt <= 4 ? 5 : vpt <= 8 ? 4 : 1; }

template <class T, int VPT>
__global__ void __launch_bounds__(256, backward_ctas(VPT)) k_route_backward(const RouteArgs a) {
  constexpr int P = (VPT + 1) / 2;  // pairs of a lane's experts, the last of one expert half empty
  extern __shared__ __align__(16) float direct[];  // [warps][32 * VPT]: what the choices add
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.experts, K = a.topk;
  float* mine = direct + warp * 32 * VPT;
#pragma unroll
  for (int j = 0; j < VPT; ++j) mine[lane * VPT + j] = 0.f;
  __syncwarp();
  const float n = fmaxf(a.stats[a.tokens], 1.f);
  const float per_count = a.d_losses ? a.d_losses[0] * (static_cast<float>(E) / static_cast<float>(K)) / n / n : 0.f;
  const float per_lse = a.d_losses ? 2.f * a.d_losses[1] / n : 0.f;
  auto load_of = [&](int j) {
    return j < VPT && lane * VPT + j < E ? per_count * static_cast<float>(a.counts[lane * VPT + j]) : 0.f;
  };
  F2 load[P];
#pragma unroll
  for (int q = 0; q < P; ++q) load[q] = f2(load_of(2 * q), load_of(2 * q + 1));
  const T* z = static_cast<const T*>(a.z);
  T* dz = static_cast<T*>(a.dz);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  // a token's data, loaded while the one before it is worked on
  float next_v[VPT], next_lse = 0.f, next_w = 0.f, next_d = 0.f;
  int next_id = -1;
  auto fetch = [&](int64_t t) {
    if (t >= a.tokens) return;
    load_row<T, VPT>(z + t * a.stride, lane, E, a.vec, -INFINITY, next_v);
    next_lse = a.stats[t];
    if (lane < K) {
      next_id = a.ids[t * K + lane];
      next_w = a.weights[t * K + lane];
      if (a.d_weights) next_d = a.d_weights[t * K + lane];
    }
  };
  int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp;
  fetch(t);
  for (; t < a.tokens; t += step) {
    F2 e[P];
#pragma unroll
    for (int q = 0; q < P; ++q) e[q] = f2(next_v[2 * q], 2 * q + 1 < VPT ? next_v[VPT == 1 ? 0 : 2 * q + 1] : -INFINITY);
    const float lse = next_lse;
    int id = next_id;
    float w = next_w, d = next_d;
    fetch(t + step);
    if (id < 0 || id >= E) id = -1, w = 0.f, d = 0.f;
    const bool any = __shfl_sync(kFull, id, 0) >= 0;
    const float wd = warp_all_sum(id >= 0 ? w * d : 0.f);
    if (id >= 0) mine[id] = a.normalize ? w * (d - wd) : w * d;
    // p is exp(z - lse) over the sum of these: lse as it was rounded has lost
    // log(sum) where the scores are large, but lies less than 14 above the largest
    F2 total2 = f2(0.f), s2 = total2;
    const F2 minus = f2(-lse), log2e = f2(kLog2e);
#pragma unroll
    for (int q = 0; q < P; ++q) {
      float lo, hi;
      f2_out(mul2(add2(e[q], minus), log2e), lo, hi);
      e[q] = f2(tc::exp2_of(lo), tc::exp2_of(hi));
      total2 = add2(total2, e[q]), s2 = fma2(e[q], load[q], s2);
    }
    float total = sum2(total2), s = sum2(s2);
    sum_both(total, s);
    const float inv = any ? reciprocal(total) : 0.f;
    s *= inv;
    if (!a.normalize) s += wd;
    const F2 by = f2(inv), shift = f2((per_lse * lse - s) * inv);
    __syncwarp();
    float extra[2 * P];
    if constexpr (VPT % 4 == 0) {
#pragma unroll
      for (int j = 0; j < VPT; j += 4) {
        const float4 q = *reinterpret_cast<const float4*>(mine + lane * VPT + j);
        extra[j] = q.x, extra[j + 1] = q.y, extra[j + 2] = q.z, extra[j + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2 * P; ++j) extra[j] = j < VPT ? mine[lane * VPT + j] : 0.f;
    }
    float v[2 * P];
#pragma unroll
    for (int q = 0; q < P; ++q)
      f2_out(fma2(e[q], fma2(load[q], by, shift), f2(extra[2 * q], extra[2 * q + 1])), v[2 * q], v[2 * q + 1]);
    if (!any) {
#pragma unroll
      for (int j = 0; j < 2 * P; ++j) v[j] = 0.f;
    }
    __syncwarp();
    if (id >= 0) mine[id] = 0.f;
    __syncwarp();  // another lane may have the same expert of the next token
    T* row = dz + t * E;
    if constexpr (VPT % 8 == 0) {
      if (a.vec) {
#pragma unroll
        for (int i = 0; i < VPT; i += 8) {
          if constexpr (sizeof(T) == 4) {
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + lane * VPT + i),
                         "f"(v[i]), "f"(v[i + 1]), "f"(v[i + 2]), "f"(v[i + 3]), "f"(v[i + 4]), "f"(v[i + 5]),
                         "f"(v[i + 6]), "f"(v[i + 7])
                         : "memory");
            continue;
          }
          const float o[8] = {v[i], v[i + 1], v[i + 2], v[i + 3], v[i + 4], v[i + 5], v[i + 6], v[i + 7]};
          Elem<T>::store8(row + lane * VPT + i, o);
        }
        continue;
      }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (lane * VPT + j < E) row[lane * VPT + j] = Elem<T>::narrow(v[j]);
  }
}

// ---------------------------------------------------------------------------
// host

template <class... P>
cudaError_t launch(void (*fn)(P...), int64_t grid, int threads, size_t smem, bool early, cudaStream_t s, P... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, args...);
  if (e == cudaSuccess) g_launches.fetch_add(1, std::memory_order_relaxed);
  return e;
}

int ctas_for(int64_t tokens, int32_t experts) {
  const int warps = warps_of((experts + 31) / 32);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kCtasMost, (tokens + warps - 1) / warps)));
}

template <class T, int VPT>
cudaError_t run_route(const RouteArgs& a, bool backward, cudaStream_t s) {
  if (backward) {
    constexpr int kWarpsHere = 8;
    const int64_t grid = std::min<int64_t>(kSMs * 8, (a.tokens + kWarpsHere - 1) / kWarpsHere);
    static_assert(kWarpsHere * 32 * VPT * 4 <= 48 * 1024, "shared memory without asking");
    return launch(&k_route_backward<T, VPT>, grid, 32 * kWarpsHere, kWarpsHere * 32 * VPT * 4, false, s, a);
  }
  constexpr int kWarps = warps_of(VPT), kMost = (kWarps + 1) * 32 * VPT * 4;
  static KernelFacts facts;
  cudaError_t e = facts.allow(reinterpret_cast<const void*>(&k_route<T, VPT>), kMost, kMost);
  if (e == cudaSuccess)
    e = launch(&k_route<T, VPT>, a.ctas, 32 * kWarps, static_cast<size_t>(kWarps + 1) * a.experts * 4, false, s, a);
  if (e == cudaSuccess && a.ctas > 1) e = launch(&k_route_finish, kFinishCtas, kThreads, 0, true, s, a);
  return e;
}

template <class T>
cudaError_t run_typed(const RouteArgs& a, bool backward, cudaStream_t s) {
  const int each = (a.experts + 31) / 32;
  return each <= 1    ? run_route<T, 1>(a, backward, s)
         : each <= 2  ? run_route<T, 2>(a, backward, s)
         : each <= 4  ? run_route<T, 4>(a, backward, s)
         : each <= 8  ? run_route<T, 8>(a, backward, s)
         : each <= 16 ? run_route<T, 16>(a, backward, s)
                      : run_route<T, 32>(a, backward, s);
}

// Rows of exactly a power of two times 32 experts on 32-byte boundaries.
bool wide_rows(int experts, int64_t stride, int bytes, const void* z, const void* dz) {
  const int each = experts / 32;
  return experts % 32 == 0 && (each & (each - 1)) == 0 && each * bytes >= 16 && stride * bytes % 32 == 0 &&
         aligned_to(z, 32) && aligned_to(dz, 32);
}

zero_status check_shape(const char* fn, int64_t tokens, int64_t stride, int32_t experts, int32_t topk, int dtype) {
  if (tokens < 0 || tokens > INT64_C(1) << 24)
    return fail(ZERO_ERR_INVALID, "%s: tokens must lie in [0, 2^24]", fn);
  if (experts < 1 || experts > kExpertsMost)
    return fail(ZERO_ERR_INVALID, "%s: n_experts must lie in [1, %d]", fn, kExpertsMost);
  if (topk < 1 || topk > experts || topk > kTopkMost)
    return fail(ZERO_ERR_INVALID, "%s: topk must lie in [1, min(n_experts, %d)]", fn, kTopkMost);
  if (!known_type(dtype)) return fail(ZERO_ERR_INVALID, "%s: unknown dtype", fn);
  if (stride < experts || stride > INT64_C(1) << 36)
    return fail(ZERO_ERR_INVALID, "%s: logits_stride must be at least n_experts", fn);
  return ZERO_OK;
}

zero_status check_ptr(const char* fn, const char* what, const void* p, int bytes, bool needed) {
  if (needed && !p) return fail(ZERO_ERR_INVALID, "%s: %s is NULL", fn, what);
  if (!aligned_to(p, bytes)) return fail(ZERO_ERR_ALIGN, "%s: %s is not aligned to %d bytes", fn, what, bytes);
  return ZERO_OK;
}

int64_t workspace_of(int64_t tokens, int32_t experts) {
  const int64_t ctas = ctas_for(tokens, experts);
  return ctas > 1 ? ctas * (experts * 2 + 2) * 4 : 0;
}

zero_status run(const char* fn, const RouteArgs& a, int dtype, bool backward, void* stream) {
  const cudaError_t pending = cudaGetLastError();
  if (pending != cudaSuccess)
    return fail(ZERO_ERR_CUDA, "%s: pending CUDA error: %s", fn, cudaGetErrorString(pending));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == ZERO_FP32   ? run_typed<float>(a, backward, s)
                        : dtype == ZERO_BF16 ? run_typed<__nv_bfloat16>(a, backward, s)
                                             : run_typed<__half>(a, backward, s);
  if (e != cudaSuccess) return fail(ZERO_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return ZERO_OK;
}

#define ROUTE_TRY(x)                \
  do {                              \
    const zero_status st_ = (x);    \
    if (st_ != ZERO_OK) return st_; \
  } while (0)

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" zero_status zero_expert_route_workspace_bytes(int64_t tokens, int32_t n_experts, int64_t* bytes) {
  const char* fn = "zero_expert_route_workspace_bytes";
  clear_error();
  if (!bytes) return fail(ZERO_ERR_INVALID, "%s: bytes is NULL", fn);
  ROUTE_TRY(check_shape(fn, tokens, n_experts, n_experts, 1, ZERO_FP32));
  *bytes = workspace_of(tokens, n_experts);
  return ZERO_OK;
}

extern "C" zero_status zero_expert_route(const void* logits, int64_t logits_stride, zero_dtype dtype, int64_t tokens,
                                         int32_t n_experts, int32_t topk, int32_t normalize, int32_t* ids,
                                         float* weights, int32_t* counts, float* losses, float* stats,
                                         void* workspace, int64_t workspace_bytes, void* stream) {
  const char* fn = "zero_expert_route";
  clear_error();
  NvtxRange range(fn);
  ROUTE_TRY(check_shape(fn, tokens, logits_stride, n_experts, topk, dtype));
  const bool any = tokens > 0;
  const int b = type_bytes(dtype);
  ROUTE_TRY(check_ptr(fn, "logits", logits, b, any));
  ROUTE_TRY(check_ptr(fn, "ids", ids, 4, any));
  ROUTE_TRY(check_ptr(fn, "weights", weights, 4, any));
  ROUTE_TRY(check_ptr(fn, "counts", counts, 4, true));
  ROUTE_TRY(check_ptr(fn, "losses", losses, 4, true));
  ROUTE_TRY(check_ptr(fn, "stats", stats, 4, true));
  const int64_t need = workspace_of(tokens, n_experts);
  ROUTE_TRY(check_ptr(fn, "workspace", workspace, 4, need > 0));
  if (workspace_bytes < need)
    return fail(ZERO_ERR_INVALID, "%s: workspace holds %" PRId64 " bytes, needs %" PRId64, fn, workspace_bytes, need);
  ROUTE_TRY(check_overlaps(fn,
                           {Extent::block("ids", ids, tokens * topk * 4), Extent::block("weights", weights, tokens * topk * 4),
                            Extent::block("counts", counts, n_experts * INT64_C(4)), Extent::block("losses", losses, 8),
                            Extent::block("stats", stats, (tokens + 1) * 4), Extent::block("workspace", need ? workspace : nullptr, need)},
                           {{"logits", logits, tokens, logits_stride * b, n_experts * INT64_C(1) * b}}));
  RouteArgs a = {};
  a.z = logits, a.tokens = tokens, a.stride = logits_stride, a.experts = n_experts, a.topk = topk;
  a.normalize = normalize != 0, a.vec = wide_rows(n_experts, logits_stride, b, logits, nullptr);
  a.ids = ids, a.weights = weights, a.counts = counts, a.losses = losses, a.stats = stats;
  a.ctas = ctas_for(tokens, n_experts);
  a.part_counts = static_cast<int32_t*>(workspace);
  a.part_sums = reinterpret_cast<float*>(a.part_counts + static_cast<int64_t>(a.ctas) * n_experts);
  a.part_ends = a.part_sums + static_cast<int64_t>(a.ctas) * n_experts;
  return run(fn, a, dtype, false, stream);
}

extern "C" zero_status zero_expert_route_backward(const void* logits, int64_t logits_stride, zero_dtype dtype,
                                                  int64_t tokens, int32_t n_experts, int32_t topk, int32_t normalize,
                                                  const int32_t* ids, const float* weights, const int32_t* counts,
                                                  const float* stats, const float* d_weights, const float* d_losses,
                                                  void* d_logits, void* stream) {
  const char* fn = "zero_expert_route_backward";
  clear_error();
  NvtxRange range(fn);
  ROUTE_TRY(check_shape(fn, tokens, logits_stride, n_experts, topk, dtype));
  const bool any = tokens > 0;
  const int b = type_bytes(dtype);
  ROUTE_TRY(check_ptr(fn, "logits", logits, b, any));
  ROUTE_TRY(check_ptr(fn, "ids", ids, 4, any));
  ROUTE_TRY(check_ptr(fn, "weights", weights, 4, any));
  ROUTE_TRY(check_ptr(fn, "counts", counts, 4, any));
  ROUTE_TRY(check_ptr(fn, "stats", stats, 4, any));
  ROUTE_TRY(check_ptr(fn, "d_weights", d_weights, 4, false));
  ROUTE_TRY(check_ptr(fn, "d_losses", d_losses, 4, false));
  ROUTE_TRY(check_ptr(fn, "d_logits", d_logits, b, any));
  if (!any) return ZERO_OK;
  ROUTE_TRY(check_overlaps(fn, {Extent::block("d_logits", d_logits, tokens * n_experts * b)},
                           {{"logits", logits, tokens, logits_stride * b, n_experts * INT64_C(1) * b},
                            Extent::block("ids", ids, tokens * topk * 4), Extent::block("weights", weights, tokens * topk * 4),
                            Extent::block("counts", counts, n_experts * INT64_C(4)),
                            Extent::block("stats", stats, (tokens + 1) * 4),
                            Extent::block("d_weights", d_weights, tokens * topk * 4),
                            Extent::block("d_losses", d_losses, 8)}));
  RouteArgs a = {};
  a.z = logits, a.tokens = tokens, a.stride = logits_stride, a.experts = n_experts, a.topk = topk;
  a.normalize = normalize != 0, a.vec = wide_rows(n_experts, logits_stride, b, logits, d_logits);
  a.ids = const_cast<int32_t*>(ids), a.weights = const_cast<float*>(weights);
  a.counts = const_cast<int32_t*>(counts), a.stats = const_cast<float*>(stats);
  a.d_weights = d_weights, a.d_losses = d_losses, a.dz = d_logits;
  return run(fn, a, dtype, true, stream);
}
