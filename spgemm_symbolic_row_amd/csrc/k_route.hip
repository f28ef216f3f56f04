// Routing of tokens to experts, and its gradient.  Row t of the logits gives
// row t of the sparse routing matrix: the k experts with the largest keys,
// columns rising, and their weights.
//
// One wave takes one row; lane l holds experts l*V .. l*V+V-1, so the lowest
// lane of a tie holds the lowest expert.  Keys are compared as ordered 32-bit
// integers; each of the k picks is one DPP maximum over the wave and one
// ballot.  All sums are in 32 bits.  A row is read once (4 to 2 bytes per
// logit) and 8 bytes per entry are written; what bounds it is the chain of
// picks (about 8 dependent steps each) at few rows, and their instructions at
// many.
#include <algorithm>

#include "expert_common.hpp"

namespace sg {
namespace {

constexpr int kRouteNT = 256;
constexpr int kRouteRows = kRouteNT / kWave;

template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* row, int E, bool vec, float z[V]) {
  const int e0 = lane_id() * V;
  if (vec && e0 + V <= E) {
    struct alignas(sizeof(T) * V) Pack { T v[V]; };
    const Pack p = *(const Pack*)(row + e0);
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] = to_f32(p.v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] = e0 + j < E ? to_f32(row[e0 + j]) : -INFINITY;
  }
}

// As the keys are defined: 0 below z = -88, where exp(-z) is beyond fp32.
__device__ __forceinline__ float sigmoid_key(float z) { return 1.0f / (1.0f + expf(-z)); }

// As the weights use it: the same value, without that overflow.
__device__ __forceinline__ float sigmoid(float z) {
  const float e = expf(-fabsf(z));
  return (z < 0.0f ? e : 1.0f) / (1.0f + e);
}

// Ordered key of an expert, 0 where it is out: a logit or a key that is
// minus infinity or NaN.
template <bool kSig>
__device__ __forceinline__ uint32_t key_of(float z, float b, bool biased) {
  float key = kSig ? sigmoid_key(z) : z;
  if (biased) key += b;
  return z > -INFINITY && key > -INFINITY ? ordered_bits(key) : 0u;
}

// The groups that may be chosen from, as a bit mask: group g's score is its
// largest key (softmax) or the sum of its two largest (sigmoid).
template <int V, bool kSig>
__device__ __forceinline__ uint64_t pick_groups(const uint32_t key[V], int per, int G, int top) {
  const int e0 = lane_id() * V;
  uint32_t score = 0;  // of group lane_id()
  for (int g = 0; g < G; ++g) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if ((e0 + j) / per == g) m = max(m, key[j]);
    const uint32_t M = wave_max_u32(m);
    uint32_t s = M;
    if (kSig && M) {
      const int first = ffs64(__ballot(m == M));
      uint32_t m2 = 0;
      bool seen = false;  // the largest key counts once, at its lowest expert
#pragma unroll
      for (int j = 0; j < V; ++j)
        if ((e0 + j) / per == g) {
          const bool skip = lane_id() == first && key[j] == M && !seen;
          if (skip) seen = true;
          else m2 = max(m2, key[j]);
        }
      const uint32_t M2 = wave_max_u32(m2);
      if (M2) s = ordered_bits(from_ordered(M) + from_ordered(M2));
    }
    if (lane_id() == g) score = s;
  }
  uint64_t chosen = 0;
  for (int i = 0; i < top; ++i) {
    const uint32_t M = wave_max_u32(score);
    if (!M) break;
    const int g = ffs64(__ballot(score == M));
    chosen |= 1ull << g;
    if (lane_id() == g) score = 0;
  }
  return chosen;
}

struct RouteArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  const uint8_t* active;
  int32_t* col;
  float* val;
  int64_t T;
  int E, k, groups, top_groups;
  bool renorm, vec;
  float scale;
};

template <typename T, int V, bool kSig>
__global__ __launch_bounds__(kRouteNT) void k_route(RouteArgs a) {
  const int64_t t = (int64_t)blockIdx.x * kRouteRows + threadIdx.x / kWave;
  if (t >= a.T) return;
  const int lane = lane_id(), e0 = lane * V;
  float z[V];
  uint32_t key[V];
  const bool active = !a.active || a.active[t];
  if (active) {
    load_logits<T, V>((const T*)a.logits + t * a.ld, a.E, a.vec, z);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] = -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float b = a.bias && e0 + j < a.E ? a.bias[e0 + j] : 0.0f;
    key[j] = key_of<kSig>(z[j], b, a.bias != nullptr);
  }
  // Softmax over every expert that is not out: its maximum and sum, before
  // keys are taken away.
  float top = 0.0f, total = 0.0f;
  if (!kSig && !a.renorm) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (key[j]) m = max(m, ordered_bits(z[j]));
    const uint32_t M = wave_max_u32(m);
    top = M ? from_ordered(M) : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (key[j]) total += expf(z[j] - top);
    total = wave_sum_f32(total);
  }
  if (a.groups > 1) {
    const int per = a.E / a.groups;
    const uint64_t chosen = pick_groups<V, kSig>(key, per, a.groups, a.top_groups);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (e0 + j < a.E && !((chosen >> ((e0 + j) / per)) & 1)) key[j] = 0;
  }
  uint32_t taken = 0;  // bit j: expert e0 + j is picked
  int count = 0;
  for (; count < a.k; ++count) {
    uint32_t m = key[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = max(m, key[j]);
    const uint32_t M = wave_max_u32(m);
    if (!M) break;
    if (lane == ffs64(__ballot(m == M))) {
      bool done = false;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (!done && key[j] == M) {
          done = true;
          key[j] = 0;
          taken |= 1u << j;
        }
    }
  }
  // Weights of the picked experts.
  float w[V];
  if (!kSig && a.renorm) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if ((taken >> j) & 1) m = max(m, ordered_bits(z[j]));
    const uint32_t M = wave_max_u32(m);
    top = M ? from_ordered(M) : 0.0f;
  }
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    w[j] = (taken >> j) & 1 ? (kSig ? sigmoid(z[j]) : expf(z[j] - top)) : 0.0f;
    sum += w[j];
  }
  if (a.renorm) {
    total = wave_sum_f32(sum);
    if (kSig) total += 1e-20f;
  } else if (kSig) {
    total = 1.0f;
  }
  // Positions: picks of lower lanes, then of lower experts in the lane.
  int at = 0;
#pragma unroll
  for (int j = 0; j < V; ++j)
    at += (int)__popcll(__ballot((taken >> j) & 1) & lanemask_lt());
#pragma unroll
  for (int j = 0; j < V; ++j)
    if ((taken >> j) & 1) {
      a.col[t * a.k + at] = e0 + j;
      a.val[t * a.k + at] = w[j] / total * a.scale;
      ++at;
    }
  if (lane >= count && lane < a.k) {
    a.col[t * a.k + lane] = -1;
    a.val[t * a.k + lane] = 0.0f;
  }
}

struct RouteGradArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  const int32_t* col;
  const float* dval;
  void* dlogits;  // T x E, contiguous
  int64_t T;
  int E, k;
  bool renorm, vec;
  float scale;
};

// The scores are computed again from the logits.  With p the scores and
// dw = scale * dval:
//   softmax over all:      dz_e = p_e ([e picked] dw_e - sum_S p_j dw_j)
//   softmax over the pick: the same with p the softmax over S, 0 outside S
//   sigmoid:               dz_i = dw_i p_i (1 - p_i)
//   sigmoid renormalised:  dz_i = (dw_i - sum_S p_j dw_j / D) / D p_i (1 - p_i),
//                          D = sum_S p_j + 1e-20
template <typename T, int V, bool kSig>
__global__ __launch_bounds__(kRouteNT) void k_route_grad(RouteGradArgs a) {
  extern __shared__ float lds[];  // per wave: dw of every expert, then a mark per expert
  const int64_t t = (int64_t)blockIdx.x * kRouteRows + threadIdx.x / kWave;
  if (t >= a.T) return;
  const int lane = lane_id(), e0 = lane * V;
  float* dws = lds + (threadIdx.x / kWave) * 2 * a.E;
  float* mark = dws + a.E;
  const int c = lane < a.k ? a.col[t * a.k + lane] : -1;
  const bool there = (uint32_t)c < (uint32_t)a.E;
  const bool any = __ballot(there) != 0;
  float d[V];
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = 0.0f;
  if (any) {
    for (int e = lane; e < a.E; e += kWave) mark[e] = 0.0f;
    // One wave's LDS accesses are performed in order.
    __builtin_amdgcn_wave_barrier();
    if (there) {
      dws[c] = a.dval[t * a.k + lane] * a.scale;
      mark[c] = 1.0f;
    }
    __builtin_amdgcn_wave_barrier();
    float z[V], p[V], dw[V];
    load_logits<T, V>((const T*)a.logits + t * a.ld, a.E, a.vec, z);
    bool in[V], pick[V];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool inside = e0 + j < a.E;
      pick[j] = inside && mark[inside ? e0 + j : 0] != 0.0f;
      dw[j] = pick[j] ? dws[e0 + j] : 0.0f;
      const float b = a.bias && inside ? a.bias[e0 + j] : 0.0f;
      in[j] = kSig || a.renorm ? pick[j] : key_of<kSig>(z[j], b, a.bias != nullptr) != 0;
      if (!kSig && in[j]) m = max(m, ordered_bits(z[j]));
    }
    const uint32_t M = wave_max_u32(m);
    const float top = M ? from_ordered(M) : 0.0f;
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      p[j] = in[j] ? (kSig ? sigmoid(z[j]) : expf(z[j] - top)) : 0.0f;
      sum += p[j];
      dot += pick[j] ? p[j] * dw[j] : 0.0f;
    }
    sum = wave_sum_f32(sum);
    dot = wave_sum_f32(dot);
    if (!kSig) {
      const float mean = dot / sum;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (in[j]) d[j] = p[j] / sum * (dw[j] - mean);
    } else {
      const float D = sum + 1e-20f, mean = dot / D;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (in[j]) d[j] = (a.renorm ? (dw[j] - mean) / D : dw[j]) * p[j] * (1.0f - p[j]);
    }
  }
  T* out = (T*)a.dlogits + t * a.E;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (e0 + j < a.E) out[e0 + j] = from_f32<T>(d[j]);
}

template <typename T, bool kSig>
void route_by_width(const RouteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + kRouteRows - 1) / kRouteRows)), nt(kRouteNT);
  if (a.E <= 64) hipLaunchKernelGGL((k_route<T, 1, kSig>), grid, nt, 0, s, a);
  else if (a.E <= 128) hipLaunchKernelGGL((k_route<T, 2, kSig>), grid, nt, 0, s, a);
  else if (a.E <= 256) hipLaunchKernelGGL((k_route<T, 4, kSig>), grid, nt, 0, s, a);
  else if (a.E <= 512) hipLaunchKernelGGL((k_route<T, 8, kSig>), grid, nt, 0, s, a);
  else hipLaunchKernelGGL((k_route<T, 16, kSig>), grid, nt, 0, s, a);
}

template <typename T, bool kSig>
void route_grad_by_width(const RouteGradArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + kRouteRows - 1) / kRouteRows)), nt(kRouteNT);
  const size_t lds = (size_t)kRouteRows * 2 * a.E * sizeof(float);
  if (a.E <= 64) hipLaunchKernelGGL((k_route_grad<T, 1, kSig>), grid, nt, lds, s, a);
  else if (a.E <= 128) hipLaunchKernelGGL((k_route_grad<T, 2, kSig>), grid, nt, lds, s, a);
  else if (a.E <= 256) hipLaunchKernelGGL((k_route_grad<T, 4, kSig>), grid, nt, lds, s, a);
  else if (a.E <= 512) hipLaunchKernelGGL((k_route_grad<T, 8, kSig>), grid, nt, lds, s, a);
  else hipLaunchKernelGGL((k_route_grad<T, 16, kSig>), grid, nt, lds, s, a);
}

int width_of(int64_t E) { return E <= 64 ? 1 : E <= 128 ? 2 : E <= 256 ? 4 : E <= 512 ? 8 : 16; }

int64_t type_bytes(spgemm_dtype t) { return t == SPGEMM_F32 ? 4 : 2; }

// Whether a lane's experts can be loaded at once.
bool can_vec(const void* p, int64_t ld, int64_t E, spgemm_dtype t) {
  const int64_t b = type_bytes(t) * width_of(E);
  return (uintptr_t)p % b == 0 && ld % width_of(E) == 0 && b <= 16;
}

spgemm_status refuse(spgemm_status st, const char* msg) {
  set_thread_error(msg);
  return st;
}

spgemm_status launched() {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return SPGEMM_OK;
  return refuse(SPGEMM_ERR_HIP, hipGetErrorString(e));
}

spgemm_status check_route(int64_t T, int64_t E, int32_t k, const void* logits, int64_t ld,
                          spgemm_dtype dtype, const spgemm_route_options* o, const void* col,
                          const void* val) {
  if (T < 0 || E < 1 || E > kMaxExperts)
    return refuse(SPGEMM_ERR_INVALID_ARG, "route: tokens < 0, or experts outside [1, 1024]");
  if (k < 1 || k > 64 || k > E)
    return refuse(SPGEMM_ERR_INVALID_ARG, "route: k outside [1, min(64, experts)]");
  if (dtype != SPGEMM_F32 && dtype != SPGEMM_BF16 && dtype != SPGEMM_F16)
    return refuse(SPGEMM_ERR_INVALID_ARG, "route: logits must be fp32, bf16 or fp16");
  if (ld < E) return refuse(SPGEMM_ERR_INVALID_ARG, "route: row stride below the expert count");
  if (!o) return refuse(SPGEMM_ERR_INVALID_ARG, "route: null options");
  const int64_t g = o->groups ? o->groups : 1, tg = o->top_groups ? o->top_groups : g;
  if (g < 1 || g > 64 || E % g || tg < 1 || tg > g)
    return refuse(SPGEMM_ERR_INVALID_ARG,
                  "route: groups outside [1, 64] or not dividing the experts, or top_groups "
                  "outside [1, groups]");
  if (k > E / g * tg)
    return refuse(SPGEMM_ERR_INVALID_ARG, "route: k above the experts of the chosen groups");
  if (T > INT32_MAX / k)
    return refuse(SPGEMM_ERR_INDEX_OVERFLOW, "route: more than 2^31 - 1 entries");
  if (T > 0 && (!logits || !col || !val))
    return refuse(SPGEMM_ERR_INVALID_ARG, "route: null array");
  return SPGEMM_OK;
}

}  // namespace
}  // namespace sg

using namespace sg;

extern "C" spgemm_status spgemm_route(int64_t T, int64_t E, int32_t k, const void* dLogits,
                                      int64_t ld, spgemm_dtype dtype, const float* dBias,
                                      const uint8_t* dActive, const spgemm_route_options* opts,
                                      int32_t* dCol, float* dVal, void* stream) {
  const spgemm_status st = check_route(T, E, k, dLogits, ld, dtype, opts, dCol, dVal);
  if (st != SPGEMM_OK || T == 0) return st;
  RouteArgs a{};
  a.logits = dLogits;
  a.ld = ld;
  a.bias = dBias;
  a.active = dActive;
  a.col = dCol;
  a.val = dVal;
  a.T = T;
  a.E = (int)E;
  a.k = k;
  a.groups = opts->groups ? opts->groups : 1;
  a.top_groups = opts->top_groups ? opts->top_groups : a.groups;
  if (a.top_groups == a.groups) a.groups = 1;  // every group is chosen
  a.renorm = !opts->no_renormalise;
  a.vec = can_vec(dLogits, ld, E, dtype);
  a.scale = opts->scale != 0.0f ? opts->scale : 1.0f;
  const hipStream_t s = (hipStream_t)stream;
  if (dtype == SPGEMM_F32)
    opts->sigmoid ? route_by_width<float, true>(a, s) : route_by_width<float, false>(a, s);
  else if (dtype == SPGEMM_BF16)
    opts->sigmoid ? route_by_width<__bf16, true>(a, s) : route_by_width<__bf16, false>(a, s);
  else
    opts->sigmoid ? route_by_width<_Float16, true>(a, s) : route_by_width<_Float16, false>(a, s);
  return launched();
}

extern "C" spgemm_status spgemm_route_backward(int64_t T, int64_t E, int32_t k,
                                               const void* dLogits, int64_t ld,
                                               spgemm_dtype dtype, const float* dBias,
                                               const spgemm_route_options* opts,
                                               const int32_t* dCol, const float* dGradVal,
                                               void* dGradLogits, void* stream) {
  const spgemm_status st = check_route(T, E, k, dLogits, ld, dtype, opts, dCol, dGradVal);
  if (st != SPGEMM_OK || T == 0) return st;
  if (!dGradLogits) return refuse(SPGEMM_ERR_INVALID_ARG, "route: null array");
  RouteGradArgs a{};
  a.logits = dLogits;
  a.ld = ld;
  a.bias = dBias;
  a.col = dCol;
  a.dval = dGradVal;
  a.dlogits = dGradLogits;
  a.T = T;
  a.E = (int)E;
  a.k = k;
  a.renorm = !opts->no_renormalise;
  a.vec = can_vec(dLogits, ld, E, dtype);
  a.scale = opts->scale != 0.0f ? opts->scale : 1.0f;
  const hipStream_t s = (hipStream_t)stream;
  if (dtype == SPGEMM_F32)
    opts->sigmoid ? route_grad_by_width<float, true>(a, s) : route_grad_by_width<float, false>(a, s);
  else if (dtype == SPGEMM_BF16)
    opts->sigmoid ? route_grad_by_width<__bf16, true>(a, s)
                  : route_grad_by_width<__bf16, false>(a, s);
  else
    opts->sigmoid ? route_grad_by_width<_Float16, true>(a, s)
                  : route_grad_by_width<_Float16, false>(a, s);
  return launched();
}
