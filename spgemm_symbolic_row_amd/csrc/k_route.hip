// Routing of tokens to experts, and its gradient.  Row t of the logits gives
// row t of the sparse routing matrix: the k experts with the largest keys,
// columns rising, and their weights.
//
// Up to 256 experts 16 lanes take a row, four rows to a wave; above, a wave
// does.  Lane l of a row holds experts l*V .. l*V+V-1, so the lowest lane of a
// tie holds the lowest expert.  Keys are compared as ordered 32-bit integers;
// each of the k picks is a maximum over the lane's keys, one over the row by
// DPP and one ballot.  The picks are then packed through LDS, so that the
// weights cost one exponential each.  All sums are in 32 bits.  A row is read
// once (4 or 2 bytes per logit) and 8 bytes per entry are written; what bounds
// it is the chain of picks at few rows (1 x 64, 6 picks: 3.3 us) and the
// instructions at many (16384 x 256 fp32, sigmoid, 8 groups, 8 picks: 20 us, 0.9
// TB/s, 1990 vector instructions for a wave's four rows, which keep the vector
// units busy 70%; a wave to a row took 33).
#include <algorithm>

#include "route_row.hpp"

namespace sg {
namespace {

constexpr int kRouteNT = 256;
constexpr int kRouteRows = kRouteNT / kWave;  // of the gradient: a wave takes a row

struct RouteArgs {
  RouteRow row;
  const void* logits;
  int64_t ld;
  const uint8_t* active;
  int32_t* col;
  float* val;
  int64_t T;
  bool vec;
};

template <typename T, int L, int V, bool kSig>
__global__ __launch_bounds__(kRouteNT) void k_route(RouteArgs a) {
  extern __shared__ uint32_t packed[];  // per row: k columns, k logits
  const int row = threadIdx.x / L, lane = threadIdx.x % L, e0 = lane * V;
  const int64_t t = (int64_t)blockIdx.x * (kRouteNT / L) + row;
  if ((int64_t)blockIdx.x * (kRouteNT / L) + threadIdx.x / kWave * (kWave / L) >= a.T)
    return;  // the whole wave
  const bool inside = t < a.T;
  float z[V];
  if (inside && (!a.active || a.active[t])) {
    load_logits<T, V>((const T*)a.logits + t * a.ld, e0, a.row.E, a.vec, z);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] = -INFINITY;
  }
  const int k = a.row.k;
  route_row<L, V, kSig>(a.row, z, packed + row * 2 * k, [&](int i, int col, float val) {
    if (inside) {
      a.col[t * k + i] = col;
      a.val[t * k + i] = val;
    }
  });
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
    load_logits<T, V>((const T*)a.logits + t * a.ld, e0, a.E, a.vec, z);
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
        if (in[j]) d[j] = (a.renorm ? (dw[j] - mean) / D : dw[j]) * sigmoid_slope(z[j]);
    }
  }
  T* out = (T*)a.dlogits + t * a.E;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (e0 + j < a.E) out[e0 + j] = from_f32<T>(d[j]);
}

// Experts of a lane, and lanes of a row.
int width_of(int64_t E) { return E <= 16 ? 1 : E <= 32 ? 2 : E <= 64 ? 4 : E <= 128 ? 8 : 16; }
int lanes_of(int64_t E) { return E <= 256 ? 16 : 64; }

// Work groups of one launch at most: a launch takes fewer than 2^32 work items.
constexpr int64_t kRouteGrid = ((int64_t)1 << 31) / kRouteNT;

template <typename T, int L, int V, bool kSig>
void launch_route(RouteArgs a, hipStream_t s) {
  constexpr int kRows = kRouteNT / L;
  for (int64_t left = a.T; left > 0; left -= a.T) {
    a.T = std::min(left, kRouteGrid * kRows);
    hipLaunchKernelGGL((k_route<T, L, V, kSig>), dim3((unsigned)((a.T + kRows - 1) / kRows)),
                       dim3(kRouteNT), (size_t)kRows * 2 * a.row.k * sizeof(uint32_t), s, a);
    a.logits = (const T*)a.logits + a.T * a.ld;
    if (a.active) a.active += a.T;
    a.col += a.T * a.row.k;
    a.val += a.T * a.row.k;
  }
}

template <typename T, bool kSig>
void route_by_width(const RouteArgs& a, hipStream_t s) {
  if (lanes_of(a.row.E) == 64) return launch_route<T, 64, 16, kSig>(a, s);
  switch (width_of(a.row.E)) {
    case 1: return launch_route<T, 16, 1, kSig>(a, s);
    case 2: return launch_route<T, 16, 2, kSig>(a, s);
    case 4: return launch_route<T, 16, 4, kSig>(a, s);
    case 8: return launch_route<T, 16, 8, kSig>(a, s);
    default: return launch_route<T, 16, 16, kSig>(a, s);
  }
}

template <typename T, int V, bool kSig>
void launch_route_grad(RouteGradArgs a, hipStream_t s) {
  for (int64_t left = a.T; left > 0; left -= a.T) {
    a.T = std::min(left, kRouteGrid * kRouteRows);
    hipLaunchKernelGGL((k_route_grad<T, V, kSig>),
                       dim3((unsigned)((a.T + kRouteRows - 1) / kRouteRows)), dim3(kRouteNT),
                       (size_t)kRouteRows * 2 * a.E * sizeof(float), s, a);
    a.logits = (const T*)a.logits + a.T * a.ld;
    a.col += a.T * a.k;
    a.dval += a.T * a.k;
    a.dlogits = (T*)a.dlogits + a.T * a.E;
  }
}

template <typename T, bool kSig>
void route_grad_by_width(const RouteGradArgs& a, hipStream_t s) {
  if (a.E <= 64) launch_route_grad<T, 1, kSig>(a, s);
  else if (a.E <= 128) launch_route_grad<T, 2, kSig>(a, s);
  else if (a.E <= 256) launch_route_grad<T, 4, kSig>(a, s);
  else if (a.E <= 512) launch_route_grad<T, 8, kSig>(a, s);
  else launch_route_grad<T, 16, kSig>(a, s);
}

int64_t type_bytes(spgemm_dtype t) { return t == SPGEMM_F32 ? 4 : 2; }

// Whether a lane's `width` experts can be loaded at once, 16 bytes at most.
bool can_vec(const void* p, int64_t ld, int64_t width, spgemm_dtype t) {
  const int64_t b = std::min<int64_t>(type_bytes(t) * width, 16);
  return (uintptr_t)p % b == 0 && ld * type_bytes(t) % b == 0;
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
  if (T < 0) return refuse(SPGEMM_ERR_INVALID_ARG, "route: tokens < 0");
  const spgemm_status st = check_route_options(E, k, o);
  if (st != SPGEMM_OK) return st;
  if (dtype != SPGEMM_F32 && dtype != SPGEMM_BF16 && dtype != SPGEMM_F16)
    return refuse(SPGEMM_ERR_INVALID_ARG, "route: logits must be fp32, bf16 or fp16");
  if (ld < E) return refuse(SPGEMM_ERR_INVALID_ARG, "route: row stride below the expert count");
  if (T > INT32_MAX / k)
    return refuse(SPGEMM_ERR_INDEX_OVERFLOW, "route: more than 2^31 - 1 entries");
  if (T > 0 && (!logits || !col || !val))
    return refuse(SPGEMM_ERR_INVALID_ARG, "route: null array");
  return SPGEMM_OK;
}

}  // namespace

spgemm_status check_route_options(int64_t E, int32_t k, const spgemm_route_options* o) {
  if (E < 1 || E > kMaxExperts)
    return refuse(SPGEMM_ERR_INVALID_ARG, "route: experts outside [1, 1024]");
  if (k < 1 || k > 64 || k > E)
    return refuse(SPGEMM_ERR_INVALID_ARG, "route: k outside [1, min(64, experts)]");
  if (!o) return refuse(SPGEMM_ERR_INVALID_ARG, "route: null options");
  const int64_t g = o->groups ? o->groups : 1, tg = o->top_groups ? o->top_groups : g;
  if (g < 1 || g > 64 || E % g || tg < 1 || tg > g)
    return refuse(SPGEMM_ERR_INVALID_ARG,
                  "route: groups outside [1, 64] or not dividing the experts, or top_groups "
                  "outside [1, groups]");
  if (k > E / g * tg)
    return refuse(SPGEMM_ERR_INVALID_ARG, "route: k above the experts of the chosen groups");
  return SPGEMM_OK;
}

}  // namespace sg

using namespace sg;

extern "C" spgemm_status spgemm_route(int64_t T, int64_t E, int32_t k, const void* dLogits,
                                      int64_t ld, spgemm_dtype dtype, const float* dBias,
                                      const uint8_t* dActive, const spgemm_route_options* opts,
                                      int32_t* dCol, float* dVal, void* stream) {
  const spgemm_status st = check_route(T, E, k, dLogits, ld, dtype, opts, dCol, dVal);
  if (st != SPGEMM_OK || T == 0) return st;
  (void)hipGetLastError();  // an error that earlier calls left is not this one's
  RouteArgs a{};
  a.row = route_row_of(E, k, *opts, dBias, width_of(E));
  a.logits = dLogits;
  a.ld = ld;
  a.active = dActive;
  a.col = dCol;
  a.val = dVal;
  a.T = T;
  a.vec = can_vec(dLogits, ld, width_of(E), dtype);
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
  (void)hipGetLastError();  // an error that earlier calls left is not this one's
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
  const int64_t width = E <= 64 ? 1 : E <= 128 ? 2 : E <= 256 ? 4 : E <= 512 ? 8 : 16;
  a.vec = can_vec(dLogits, ld, width, dtype);
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
