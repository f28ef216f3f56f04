// One row of routing, from its logits to its picks, by L = 16 or 64 lanes of a wave:
// lane l holds experts l*V .. l*V+V-1, so the lowest lane of a tie holds the lowest
// expert.  Keys are compared as ordered 32-bit integers; each of the k picks is a
// maximum over the lane's keys, one over the row by DPP and one ballot.  The picks
// are then packed through LDS, so that the weights cost one exponential each.
#pragma once
#include "expert_common.hpp"

namespace sg {

template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* row, int e0, int E, bool vec, float z[V]) {
  if (vec && e0 + V <= E) {
    constexpr int kOnce = V * sizeof(T) > 16 ? 16 / sizeof(T) : V;  // values of one load
    struct alignas(sizeof(T) * kOnce) Pack { T v[kOnce]; };
#pragma unroll
    for (int i = 0; i < V / kOnce; ++i) {
      const Pack p = ((const Pack*)(row + e0))[i];
#pragma unroll
      for (int j = 0; j < kOnce; ++j) z[i * kOnce + j] = to_f32(p.v[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] = e0 + j < E ? to_f32(row[e0 + j]) : -INFINITY;
  }
}

// Maximum and sum over the L lanes of a row, in all of them.
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  if constexpr (L == 64) return wave_max_u32(x);
  x = max(x, dpp_or_zero<0x128, 0xf>(x));  // row_ror:8
  x = max(x, dpp_or_zero<0x124, 0xf>(x));
  x = max(x, dpp_or_zero<0x122, 0xf>(x));
  return max(x, dpp_or_zero<0x121, 0xf>(x));
}
template <int L>
__device__ __forceinline__ float row_sum(float x) {
  if constexpr (L == 64) return wave_sum_f32(x);
  x = dpp_add<0x128, 0xf>(x);
  x = dpp_add<0x124, 0xf>(x);
  x = dpp_add<0x122, 0xf>(x);
  return dpp_add<0x121, 0xf>(x);
}
// First lane of the row, counted from its start, for which `is` holds.
template <int L>
__device__ __forceinline__ int row_first(bool is) {
  const uint64_t m = __ballot(is);
  if constexpr (L == 64) return ffs64(m);
  return __ffs((int)(uint32_t)(m >> (lane_id() & 48)) & 0xffff) - 1;
}
// Sum over the row's lower lanes.
template <int L>
__device__ __forceinline__ int row_excl_scan(int x) {
  if constexpr (L == 64) return wave_incl_scan(x) - x;
  uint32_t s = x;
  s += dpp_or_zero<0x111, 0xf>(s);  // row_shr:1
  s += dpp_or_zero<0x112, 0xf>(s);
  s += dpp_or_zero<0x114, 0xf>(s);
  s += dpp_or_zero<0x118, 0xf>(s);
  return (int)s - x;
}

// As the keys are defined: 0 below z = -88, where exp(-z) is beyond fp32.
__device__ __forceinline__ float sigmoid_key(float z) { return 1.0f / (1.0f + expf(-z)); }

// As the weights use it: the same value, without that overflow.
__device__ __forceinline__ float sigmoid(float z) {
  const float e = expf(-fabsf(z));
  return (z < 0.0f ? e : 1.0f) / (1.0f + e);
}

// Its slope s (1 - s) = e / (1 + e)^2 with e = exp(-|z|): 1 - s would keep few bits
// where s is near 1.
__device__ __forceinline__ float sigmoid_slope(float z) {
  const float e = expf(-fabsf(z)), d = 1.0f / (1.0f + e);
  return e * d * d;
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
// largest key (softmax) or the sum of its two largest (sigmoid).  Where a group
// is `span` = a power of two whole lanes, all groups are reduced at once by
// exchanges inside them; else one after the other.
template <int L, int V, bool kSig>
__device__ __forceinline__ uint64_t pick_groups(const uint32_t key[V], int per, int G, int top,
                                                int span) {
  const int lane = lane_id() % L, e0 = lane * V;
  constexpr int kSlots = 64 / L;  // lane l holds the scores of groups l, l + L, ..
  uint32_t score[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) score[i] = 0;
  auto score_of = [](uint32_t m, uint32_t m2) {
    return kSig && m2 ? ordered_bits(from_ordered(m) + from_ordered(m2)) : m;
  };
  if (span) {
    uint32_t m = 0, m2 = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      m2 = max(m2, min(m, key[j]));
      m = max(m, key[j]);
    }
    for (int d = 1; d < span; d <<= 1) {
      const uint32_t o = __shfl_xor(m, d), o2 = __shfl_xor(m2, d);
      m2 = max(max(m2, o2), min(m, o));
      m = max(m, o);
    }
    const uint32_t s = score_of(m, m2);
    // At most L groups here.
    const uint32_t mine = __shfl(s, (lane_id() & ~(L - 1)) + lane * span % L);
    score[0] = lane < G ? mine : 0;
  } else {
    for (int g = 0; g < G; ++g) {
      uint32_t m = 0, m2 = 0;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if ((e0 + j) / per == g) {
          m2 = max(m2, min(m, key[j]));
          m = max(m, key[j]);
        }
      const uint32_t M = row_max<L>(m);
      uint32_t s = M;
      if constexpr (kSig) {
        // The row's second key: the first holder of the largest gives its own second.
        const int first = row_first<L>(m == M);
        s = score_of(M, row_max<L>(lane == first ? m2 : m));
      }
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        if (lane + i * L == g) score[i] = s;
    }
  }
  uint64_t chosen = 0;
  for (int n = 0; n < top; ++n) {
    uint32_t m = score[0];
#pragma unroll
    for (int i = 1; i < kSlots; ++i) m = max(m, score[i]);
    const uint32_t M = row_max<L>(m);
    bool done = false;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int l = row_first<L>(score[i] == M && M);
      if (!done && l >= 0) {
        done = true;
        chosen |= 1ull << (l + i * L);
        if (lane == l) score[i] = 0;
      }
    }
  }
  return chosen;
}

struct RouteRow {
  const float* bias;
  int E, k, groups, top_groups, span;
  bool renorm;
  float scale;
};

// The options of a row by L lanes of V experts each.
inline RouteRow route_row_of(int64_t E, int32_t k, const spgemm_route_options& o,
                             const float* bias, int width) {
  RouteRow a{};
  a.bias = bias;
  a.E = (int)E;
  a.k = k;
  a.groups = o.groups ? o.groups : 1;
  a.top_groups = o.top_groups ? o.top_groups : a.groups;
  if (a.top_groups == a.groups) a.groups = 1;  // every group is chosen
  a.renorm = !o.no_renormalise;
  const int64_t per = E / a.groups, lanes = per / width;
  if (per % width == 0 && (lanes & (lanes - 1)) == 0) a.span = (int)lanes;
  a.scale = o.scale != 0.0f ? o.scale : 1.0f;
  return a;
}

// Checks what a row of logits does not say (in k_route.hip).
spgemm_status check_route_options(int64_t E, int32_t k, const spgemm_route_options* o);

// store(i, column, weight) is called for every slot i < k by one lane.  `cols` is
// LDS of 2 k words for the row.  z is minus infinity where there is no expert and
// in a row that is not routed.
template <int L, int V, bool kSig, typename Store>
__device__ __forceinline__ void route_row(const RouteRow& a, const float (&z)[V], uint32_t* cols,
                                          Store store) {
  const int lane = lane_id() % L, e0 = lane * V;
  uint32_t key[V];
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
    const uint32_t M = row_max<L>(m);
    top = M ? from_ordered(M) : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (key[j]) total += expf(z[j] - top);
    total = row_sum<L>(total);
  }
  if (a.groups > 1) {
    const int per = a.E / a.groups;
    const uint64_t chosen = pick_groups<L, V, kSig>(key, per, a.groups, a.top_groups, a.span);
    if (a.span) {  // a lane's experts are of one group
      const bool keep = e0 < a.E && (chosen >> (e0 / per)) & 1;
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = keep ? key[j] : 0;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (e0 + j < a.E && !((chosen >> ((e0 + j) / per)) & 1)) key[j] = 0;
    }
  }
  uint32_t taken = 0;  // bit j: expert e0 + j is picked
  for (int n = 0; n < a.k; ++n) {
    uint32_t m = key[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = max(m, key[j]);
    const uint32_t M = row_max<L>(m);
    if (L == 64 && !M) break;
    if (M && lane == row_first<L>(m == M)) {
      uint32_t bits = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) bits |= (key[j] == M ? 1u : 0u) << j;
      bits &= -bits;
      taken |= bits;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if ((bits >> j) & 1) key[j] = 0;
    }
  }
  // Pack the picks: those of lower lanes first, then of lower experts.
  float* zs = (float*)(cols + a.k);
  const int mine = __popc(taken), before = row_excl_scan<L>(mine);
  int at = before;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if ((taken >> j) & 1) {
      cols[at] = e0 + j;
      zs[at] = z[j];
      ++at;
    }
  const int count = __shfl(before + mine, (lane_id() & ~(L - 1)) + L - 1);
  __builtin_amdgcn_wave_barrier();  // one wave's LDS accesses are performed in order
  // Weights: entry i of the row in lane i % L.
  constexpr int kMost = 64 / L;
  float w[kMost], sum = 0.0f;
  if (!kSig && a.renorm) {
    uint32_t m = 0;
#pragma unroll
    for (int n = 0; n < kMost; ++n)
      if (lane + n * L < count) m = max(m, ordered_bits(zs[lane + n * L]));
    const uint32_t M = row_max<L>(m);
    top = M ? from_ordered(M) : 0.0f;
  }
#pragma unroll
  for (int n = 0; n < kMost; ++n) {
    w[n] = 0.0f;
    if (lane + n * L < count) {
      const float x = zs[lane + n * L];
      w[n] = kSig ? sigmoid(x) : expf(x - top);
      sum += w[n];
    }
  }
  if (a.renorm) {
    total = row_sum<L>(sum);
    if (kSig) total += 1e-20f;
  } else if (kSig) {
    total = 1.0f;
  }
#pragma unroll
  for (int n = 0; n < kMost; ++n) {
    const int i = lane + n * L;
    if (i < a.k) store(i, i < count ? (int)cols[i] : -1, i < count ? w[n] / total * a.scale : 0.0f);
  }
}

}  // namespace sg
