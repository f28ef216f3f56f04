// A whole expert layer for a few tokens, in two launches: the router's logits,
// then everything else.
//
// Up to 16 tokens are the 16 columns of a 16x16x32 MFMA, so every expert that any
// token picked is one tile of rows, whichever tokens those are: its weights are
// read once, straight from memory to registers, and bound the layer.
//
// The logits: a work group to an expert; sums in 64 bits, so that the choice among
// close experts does not depend on their order.
//
// The rest is one launch.  Every work group routes all tokens itself (a wave to a
// token, up to two of them each), which costs less than waiting for another to do
// it.  Then work groups take numbers from a counter: first the tiles of W_in, whose
// results go to memory, then those of W_out, which wait until all the former are
// there, their first weights already loaded.  A work group waits only for numbers
// below its own, whose holders run and never wait for higher ones: however few work
// groups are on the chip at a time, every wait ends.
#include <algorithm>
#include <type_traits>

#include "route_row.hpp"
#include "rows8.hpp"

namespace sg {
namespace {

constexpr int kTokens = 16;  // columns of a tile
constexpr int kNT = 512, kWaves = kNT / kWave;
constexpr int kStep = 64;    // K of one step: 16 for each quarter of a wave
constexpr int kBlock = 128;  // rows and columns that share a scale

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma16(__bf16, s16x8 a, s16x8 b, f32x4 c) {
  typedef __bf16 v8 __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a),
                                                 __builtin_bit_cast(v8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(_Float16, s16x8 a, s16x8 b, f32x4 c) {
  typedef _Float16 v8 __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a),
                                                __builtin_bit_cast(v8, b), c, 0, 0, 0);
}

// ---- the router's logits ----

struct Counters {
  uint32_t ticket;  // the next tile's number
  uint32_t done;    // tiles of W_in whose results are in memory
};

struct LogitArgs {
  const void* x;
  int64_t x_ld;
  const void* router;  // E x D, fp32 or x's type
  float* logits;       // T x E
  Counters* counters;
  int T, E, D;
  bool w32;
};

template <typename T, int TB>
__global__ __launch_bounds__(256) void k_step_logits(LogitArgs a) {
  __shared__ double part[TB][256];
  const int e = blockIdx.x;
  if (e == 0 && threadIdx.x == 0) *a.counters = Counters{0, 0};
  double acc[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) acc[t] = 0.0;
  for (int c = threadIdx.x * 8; c < a.D; c += 256 * 8) {
    const int64_t at = (int64_t)e * a.D + c;
    float w[8];
    if (a.w32) load8_any((const float*)a.router + at, a.D - c, w);
    else load8_any((const T*)a.router + at, a.D - c, w);
    float x[TB][8];
#pragma unroll
    for (int t = 0; t < TB; ++t)
      load8_any((const T*)a.x + min(t, a.T - 1) * a.x_ld + c, a.D - c, x[t]);
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[t] = fma((double)w[j], (double)x[t][j], acc[t]);
  }
#pragma unroll
  for (int t = 0; t < TB; ++t) part[t][threadIdx.x] = acc[t];
  __syncthreads();
  const int wave = threadIdx.x / kWave, l = lane_id();
  for (int t = wave; t < a.T; t += 256 / kWave) {
    double s = (part[t][l] + part[t][l + 64]) + (part[t][l + 128] + part[t][l + 192]);
    s = wave_sum(s);
    if (l == 0) a.logits[(int64_t)t * a.E + e] = (float)s;
  }
}

// ---- weights ----

// A lane's share of one step of its row: 16 values from k = 64 s + 16 (l / 16), at
// a uniform address plus the lane's offset.  16-bit weights are the operands as
// they are; 8-bit ones are decoded when used, exactly, to x's type.
template <typename T, bool k8>
struct Share {
  static constexpr int kBytes = 2;
  s16x8 v[2];
  __device__ void load(const char* base, uint32_t off) { __builtin_memcpy(v, base + off, 32); }
  // The n values that the row still has; zeros beyond.
  __device__ void load_end(const char* base, uint32_t off, int n) {
    const short* p = (const short*)(base + off);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j / 8][j % 8] = j < n ? p[j] : (short)0;
  }
  __device__ s16x8 half(int h) const { return v[h]; }
};

template <typename T>
struct Share<T, true> {
  static constexpr int kBytes = 1;
  uint32_t v[4];
  __device__ void load(const char* base, uint32_t off) { __builtin_memcpy(v, base + off, 16); }
  __device__ void load_end(const char* base, uint32_t off, int n) {
    const uint8_t* p = (const uint8_t*)(base + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * i + j < n) v[i] |= (uint32_t)p[4 * i + j] << (8 * j);
    }
  }
  __device__ s16x8 half(int h) const {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (__is_same(T, __bf16)) {
        r[2 * i] = __builtin_bit_cast(
            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * h + i], 1.0f, false));
        r[2 * i + 1] = __builtin_bit_cast(
            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * h + i], 1.0f, true));
      } else {
        r[2 * i] = __builtin_bit_cast(
            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * h + i], 1.0f, false));
        r[2 * i + 1] = __builtin_bit_cast(
            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * h + i], 1.0f, true));
      }
    }
    return __builtin_bit_cast(s16x8, r);
  }
};

struct LayerArgs {
  RouteRow row;
  const void* x;
  int64_t x_ld;
  const uint8_t* active;
  const void* w_in;
  const void* w_out;
  const float* in_scale;   // E x ceil(2F / 128) x ceil(D / 128), of 8-bit weights
  const float* out_scale;  // E x ceil(D / 128) x ceil(F / 128)
  const float* logits;
  Counters* counters;
  uint16_t* h;             // by entry t k + i, rows of h_ld
  void* y;
  int32_t* col;
  float* val;
  int T, D, F, h_ld;
  int most;                // experts that the tokens can pick together
  bool sigmoid;
};

// The rows of a tile of 8-bit weights lie in one or two rows of blocks: those below
// `edge` (an index into the tile) take the scale of the first.
struct Scales {
  const float* first;
  const float* second;
  int edge;
};
__device__ __forceinline__ Scales scales_of(const float* scale, int64_t expert, int row0, int rows,
                                            int cols) {
  const int per = (cols + kBlock - 1) / kBlock, r = row0 / kBlock;
  const int all = (rows + kBlock - 1) / kBlock;
  const float* p = scale + (expert * all + r) * per;
  return {p, r + 1 < all ? p + per : p, (r + 1) * kBlock - row0};
}

// acc += the products of one step's halves, times the scales of its rows.
template <typename T, bool k8>
__device__ __forceinline__ void multiply(const Share<T, k8>& w, const s16x8 (&x)[2],
                                         const Scales& sc, int block, f32x4& acc) {
  if constexpr (!k8) {
    acc = mfma16(T{}, w.half(0), x[0], acc);
    acc = mfma16(T{}, w.half(1), x[1], acc);
  } else {
    f32x4 p = {0, 0, 0, 0};
    p = mfma16(T{}, w.half(0), x[0], p);
    p = mfma16(T{}, w.half(1), x[1], p);
    const float s1 = sc.first[block], s2 = sc.second[block];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc[j] += ((lane_id() >> 4) * 4 + j < sc.edge ? s1 : s2) * p[j];
  }
}

template <typename T, bool k8, int V>
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(4, 4))) void k_step(
    LayerArgs a) {
  typedef Share<T, k8> W;
  extern __shared__ uint32_t lds[];
  const int k = a.row.k, n = a.T * k, E = a.row.E;
  int32_t* cols = (int32_t*)lds;                      // n
  float* vals = (float*)(cols + n);                   // n
  uint32_t* packed = (uint32_t*)(vals + n);           // 2 k for each wave
  uint32_t* picked = packed + kWaves * 2 * k;         // a bit for each of 1024 experts
  uint16_t* expert = (uint16_t*)(picked + 32);        // picked experts, rising
  int16_t* slot = (int16_t*)(expert + (a.most + 1) / 2 * 2);  // slot of expert u's entry of token t, or -1
  __shared__ float part[kWaves][2][16][kTokens + 1];
  __shared__ uint32_t ticket;
  const int tid = threadIdx.x, l = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);

  if (tid == 0) ticket = __hip_atomic_fetch_add(&a.counters->ticket, 1u, __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT);
  if (tid < 32) picked[tid] = 0;
  for (int i = tid; i < a.most * kTokens; i += kNT) slot[i] = -1;
  for (int t = wave; t < a.T; t += kWaves) {
    float z[V];
    const bool on = !a.active || a.active[t];
#pragma unroll
    for (int j = 0; j < V; ++j)
      z[j] = on && l * V + j < E ? a.logits[(int64_t)t * E + l * V + j] : -INFINITY;
    auto store = [&](int i, int c, float v) {
      cols[t * k + i] = c;
      vals[t * k + i] = v;
      if (blockIdx.x == 0) {
        a.col[t * k + i] = c;
        a.val[t * k + i] = v;
      }
    };
    if (a.sigmoid) route_row<64, V, true>(a.row, z, packed + wave * 2 * k, store);
    else route_row<64, V, false>(a.row, z, packed + wave * 2 * k, store);
  }
  __syncthreads();
  for (int i = tid; i < n; i += kNT)
    if (cols[i] >= 0) atomicOr(&picked[cols[i] / 32], 1u << (cols[i] % 32));
  __syncthreads();
  // Place of expert e among the picked ones.
  auto rank_of = [&](int e) {
    int r = __popc(picked[e / 32] & ((1u << (e % 32)) - 1));
    for (int i = 0; i < e / 32; ++i) r += __popc(picked[i]);
    return r;
  };
  int used = 0;
  for (int i = 0; i < (E + 31) / 32; ++i) used += __popc(picked[i]);
  used = __builtin_amdgcn_readfirstlane(used);
  for (int i = tid; i < n; i += kNT) {
    if (cols[i] < 0) continue;
    const int u = rank_of(cols[i]);
    expert[u] = (uint16_t)cols[i];
    slot[u * kTokens + i / k] = (int16_t)(i % k);
  }
  __syncthreads();

  const int in_cols = (a.F + 15) / 16, out_cols = (a.D + 15) / 16;
  const uint32_t in_tiles = (uint32_t)used * in_cols, all = in_tiles + out_cols;
  const int quarter = l >> 4, column = l & 15;
  uint32_t tile = __builtin_amdgcn_readfirstlane(ticket);
  // The number of the tile after this one, taken early.
  auto take = [&]() {
    __syncthreads();  // `ticket` and `part` have been read
    if (tid == 0) ticket = __hip_atomic_fetch_add(&a.counters->ticket, 1u, __ATOMIC_RELAXED,
                                                  __HIP_MEMORY_SCOPE_AGENT);
  };
  while (tile < in_tiles) {
      take();
      // h of expert u's tokens, 16 columns.
      const int u = tile / in_cols, f0 = (int)(tile % in_cols) * 16;
      const int e = __builtin_amdgcn_readfirstlane(expert[u]);
      const int64_t row_bytes = (int64_t)a.D * W::kBytes;
      const char* gate = (const char*)a.w_in + ((int64_t)e * 2 * a.F + f0) * row_bytes;
      const char* up = gate + a.F * row_bytes;
      const uint32_t off =
          (uint32_t)min(column, a.F - 1 - f0) * (uint32_t)row_bytes + quarter * 16 * W::kBytes;
      Scales sg{}, su{};
      if constexpr (k8) {
        sg = scales_of(a.in_scale, e, f0, 2 * a.F, a.D);
        su = scales_of(a.in_scale, e, a.F + f0, 2 * a.F, a.D);
      }
      const T* x = (const T*)a.x + min(column, a.T - 1) * a.x_ld + quarter * 16;
      f32x4 g = {0, 0, 0, 0}, v = {0, 0, 0, 0};
      const int full = a.D / kStep;
      int s = wave;
      // B steps at once.
      auto batches = [&](auto count) {
        constexpr int B = decltype(count)::value;
        for (; s + (B - 1) * kWaves < full; s += B * kWaves) {
          W w1[B], w2[B];
          s16x8 xf[B][2];
#pragma unroll
          for (int i = 0; i < B; ++i) {
            const int64_t at = (int64_t)s * (kStep * W::kBytes) + i * kWaves * kStep * W::kBytes;
            w1[i].load(gate + at, off);
            w2[i].load(up + at, off);
          }
#pragma unroll
          for (int i = 0; i < B; ++i) __builtin_memcpy(xf[i], x + (s + i * kWaves) * kStep, 32);
          __builtin_amdgcn_sched_barrier(0);  // all loads before the first product
#pragma unroll
          for (int i = 0; i < B; ++i) {
            const int block = (s + i * kWaves) * kStep / kBlock;
            multiply<T, k8>(w1[i], xf[i], sg, block, g);
            multiply<T, k8>(w2[i], xf[i], su, block, v);
          }
        }
      };
      batches(std::integral_constant<int, 4>{});
      batches(std::integral_constant<int, 2>{});
      batches(std::integral_constant<int, 1>{});
      if (full * kStep < a.D && wave == full % kWaves) {
        const int left = a.D - full * kStep - quarter * 16;
        W w;
        Share<T, false> xe;
        xe.load_end((const char*)(x + full * kStep), 0, left);
        w.load_end(gate + full * kStep * W::kBytes, off, left);
        multiply<T, k8>(w, xe.v, sg, full * kStep / kBlock, g);
        w.load_end(up + full * kStep * W::kBytes, off, left);
        multiply<T, k8>(w, xe.v, su, full * kStep / kBlock, v);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        part[wave][0][quarter * 4 + j][column] = g[j];
        part[wave][1][quarter * 4 + j][column] = v[j];
      }
      __syncthreads();
      // A pair of columns to a thread.
      const int t = tid / 8, c = tid % 8 * 2;
      const int i = t < a.T ? slot[u * kTokens + t] : -1;
      if (i >= 0 && f0 + c < a.h_ld) {
        uint32_t pair = 0;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float gs = 0.0f, us = 0.0f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            gs += part[w][0][c + q][t];
            us += part[w][1][c + q][t];
          }
          const float hv = f0 + c + q < a.F ? gs / (1.0f + expf(-gs)) * us : 0.0f;
          pair |= (uint32_t)__builtin_bit_cast(uint16_t, from_f32<T>(hv)) << (16 * q);
        }
        __hip_atomic_store((uint32_t*)(a.h + (int64_t)(t * k + i) * a.h_ld + f0 + c), pair,
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      // The stores are written through and done before the tile is counted.  A release
      // at this scope would also write the L2's other lines back.
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (tid == 0)
        __hip_atomic_fetch_add(&a.counters->done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      tile = __builtin_amdgcn_readfirstlane(ticket);
  }
  bool ready = false;  // all of h is there
  while (tile < all) {
      take();
      // 16 columns of y: the steps of all picked experts in one row, of which a
      // wave takes every eighth.
      const int n0 = (int)(tile - in_tiles) * 16;
      const int full = a.F / kStep;
      const int64_t row_bytes = (int64_t)a.F * W::kBytes;
      const uint32_t off =
          (uint32_t)min(column, a.D - 1 - n0) * (uint32_t)row_bytes + quarter * 16 * W::kBytes;
      auto rows_of = [&](int u) {
        const int e = __builtin_amdgcn_readfirstlane(expert[u]);
        return (const char*)a.w_out + ((int64_t)e * a.D + n0) * row_bytes;
      };
      // Step s of expert u; beyond the last one there is none.
      struct Place { int u, s; };
      auto settle = [&](Place& p) {
        while (p.s >= full && p.u < used) p.s -= full, ++p.u;
      };
      constexpr int kBatch = 8, kHalf = 4;
      auto fetch = [&](Place p, W (&w)[kBatch]) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          settle(p);
          const bool there = p.u < used;  // else the last one again
          w[i].load(rows_of(there ? p.u : used - 1) +
                        (int64_t)(there ? p.s : full - 1) * (kStep * W::kBytes), off);
          p.s += kWaves;
        }
      };
      auto wait = [&]() {
        if (ready) return;
        if (tid == 0)
          while (__hip_atomic_load(&a.counters->done, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) <
                 in_tiles)
            __builtin_amdgcn_s_sleep(1);
        __syncthreads();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        ready = true;
      };
      f32x4 sum = {0, 0, 0, 0};
      // The token's row of h for expert u, and its value; null where it did not pick it.
      struct Row { const uint16_t* h; float value; };
      auto row_of = [&](int u) {
        const int i = column < a.T ? slot[u * kTokens + column] : -1;
        const int entry = i < 0 ? 0 : column * k + i;
        return Row{i < 0 ? nullptr : a.h + (int64_t)entry * a.h_ld + quarter * 16, vals[entry]};
      };
      auto add = [&](const W& w, const s16x8 (&h)[2], const Row& r, int u, int s) {
        Scales sc{};
        if constexpr (k8)
          sc = scales_of(a.out_scale, __builtin_amdgcn_readfirstlane(expert[u]), n0, a.D, a.F);
        f32x4 acc = {0, 0, 0, 0};
        multiply<T, k8>(w, h, sc, s * kStep / kBlock, acc);
        // What a token did not pick adds nothing, whatever its weights hold.
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] += r.h ? r.value * acc[j] : 0.0f;
      };
      if (full && used) {
        W w[kBatch];
        Place at{0, wave};
        settle(at);
        fetch(at, w);
        __builtin_amdgcn_sched_barrier(0);
        wait();
        while (true) {
#pragma unroll
          for (int i0 = 0; i0 < kBatch; i0 += kHalf) {
            Place p[kHalf];
            Row r[kHalf];
            s16x8 h[kHalf][2];
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
              p[i] = at;
              r[i] = row_of(min(at.u, used - 1));
              h[i][0] = h[i][1] = s16x8{0, 0, 0, 0, 0, 0, 0, 0};
              if (r[i].h && at.u < used) __builtin_memcpy(h[i], r[i].h + at.s * kStep, 32);
              at.s += kWaves;
              settle(at);
            }
#pragma unroll
            for (int i = 0; i < kHalf; ++i)
              if (p[i].u < used) add(w[i0 + i], h[i], r[i], p[i].u, p[i].s);
          }
          if (at.u >= used) break;
          fetch(at, w);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        wait();
      }
      if (full * kStep < a.F)
        for (int u = wave; u < used; u += kWaves) {
          const int left = a.F - full * kStep - quarter * 16;
          W we;
          Share<T, false> he;
          const Row r = row_of(u);
          he.load_end((const char*)(r.h + full * kStep), 0, r.h ? left : 0);
          we.load_end(rows_of(u) + full * kStep * W::kBytes, off, left);
          add(we, he.v, r, u, full);
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) part[wave][0][quarter * 4 + j][column] = sum[j];
      __syncthreads();
      const int t = tid / 16, c = tid % 16;
      if (t < a.T && n0 + c < a.D) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) v += part[i][0][c][t];
        ((T*)a.y)[(int64_t)t * a.D + n0 + c] = from_f32<T>(v);
      }
      tile = __builtin_amdgcn_readfirstlane(ticket);
  }
}

// ---- host ----

constexpr int kGroups = 512;  // two to a compute unit

int64_t hidden_pitch(int64_t F) { return (F + 7) / 8 * 8; }

struct Work {
  Counters* counters;
  float* logits;
  uint16_t* h;
};
Work take_work(Carver& c, const spgemm_expert_step_desc& d) {
  Work w{};
  w.counters = c.take<Counters>(1);
  w.logits = c.take<float>(d.tokens * d.experts);
  w.h = c.take<uint16_t>(d.tokens * d.k * hidden_pitch(d.hidden));
  return w;
}

spgemm_status refuse(spgemm_status st, const char* msg) {
  set_thread_error(msg);
  return st;
}

spgemm_status check_desc(const spgemm_expert_step_desc* d) {
  if (!d) return refuse(SPGEMM_ERR_INVALID_ARG, "expert_step: null description");
  if (d->dtype != SPGEMM_BF16 && d->dtype != SPGEMM_F16)
    return refuse(SPGEMM_ERR_INVALID_ARG, "expert_step: x must be bf16 or fp16");
  if (d->weight_dtype != d->dtype && d->weight_dtype != SPGEMM_E4M3)
    return refuse(SPGEMM_ERR_INVALID_ARG, "expert_step: weights must be of x's type or e4m3");
  if (d->router_dtype != d->dtype && d->router_dtype != SPGEMM_F32)
    return refuse(SPGEMM_ERR_INVALID_ARG, "expert_step: the router must be fp32 or of x's type");
  if (d->tokens < 0 || d->tokens > kTokens)
    return refuse(SPGEMM_ERR_INVALID_ARG, "expert_step: tokens outside [0, 16]");
  if (d->width < 1 || d->hidden < 1 || d->x_ld < d->width)
    return refuse(SPGEMM_ERR_INVALID_ARG, "expert_step: empty width, or a row stride below it");
  if (d->width > 1 << 22 || d->hidden > 1 << 22 || d->x_ld >= 1 << 30)
    return refuse(SPGEMM_ERR_INDEX_OVERFLOW, "expert_step: a width above 2^22, or a stride of 2^30 or more");
  return check_route_options(d->experts, d->k, &d->route);
}

template <typename T>
void logits(const LogitArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.E), nt(256);
  if (a.T == 1) hipLaunchKernelGGL((k_step_logits<T, 1>), grid, nt, 0, s, a);
  else if (a.T <= 4) hipLaunchKernelGGL((k_step_logits<T, 4>), grid, nt, 0, s, a);
  else hipLaunchKernelGGL((k_step_logits<T, kTokens>), grid, nt, 0, s, a);
}

template <typename T, bool k8>
void layer(const LayerArgs& a, hipStream_t s) {
  const int n = a.T * a.row.k;
  const size_t lds = (2 * n + kWaves * 2 * a.row.k + 32) * 4 + (a.most + 1) / 2 * 4 +
                     (size_t)a.most * kTokens * 2;
  const int64_t tiles = (int64_t)a.most * ((a.F + 15) / 16) + (a.D + 15) / 16;
  const dim3 grid((unsigned)std::min<int64_t>(tiles, kGroups));
  if (a.row.E <= 256) hipLaunchKernelGGL((k_step<T, k8, 4>), grid, dim3(kNT), lds, s, a);
  else hipLaunchKernelGGL((k_step<T, k8, 16>), grid, dim3(kNT), lds, s, a);
}

}  // namespace
}  // namespace sg

using namespace sg;

extern "C" spgemm_status spgemm_expert_step_workspace(const spgemm_expert_step_desc* desc,
                                                      int64_t* bytes) {
  const spgemm_status st = check_desc(desc);
  if (st != SPGEMM_OK) return st;
  if (!bytes) return refuse(SPGEMM_ERR_INVALID_ARG, "expert_step: null size");
  Carver c(nullptr);
  take_work(c, *desc);
  *bytes = c.used;
  return SPGEMM_OK;
}

extern "C" spgemm_status spgemm_expert_step(
    const spgemm_expert_step_desc* desc, const void* dX, const void* dRouter, const float* dBias,
    const uint8_t* dActive, const void* dWIn, const float* dInScale, const void* dWOut,
    const float* dOutScale, void* dY, int32_t* dCol, float* dVal, void* dWork, int64_t work_bytes,
    void* stream) {
  const spgemm_status st = check_desc(desc);
  if (st != SPGEMM_OK || desc->tokens == 0) return st;
  const spgemm_expert_step_desc& d = *desc;
  const bool scaled = d.weight_dtype == SPGEMM_E4M3;
  if (!dX || !dRouter || !dWIn || !dWOut || !dY || !dCol || !dVal || !dWork ||
      (scaled && (!dInScale || !dOutScale)))
    return refuse(SPGEMM_ERR_INVALID_ARG, "expert_step: null array");
  Carver c(dWork);
  const Work w = take_work(c, d);
  if (work_bytes < c.used)
    return refuse(SPGEMM_ERR_INVALID_ARG, "expert_step: workspace too small");
  LogitArgs z{};
  z.x = dX;
  z.x_ld = d.x_ld;
  z.router = dRouter;
  z.logits = w.logits;
  z.counters = w.counters;
  z.T = (int)d.tokens;
  z.E = (int)d.experts;
  z.D = (int)d.width;
  z.w32 = d.router_dtype == SPGEMM_F32;
  LayerArgs a{};
  a.row = route_row_of(d.experts, d.k, d.route, dBias, d.experts <= 256 ? 4 : 16);
  a.sigmoid = d.route.sigmoid != 0;
  a.x = dX;
  a.x_ld = d.x_ld;
  a.active = dActive;
  a.w_in = dWIn;
  a.w_out = dWOut;
  a.in_scale = dInScale;
  a.out_scale = dOutScale;
  a.logits = w.logits;
  a.counters = w.counters;
  a.h = w.h;
  a.y = dY;
  a.col = dCol;
  a.val = dVal;
  a.T = z.T;
  a.D = z.D;
  a.F = (int)d.hidden;
  a.h_ld = (int)hidden_pitch(d.hidden);
  a.most = (int)std::min<int64_t>(d.experts, d.tokens * d.k);
  (void)hipGetLastError();  // an error that earlier calls left is not this one's
  const hipStream_t s = (hipStream_t)stream;
  if (d.dtype == SPGEMM_BF16) {
    logits<__bf16>(z, s);
    scaled ? layer<__bf16, true>(a, s) : layer<__bf16, false>(a, s);
  } else {
    logits<_Float16>(z, s);
    scaled ? layer<_Float16, true>(a, s) : layer<_Float16, false>(a, s);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SPGEMM_OK : refuse(SPGEMM_ERR_HIP, hipGetErrorString(e));
}
