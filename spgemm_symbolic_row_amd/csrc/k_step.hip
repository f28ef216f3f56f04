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

// A line of memory to each: the chip makes one atomic operation on a line in about
// 11 ns.
constexpr int kDone = 8;
struct Counters {
  struct alignas(256) Line { uint32_t n; };
  Line ticket;       // the next tile's number
  Line done[kDone];  // tiles of W_in whose results are in memory, by number % kDone
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
  if (e == 0 && threadIdx.x <= kDone) (&a.counters->ticket)[threadIdx.x].n = 0;
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

struct StepArgs {
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
  int cut;                 // parts that a tile of W_out cuts K into
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

__device__ __forceinline__ uint32_t take_ticket(Counters* c) {
  return __hip_atomic_fetch_add(&c->ticket.n, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <typename T, bool k8, int L, int V>
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_step(
    StepArgs a) {
  typedef Share<T, k8> W;
  extern __shared__ uint32_t lds[];
  const int k = a.row.k, n = a.T * k, E = a.row.E;
  int32_t* cols = (int32_t*)lds;                      // n
  float* vals = (float*)(cols + n);                   // n
  uint32_t* packed = (uint32_t*)(vals + n);           // 2 k for each row routed at a time
  uint32_t* picked = packed + kNT / L * 2 * k;        // a bit for each of 1024 experts
  uint16_t* expert = (uint16_t*)(picked + 32);        // picked experts, rising
  int16_t* slot = (int16_t*)(expert + (a.most + 1) / 2 * 2);  // of expert u's entry of token t, or -1
  __shared__ float part[kWaves][4][16][kTokens + 1];
  __shared__ uint32_t ticket[2];
  const int tid = threadIdx.x, l = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  // Takes the numbers: a thread of a wave that has no row to route unless all have.
  const bool taker = tid == kNT - kWave;

  uint32_t mine[2] = {0, 0};
  if (taker) {
    mine[0] = take_ticket(a.counters);
    mine[1] = take_ticket(a.counters);
  }
  if (tid < 32) picked[tid] = 0;
  for (int i = tid; i < a.most * kTokens; i += kNT) slot[i] = -1;
  for (int t0 = 0; t0 < a.T; t0 += kNT / L) {
    const int t = t0 + tid / L, e0 = tid % L * V;
    if (t0 + wave * (kWave / L) >= a.T) break;  // the whole wave
    float z[V];
    const bool inside = t < a.T, on = inside && (!a.active || a.active[t]);
#pragma unroll
    for (int j = 0; j < V; ++j)
      z[j] = on && e0 + j < E ? a.logits[(int64_t)t * E + e0 + j] : -INFINITY;
    auto store = [&](int i, int c, float v) {
      if (!inside) return;
      cols[t * k + i] = c;
      vals[t * k + i] = v;
      if (blockIdx.x == 0) {
        a.col[t * k + i] = c;
        a.val[t * k + i] = v;
      }
    };
    if (a.sigmoid) route_row<L, V, true>(a.row, z, packed + tid / L * 2 * k, store);
    else route_row<L, V, false>(a.row, z, packed + tid / L * 2 * k, store);
  }
  if (taker) ticket[0] = mine[0], ticket[1] = mine[1];
  __syncthreads();
  for (int i = tid; i < n; i += kNT)
    if (cols[i] >= 0) atomicOr(&picked[cols[i] / 32], 1u << (cols[i] % 32));
  __syncthreads();
  int used = 0;
  for (int i = 0; i < (E + 31) / 32; ++i) used += __popc(picked[i]);
  used = __builtin_amdgcn_readfirstlane(used);
  for (int i = tid; i < n; i += kNT) {
    const int e = cols[i];
    if (e < 0) continue;
    // Its place among the picked ones.
    int u = __popc(picked[e / 32] & ((1u << (e % 32)) - 1));
    for (int j = 0; j < e / 32; ++j) u += __popc(picked[j]);
    expert[u] = (uint16_t)e;
    slot[u * kTokens + i / k] = (int16_t)(i % k);
  }
  __syncthreads();

  // Columns of y to a tile, and parts that its sums are cut into: see below.
  const int cut = a.cut, out_width = 16 / cut;
  const int in_cols = (a.F + 31) / 32;
  const uint32_t in_tiles = (uint32_t)used * in_cols;
  const uint32_t all = in_tiles + (a.D + out_width - 1) / out_width;
  const int quarter = l >> 4, column = l & 15;
  uint32_t tile = __builtin_amdgcn_readfirstlane(ticket[0]);
  uint32_t next = __builtin_amdgcn_readfirstlane(ticket[1]);

  // ---- tiles of W_in: h of expert u's tokens, 32 columns ----
  if (tile < in_tiles) {
    const int64_t row_bytes = (int64_t)a.D * W::kBytes;
    const T* x = (const T*)a.x + min(column, a.T - 1) * a.x_ld + quarter * 16;
    const int full = a.D / kStep;
    struct Place {
      int u, f0, e;
      const char* rows[2];  // gate, up
      uint32_t off[2];      // of the first and the second 16 rows
    };
    auto place_of = [&](uint32_t tile) {
      Place p;
      p.u = tile / in_cols;
      p.f0 = (int)(tile % in_cols) * 32;
      p.e = __builtin_amdgcn_readfirstlane(expert[p.u]);
      p.rows[0] = (const char*)a.w_in + ((int64_t)p.e * 2 * a.F + p.f0) * row_bytes;
      p.rows[1] = p.rows[0] + a.F * row_bytes;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        p.off[j] = (uint32_t)min(16 * j + column, a.F - 1 - p.f0) * (uint32_t)row_bytes +
                   quarter * 16 * W::kBytes;
      return p;
    };
    constexpr int kBatch = 4;
    W w[kBatch][2][2];  // [][gate, up][rows]
    s16x8 xf[kBatch][2];
    // Steps s, s + kWaves, ..; beyond the last one that again.
    auto load = [&](const Place& p, int s) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t at = min(s + i * kWaves, full - 1);
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            w[i][o][j].load(p.rows[o] + at * (kStep * W::kBytes), p.off[j]);
        __builtin_memcpy(xf[i], x + at * kStep, 32);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    Place p = place_of(tile);
    if (full) load(p, wave);
    // A tile's first loads are on their way while the one before it is joined.
    while (true) {
      uint32_t later = 0;
      if (taker) later = take_ticket(a.counters);
      Scales sc[2][2]{};
      if constexpr (k8) {
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            sc[o][j] = scales_of(a.in_scale, p.e, min(o * a.F + p.f0 + 16 * j, 2 * a.F - 1),
                                 2 * a.F, a.D);
      }
      f32x4 acc[2][2];
#pragma unroll
      for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[o][j] = f32x4{0, 0, 0, 0};
      for (int s = wave; s < full;) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int at = s + i * kWaves;
          if (at < full) {
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                multiply<T, k8>(w[i][o][j], xf[i], sc[o][j], at * kStep / kBlock, acc[o][j]);
          }
        }
        s += kBatch * kWaves;
        if (s < full) load(p, s);
      }
      if (full * kStep < a.D && wave == full % kWaves) {
        const int left = a.D - full * kStep - quarter * 16;
        Share<T, false> xe;
        xe.load_end((const char*)(x + full * kStep), 0, left);
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            W we;
            we.load_end(p.rows[o] + full * kStep * W::kBytes, p.off[j], left);
            multiply<T, k8>(we, xe.v, sc[o][j], full * kStep / kBlock, acc[o][j]);
          }
      }
      const bool more = next < in_tiles;
      const int u = p.u, f0 = p.f0;
      if (more) {
        p = place_of(next);
        if (full) load(p, wave);
      }
#pragma unroll
      for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[wave][2 * o + i][quarter * 4 + j][column] = acc[o][i][j];
      if (taker) ticket[0] = later;
      __syncthreads();
      // A pair of columns to a thread.
      const int t = tid / 16, c = tid % 16 * 2;
      const int i = t < a.T ? slot[u * kTokens + t] : -1;
      if (i >= 0 && f0 + c < a.h_ld) {
        uint32_t pair = 0;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float gs = 0.0f, us = 0.0f;
#pragma unroll
          for (int v = 0; v < kWaves; ++v) {
            gs += part[v][c / 16][c % 16 + q][t];
            us += part[v][2 + c / 16][c % 16 + q][t];
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
      const uint32_t after = __builtin_amdgcn_readfirstlane(ticket[0]);
      __syncthreads();
      if (tid == 0)
        __hip_atomic_fetch_add(&a.counters->done[tile % kDone].n, 1u, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
      tile = next;
      next = after;
      if (!more) break;
    }
  }

  // ---- tiles of W_out: 16 / cut columns of y ----
  // With T tokens only T of the 16 columns of a product are of use.  Where 2 T <= 16,
  // row r and column c of a tile stand for part r / width and c / width of K, so
  // that its 16 rows are `cut` parts of `width` rows of W_out and there are `cut`
  // times as many tiles; only the products of equal parts are taken.  The steps of
  // all picked experts are one row, q being step q % full of expert q / full, and
  // part i of a wave's step takes the i-th of `cut` neighbours.
  if (tile >= all) return;
  const int full = a.F / kStep, steps = used * full;
  const int sub = column % out_width, my_part = column / out_width;
  const float per = full ? 1.0f / (float)full : 0.0f;
  bool ready = false;  // all of h is there
  while (tile < all) {
    const int n0 = (int)(tile - in_tiles) * out_width, row = min(n0 + sub, a.D - 1);
    uint32_t later = 0;
    if (taker) later = take_ticket(a.counters);
    struct Place { int u, s; };
    auto place_of = [&](int q) {
      Place p;
      p.u = (int)((float)q * per);
      p.s = q - p.u * full;
      if (p.s < 0) --p.u, p.s += full;
      if (p.s >= full) ++p.u, p.s -= full;
      return p;
    };
    auto weights_at = [&](const Place& p) {
      return (const char*)a.w_out +
             (((int64_t)expert[p.u] * a.D + row) * a.F + p.s * kStep + quarter * 16) * W::kBytes;
    };
    constexpr int kBatch = 6, kHalf = 3;
    W w[2][kBatch];
    auto fetch = [&](int q, W (&w)[kBatch]) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        w[i].load(weights_at(place_of(min(q + i * kWaves * cut, steps - 1))), 0);
      __builtin_amdgcn_sched_barrier(0);
    };
    f32x4 sum = {0, 0, 0, 0};
    // The token's row of h for expert u, and its value; null where it did not pick it.
    struct Row { const uint16_t* h; float value; };
    auto row_of = [&](int u) {
      const int i = sub < a.T ? slot[u * kTokens + sub] : -1;
      const int entry = i < 0 ? 0 : sub * k + i;
      return Row{i < 0 ? nullptr : a.h + (int64_t)entry * a.h_ld + quarter * 16, vals[entry]};
    };
    // A lane's scale is that of its column's part, the only one whose products count.
    auto add = [&](const W& w, const s16x8 (&h)[2], const Row& r, const Place& p) {
      Scales sc{};
      float one = 1.0f;
      if constexpr (k8) {
        const int cols = (a.F + kBlock - 1) / kBlock, rows = (a.D + kBlock - 1) / kBlock;
        one = a.out_scale[((int64_t)expert[p.u] * rows + n0 / kBlock) * cols + p.s * kStep / kBlock];
      }
      f32x4 acc = {0, 0, 0, 0};
      acc = mfma16(T{}, w.half(0), h[0], acc);
      acc = mfma16(T{}, w.half(1), h[1], acc);
      // What a token did not pick adds nothing, whatever its weights hold.
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += r.h ? r.value * one * acc[j] : 0.0f;
    };
    auto use = [&](int q0, const W (&w)[kBatch]) {
#pragma unroll
      for (int i0 = 0; i0 < kBatch; i0 += kHalf) {
        Place p[kHalf];
        Row r[kHalf];
        s16x8 h[kHalf][2];
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
          const int q = q0 + (i0 + i) * kWaves * cut;
          p[i] = place_of(min(q, steps - 1));
          r[i] = row_of(p[i].u);
          if (q >= steps) r[i].h = nullptr;
          h[i][0] = h[i][1] = s16x8{0, 0, 0, 0, 0, 0, 0, 0};
          if (r[i].h) __builtin_memcpy(h[i], r[i].h + p[i].s * kStep, 32);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kHalf; ++i) add(w[i0 + i], h[i], r[i], p[i]);
      }
    };
    const int stride = kBatch * kWaves * cut;
    int q = wave * cut + my_part;
    if (steps) fetch(q, w[0]);
    if (wave * cut + stride < steps) fetch(q + stride, w[1]);
    if (!ready) {
      if (wave == 0)
        while (true) {
          uint32_t c = 0;
          if (l < kDone)
            c = __hip_atomic_load(&a.counters->done[l].n, __ATOMIC_RELAXED,
                                  __HIP_MEMORY_SCOPE_AGENT);
          if (wave_sum(c) >= in_tiles) break;
          __builtin_amdgcn_s_sleep(4);
        }
      __syncthreads();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      ready = true;
    }
    // The first part's place decides, for the whole wave.
    for (int q1 = wave * cut; q1 < steps; q1 += 2 * stride, q += 2 * stride) {
      use(q, w[0]);
      if (q1 + 2 * stride < steps) fetch(q + 2 * stride, w[0]);
      if (q1 + stride < steps) {
        use(q + stride, w[1]);
        if (q1 + 3 * stride < steps) fetch(q + 3 * stride, w[1]);
      }
    }
    if (full * kStep < a.F)
      for (int u0 = wave * cut; u0 < used; u0 += kWaves * cut) {
        const int u = min(u0 + my_part, used - 1), left = a.F - full * kStep - quarter * 16;
        W we;
        Share<T, false> he;
        Row r = row_of(u);
        if (u0 + my_part >= used) r.h = nullptr;
        he.load_end((const char*)(r.h + full * kStep), 0, r.h ? left : 0);
        we.load_end(weights_at(Place{u, full}), 0, left);
        add(we, he.v, r, Place{u, full});
      }
    __syncthreads();  // `part` and `ticket` of the tile before have been read
#pragma unroll
    for (int j = 0; j < 4; ++j) part[wave][0][quarter * 4 + j][column] = sum[j];
    if (taker) ticket[0] = later;
    __syncthreads();
    const int t = tid / out_width, c = tid % out_width;
    if (t < a.T && n0 + c < a.D) {
      float v = 0.0f;
      for (int i = 0; i < cut; ++i)
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += part[w][0][i * out_width + c][i * out_width + t];
      ((T*)a.y)[(int64_t)t * a.D + n0 + c] = from_f32<T>(v);
    }
    tile = next;
    next = __builtin_amdgcn_readfirstlane(ticket[0]);
  }
}

// ---- host ----

constexpr int kGroups = 256;  // one to a compute unit

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
  if (d->width > 1 << 20 || d->hidden > 1 << 20 || d->x_ld >= 1 << 30)
    return refuse(SPGEMM_ERR_INDEX_OVERFLOW, "expert_step: a width above 2^20, or a stride of 2^30 or more");
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
void layer(const StepArgs& a, hipStream_t s) {
  const int n = a.T * a.row.k;
  const int64_t tiles =
      (int64_t)a.most * ((a.F + 31) / 32) + (a.D + 16 / a.cut - 1) / (16 / a.cut);
  const dim3 grid((unsigned)std::min<int64_t>(tiles, kGroups));
  const int rows = a.row.E <= 256 ? kNT / 16 : kWaves;  // routed at a time
  const size_t lds = (2 * n + rows * 2 * a.row.k + 32) * 4 + (a.most + 1) / 2 * 4 +
                     (size_t)a.most * kTokens * 2;
  if (a.row.E <= 64) hipLaunchKernelGGL((k_step<T, k8, 16, 4>), grid, dim3(kNT), lds, s, a);
  else if (a.row.E <= 256) hipLaunchKernelGGL((k_step<T, k8, 16, 16>), grid, dim3(kNT), lds, s, a);
  else hipLaunchKernelGGL((k_step<T, k8, 64, 16>), grid, dim3(kNT), lds, s, a);
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
  StepArgs a{};
  a.row = route_row_of(d.experts, d.k, d.route, dBias, d.experts <= 64 ? 4 : 16);
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
  // Parts as the tokens leave room for them, while there are fewer tiles than work groups.
  a.cut = 1;
  while (2 * a.cut * a.T <= kTokens && (d.width + 15) / 16 * 2 * a.cut <= kGroups) a.cut *= 2;
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
