// A whole expert layer for a few tokens, in two launches: the router's logits,
// then everything else.
//
// Up to 16 tokens are the 16 columns of a 16x16x32 MFMA, so every expert that any
// token picked is one tile of rows, whichever tokens those are: its weights are
// read once, straight from memory to registers, and bound the layer.
//
// The hidden vector is kept in two terms of x's type, the second being what the
// rounding to the first leaves: rounded once, its error would add to that of y's own
// rounding and make y 1.4 times as far off (1.5 and more for few entries).  The
// second products cost 1 us of 64 (5 tokens, 19 experts of 2040 x 1400 in 8 bits) and
// 16 of 135 (16 tokens, 55 experts of 2048 x 768).
//
// The logits: a work group to an expert and up to four tokens (16 tokens by one: 12 us
// for 128 experts of 2048, by four 5.5); sums in 64 bits, so that the choice among close
// experts does not depend on their order.
//
// The rest is one launch.  Every work group routes all tokens itself, which costs
// less than waiting for another to do it.  Then work groups take tiles of W_in by
// numbers from a counter; the results go to memory.  A work group that finds no
// number left goes on to its tiles of W_out, loads their first weights and waits
// until all results are there.  It waits only when every tile of W_in has been taken
// by a work group that runs and that waits for nothing: however few work groups
// are on the chip at a time, every wait ends.
//
// One token with 6 of 64 experts of 2048 x 1024 takes 30 us where a copy of its 76 MB
// takes 15: the logits' launch 3, routing and tables 6, W_in 11 (5 TB/s), the wait for
// the slowest result 3, W_out, whose weights are there by then, 5.  16 tokens with 55
// of 128 experts of 2048 x 768 take 144 to 150 us for 519 MB: W_in runs at 5.1 TB/s, W_out
// at 3.3: a step there has eight accesses of h to two of weights.  The unit of the vector
// memory path that takes the addresses is busy 71% of the whole kernel, the one that
// returns the data 85%, 60 of them waiting for the caches; neither the waits of the loop
// nor its addresses bound it (without conditions between steps, 32-bit addresses: 145
// against 144, side by side).
//
// route, the router's product and experts, the calls that this joins, take longer at 1, 4
// and 8 tokens and less at 2 and from 12 on, by up to 9% (12 tokens, 6 of 64 experts of
// 2048 x 1024: 126 against 133 us); they round the hidden vector once.  16 tokens are what
// the columns of a product hold.
//
// The hand-over of h below is written for gfx950's caches: stores of agent scope are
// written through and done once vmcnt is 0.  No other target has the products and
// conversions used here, so that the file is not built for one.
//
// A work group of 8 waves has a compute unit: two of them, with half the registers,
// spill or have half the loads on their way (W_in's tiles 16 against 11 us).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "route_row.hpp"
#include "rows8.hpp"

namespace sg {
namespace {

constexpr int kTokens = 16;  // columns of a tile
constexpr int kNT = 512, kWaves = kNT / kWave;
constexpr int kPitch = 20;   // of 16 floats in LDS
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
  const int e = blockIdx.x, t0 = (int)blockIdx.y * TB;
  if (e == 0 && t0 == 0 && threadIdx.x <= kDone) (&a.counters->ticket)[threadIdx.x].n = 0;
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
      load8_any((const T*)a.x + min(t0 + t, a.T - 1) * a.x_ld + c, a.D - c, x[t]);
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[t] = fma((double)w[j], (double)x[t][j], acc[t]);
  }
#pragma unroll
  for (int t = 0; t < TB; ++t) part[t][threadIdx.x] = acc[t];
  __syncthreads();
  const int wave = threadIdx.x / kWave, l = lane_id();
  for (int t = wave; t < TB && t0 + t < a.T; t += 256 / kWave) {
    double s = (part[t][l] + part[t][l + 64]) + (part[t][l + 128] + part[t][l + 192]);
    s = wave_sum(s);
    if (l == 0) a.logits[(int64_t)(t0 + t) * a.E + e] = (float)s;
  }
}

// ---- weights ----

// A lane's share of one step of its row: 16 values.  In step s lane l has those from
// k = 64 s + 16 (l / 16); one whose values reach past the end of K takes the last 16
// there are and drops those that other lanes have.
__device__ __forceinline__ int k_of(int s, int K) {
  return min(s * kStep + (lane_id() >> 4) * 16, K - 16);
}
__device__ __forceinline__ int dropped(int s, int K) {
  return min(s * kStep + (lane_id() >> 4) * 16 - k_of(s, K), 16);
}

// Loads at addresses that are no multiple of 4 bytes make a whole call 2.4 times as long
// (1025 x 1025 bfloat16 240 us, 1026 x 1026 98), so unless `even` the words that hold
// the values are loaded, all of which are at least in part the row's, and shifted
// when they are used.  16-bit values are the operands as they are; 8-bit ones are
// decoded when used, exactly, to x's type.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 any_u32x4 __attribute__((aligned(1)));
typedef u32x4 word_u32x4 __attribute__((aligned(4)));

// Without the first n of a word's values of kBytes, beginning with value `first`.
template <int kBytes>
__device__ __forceinline__ u32x4 without(u32x4 v, int first, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int gone = (n - first) * kBytes - 4 * i;  // bytes
    v[i] &= gone <= 0 ? ~0u : gone >= 4 ? 0u : ~0u << (8 * gone);
  }
  return v;
}
__device__ __forceinline__ u32x4 shifted(u32x4 v, uint32_t next, uint32_t off) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __builtin_amdgcn_alignbyte(i < 3 ? v[(i + 1) & 3] : next, v[i], off);
  return r;
}
// The words that begin at or before p and hold 16 values of kBytes: lo, hi where
// values have 2 bytes, and one more unless `even`.
template <int kBytes>
__device__ __forceinline__ void load_words(const char* p, bool even, u32x4& lo, u32x4& hi,
                                           uint32_t& more) {
  if (even) {
    lo = *(const any_u32x4*)p;
    if constexpr (kBytes == 2) hi = *(const any_u32x4*)(p + 16);
  } else {
    const uint32_t off = (uint32_t)(uintptr_t)p & 3;
    const char* q = p - off;
    lo = *(const word_u32x4*)q;
    if constexpr (kBytes == 2) hi = *(const word_u32x4*)(q + 16);
    more = *(const uint32_t*)(q + (off ? 16 * kBytes : 16 * kBytes - 4));
  }
}

template <typename T, bool k8>
struct Share {
  static constexpr int kBytes = 2;
  u32x4 lo, hi;
  uint32_t more;
  __device__ void load(const char* p, bool even) { load_words<2>(p, even, lo, hi, more); }
  // Of a load at a multiple of 4 bytes plus off.
  __device__ void shift(uint32_t off) {
    lo = shifted(lo, hi[0], off);
    hi = shifted(hi, more, off);
  }
  // Without the first n values.
  __device__ void drop(int n) {
    lo = without<2>(lo, 0, n);
    hi = without<2>(hi, 8, n);
  }
  __device__ s16x8 half(int h) const { return __builtin_bit_cast(s16x8, h ? hi : lo); }
};

template <typename T>
struct Share<T, true> {
  static constexpr int kBytes = 1;
  u32x4 lo;
  uint32_t more;
  __device__ void load(const char* p, bool even) {
    u32x4 none;
    load_words<1>(p, even, lo, none, more);
  }
  __device__ void shift(uint32_t off) { lo = shifted(lo, more, off); }
  __device__ void drop(int n) { lo = without<1>(lo, 0, n); }
  __device__ s16x8 half(int h) const {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t q = h ? lo[2 + i] : lo[i];
      if constexpr (__is_same(T, __bf16)) {
        r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, 1.0f, false));
        r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, 1.0f, true));
      } else {
        r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q, 1.0f, false));
        r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q, 1.0f, true));
      }
    }
    return __builtin_bit_cast(s16x8, r);
  }
};

// What the second term of the hidden vector is multiplied by.  fp16 has no steps below
// 2^-24: as it is, the second term of values below 2^-3 would lose bits, and below 2^-14
// all of them.  The largest one is 2^4, so that its units fit the type.
template <typename T>
constexpr float kRestUnit = __is_same(T, __bf16) ? 1.0f : 2048.0f;

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
  uint16_t* h;             // by entry t k + i, rows of h_ld; then what they leave of h
  void* y;
  int32_t* col;
  float* val;
  int T, D, F, h_ld;
  int most;                // experts that the tokens can pick together
  int cut;                 // parts that a tile of W_out cuts K into
  int xs_at, xs_ld;        // where the rows of x begin in LDS, and their pitch; 0: they are not there
  bool sigmoid;
  bool even_x, even_in, even_out;  // rows begin at multiples of 4 bytes
};

__device__ __forceinline__ uint32_t take_ticket(Counters* c) {
  return __hip_atomic_fetch_add(&c->ticket.n, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <typename T, bool k8, int L, int V>
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_step(
    StepArgs a) {
  typedef Share<T, k8> W;
  // 16 bytes: x is read from here by that, from offsets that the host aligns.
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  const int k = a.row.k, n = a.T * k, E = a.row.E;
  int32_t* cols = (int32_t*)lds;                      // n
  float* vals = (float*)(cols + n);                   // n
  uint32_t* packed = (uint32_t*)(vals + n);           // 2 k for each row routed at a time
  uint32_t* picked = packed + kNT / L * 2 * k;        // a bit for each of 1024 experts
  uint16_t* expert = (uint16_t*)(picked + 32);        // picked experts, rising
  int16_t* entry_of = (int16_t*)(expert + (a.most + 1) / 2 * 2);  // token t's for expert u, or -1
  float* value_of = (float*)(entry_of + a.most * kTokens);        // and its value
  uint16_t* xs = (uint16_t*)((char*)lds + a.xs_at);  // rows of x, as the lanes take them, if there is room
  __shared__ __attribute__((aligned(16))) float part[kWaves][4][16][kPitch];  // [][gate or up, rows][column][row]
  __shared__ float joined[2][kTokens][33];
  __shared__ uint32_t ticket[2];
  const int tid = threadIdx.x, l = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  // Takes the numbers: a thread of a wave that has no row to route unless all have.
  const bool taker = tid == kNT - kWave;

  // The second number is taken when every work group has surely taken its first.
  uint32_t mine[2] = {0, 0};
  if (taker) mine[0] = take_ticket(a.counters);
  if (tid < 32) picked[tid] = 0;
  for (int i = tid; i < a.most * kTokens; i += kNT) entry_of[i] = -1;
  if (a.xs_ld) {
    const int per = (a.D + kStep - 1) / kStep * (kStep / 8);  // eights of a row
    for (int i = tid; i < a.T * per; i += kNT) {
      const int t = i / per, c = i % per * 8, k0 = c / 16 * 16, at = min(k0, a.D - 16);
      const int n = k0 - at - c % 16;  // values that other lanes have
      *(u32x4*)(xs + t * a.xs_ld + c) =
          without<2>(*(const any_u32x4*)((const uint16_t*)a.x + t * a.x_ld + at + c % 16), 0, n);
    }
  }
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
  if (taker) ticket[0] = mine[0];
  __syncthreads();
  if (taker) mine[1] = take_ticket(a.counters);
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
    entry_of[u * kTokens + i / k] = (int16_t)i;
    value_of[u * kTokens + i / k] = vals[i];
  }
  __syncthreads();

  // Columns of y to a tile, and parts that its sums are cut into: see below.
  const int cut = a.cut, out_width = 16 / cut;
  const int in_cols = (a.F + 31) / 32;
  const uint32_t in_tiles = (uint32_t)used * in_cols;
  const int quarter = l >> 4, column = l & 15;
  uint32_t tile = __builtin_amdgcn_readfirstlane(ticket[0]);

  // ---- tiles of W_in: h of expert u's tokens, 32 columns ----
  // Each wave takes every eighth step.  Four steps of a wave are on their way: as soon
  // as one is used, the one four further on is loaded in its place, which at the end
  // of a tile is one of the next.
  if (tile < in_tiles) {
    constexpr int kRing = 4;
    const uint32_t row_bytes = (uint32_t)a.D * W::kBytes;
    const char* x = (const char*)((const T*)a.x + min(column, a.T - 1) * a.x_ld);
    const int steps = (a.D + kStep - 1) / kStep;
    const int rounds = (steps + kRing * kWaves - 1) / (kRing * kWaves);
    const int scale_cols = (a.D + kBlock - 1) / kBlock, scale_rows = (2 * a.F + kBlock - 1) / kBlock;
    struct Place {
      int u, f0, e;
      const char* rows[2];  // gate, up
    };
    auto place_of = [&](uint32_t tile) {
      Place p;
      p.u = tile / in_cols;
      p.f0 = (int)(tile % in_cols) * 32;
      p.e = __builtin_amdgcn_readfirstlane(expert[p.u]);
      p.rows[0] = (const char*)a.w_in + ((int64_t)p.e * 2 * a.F + p.f0) * row_bytes;
      p.rows[1] = p.rows[0] + (int64_t)a.F * row_bytes;
      return p;
    };
    // The lane's row of the first or second 16, from the tile's first.
    auto row_of = [&](const Place& p, int j) {
      return (uint32_t)min(16 * j + column, a.F - 1 - p.f0) * row_bytes;
    };
    const uint16_t* xl = xs + min(column, a.T - 1) * a.xs_ld + quarter * 16;
    struct Slot {
      W w[2][2];  // [gate, up][rows]
      Share<T, false> x;  // where it is not in LDS
      // Of 8-bit weights: 16 rows lie in one or two rows of blocks, whose scales lane
      // o + 2 j and lane 4 + o + 2 j hold.
      float scales;
    };
    Slot slots[kRing];
    auto load = [&](Slot& s, const Place& p, int step) {
      const int at = k_of(step, a.D);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int o = 0; o < 2; ++o)
          s.w[o][j].load(p.rows[o] + (row_of(p, j) + (uint32_t)at * W::kBytes), a.even_in);
      if (!a.xs_ld) s.x.load(x + at * 2, a.even_x);
      if constexpr (k8)
        if (l < 8) {
          const int row = (l & 1) * a.F + p.f0 + (l & 2) * 8 + (l & 4 ? 15 : 0);
          s.scales = a.in_scale[((int64_t)p.e * scale_rows + min(row, 2 * a.F - 1) / kBlock) * scale_cols +
                                step * kStep / kBlock];
        }
      __builtin_amdgcn_sched_barrier(0);
    };
    Place p = place_of(tile);
#pragma unroll
    for (int i = 0; i < kRing; ++i)
      if (wave + i * kWaves < steps) load(slots[i], p, wave + i * kWaves);
    if (taker) ticket[1] = mine[1];
    __syncthreads();
    uint32_t next = __builtin_amdgcn_readfirstlane(ticket[1]);
#pragma unroll 1
    while (true) {
      uint32_t later = 0;
      if (taker) later = take_ticket(a.counters);
      const bool more = next < in_tiles;
      const Place following = place_of(more ? next : tile);
      f32x4 acc[2][2];
#pragma unroll
      for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[o][j] = f32x4{0, 0, 0, 0};
      auto use = [&](Slot& s, int step) {
        const int at = k_of(step, a.D), n = dropped(step, a.D);
        const bool end = step * kStep + kStep > a.D;
        s16x8 xf[2];
        if (a.xs_ld) {
          xf[0] = *(const s16x8*)(xl + step * kStep);
          xf[1] = *(const s16x8*)(xl + step * kStep + 8);
        } else {
          if (!a.even_x) s.x.shift((uint32_t)(uintptr_t)(x + at * 2) & 3);
          if (end) s.x.drop(n);
          xf[0] = s.x.half(0), xf[1] = s.x.half(1);
        }
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            W& w = s.w[o][j];
            if (!a.even_in)
              w.shift(((uint32_t)(uintptr_t)p.rows[o] + row_of(p, j) + at * W::kBytes) & 3);
            if (end) w.drop(n);
            if constexpr (!k8) {
              acc[o][j] = mfma16(T{}, w.half(0), xf[0], acc[o][j]);
              acc[o][j] = mfma16(T{}, w.half(1), xf[1], acc[o][j]);
            } else {
              f32x4 q = {0, 0, 0, 0};
              q = mfma16(T{}, w.half(0), xf[0], q);
              q = mfma16(T{}, w.half(1), xf[1], q);
              auto scale = [&](int lane) {
                return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(s.scales), lane));
              };
              const float first = scale(o + 2 * j), second = scale(4 + o + 2 * j);
              const int edge = kBlock - (o * a.F + p.f0 + 16 * j) % kBlock;  // rows of the first block
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[o][j][i] += (quarter * 4 + i < edge ? first : second) * q[i];
            }
          }
      };
#pragma unroll 1
      for (int r = 0; r < rounds; ++r) {
        const bool last = r + 1 == rounds;
        Place from = p;
        if (last) from = following;
#pragma unroll
        for (int i = 0; i < kRing; ++i) {
          const int step = wave + (r * kRing + i) * kWaves;
          const int ahead = last ? wave + i * kWaves : step + kRing * kWaves;
          if (step < steps) use(slots[i], step);
          if ((!last || more) && ahead < steps) load(slots[i], from, ahead);
        }
      }
      // The waves' sums are joined and h is stored.
      {
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
          for (int j = 0; j < 2; ++j) *(f32x4*)&part[wave][2 * o + j][column][quarter * 4] = acc[o][j];
        if (taker) ticket[0] = later;
        __syncthreads();
        // Sums of gate and up: token, column.
        {
          const int t = tid / 32, c = tid % 32;
          float v[2] = {0.0f, 0.0f};
#pragma unroll 4
          for (int i = 0; i < kWaves; ++i)
#pragma unroll
            for (int o = 0; o < 2; ++o) v[o] += part[i][2 * o + c / 16][t][c % 16];
          joined[0][t][c] = v[0];
          joined[1][t][c] = v[1];
        }
        __syncthreads();
        // A pair of columns to a thread.
        const int t = tid / 16, c = tid % 16 * 2;
        const int i = t < a.T ? entry_of[p.u * kTokens + t] : -1;
        if (i >= 0 && p.f0 + c < a.h_ld) {
          uint32_t pair[2] = {0, 0};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float gs = joined[0][t][c + q], us = joined[1][t][c + q];
            const float hv = p.f0 + c + q < a.F ? gs / (1.0f + expf(-gs)) * us : 0.0f;
            const T first = from_f32<T>(hv);
            // Nothing is left of a value beyond the type, or y were inf - inf.
            const bool finite = fabsf(to_f32(first)) < INFINITY;
            const T rest = from_f32<T>(finite ? (hv - to_f32(first)) * kRestUnit<T> : 0.0f);
            pair[0] |= (uint32_t)__builtin_bit_cast(uint16_t, first) << (16 * q);
            pair[1] |= (uint32_t)__builtin_bit_cast(uint16_t, rest) << (16 * q);
          }
          uint32_t* to = (uint32_t*)(a.h + (int64_t)i * a.h_ld + p.f0 + c);
          __hip_atomic_store(to, pair[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __hip_atomic_store(to + (int64_t)n * a.h_ld / 2, pair[1], __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_AGENT);
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
      }
      if (!more) break;
      p = following;
    }
  }

  // ---- tiles of W_out: 16 / cut columns of y ----
  // A tile's 16 rows are `cut` parts of K of `width` columns of y, so that there are
  // tiles for every compute unit.  The 16 columns of a product are parts and tokens,
  // and only the products of equal parts are taken; where parts and tokens do not
  // fit 16 columns, a second product has the other half of the parts.  The steps
  // of all picked experts are one row, q being step q % per of expert q / per, and
  // part i of a wave's step takes the i-th of `cut` neighbours.
  const int out_tiles = (a.D + out_width - 1) / out_width;
  const int per = (a.F + kStep - 1) / kStep, steps = used * per;
  const int passes = cut * a.T > 16 ? 2 : 1, room = 16 * passes / cut;  // columns for tokens
  const int sub = column % out_width;  // as a row of the weights
  const int token = min(column % room, a.T - 1);  // as a column of h, some of which are not used
  struct Place { int u, s; };
  // Of kWaves * cut steps.
  const int ahead_u = kWaves * cut / per, ahead_s = kWaves * cut % per;
  auto advance = [&](Place& p) {
    p.u += ahead_u;
    p.s += ahead_s;
    if (p.s >= per) p.s -= per, ++p.u;
  };
  auto start_of = [&](int part) {
    const int q = wave * cut + part;
    return Place{q / per, q % per};
  };
  const int w_part = column / out_width, h_part = column / room;
  // Steps of this wave, the last of which may lack some parts.
  const int count = (steps - wave * cut + kWaves * cut - 1) / (kWaves * cut);
  const bool ragged = a.F % kStep != 0;
  const int64_t rest_at = (int64_t)n * a.h_ld;  // h's second terms, from its first
  bool ready = false;  // all of h is there
#pragma unroll 1
  for (int out = blockIdx.x; out < out_tiles; out += gridDim.x) {
    const int n0 = out * out_width;
    const char* rows = (const char*)a.w_out + (int64_t)min(n0 + sub, a.D - 1) * a.F * W::kBytes;
    const uint64_t expert_bytes = (uint64_t)a.D * a.F * W::kBytes;
    const int scale_cols = (a.F + kBlock - 1) / kBlock;
    const uint64_t scale_stride = (uint64_t)((a.D + kBlock - 1) / kBlock) * scale_cols;
    const float* scales = a.out_scale + n0 / kBlock * (int64_t)scale_cols;
    constexpr int kRing = 3;  // steps on their way
    struct Slot {
      W w;
      uint32_t off;  // of its address, from a multiple of 4 bytes
      int drop;
    };
    struct Hidden {
      Share<T, false> h, rest;
      float value;  // of the token for the step's expert
      float scale;  // of 8-bit weights: that of the column's part, whose products count
      int drop;     // or -1: what it did not pick adds nothing, whatever its weights hold
    };
    Slot w[kRing];
    Hidden h[2][kRing];
    Place pw = start_of(w_part), ph[2] = {start_of(h_part), start_of(h_part + cut / 2)};
    auto load_w = [&](Slot& s) {
      const char* from = rows + expert[min(pw.u, used - 1)] * expert_bytes +
                         (uint32_t)(k_of(pw.s, a.F) * W::kBytes);
      s.w.load(from, a.even_out);
      s.off = (uint32_t)(uintptr_t)from & 3;
      s.drop = dropped(pw.s, a.F);
      advance(pw);
    };
    auto load_h = [&](Hidden& h, Place& p) {
      const int u = min(p.u, used - 1), at = u * kTokens + token;
      const int i = entry_of[at];
      const bool there = i >= 0 && p.u < used;
      h.value = value_of[at];
      h.drop = there ? dropped(p.s, a.F) : -1;
      if constexpr (k8)
        h.scale = scales[expert[u] * scale_stride + (uint32_t)(p.s * kStep / kBlock)];
      // Rows that are not there are read as those of entry 0, and not used.
      const uint16_t* from = a.h + (uint64_t)(uint32_t)max(i, 0) * (uint32_t)a.h_ld + (uint32_t)k_of(p.s, a.F);
      h.h.load((const char*)from, true);
      h.rest.load((const char*)(from + rest_at), true);
      advance(p);
    };
    auto load_both = [&](int i) {
      load_h(h[0][i], ph[0]);
      if (passes == 2) load_h(h[1][i], ph[1]);
    };
    f32x4 sum[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    auto add = [&](const W& w, Hidden& h, f32x4& sum) {
      if (ragged && __ballot(h.drop > 0)) h.h.drop(h.drop), h.rest.drop(h.drop);
      f32x4 acc = {0, 0, 0, 0};
      acc = mfma16(T{}, w.half(0), h.rest.half(0), acc);
      acc = mfma16(T{}, w.half(1), h.rest.half(1), acc);
      if constexpr (kRestUnit<T> != 1.0f)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] *= 1.0f / kRestUnit<T>;
      acc = mfma16(T{}, w.half(0), h.h.half(0), acc);
      acc = mfma16(T{}, w.half(1), h.h.half(1), acc);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        sum[j] += h.drop >= 0 ? (k8 ? h.value * h.scale : h.value) * acc[j] : 0.0f;
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i)
      if (i < count) load_w(w[i]);
    __builtin_amdgcn_sched_barrier(0);
    if (!ready) {
      // One wave acquires for all: each invalidation of the caches holds the others up,
      // 15 us where all eight waves of 256 work groups made one.
      if (wave == 0) {
        while (true) {
          uint32_t c = 0;
          if (l < kDone)
            c = __hip_atomic_load(&a.counters->done[l].n, __ATOMIC_RELAXED,
                                  __HIP_MEMORY_SCOPE_AGENT);
          if (wave_sum(c) >= in_tiles) break;
          __builtin_amdgcn_s_sleep(4);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      }
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int i = 0; i < kRing; ++i)
      if (i < count) load_both(i);
    __builtin_amdgcn_sched_barrier(0);
    auto use = [&](int i) {
      if (!a.even_out) w[i].w.shift(w[i].off);
      // Only the last step of an expert has values to drop.
      if (ragged && __ballot(w[i].drop > 0)) w[i].w.drop(w[i].drop);
      add(w[i].w, h[0][i], sum[0]);
      if (passes == 2) add(w[i].w, h[1][i], sum[1]);
    };
#pragma unroll 1
    for (int j = 0; j < count; j += kRing) {
#pragma unroll
      for (int i = 0; i < kRing; ++i) {
        if (j + i < count) use(i);
        if (j + i + kRing < count) {
          load_w(w[i]);
          load_both(i);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();  // `part` of the tile before has been read
#pragma unroll
    for (int i = 0; i < 2; ++i) *(f32x4*)&part[wave][i][column][quarter * 4] = sum[i];
    __syncthreads();
    const int t = tid / out_width, c = tid % out_width;
    if (t < a.T && n0 + c < a.D) {
      float v = 0.0f;
      const int parts = cut / passes;  // of a product
#pragma unroll 1
      for (int i = 0; i < cut; ++i)
#pragma unroll 4
        for (int w = 0; w < kWaves; ++w)
          v += part[w][i / parts][i % parts * room + t][i * out_width + c];
      ((T*)a.y)[(int64_t)t * a.D + n0 + c] = from_f32<T>(v);
    }
  }
}

// ---- host ----

constexpr int kGroups = 256;  // one to a compute unit
// Dynamic LDS of a work group at most: what its static arrays leave.
constexpr size_t kMostLds = kLdsPerGroup - 46 * 1024;

int64_t hidden_pitch(int64_t F) { return (F + 7) / 8 * 8; }

struct Work {
  Counters* counters;
  float* logits;
  uint16_t* h;
};
Work take_work(Carver& c, const spgemm_expert_step_desc& d) {
  Work w{};
  w.logits = c.take<float>(d.tokens * d.experts);
  w.h = c.take<uint16_t>(2 * d.tokens * d.k * hidden_pitch(d.hidden));
  w.counters = c.take<Counters>(1);
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
  if (d->width < 16 || d->hidden < 16 || d->x_ld < d->width)
    return refuse(SPGEMM_ERR_INVALID_ARG, "expert_step: a width below 16, or a row stride below the width");
  if (d->width > 1 << 20 || d->hidden > 1 << 20 || d->x_ld >= 1 << 30)
    return refuse(SPGEMM_ERR_INDEX_OVERFLOW, "expert_step: a width above 2^20, or a stride of 2^30 or more");
  return check_route_options(d->experts, d->k, &d->route);
}

template <typename T>
void logits(const LogitArgs& a, hipStream_t s) {
  if (a.T == 1)
    hipLaunchKernelGGL((k_step_logits<T, 1>), dim3((unsigned)a.E), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_step_logits<T, 4>), dim3((unsigned)a.E, (unsigned)((a.T + 3) / 4)),
                       dim3(256), 0, s, a);
}

template <typename T, bool k8>
void layer(StepArgs a, hipStream_t s) {
  const int n = a.T * a.row.k;
  const int64_t tiles =
      std::max((int64_t)a.most * ((a.F + 31) / 32), ((int64_t)a.D + 16 / a.cut - 1) / (16 / a.cut));
  const dim3 grid((unsigned)std::min<int64_t>(tiles, kGroups));
  const int rows = a.row.E <= 256 ? kNT / 16 : kWaves;  // routed at a time
  size_t lds = (2 * n + rows * 2 * a.row.k + 32) * 4 + (a.most + 1) / 2 * 4 +
               (size_t)a.most * kTokens * 6;
  // The rows of x, where they fit: an access of 16 bytes takes the vector memory path a
  // cycle, and those of x half as many again as 8-bit weights (8 tokens, 34 experts of
  // 2048 x 1408: W_in 69 -> 48 us).  8 more values to a row spread its columns over
  // the banks.
  const int ld = (a.D + kStep - 1) / kStep * kStep + 8;
  const size_t at = (lds + 15) / 16 * 16, rows_bytes = (size_t)a.T * ld * 2;
  if (at + rows_bytes <= kMostLds) {
    a.xs_at = (int)at;
    a.xs_ld = ld;
    lds = at + rows_bytes;
  }
  const int row_kind = a.row.E <= 64 ? 0 : a.row.E <= 128 ? 1 : a.row.E <= 256 ? 2 : 3;
  static std::atomic<uint64_t> allowed[4] = {};  // by kernel: devices whose LDS limit is set
  auto launch = [&](auto kernel) {
    int device = 0;
    // After a failure nothing more is launched, and setting the limit, which leaves
    // the error state clear, does not lose it: the caller's last look reports it.
    if (hipPeekAtLastError() != hipSuccess || hipGetDevice(&device) != hipSuccess) return;
    const uint64_t bit = 1ull << (device & 63);
    if (!(allowed[row_kind].load() & bit)) {
      allow_max_dynamic_lds((const void*)kernel);
      allowed[row_kind].fetch_or(bit);
    }
    hipLaunchKernelGGL(kernel, grid, dim3(kNT), lds, s, a);
  };
  switch (row_kind) {
    case 0: return launch(k_step<T, k8, 16, 4>);
    case 1: return launch(k_step<T, k8, 16, 8>);
    case 2: return launch(k_step<T, k8, 16, 16>);
    default: return launch(k_step<T, k8, 64, 16>);
  }
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
  if ((uintptr_t)dWork % 4)  // its counters and h are accessed by atomic operations
    return refuse(SPGEMM_ERR_INVALID_ARG, "expert_step: workspace not at a multiple of 4 bytes");
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
  a.row = route_row_of(d.experts, d.k, d.route, dBias, d.experts <= 64 ? 4 : d.experts <= 128 ? 8 : 16);
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
  const int64_t wb = scaled ? 1 : 2;
  a.even_x = (uintptr_t)dX % 4 == 0 && d.x_ld % 2 == 0;
  a.even_in = (uintptr_t)dWIn % 4 == 0 && d.width * wb % 4 == 0;
  a.even_out = (uintptr_t)dWOut % 4 == 0 && d.hidden * wb % 4 == 0;
  // Parts as the tokens leave room for them in two products, so that the compute units
  // have the fewest columns to do one after the other.
  auto turns = [&](int64_t cut) { return ((d.width * cut + 15) / 16 + kGroups - 1) / kGroups; };
  a.cut = 1;
  for (int cut = 2; cut <= 16 && cut * a.T <= 2 * kTokens; cut *= 2)
    if (turns(cut) * a.cut < turns(a.cut) * cut) a.cut = cut;
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
