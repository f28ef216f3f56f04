// The experts' products.  With R the routing matrix (entries (t, e, w)), every
// entry is one row of a set of products grouped by expert:
//   g = W_gate[e] x_t,  u = W_up[e] x_t,  h = silu(g) * u,  y_t = sum_e w W_out[e] h
// and, given dy,
//   q = W_out[e]^T dy_t,  dw = <h, q>,  dh = w q,
//   dg = dh u s(g) (1 + g (1 - s(g))),  du = dh silu(g),
//   dx_t = sum_e W_in[e]^T [dg; du],  dW_in[e] = sum_t [dg; du] x_t^T,
//   dW_out[e] = sum_t dy_t (w h)^T.
//
// One kernel makes all six products.  A work group computes a BM x BN tile
// from K-slices of 64 staged in LDS; its four waves, one to a SIMD, multiply
// 32x32x16 MFMA blocks with fp32 accumulators.  At 256 x 256 a wave's part is
// 128 x 128: of a slice's 2048 cycles of products LDS reads and writes take
// 770, where eight waves of 128 x 64 would read half as much again; one wave to
// a SIMD issues at most an instruction in 4 cycles, so the loop is kept to 4
// instructions per 32-cycle product.  A slice takes about 2300 cycles (2800 in
// the weight gradients), the rest of a tile 15,000-20,000.  At 131,072 rows of
// 64 experts, 2048 x 1024, W_in's product runs at 1.1 PFLOP/s and 1.76 GHz with
// the matrix cores busy 67%; the clock falls under the load, and further as
// they are kept busier.  An operand tile lies in LDS in one of two forms, both
// filled by 16-byte global-to-LDS loads whose lane-linear destination is
// permuted by choosing the source address:
//   row form (K contiguous in memory): [row][64 k], 16-byte chunk c of row r
//     at slot c ^ (r >> 1 & 7); fragments are ds_read_b128.  With r & 7 the
//     reads run at 54% of the rate, without the xor at 14%.
//   column form (K strided): [k][column], the 32-byte segment s of row k at
//     segment s ^ 2 (k & 3); fragments are two transposing 8-byte reads.  With
//     (k & 3) | (k >> 3 & 1) << 2 they run at 50%, without the xor at 26%.
// K beyond its end is read from a block of zeros.  Rows that a tile has not are
// its last row again; what they give is not stored.
#include <algorithm>
#include <atomic>
#include <type_traits>
#include <utility>

#include "rows8.hpp"

namespace sg {
namespace {

constexpr int kBK = 64;    // K of one slice: a 128-byte line of a row
constexpr int kWaves = 4;  // 2 x 2, each a quarter of the tile
constexpr int kNT = kWaves * kWave;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_char;

// c += a b (32 x 32 x 16), c in accumulation registers.  Written out because
// the compiler, with 256 accumulators and two sets of fragments, moves
// accumulators between the register files inside the loop.  It does not know
// the instruction here, so the two wait states that a vector write of a, b or c
// needs before it are part of it, and settle() stands between the last one and
// reads of c.
//
// The forms with a load also send 64 lanes x 16 bytes from each lane's address
// to LDS, lane-linear from lds + at (uniform).  Nothing waits for such a load
// but wait_loads() and wait_slice(): the compiler, which would wait before the
// next LDS read, does not see it.  The product stands between the write of M0
// and the load, which must not follow at once.
#define SG_MFMA_FORMS(T, NAME)                                                                  \
  __device__ __forceinline__ void mfma(T, s16x8 a, s16x8 b, f32x16& c) {                        \
    asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_" NAME " %0, %1, %2, %0"                       \
                 : "+a"(c)                                                                      \
                 : "v"(a), "v"(b));                                                             \
  }                                                                                             \
  template <int kAt>                                                                            \
  __device__ __forceinline__ void mfma_load(T, s16x8 a, s16x8 b, f32x16& c, uint32_t lds,       \
                                            const void* p) {                                    \
    asm volatile("s_add_u32 m0, %3, %5\n\ts_nop 0\n\tv_mfma_f32_32x32x16_" NAME               \
                 " %0, %1, %2, %0\n\tglobal_load_lds_dwordx4 %4, off"                           \
                 : "+a"(c)                                                                      \
                 : "v"(a), "v"(b), "s"(lds), "v"(p), "n"(kAt)                                   \
                 : "memory", "scc");                                                            \
  }                                                                                             \
  template <int kAt>                                                                            \
  __device__ __forceinline__ void mfma_load(T, s16x8 a, s16x8 b, f32x16& c, uint32_t lds,       \
                                            const void* base, uint32_t off) {                   \
    asm volatile("s_add_u32 m0, %3, %6\n\ts_nop 0\n\tv_mfma_f32_32x32x16_" NAME               \
                 " %0, %1, %2, %0\n\tglobal_load_lds_dwordx4 %4, %5"                            \
                 : "+a"(c)                                                                      \
                 : "v"(a), "v"(b), "s"(lds), "v"(off), "s"(base), "n"(kAt)                      \
                 : "memory", "scc");                                                            \
  }
SG_MFMA_FORMS(__bf16, "bf16")
SG_MFMA_FORMS(_Float16, "f16")
#undef SG_MFMA_FORMS

template <int MT, int NT>
__device__ __forceinline__ void settle(f32x16 (&c)[MT][NT]) {
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) asm volatile("" : "+a"(c[m][n]));
}

// The load alone.
__device__ __forceinline__ void load_to_lds(uint32_t lds, const void* p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds),
               "v"(p)
               : "memory");
}
// All but the wave's last kLeft vector memory operations are done; then all
// waves' are.
template <int kLeft>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLeft) : "memory");
}
// The same, and the wave's LDS reads are done.
template <int kLeft>
__device__ __forceinline__ void wait_slice() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLeft) : "memory");
}

// 1 / (1 + exp(-g)) by the native base-2 exponential and reciprocal, each within an
// ulp (2^-23): with the rounding of the exponent (1.5 |g| 2^-24) and of the sum,
// within (5 + 1.5 |g|) 2^-24 of its value.  0 below g = -88, where the value is
// subnormal.
__device__ __forceinline__ float fast_sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * g));
}

// 1 / x of a power of two with exponent in [-126, 126].
__device__ __forceinline__ float inverse_power(float x) {
  return __uint_as_float((254u << 23) - __float_as_uint(x));
}

static __device__ __align__(16) const uint32_t zeros16[4] = {0, 0, 0, 0};

// ---- operand tiles ----
// Where a lane's share of a tile lies.  Load i of wave w fills bytes
// (i * kWaves + w) * 1024 .. of the tile, 16 for each lane.

// Row form: rows of kBK consecutive K; a load covers 8 rows.
struct RowForm {
  __device__ static int row(int i) {
    return (i * kWaves + (int)threadIdx.x / kWave) * 8 + lane_id() / 8;
  }
  __device__ static int k() { return ((lane_id() & 7) ^ ((row(0) >> 1) & 7)) * 8; }
  // Fragments: rows row0 + 32 m + lane % 32, k 16 kb + lane / 32 * 8 .. + 7.
  uint32_t at[4];  // by kb
  __device__ void frag_init(int row0) {
    const int l = lane_id();
#pragma unroll
    for (int kb = 0; kb < 4; ++kb)
      at[kb] = (row0 + (l & 31)) * (kBK * 2) + (((kb * 2 + (l >> 5)) ^ ((l >> 1) & 7)) * 16);
  }
  __device__ s16x8 frag(uint32_t lds, int m, int kb) const {
    return *(const __attribute__((address_space(3))) s16x8*)((const lds_char*)(lds + at[kb]) +
                                                             m * 32 * kBK * 2);
  }
};

// Column form: kBK k-rows of COLS columns.
template <int COLS>
struct ColForm {
  static constexpr int kRowBytes = COLS * 2;
  static constexpr int kRowsPerLoad = 1024 / kRowBytes;
  static_assert(kRowsPerLoad >= 1, "a load covers whole rows");
  __device__ static int f(int k) { return (k & 3) * 2; }
  __device__ static int row(int i) {
    return (i * kWaves + (int)threadIdx.x / kWave) * kRowsPerLoad + lane_id() * 16 / kRowBytes;
  }
  // First column of the lane's chunk, the same in every load.
  __device__ static int col() {
    const int c = lane_id() % (kRowBytes / 16);
    const int seg = c >> 1;
    return (((seg & ~7) | ((seg ^ f(row(0))) & 7)) * 2 + (c & 1)) * 8;
  }
  // Fragments: columns col0 + 32 m + lane % 32, k as in the row form.  A lane
  // gives the address of 4 columns of one k-row and gets 4 k of one column.
  uint32_t at[4];  // by m
  __device__ void frag_init(int col0) {
    const int l = lane_id(), k = (l >> 5) * 8 + ((l & 15) >> 2);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int seg = col0 / 16 + 2 * m + ((l >> 4) & 1);
      at[m] = k * kRowBytes + ((seg & ~7) | ((seg ^ f(k)) & 7)) * 32 + (l & 3) * 8;
    }
  }
  __device__ s16x8 frag(uint32_t lds, int m, int kb) const {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    lds_char* p = (lds_char*)(lds + at[m]) + kb * 16 * kRowBytes;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * kRowBytes));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// ---- the six products ----

enum Kind {
  kIn,        // [g, u] rows of x, W_in      -> h (and g, u)
  kOut,       // h, W_out                    -> rows of y before their sum
  kGradH,     // rows of dy, W_out           -> dg, du, w h, dw partial sums
  kGradX,     // [dg, du], W_in              -> rows of dx before their sum
  kGradWOut,  // dy^T, w h                   -> dW_out
  kGradWIn,   // [dg, du]^T, x               -> dW_in
};

struct ProductArgs {
  const void* a;  // left operand's rows (per entry or per token)
  const void* b;  // right operand: weights, or rows per entry or token
  int64_t lda, ldb;
  int64_t b_expert;  // elements between experts' weights
  Dispatch d;
  int E, M, N, K;    // M: rows of the result per expert (weight gradients)
  int Npad;          // readable columns of the right operand's rows
  int Mpad;
  int Kpad;
  int F, Fpad;
  void* c;           // 16-bit or fp32 result
  int64_t ldc, c_expert;
  float* g;          // fp32 pre-activations, Fpad to a row
  float* u;
  void* hw;          // w h
  float* dval_part;  // per entry: one partial sum of each wave's columns
  int parts;
  const float* size;   // by expert (kScaled): of the values (hidden gradient), or the unit of
                       // the rows that a weight gradient sums
  int k;               // slots of a row of the routing matrix
  const int32_t* col;  // and its entries, where they are taken unsorted
  const float* val;
};

// float16 ends at 2^-24 and 65504, where incoming gradients and values may be of
// any size, so [dg, du] and w h are held in units that are powers of two, undone
// in fp32 after the products:
//   [dg, du] for dx: the row's largest finite magnitude at 2^14 .. 2^15;
//   [dg, du] for dW_in, which sums over rows: that of the expert's largest row;
//   w h: |w| below 1 for the expert's largest.
// An element keeps 11 bits down to 2^-28 of that magnitude, and an error of 2^-39
// of it below.  bfloat16 has the range of fp32 and needs none.  The units of
// [dg, du] are known only when a row is done, so it passes through fp32: 8192
// tokens with 8 of 64 experts, 2048 x 1024, take 3541 us forward and backward,
// where bfloat16 takes 3085.
template <typename T>
constexpr bool kScaled = std::is_same<T, _Float16>::value;

constexpr int kFewRows = 16;  // rows of a tile of the few-rows products

// 8 values to p at once where it is aligned to them (vec) and n >= 8; else the
// first n one by one.
template <typename T>
__device__ __forceinline__ void store8(T* p, bool vec, int n, const float v[8]) {
  if (vec && n >= 8) {
    struct alignas(16) Pack { T v[16 / sizeof(T)]; };
    constexpr int V = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) {
      Pack q;
#pragma unroll
      for (int j = 0; j < V; ++j) q.v[j] = from_f32<T>(v[i * V + j]);
      ((Pack*)p)[i] = q;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = from_f32<T>(v[j]);
  }
}
__device__ __forceinline__ void load8(const float* p, float v[8]) {
  const f32x4 a = ((const f32x4*)p)[0], b = ((const f32x4*)p)[1];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = a[j], v[j + 4] = b[j];
}

template <typename T>
__device__ __forceinline__ void store4(T* p, bool vec, int n, const float v[4]) {
  if (vec && n >= 4) {
    struct alignas(4 * sizeof(T)) Pack { T v[4]; };
    Pack q;
#pragma unroll
    for (int j = 0; j < 4; ++j) q.v[j] = from_f32<T>(v[j]);
    *(Pack*)p = q;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) p[j] = from_f32<T>(v[j]);
  }
}

// Tile number `lin` -> row tile and column tile: groups of 8 row tiles by all
// column tiles, so that the work groups of one XCD, which take consecutive
// numbers, share rows and weights in its L2.
__device__ __forceinline__ void tile_at(int lin, int rows, int cols, int& tr, int& tc) {
  const int group = lin / (8 * cols), r = lin % (8 * cols);
  const int gr = min(8, rows - group * 8);
  tr = group * 8 + r % gr;
  tc = r / gr;
}

// What a work group needs to know about its tile.
struct Tile {
  int expert;
  int row0, rows;  // first sorted position and how many (weight gradients: the K)
  int m0, n0;      // first row (weight gradients) and column of the result
};

// Positions of the sorted token list that a weight gradient keeps in LDS.
constexpr int kListLen = 4096;

// Sum over kLanes = 8 or 16 consecutive lanes, in all of them.
template <int kLanes>
__device__ __forceinline__ float sum_of_lanes(float x) {
  x = dpp_add<0xb1, 0xf>(x);
  x = dpp_add<0x4e, 0xf>(x);
  x = dpp_add<0x141, 0xf>(x);
  if constexpr (kLanes == 16) x = dpp_add<0x140, 0xf>(x);  // row_mirror
  return x;
}

template <typename F, int... kI>
__device__ __forceinline__ void for_each_index(F& f, std::integer_sequence<int, kI...>) {
  (f(std::integral_constant<int, kI>{}), ...);
}
template <int kN, typename F>
__device__ __forceinline__ void for_each_index(F& f) {
  for_each_index(f, std::make_integer_sequence<int, kN>{});
}

// LDS stages of the operands.  160 KB hold five of 32 KB: the left operand
// has three, which gives its loads half a slice more.  A weight gradient
// keeps its token list there instead.
template <int KIND, int BM, int BN>
struct Stages {
  static constexpr bool kWGrad = KIND == kGradWOut || KIND == kGradWIn;
  static constexpr int kA = kWGrad ? 2 : 3, kB = !kWGrad && BM < BN ? 3 : 2;
};

// Whether a work group takes tiles in turn, or there is one for every tile.  In
// turn, at 64 experts of 2048 x 1024: the weight gradients 741 -> 638 us and 355
// -> 328 us (1024 rows to an expert, whose unequal shares are evened out), W_in's
// product 1108 -> 970-990 us (2048 rows); not the hidden gradient, whose loop leaves
// too few registers (434 -> 498 us).  dx's product (582 -> 596 us) and W_out's (362
// -> 352 us) hardly care.
template <int KIND>
constexpr bool kTurns = KIND == kIn || KIND == kGradWOut || KIND == kGradWIn;

// kFar: the gathered rows span 4 GB or more, so that their offsets are 64-bit
// pointers; those cost 7% of the main loop.
template <typename T, int KIND, int BM, int BN, bool kFar>
__global__ __launch_bounds__(kNT) __attribute__((amdgpu_waves_per_eu(1, 1))) void k_product(
    ProductArgs a) {
  constexpr int HM = BM / 2, HN = BN / 2, MT = HM / 32, NT = HN / 32;
  constexpr bool kWGrad = KIND == kGradWOut || KIND == kGradWIn;
  constexpr bool kACol = kWGrad, kBCol = kWGrad || KIND == kGradH || KIND == kGradX;
  constexpr bool kAGather = KIND == kIn || KIND == kGradH || KIND == kGradWOut;
  constexpr bool kBGather = KIND == kGradWIn;
  constexpr int kABytes = BM * kBK * 2, kBBytes = BN * kBK * 2;
  constexpr int AL = BM / 32, BL = BN / 32;  // loads of a wave per slice
  constexpr int AS = Stages<KIND, BM, BN>::kA, BS = Stages<KIND, BM, BN>::kB;
  constexpr int kNStep = KIND == kIn ? BN / 2 : BN;
  extern __shared__ char smem[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char*)smem;
  int32_t* list = (int32_t*)(smem + AS * kABytes + BS * kBBytes);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int wm = wave >> 1, wn = wave & 1, l = lane_id();

  const int cols = (a.N + kNStep - 1) / kNStep;
  const int row_tiles = kWGrad ? a.E * ((a.M + BM - 1) / BM) : *a.d.ntiles;
  // Work groups go round-robin to the XCDs: XCD x takes a contiguous share of
  // the tiles, and its work groups take them in turn.  The tiles of a weight
  // gradient cost their expert's rows, so there the shares are of rows, where
  // more tiles than work groups repay the look-ups (about 5 us).
  const int total = row_tiles * cols, xcd = (int)blockIdx.x % kXcds;
  auto share_start = [&](int x) {
    if (!kWGrad || total <= (int)gridDim.x)
      return min(total, x * ((total + kXcds - 1) / kXcds));
    if (x == 0) return 0;
    if (x == kXcds) return total;
    const int32_t* rp = a.d.row_ptr;
    const int64_t at = (int64_t)rp[a.E] * x / kXcds;
    const int64_t e = wave_last_le(rp, (int64_t)0, (int64_t)a.E, at);
    const int64_t rows = rp[e + 1] - rp[e], per = total / a.E;
    return (int)(e * per + (rows ? (at - rp[e]) * per / rows : 0));
  };
  const int last = __builtin_amdgcn_readfirstlane(share_start(xcd + 1));
  int lin = __builtin_amdgcn_readfirstlane(share_start(xcd)) + (int)blockIdx.x / kXcds;
#pragma unroll 1
  for (; lin < last; lin += (int)gridDim.x / kXcds) {
  if constexpr (kTurns<KIND>) __syncthreads();  // the last tile's rows have left LDS

  Tile t;
  {
    int tr, tc;
    tile_at(lin, row_tiles, cols, tr, tc);
    if constexpr (kWGrad) {
      const int mts = (a.M + BM - 1) / BM;
      t.expert = tr / mts;
      t.m0 = tr % mts * BM;
      t.row0 = a.d.row_ptr[t.expert];
      t.rows = a.d.row_ptr[t.expert + 1] - t.row0;
    } else {
      t.expert = a.d.tiles[2 * tr];
      t.row0 = a.d.tiles[2 * tr + 1];
      t.rows = min(BM, a.d.row_ptr[t.expert + 1] - t.row0);
      t.m0 = 0;
    }
    t.n0 = tc * kNStep;
  }
  const int K = kWGrad ? t.rows : a.K;
  const int steps = (K + kBK - 1) / kBK;

  // Operand addresses: uniform base of the next slice to load, and offsets in
  // bytes that stay; or, where rows are gathered, pointers.  Rows and columns
  // outside the result are clamped: what they give is not stored.  K outside
  // is read from zeros.
  const T* abase = (const T*)a.a;
  const T* bbase = (const T*)a.b + (kWGrad ? 0 : t.expert * a.b_expert);
  if constexpr (kWGrad && !kAGather) abase += (int64_t)t.row0 * a.lda;
  if constexpr (kWGrad && !kBGather) bbase += (int64_t)t.row0 * a.ldb;
  if constexpr (!kWGrad && !kAGather) abase += (int64_t)t.row0 * a.lda;
  RowForm ar, br;
  ColForm<BM> ac;
  ColForm<BN> bc;
  uint32_t aoff[AL], boff[BL];
  const char* aptr[AL];
  uint32_t aidx[AL], bidx[BL];  // tokens of the next slice to load (weight gradients)
  uint32_t acol = 0, bcol = 0;
  if constexpr (!kACol) {
#pragma unroll
    for (int i = 0; i < AL; ++i) {
      const int r = min(ar.row(i), t.rows - 1);
      const uint32_t at = kAGather ? a.d.tok[t.row0 + r] : r;
      if constexpr (kFar) aptr[i] = (const char*)(abase + (int64_t)at * a.lda + ar.k());
      else aoff[i] = (at * (uint32_t)a.lda + ar.k()) * 2;
    }
    ar.frag_init(wm * HM);
  } else {
    const int c = t.m0 + ac.col();
    acol = (c < a.Mpad ? c : 0) * 2;
#pragma unroll
    for (int i = 0; i < AL; ++i) {
      aoff[i] = (uint32_t)ac.row(i) * (uint32_t)a.lda * 2 + acol;
    }
    ac.frag_init(wm * HM);
  }
  if constexpr (!kBCol) {
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int r = br.row(i);
      int n;
      if constexpr (KIND == kIn) {
        // Each wave's columns: half gate rows, then the same rows of up.
        constexpr int H = HN / 2;
        n = min(t.n0 + r / HN * H + r % H, a.N - 1) + (r % HN < H ? 0 : a.N);
      } else {
        n = min(t.n0 + r, a.N - 1);
      }
      boff[i] = ((uint32_t)n * (uint32_t)a.ldb + br.k()) * 2;
    }
    br.frag_init(wn * HN);
  } else {
    const int c = t.n0 + bc.col();
    bcol = (c < a.Npad ? c : 0) * 2;
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      boff[i] = (uint32_t)bc.row(i) * (uint32_t)a.ldb * 2 + bcol;
    }
    bc.frag_init(wn * HN);
  }

  const char* acols = (const char*)abase + acol;  // gathered rows: the lane's columns
  const char* bcols = (const char*)bbase + bcol;
  // Address of load i of slice s.
  auto addr_a = [&](int s, int i) -> const char* {
    if constexpr (kWGrad && kAGather) return acols + (uint64_t)aidx[i] * ((uint32_t)a.lda * 2);
    else if constexpr (kFar) return aptr[i];
    else return (const char*)abase + aoff[i];
  };
  auto addr_b = [&](int s, int i) -> const char* {
    if constexpr (kBGather) return bcols + (uint64_t)bidx[i] * ((uint32_t)a.ldb * 2);
    else return (const char*)bbase + boff[i];
  };
  // Whether its K is inside.
  auto inside_a = [&](int s, int i) {
    return kACol ? s * kBK + ac.row(i) < K : s * kBK + ar.k() < a.Kpad;
  };
  auto inside_b = [&](int s, int i) {
    return kBCol ? s * kBK + bc.row(i) < K : s * kBK + br.k() < a.Kpad;
  };
  auto next_a = [&]() {
    if constexpr (kACol) {
      if constexpr (!kAGather) abase += (int64_t)kBK * a.lda;
    } else if constexpr (!kFar) {
      abase += kBK;  // far pointers move as they are used
    }
  };
  auto next_b = [&]() {
    if constexpr (kBCol) {
      if constexpr (!kBGather) bbase += (int64_t)kBK * a.ldb;
    } else {
      bbase += kBK;
    }
  };
  // The part of the token list that begins at slice s, and the tokens of
  // slice s from it.
  auto fill_list = [&](int s) {
    if constexpr (kWGrad) {
      __syncthreads();
      for (int i = threadIdx.x; i < min(kListLen, K - s * kBK); i += kNT)
        list[i] = a.d.tok[t.row0 + s * kBK + i];
      __syncthreads();
    }
  };
  // Tokens of half h of slice s.
  auto fetch_tokens = [&](int s, int h) {
    const int32_t* from = list + s * kBK % kListLen;
    if constexpr (kWGrad && kAGather) {
#pragma unroll
      for (int i = h * AL / 2; i < (h + 1) * AL / 2; ++i) aidx[i] = from[ac.row(i)];
    }
    if constexpr (kBGather) {
#pragma unroll
      for (int i = h * BL / 2; i < (h + 1) * BL / 2; ++i) bidx[i] = from[bc.row(i)];
    }
  };
  auto stage_a = [&](int s) { return lds0 + (uint32_t)(s % AS) * kABytes; };
  auto stage_b = [&](int s) { return lds0 + AS * kABytes + (uint32_t)(s % BS) * kBBytes; };
  auto frag_a = [&](uint32_t lds, int m, int kb) {
    if constexpr (kACol) return ac.frag(lds, m, kb);
    else return ar.frag(lds, m, kb);
  };
  auto frag_b = [&](uint32_t lds, int n, int kb) {
    if constexpr (kBCol) return bc.frag(lds, n, kb);
    else return br.frag(lds, n, kb);
  };

  f32x16 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[m][n][j] = 0.0f;

  if (steps > 0) {
    fill_list(0);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      fetch_tokens(s, 0);
      fetch_tokens(s, 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = h * AL / 2; i < (h + 1) * AL / 2; ++i)
          load_to_lds(stage_a(s) + (i * kWaves + wave) * 1024,
                      inside_a(s, i) ? (const void*)addr_a(s, i) : (const void*)zeros16);
#pragma unroll
        for (int i = h * BL / 2; i < (h + 1) * BL / 2; ++i)
          load_to_lds(stage_b(s) + (i * kWaves + wave) * 1024,
                      inside_b(s, i) ? (const void*)addr_b(s, i) : (const void*)zeros16);
      }
      if constexpr (kFar) {
#pragma unroll
        for (int i = 0; i < AL; ++i) aptr[i] += kBK * 2;
      }
      next_a();
      next_b();
    }
    fetch_tokens(2, 0);
    // A slice has two halves of 32 k.  Half 0 multiplies the fragments of its
    // own k, read before, and reads those of half 1.  Then the slice is no
    // longer needed in LDS, and the next one has to be there.  Half 1
    // multiplies its fragments and reads the next slice's first ones.  The
    // loads of the slice after that go into half 0 where the operand has a
    // third stage, into half 1 where it takes the place of this slice.  In a
    // weight gradient the halves of a slice are k-rows of their own, so each
    // takes the place of its like as soon as that has been read: four stages of
    // half a slice, with a barrier after either half.
    s16x8 fa[2][2][MT], fb[2][2][NT];  // [half][16 k of it][]
    wait_loads<AL + BL>();
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int n = 0; n < NT; ++n) fb[0][kb][n] = frag_b(stage_b(0), n, kb);
#pragma unroll
      for (int m = 0; m < MT; ++m) fa[0][kb][m] = frag_a(stage_a(0), m, kb);
    }
    // Half 0 of a weight gradient loads over what all waves have just read.
    if constexpr (kWGrad) wait_slice<AL + BL>();
    // LDS offsets of slices s, s + 1, s + 2.
    uint32_t la[3] = {stage_a(0), stage_a(1), stage_a(2)};
    uint32_t lb[3] = {stage_b(0), stage_b(1), stage_b(2)};
    // Loads of slice s + 2: all of it is there, its end has to be looked for,
    // or there is no such slice.
    enum { kInside, kChecked, kNone };
    auto half = [&](int s, auto which, auto loads) {
      constexpr int P = decltype(which)::value, Q = 1 - P;
      constexpr bool kCheck = decltype(loads)::value == kChecked;
      constexpr bool kAny = decltype(loads)::value != kNone;
      constexpr bool kLoadA = kAny && (kWGrad || (P == 0 ? AS == 3 : AS == 2));
      constexpr bool kLoadB = kAny && (kWGrad || (P == 0 ? BS == 3 : BS == 2));
      constexpr int kShare = kWGrad ? 2 : 1;
      constexpr int kLoadsA = kLoadA ? AL / kShare : 0;
      constexpr int kLoads = kLoadsA + (kLoadB ? BL / kShare : 0);
      // Tokens that the next half's loads need.
      if constexpr (kAny) {
        if constexpr (P == 0) fetch_tokens(s + 2, 1);
        else fetch_tokens(s + 3, 0);
      }
      const uint32_t ra = la[P], rb = lb[P];
      const uint32_t wa = la[2] + wave * 1024, wb = lb[2] + wave * 1024;
      constexpr int kAll = 2 * MT * NT, kReads = 2 * (MT + NT);
      // Products that reads and loads go between; a product takes one load at most.
      constexpr int kSpan = kAll * 3 / 4 > kLoads ? kAll * 3 / 4 : kLoads;
      static_assert(kSpan <= kAll, "a half has products for all its loads");
      auto step = [&](auto index) {
        constexpr int i = decltype(index)::value;
        constexpr int kb = i / (MT * NT), m = i / NT % MT, n = i % NT;
        constexpr int x = i * kLoads / kSpan;
        if constexpr (x < kLoads && x != (i + 1) * kLoads / kSpan) {
          constexpr bool kA = x < kLoadsA;
          constexpr int y = (kA ? x : x - kLoadsA) + (kWGrad ? P * (kA ? AL : BL) / 2 : 0);
          if constexpr (kCheck) {
            const char* p = kA ? addr_a(s + 2, y) : addr_b(s + 2, y);
            asm volatile("" : "+v"(p));  // both sides at hand: a select, no branch
            if (!(kA ? inside_a(s + 2, y) : inside_b(s + 2, y))) p = (const char*)zeros16;
            mfma_load<y * kWaves * 1024>(T{}, fb[P][kb][n], fa[P][kb][m], acc[m][n], kA ? wa : wb,
                                         p);
          } else if constexpr (kA ? kFar || (kACol && kAGather) : kBGather) {
            mfma_load<y * kWaves * 1024>(T{}, fb[P][kb][n], fa[P][kb][m], acc[m][n], kA ? wa : wb,
                                         kA ? addr_a(s + 2, y) : addr_b(s + 2, y));
          } else {
            mfma_load<y * kWaves * 1024>(T{}, fb[P][kb][n], fa[P][kb][m], acc[m][n], kA ? wa : wb,
                                         kA ? abase : bbase, kA ? aoff[y] : boff[y]);
          }
          if constexpr (kA && kFar) aptr[y] += kBK * 2;
        } else {
          mfma(T{}, fb[P][kb][n], fa[P][kb][m], acc[m][n]);
        }
#pragma unroll
        for (int z = i * kReads / kSpan; z < (i + 1) * kReads / kSpan && z < kReads; ++z) {
          const int k2 = z / (MT + NT), w = z % (MT + NT);
          if (w == 0) fa[Q][k2][0] = frag_a(ra, 0, 2 * Q + k2);
          else if (w <= NT) fb[Q][k2][w - 1] = frag_b(rb, w - 1, 2 * Q + k2);
          else fa[Q][k2][w - NT] = frag_a(ra, w - NT, 2 * Q + k2);
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      for_each_index<kAll>(step);
      if constexpr (kLoadA && (P == 1 || !kWGrad)) next_a();
      if constexpr (kLoadB && (P == 1 || !kWGrad)) next_b();
    };
    const int full = K / kBK;  // slices without an end of K
    auto slice = [&](int s, auto loads) {
      constexpr bool kAny = decltype(loads)::value != kNone;
      constexpr int kLeft =
          !kAny ? 0 : kWGrad ? AL + BL : (AS == 3 ? AL : 0) + (BS == 3 ? BL : 0);
      half(s, std::integral_constant<int, 0>{}, loads);
      wait_slice<kLeft>();
      if constexpr (kWGrad && kAny) {
        if (((s + 3) * kBK) % kListLen == 0) fill_list(s + 3);
      }
      half(s, std::integral_constant<int, 1>{}, loads);
      if constexpr (kWGrad) wait_slice<kLeft>();
      const uint32_t fa0 = AS == 3 ? la[0] : la[1], fb0 = BS == 3 ? lb[0] : lb[1];
      la[0] = la[1], la[1] = la[2], la[2] = fa0;
      lb[0] = lb[1], lb[1] = lb[2], lb[2] = fb0;
    };
    int s = 0;
    for (; s + 2 < full; ++s) slice(s, std::integral_constant<int, kInside>{});
    for (; s + 2 < steps; ++s) slice(s, std::integral_constant<int, kChecked>{});
    for (; s < steps; ++s) slice(s, std::integral_constant<int, kNone>{});
    settle(acc);
  }

  // The result goes through LDS, 32 rows of the wave's part at a time, so that
  // every store writes whole stretches of a row.  Stored from the products'
  // layout, 16 bytes of each of 32 rows at once, the weight gradients took
  // twice the time.
  // acc[m][n][4 g + j]: row wm*HM + 32 m + l % 32, column wn*HN + 32 n + 8 g +
  // l / 32 * 4 + j.
  constexpr int kPitch = HN + 4;
  constexpr int kCols = KIND == kIn ? HN / 2 : HN;      // of the wave's part of the result
  constexpr int kLanes = kCols / 8, R = kWave / kLanes;  // 8 columns to a lane, R rows at once
  constexpr int kPass = 32 / R;
  float* stg = (float*)smem + wave * 32 * kPitch;
  const int lr = l / kLanes, lc = l % kLanes * 8;
  const float* src = stg + lr * kPitch + lc;
  auto stage_block = [&](auto block) {
    constexpr int m = decltype(block)::value;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = acc[m][n][4 * q + j];
        *(f32x4*)(stg + (l & 31) * kPitch + n * 32 + q * 8 + (l >> 5) * 4) = v;
      }
    __builtin_amdgcn_wave_barrier();
  };
  // Rows and columns of the result that this tile may write, from the wave's
  // first; all the wave's columns and rows in a full tile, whose code has no
  // branches, so that its LDS reads and stores overlap (one wave to a SIMD
  // hides nothing otherwise).
  const int xw = t.n0 + wn * kCols;  // the wave's first column
  const int rows_left = (kWGrad ? a.M - t.m0 : t.rows) - wm * HM;
  const int cols_all = KIND == kIn || KIND == kGradH ? a.Fpad
                       : KIND == kOut || KIND == kGradX ? (int)a.ldc : a.N;
  const int cols_left = cols_all - xw;
  const bool vec = kWGrad ? a.ldc % 8 == 0 && (uintptr_t)a.c % 16 == 0
                   : KIND == kGradH || KIND == kIn ? a.F % 8 == 0 : true;
  const bool full = rows_left >= HM && cols_left >= kCols && vec;
  // First row of the wave in the result.
  const int64_t row_w = (kWGrad ? t.m0 : t.row0) + wm * HM;
  if constexpr (KIND == kGradH) {
    // g, u and w of the next 4 passes are loaded while these 4 are worked on.
    constexpr int kUnit = 4, kUnits = MT * kPass / kUnit;
    auto epilogue = [&](auto is_full) {
      constexpr bool kFull = decltype(is_full)::value;
      float g[2][kUnit][8], u[2][kUnit][8], w[2][kUnit];
      const float w_unit = kScaled<T> ? inverse_power(a.size[t.expert]) : 1.0f;
      // A wave all of whose rows are outside reads the tile's last one.
      const int rmax = rows_left - 1;
      const uint32_t lane_at = (uint32_t)(lr * a.Fpad + lc);
      auto fetch = [&](int unit, int buf) {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          const int r0 = (unit * kUnit + i) * R;
          if constexpr (kFull) {
            const int64_t base = (row_w + r0) * a.Fpad + xw;
            load8(a.g + base + lane_at, g[buf][i]);
            load8(a.u + base + lane_at, u[buf][i]);
            w[buf][i] = a.d.w[row_w + r0 + lr];
          } else {
            const int64_t row = row_w + min(r0 + lr, rmax);
            const int64_t at = row * a.Fpad + min(xw + lc, a.Fpad - 8);
            load8(a.g + at, g[buf][i]);
            load8(a.u + at, u[buf][i]);
            w[buf][i] = a.d.w[row];
          }
        }
      };
      fetch(0, 0);
      wait_slice<63>();
      auto unit = [&](auto index) {
        constexpr int c = decltype(index)::value, buf = c % 2, m = c * kUnit / kPass;
        typedef std::conditional_t<kScaled<T>, float, T> G;
        if constexpr (c + 1 < kUnits) fetch(c + 1, 1 - buf);
        if constexpr (c * kUnit % kPass == 0) stage_block(std::integral_constant<int, m>{});
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          const int p = c * kUnit % kPass + i, r = (c * kUnit + i) * R;
          const bool inside = kFull || (r + lr < rows_left && lc < cols_left);
          float v[8], dg[8], du[8], hv[8], dot = 0.0f;
          load8(src + p * R * kPitch, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float gj = g[buf][i][j], uj = u[buf][i][j], ww = w[buf][i];
            const float s = fast_sigmoid(gj);
            const float silu = gj * s, h = silu * uj, dh = ww * v[j];
            dot += h * v[j];
            dg[j] = dh * uj * s * (1.0f + gj * (1.0f - s));
            du[j] = dh * silu;
            hv[j] = kScaled<T> ? ww * w_unit * h : ww * h;
          }
          if (inside) {
            const int64_t row = row_w + r + lr;
            G* o = (G*)a.c + row * a.ldc + xw + lc;
            store8((T*)a.hw + row * a.Fpad + xw + lc, true, 8, hv);
            store8(o, vec, a.F - xw - lc, dg);
            store8(o + a.F, vec, a.F - xw - lc, du);
          } else {
            dot = 0.0f;
          }
          dot = sum_of_lanes<kLanes>(dot);
          const int part = t.n0 / HN + wn;
          if (lc == 0 && r + lr < rows_left && part < a.parts)
            a.dval_part[(row_w + r + lr) * a.parts + part] = dot;
        }
      };
      for_each_index<kUnits>(unit);
    };
    if (full) epilogue(std::true_type{});
    else epilogue(std::false_type{});
  } else {
    wait_slice<0>();
    auto epilogue = [&](auto is_full) {
      constexpr bool kFull = decltype(is_full)::value;
      const int64_t ld = KIND == kIn ? a.Fpad : a.ldc;
      const uint32_t lane_at = (uint32_t)lr * (uint32_t)ld + lc;
      const float unit = kWGrad && kScaled<T> ? a.size[t.expert] : 1.0f;
      auto block = [&](auto index) {
        constexpr int m = decltype(index)::value;
        stage_block(index);
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
          const int r = m * 32 + p * R;
          const bool inside = kFull || (r + lr < rows_left && lc < cols_left);
          const int64_t base = (row_w + r) * ld + xw + (kWGrad ? t.expert * a.c_expert : 0);
          float v[8];
          load8(src + p * R * kPitch, v);
          if constexpr (KIND == kIn) {
            float u[8], h[8];
            load8(src + p * R * kPitch + kCols, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              // Columns that fill a row up hold zeros.
              if (!kFull && xw + lc + j >= a.F) v[j] = u[j] = 0.0f;
              h[j] = v[j] * fast_sigmoid(v[j]) * u[j];
            }
            if (inside) {
              store8((T*)a.c + base + lane_at, true, 8, h);
              if (a.g) {
                store8(a.g + base + lane_at, true, 8, v);
                store8(a.u + base + lane_at, true, 8, u);
              }
            }
          } else if constexpr (KIND == kOut || KIND == kGradX) {
            if (inside) store8((float*)a.c + base + lane_at, true, 8, v);
          } else {
            if constexpr (kScaled<T>) {
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] *= unit;
            }
            if (inside) store8((T*)a.c + base + lane_at, vec, cols_left - lc, v);
          }
        }
      };
      for_each_index<MT>(block);
    };
    if (full) epilogue(std::true_type{});
    else epilogue(std::false_type{});
  }
  if constexpr (!kTurns<KIND>) break;
  }  // tiles
}

template <typename T, int KIND, int BM, int BN, bool kFar = false>
void launch_product(const ProductArgs& a, int64_t row_tiles, hipStream_t s) {
  auto kernel = k_product<T, KIND, BM, BN, kFar>;
  static std::atomic<uint64_t> allowed{0};  // devices whose LDS limit is set
  int device = 0;
  // After a failure nothing more is launched, and setting the limit, which leaves
  // the error state clear, does not lose it: the caller's last look reports it.
  if (hipPeekAtLastError() != hipSuccess || hipGetDevice(&device) != hipSuccess) return;
  const uint64_t bit = 1ull << (device & 63);
  if (!(allowed.load() & bit)) {
    allow_max_dynamic_lds((const void*)kernel);
    allowed.fetch_or(bit);
  }
  const int64_t step = KIND == kIn ? BN / 2 : BN;
  const int64_t tiles = row_tiles * ((a.N + step - 1) / step);
  if (tiles == 0) return;
  int64_t grid = (tiles + kXcds - 1) / kXcds * kXcds;
  // In turn: a work group for every compute unit, or the two that fit one.
  if (kTurns<KIND>) grid = std::min<int64_t>(grid, BN == 256 ? 256 : 512);
  typedef Stages<KIND, BM, BN> S;
  const size_t lds =
      (S::kA * BM + S::kB * BN) * kBK * 2 + (S::kWGrad ? kListLen * sizeof(int32_t) : 0);
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(kNT), lds, s, a);
}

// ---- few rows: products that stream the weights ----
// With a few rows to an expert every weight is used once and its bytes bound
// the product.  A wave takes 16 weight rows straight from memory to registers
// (16x16x32 MFMA, the weights as the left operand, up to 16 rows of x as the
// right one), 8 loads in flight, and the waves of a work group share K, so that
// many small work groups keep the memory busy: 48 tokens with 8 of 128 experts of
// 2048 x 768 read W_in at 5.9 and W_out at 6.4 TB/s (some of it from the
// memory-side cache), one token with 6 of 64 of 2048 x 1024 takes 14.5 + 9.3 us,
// bound by the latency of its two launches.  16 loads in flight gained nothing.

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

// Rows of a few-rows tile: of its own entry where entries are not sorted (a
// tile is an entry, in their order), else of the sorted list.
struct FewTile {
  int expert, row0, rows;
};
template <bool kDirect>
__device__ __forceinline__ bool few_tile(const ProductArgs& a, int tile, FewTile& t) {
  if constexpr (kDirect) {
    t.expert = a.col[tile];
    t.row0 = tile;
    t.rows = 1;
    return (uint32_t)t.expert < (uint32_t)a.E;
  } else {
    if (tile >= *a.d.ntiles) return false;
    t.expert = a.d.tiles[2 * tile];
    t.row0 = a.d.tiles[2 * tile + 1];
    t.rows = min(kFewRows, a.d.row_ptr[t.expert + 1] - t.row0);
    return true;
  }
}

// The lane's share of K step s: 8 values of its row from k = 32 s + l / 16 * 8,
// zeros beyond K.
__device__ __forceinline__ s16x8 few_load(const void* row, int s, int K) {
  const int k = s * 32 + (lane_id() >> 4) * 8;
  s16x8 v = *(const s16x8*)((const char*)row + (k < K ? k : 0) * 2);
  if (k >= K) v = s16x8{0, 0, 0, 0, 0, 0, 0, 0};
  return v;
}

constexpr int kFewBatch = 8;

// acc[o] += W rows of operand o times x rows, K steps first, first + step, ..
template <typename T, int kOps>
__device__ __forceinline__ void few_products(const void* const (&w)[kOps], const void* x,
                                             int first, int step, int steps, int K,
                                             f32x4 (&acc)[kOps]) {
  for (int s = first; s < steps; s += step * kFewBatch) {
    s16x8 wf[kFewBatch][kOps], xf[kFewBatch];
#pragma unroll
    for (int i = 0; i < kFewBatch; ++i) {
      const int at = s + i * step;
      if (at >= steps) break;
#pragma unroll
      for (int o = 0; o < kOps; ++o) wf[i][o] = few_load(w[o], at, K);
      xf[i] = few_load(x, at, K);
    }
#pragma unroll
    for (int i = 0; i < kFewBatch; ++i) {
      if (s + i * step >= steps) break;
#pragma unroll
      for (int o = 0; o < kOps; ++o) acc[o] = mfma16(T{}, wf[i][o], xf[i], acc[o]);
    }
  }
}

// h of one tile's rows, 16 columns to a work group.
template <typename T, bool kDirect>
__global__ __launch_bounds__(kNT) void k_few_in(ProductArgs a) {
  const int cols = (a.Fpad + 15) / 16;
  FewTile t;
  if (!few_tile<kDirect>(a, blockIdx.x / cols, t)) return;
  const int f0 = blockIdx.x % cols * 16, l = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const T* W = (const T*)a.b + t.expert * a.b_expert;
  const int f = min(f0 + (l & 15), a.F - 1);
  const void* w[2] = {W + (int64_t)f * a.ldb, W + (int64_t)(a.F + f) * a.ldb};
  const int at = t.row0 + min(l & 15, t.rows - 1);
  const void* x = (const T*)a.a + (int64_t)(kDirect ? at / a.k : a.d.tok[at]) * a.lda;
  f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  few_products<T, 2>(w, x, wave, kWaves, (a.Kpad + 31) / 32, a.Kpad, acc);
  __shared__ float part[kWaves][2][16][17];
#pragma unroll
  for (int o = 0; o < 2; ++o)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[wave][o][(l >> 4) * 4 + j][l & 15] = acc[o][j];
  __syncthreads();
  const int r = threadIdx.x / 16, c = threadIdx.x % 16;  // row, column
  if (r >= t.rows || f0 + c >= a.Fpad) return;
  float g = 0.0f, u = 0.0f;
#pragma unroll
  for (int v = 0; v < kWaves; ++v) {
    g += part[v][0][c][r];
    u += part[v][1][c][r];
  }
  const float h = f0 + c < a.F ? g * fast_sigmoid(g) * u : 0.0f;
  ((T*)a.c)[(int64_t)(t.row0 + r) * a.Fpad + f0 + c] = from_f32<T>(h);
}

// Rows of y before their sum, 32 columns to a work group.
template <typename T>
__global__ __launch_bounds__(kNT) void k_few_out(ProductArgs a) {
  const int cols = (a.N + 31) / 32;
  FewTile t;
  if (!few_tile<false>(a, blockIdx.x / cols, t)) return;
  const int n0 = blockIdx.x % cols * 32, l = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const T* W = (const T*)a.b + t.expert * a.b_expert;
  const void* w[2] = {W + (int64_t)min(n0 + (l & 15), a.N - 1) * a.ldb,
                      W + (int64_t)min(n0 + 16 + (l & 15), a.N - 1) * a.ldb};
  const void* x = (const T*)a.a + (int64_t)(t.row0 + min(l & 15, t.rows - 1)) * a.lda;
  f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  few_products<T, 2>(w, x, wave, kWaves, (a.Kpad + 31) / 32, a.Kpad, acc);
  __shared__ float part[kWaves][32][17];
#pragma unroll
  for (int o = 0; o < 2; ++o)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[wave][o * 16 + (l >> 4) * 4 + j][l & 15] = acc[o][j];
  __syncthreads();
  const int c = threadIdx.x % 32;
  for (int r = threadIdx.x / 32; r < t.rows; r += kNT / 32) {
    if (n0 + c >= a.ldc) break;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) v += part[i][c][r];
    ((float*)a.c)[(int64_t)(t.row0 + r) * a.ldc + n0 + c] = v;
  }
}

// y of one token straight from its entries' h (entry order), 16 columns to a
// work group of 8 waves that share each entry's K.
constexpr int kFewTokenWaves = 8;
template <typename T>
__global__ __launch_bounds__(kFewTokenWaves * kWave) void k_few_token(ProductArgs a) {
  const int cols = (a.N + 15) / 16;
  const int64_t t = blockIdx.x / cols;
  const int n0 = blockIdx.x % cols * 16, l = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int n = min(n0 + (l & 15), a.N - 1);
  // K steps of all entries in one row: step q is step q % per of entry q / per.
  const int per = (a.Kpad + 31) / 32, all = per * a.k;
  f32x4 sum = {0, 0, 0, 0}, acc = {0, 0, 0, 0};
  float weight = 0.0f;
  int entry = -1;
  for (int q0 = wave; q0 < all; q0 += kFewTokenWaves * kFewBatch) {
    s16x8 wf[kFewBatch], xf[kFewBatch];
    int from[kFewBatch];
    float wt[kFewBatch];
#pragma unroll
    for (int i = 0; i < kFewBatch; ++i) {
      const int q = min(q0 + i * kFewTokenWaves, all - 1);
      const int e = q / per, s = q0 + i * kFewTokenWaves < all ? q - e * per : per;
      const int64_t at = t * a.k + e;
      const int c = a.col[at];
      const bool there = (uint32_t)c < (uint32_t)a.E;
      from[i] = e;
      wt[i] = there ? a.val[at] : 0.0f;
      const int K = there ? a.Kpad : 0;
      wf[i] = few_load((const T*)a.b + (there ? c : 0) * a.b_expert + (int64_t)n * a.ldb, s, K);
      xf[i] = few_load((const T*)a.a + at * a.lda, s, K);
    }
#pragma unroll
    for (int i = 0; i < kFewBatch; ++i) {
      if (from[i] != entry) {
        sum += weight * acc;
        acc = f32x4{0, 0, 0, 0};
        entry = from[i];
        weight = wt[i];
      }
      acc = mfma16(T{}, wf[i], xf[i], acc);
    }
  }
  sum += weight * acc;
  __shared__ float part[kFewTokenWaves][16];
  if ((l & 15) == 0)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[wave][(l >> 4) * 4 + j] = sum[j];
  __syncthreads();
  const int c = threadIdx.x;
  if (c >= 16 || n0 + c >= a.N) return;
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < kFewTokenWaves; ++i) v += part[i][c];
  ((T*)a.c)[t * a.N + n0 + c] = from_f32<T>(v);
}

// ---- sums over a token's entries ----

// out[t] = sum over its entries of w * rows[pos], in the entries' order, in fp32,
// rounded once; w is the entry's val, or the row's unit, or 1.  8 columns to a
// thread.  The rows' bytes bound it: 131,072 rows of 2048 in 220-240 us, 4.7-5.2
// TB/s.
template <typename T>
__global__ __launch_bounds__(256) void k_combine(int64_t Tn, int k, int D, int Dpad,
                                                 const float* __restrict__ rows,
                                                 const int32_t* __restrict__ pos,
                                                 const float* __restrict__ val,
                                                 const float* __restrict__ unit,
                                                 T* __restrict__ out) {
  const int per = Dpad / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = i / per;
  if (t >= Tn) return;
  const int x = (int)(i - t * per) * 8;
  float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
  for (int e = 0; e < k; ++e) {
    const int p = pos[t * k + e];
    const int64_t row = max(p, 0);  // read in any case, so that the loads do not wait
    float v[8];
    const float w = val ? val[t * k + e] : unit ? unit[row] : 1.0f;
    load8(rows + row * Dpad + x, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += p < 0 ? 0.0f : w * v[j];
  }
  store8(out + t * D + x, D % 8 == 0 && (uintptr_t)out % 16 == 0, D - x, s);
}

// dval[entry] = the sum of its partial sums, in order; 0 where there is none.
__global__ __launch_bounds__(256) void k_dval(int64_t n, int parts,
                                              const int32_t* __restrict__ pos,
                                              const float* __restrict__ part,
                                              float* __restrict__ dval) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= n) return;
  const int p = pos[e];
  float s = 0.0f;
  if (p >= 0)
    for (int i = 0; i < parts; ++i) s += part[(int64_t)p * parts + i];
  dval[e] = s;
}

// ---- units of the float16 gradients ----

// size[e]: the power of two at the expert's largest finite |src| (above 0), or
// the next one (1).  A work group to an expert.
__global__ __launch_bounds__(1024) void k_expert_size(const int32_t* __restrict__ row_ptr,
                                                      const float* __restrict__ src, int above,
                                                      float* __restrict__ size) {
  __shared__ uint32_t most[1024 / kWave];
  uint32_t m = 0;
  const int end = row_ptr[blockIdx.x + 1];
  for (int64_t i = (int64_t)row_ptr[blockIdx.x] + threadIdx.x; i < end; i += 1024) {
    const uint32_t b = __float_as_uint(src[i]) & 0x7fffffffu;
    m = max(m, b < 0x7f800000u ? b : 0u);
  }
  m = wave_max_u32(m);
  if (lane_id() == 0) most[threadIdx.x / kWave] = m;
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < 1024 / kWave; ++w) m = max(m, most[w]);
  // Exponents whose inverse is a normal number, too.
  size[blockIdx.x] = __uint_as_float(min(max(m >> 23, 1u) + above, 253u) << 23);
}

// Rows of [dg, du] from fp32 (2 F of the S2 columns) to float16 (S2 columns, zeros at
// the end) in units of their own, which go to unit[row].  A wave to a row.
__global__ __launch_bounds__(256) void k_scale_rows(const int32_t* __restrict__ rows, int cols,
                                                    int S2, const float* __restrict__ src,
                                                    _Float16* __restrict__ dst,
                                                    float* __restrict__ unit) {
  const int64_t step = (int64_t)gridDim.x * (256 / kWave), n = *rows;
  for (int64_t r = (int64_t)blockIdx.x * (256 / kWave) + threadIdx.x / kWave; r < n; r += step) {
    const float* from = src + r * S2;
    auto load = [&](int c, float v[8]) {
      load8(from + c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j >= cols) v[j] = 0.0f;
    };
    uint32_t m = 0;
    for (int c = lane_id() * 8; c < S2; c += kWave * 8) {
      float v[8];
      load(c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b = __float_as_uint(v[j]) & 0x7fffffffu;
        m = max(m, b < 0x7f800000u ? b : 0u);
      }
    }
    // The exponent is kept where both powers of two are normal.
    const uint32_t e = min(max(wave_max_u32(m) >> 23, 15u), 254u);
    const float up = __uint_as_float((268u - e) << 23);
    if (lane_id() == 0) unit[r] = __uint_as_float((e - 14u) << 23);
    for (int c = lane_id() * 8; c < S2; c += kWave * 8) {
      float v[8];
      load(c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= up;
      store8(dst + r * S2 + c, true, 8, v);
    }
  }
}

// The same rows in the unit of their expert.  A wave to a row.
__global__ __launch_bounds__(256) void k_unit_rows(const int32_t* __restrict__ row_ptr, int E,
                                                   int S2, const _Float16* __restrict__ src,
                                                   const float* __restrict__ unit,
                                                   const float* __restrict__ size,
                                                   _Float16* __restrict__ dst) {
  const int64_t step = (int64_t)gridDim.x * (256 / kWave), n = row_ptr[E];
  for (int64_t r = (int64_t)blockIdx.x * (256 / kWave) + threadIdx.x / kWave; r < n; r += step) {
    const int64_t expert = wave_last_le(row_ptr, (int64_t)0, (int64_t)E, r);
    // Both are powers of two and the row's is not the larger one.
    const int e = (int)(__float_as_uint(unit[r]) >> 23) - (int)(__float_as_uint(size[expert]) >> 23);
    const float f = __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
    for (int c = lane_id() * 8; c < S2; c += kWave * 8) {
      struct alignas(16) Pack { _Float16 v[8]; };
      const Pack q = *(const Pack*)(src + r * S2 + c);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)q.v[j] * f;
      store8(dst + r * S2 + c, true, 8, v);
    }
  }
}

// Copies rows of `cols` 16-bit values to rows of `pad`, filled up with zeros:
// for operands whose rows do not begin at 16-byte boundaries.
__global__ __launch_bounds__(256) void k_pad_rows(int64_t rows, int cols, int64_t ld, int pad,
                                                  const uint16_t* __restrict__ src,
                                                  uint16_t* __restrict__ dst) {
  const int64_t all = rows * pad;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / pad;
    const int c = (int)(i - r * pad);
    dst[i] = c < cols ? src[r * ld + c] : (uint16_t)0;
  }
}

__global__ __launch_bounds__(256) void k_zero16(uint16_t* __restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = 0;
}

unsigned grid_for(int64_t n) { return (unsigned)std::min<int64_t>((n + 255) / 256, 8192); }

// ---- sizes and buffers ----

int64_t round8(int64_t x) { return (x + 7) / 8 * 8; }

struct Sizes {
  int64_t T, E, D, F, n, Dp, Fp, S2;  // S2: row of [dg, du]
  int k;
};

Sizes sizes_of(const spgemm_experts_desc& d) {
  Sizes z{};
  z.T = d.tokens;
  z.E = d.experts;
  z.D = d.width;
  z.F = d.hidden;
  z.k = d.k;
  z.n = z.T * z.k;
  z.Dp = round8(z.D);
  z.Fp = round8(z.F);
  z.S2 = round8(2 * z.F);
  return z;
}

// How a forward pass goes: by entries in their own order, by tiles of a few
// rows, or by large tiles.
enum Path { kPathDirect, kPathFew, kPathTiles };

// Fewer than 2^32 work items, as a launch takes them.
bool launchable(int64_t groups, int64_t size) { return groups * size < (int64_t)1 << 32; }

Path path_of(const Sizes& z, bool keep) {
  // Unsorted entries read the weights of a shared expert once each, but save
  // the dispatch and the sum: 2 tokens of 8 picks among 128 experts 43 against
  // 46 us, 8 tokens 118 against 105 us.
  const bool direct = z.T == 1 || z.n <= z.E / 4;
  // 16 rows to a tile against 128: 3 entries to an expert 209 against 237 us, 4.5
  // 180 against 194, 6 186 against 228, 9 217 against 209.
  if (keep || !(direct || z.n <= 6 * z.E)) return kPathTiles;
  const int64_t tiles = direct ? z.n : dispatch_max_tiles(z.n, z.E, kFewRows);
  if (!launchable(tiles * ((z.Fp + 15) / 16), kNT) ||
      !(direct ? launchable(z.T * ((z.D + 15) / 16), kFewTokenWaves * kWave)
               : launchable(tiles * ((z.D + 31) / 32), kNT)))
    return kPathTiles;
  return direct ? kPathDirect : kPathFew;
}

// Rows of a tile: 256 when the experts' rows fill such tiles to more than
// about half on average, else 128.
int tile_rows(const Sizes& z) { return z.n > 256 * z.E ? 256 : 128; }

// Whether rows of x are kept in 8 bits.  Any other value is one that a caller from before the
// field may have left there.
bool keeps_codes(const spgemm_experts_desc& d) { return d.kept_form == SPGEMM_KEPT_E4M3; }

// What the forward pass leaves for the backward pass: the dispatch, and the
// pre-activations (8 F bytes to an entry) or, by keeps_codes, the rows of x in 8 bits,
// from which the backward pass makes them again.  8192 tokens with 8 of 64 experts,
// 2048 x 1024: 538 or 18 MB.
struct Kept {
  Dispatch d;
  float* g;
  float* u;
  uint8_t* code;
  uint8_t* scale;
};

void take_dispatch(Carver& c, const Sizes& z, Dispatch& d) {
  d.row_ptr = c.take<int32_t>(z.E + 1);
  d.ent = c.take<int32_t>(z.n);
  d.tok = c.take<int32_t>(z.n);
  d.w = c.take<float>(z.n);
  d.pos = c.take<int32_t>(z.n);
  d.tiles = c.take<int32_t>(2 * dispatch_max_tiles(z.n, z.E, kFewRows));
  d.ntiles = c.take<int32_t>(1);
}

Kept take_kept(Carver& c, const Sizes& z, bool codes) {
  Kept k{};
  take_dispatch(c, z, k.d);
  if (codes) {
    k.code = c.take<uint8_t>(z.T * kept_pitch(z.D));
    k.scale = c.take<uint8_t>(z.T * kept_blocks(z.D));
    return k;
  }
  k.g = c.take<float>(z.n * z.Fp);
  k.u = c.take<float>(z.n * z.Fp);
  return k;
}

// Copies of operands whose rows are not 16-byte aligned.
struct Padded {
  uint16_t *x, *w_in, *w_out, *dy;
};

Padded take_padded(Carver& c, const Sizes& z, bool grad) {
  Padded p{};
  p.x = c.take<uint16_t>(z.T * z.Dp);
  p.w_in = c.take<uint16_t>(z.E * 2 * z.F * z.Dp);
  p.w_out = c.take<uint16_t>(z.E * z.D * z.Fp);
  if (grad) p.dy = c.take<uint16_t>(z.T * z.Dp);
  return p;
}

struct ForwardWork {
  Dispatch d;
  int32_t* tmp;
  uint16_t* h;
  float* rows;
  Padded pad;
};

ForwardWork take_forward(Carver& c, const Sizes& z, bool keep, bool padded) {
  ForwardWork w{};
  if (!keep) take_dispatch(c, z, w.d);
  w.tmp = c.take<int32_t>(dispatch_tmp_elems(z.n, z.E));
  w.h = c.take<uint16_t>(z.n * z.Fp);
  w.rows = c.take<float>(z.n * z.Dp);
  if (padded) w.pad = take_padded(c, z, false);
  return w;
}

struct BackwardWork {
  uint16_t* dgu;
  uint16_t* hw;
  float* rows;
  // Of float16 gradients: [dg, du] in fp32, and then in units of the experts;
  // the unit of each row of dgu; units by expert of [dg, du] and of w h.
  float* dgu32;
  float* row_unit;
  float* dgu_size;
  float* w_size;
  float* part;
  // Of rows kept in 8 bits: what they stand for, and the pre-activations.
  uint16_t* x;
  float* g;
  float* u;
  Padded pad;
};

// Partial sums of a value's gradient: one for each wave's columns.
int dval_parts(const Sizes& z, int cols) { return (int)((z.Fp + cols - 1) / cols); }

BackwardWork take_backward(Carver& c, const Sizes& z, bool scaled, bool codes, bool padded) {
  BackwardWork w{};
  w.dgu = c.take<uint16_t>(z.n * z.S2);
  w.hw = c.take<uint16_t>(z.n * z.Fp);
  w.rows = c.take<float>(z.n * z.Dp);
  w.part = c.take<float>(z.n * dval_parts(z, 64));
  if (scaled) {
    w.dgu32 = c.take<float>(z.n * z.S2);
    w.row_unit = c.take<float>(z.n);
    w.dgu_size = c.take<float>(z.E);
    w.w_size = c.take<float>(z.E);
  }
  if (codes) {
    w.x = c.take<uint16_t>(z.T * z.Dp);
    w.g = c.take<float>(z.n * z.Fp);
    w.u = c.take<float>(z.n * z.Fp);
  }
  if (padded) w.pad = take_padded(c, z, true);
  return w;
}

// An operand's rows as the products read them.
struct Rows {
  const void* p;
  int64_t ld;
};

Rows padded_rows(const void* p, int64_t ld, int64_t rows, int64_t cols, uint16_t* dst,
                 hipStream_t s) {
  if ((uintptr_t)p % 16 == 0 && ld % 8 == 0 && cols % 8 == 0) return {p, ld};
  const int64_t pad = round8(cols);
  hipLaunchKernelGGL(k_pad_rows, dim3(grid_for(rows * pad)), dim3(256), 0, s, rows, (int)cols, ld,
                     (int)pad, (const uint16_t*)p, dst);
  return {dst, pad};
}

bool needs_padding(const spgemm_experts_desc& d, const void* x, const void* w_in,
                   const void* w_out, const void* dy) {
  return d.width % 8 || d.hidden % 8 || d.x_ld % 8 || (dy && d.grad_ld % 8) ||
         ((uintptr_t)x | (uintptr_t)w_in | (uintptr_t)w_out | (uintptr_t)dy) % 16;
}

// Up to this many tiles a product takes smaller ones, so that more of the 256
// compute units have one.  Measured, forward pass: 76 tiles 36 -> 29 us, 120
// tiles 46 -> 38 us, but 195 tiles 59 -> 66 us and 256 tiles 81 -> 106 us, where
// the smaller ones take two rounds.
constexpr int64_t kFewTiles = 128;

// Whether a product of N columns (of pairs: gate and up) by row tiles of 128
// takes them.
bool narrow_tiles(const Sizes& z, int64_t N, bool pairs) {
  const int64_t step = pairs ? 128 : 256;
  return dispatch_max_tiles(z.n, z.E, 128) * ((N + step - 1) / step) <= kFewTiles;
}

template <typename T, int KIND, bool kFar>
void product_by_size(const ProductArgs& a, const Sizes& z, hipStream_t s) {
  const int bm = tile_rows(z);
  const int64_t tiles = dispatch_max_tiles(z.n, z.E, bm);
  if (bm == 256) launch_product<T, KIND, 256, 256, kFar>(a, tiles, s);
  else if (narrow_tiles(z, a.N, KIND == kIn)) launch_product<T, KIND, 128, 128, kFar>(a, tiles, s);
  else launch_product<T, KIND, 128, 256, kFar>(a, tiles, s);
}

template <typename T, int KIND>
void product_by_rows(const ProductArgs& a, const Sizes& z, hipStream_t s) {
  if constexpr (KIND == kIn || KIND == kGradH)
    if (z.T * a.lda >= (int64_t)1 << 31) return product_by_size<T, KIND, true>(a, z, s);
  product_by_size<T, KIND, false>(a, z, s);
}

template <typename T, int KIND>
void weight_gradient(const ProductArgs& a, const Sizes& z, hipStream_t s) {
  auto up = [](int64_t x, int64_t t) { return (x + t - 1) / t; };
  if (z.E * up(a.M, 256) * up(a.N, 256) <= kFewTiles)
    launch_product<T, KIND, 128, 128>(a, z.E * up(a.M, 128), s);
  else
    launch_product<T, KIND, 256, 256>(a, z.E * up(a.M, 256), s);
}

ProductArgs base_args(const Sizes& z, const Dispatch& d) {
  ProductArgs a{};
  a.d = d;
  a.E = (int)z.E;
  a.F = (int)z.F;
  a.Fpad = (int)z.Fp;
  return a;
}

// Of the first product: h to c, the pre-activations to g and u unless NULL.
ProductArgs in_args(const Sizes& z, const Dispatch& d, const Rows& x, const Rows& w_in, void* h,
                    float* g, float* u) {
  ProductArgs a = base_args(z, d);
  a.a = x.p;
  a.lda = x.ld;
  a.b = w_in.p;
  a.ldb = w_in.ld;
  a.b_expert = 2 * z.F * w_in.ld;
  a.N = (int)z.F;
  a.K = (int)z.D;
  a.Kpad = (int)z.Dp;
  a.c = h;
  a.g = g;
  a.u = u;
  return a;
}

template <typename T>
void combine(const Sizes& z, const float* rows, const int32_t* pos, const float* val,
             const float* unit, void* out, hipStream_t s) {
  hipLaunchKernelGGL((k_combine<T>), dim3((unsigned)((z.T * (z.Dp / 8) + 255) / 256)), dim3(256), 0,
                     s, z.T, z.k, (int)z.D, (int)z.Dp, rows, pos, val, unit, (T*)out);
}

template <typename T>
void forward(const spgemm_experts_desc& desc, const void* x, const void* w_in, const void* w_out,
             const int32_t* col, const float* val, void* y, void* kept, const ForwardWork& w,
             hipStream_t s) {
  const Sizes z = sizes_of(desc);
  Kept kp{};
  if (kept) {
    Carver c(kept);
    kp = take_kept(c, z, keeps_codes(desc));
    if (keeps_codes(desc))
      launch_rows_encode(desc.dtype, z.T, z.D, desc.x_ld, x, kp.code, kp.scale, s);
  } else {
    kp.d = w.d;
  }
  const Path path = path_of(z, kept != nullptr);
  if (path != kPathDirect)
    launch_dispatch(col, val, z.n, z.k, z.E, path == kPathFew ? kFewRows : tile_rows(z), kp.d,
                    w.tmp, s);
  const Rows xr = padded_rows(x, desc.x_ld, z.T, z.D, w.pad.x, s);
  const Rows w1 = padded_rows(w_in, z.D, z.E * 2 * z.F, z.D, w.pad.w_in, s);
  const Rows w2 = padded_rows(w_out, z.F, z.E * z.D, z.F, w.pad.w_out, s);
  ProductArgs a = in_args(z, kp.d, xr, w1, w.h, kp.g, kp.u);
  a.k = z.k;
  a.col = col;
  const int64_t few = path == kPathDirect ? z.n : dispatch_max_tiles(z.n, z.E, kFewRows);
  const dim3 in_grid((unsigned)(few * ((z.Fp + 15) / 16)));
  if (path == kPathDirect)
    hipLaunchKernelGGL((k_few_in<T, true>), in_grid, dim3(kNT), 0, s, a);
  else if (path == kPathFew)
    hipLaunchKernelGGL((k_few_in<T, false>), in_grid, dim3(kNT), 0, s, a);
  else
    product_by_rows<T, kIn>(a, z, s);
  a = base_args(z, kp.d);
  a.a = w.h;
  a.lda = z.Fp;
  a.b = w2.p;
  a.ldb = w2.ld;
  a.b_expert = z.D * w2.ld;
  a.N = (int)z.D;
  a.K = (int)z.F;
  a.Kpad = (int)z.Fp;
  a.c = w.rows;
  a.ldc = z.Dp;
  if (path == kPathDirect) {
    a.c = y;
    a.k = z.k;
    a.col = col;
    a.val = val;
    hipLaunchKernelGGL((k_few_token<T>), dim3((unsigned)(z.T * ((z.D + 15) / 16))),
                       dim3(kFewTokenWaves * kWave), 0, s, a);
    return;
  }
  if (path == kPathFew)
    hipLaunchKernelGGL((k_few_out<T>), dim3((unsigned)(few * ((z.D + 31) / 32))), dim3(kNT), 0, s,
                       a);
  else
    product_by_rows<T, kOut>(a, z, s);
  combine<T>(z, w.rows, kp.d.pos, val, nullptr, y, s);
}

template <typename T>
void backward(const spgemm_experts_desc& desc, const void* x, const void* w_in,
              const void* w_out, const void* dy, const void* kept, void* dx,
              void* dw_in, void* dw_out, float* dval, const BackwardWork& w, hipStream_t s) {
  const Sizes z = sizes_of(desc);
  Carver kc((void*)kept);
  Kept kp = take_kept(kc, z, keeps_codes(desc));
  Rows xr{w.x, z.Dp};
  if (keeps_codes(desc))
    launch_rows_decode(desc.dtype, z.T, z.D, kp.code, kp.scale, w.x, s);
  else
    xr = padded_rows(x, desc.x_ld, z.T, z.D, w.pad.x, s);
  const Rows gr = padded_rows(dy, desc.grad_ld, z.T, z.D, w.pad.dy, s);
  const Rows w1 = padded_rows(w_in, z.D, z.E * 2 * z.F, z.D, w.pad.w_in, s);
  const Rows w2 = padded_rows(w_out, z.F, z.E * z.D, z.F, w.pad.w_out, s);
  if constexpr (kScaled<T>)
    hipLaunchKernelGGL(k_expert_size, dim3((unsigned)z.E), dim3(1024), 0, s, kp.d.row_ptr, kp.d.w,
                       1, w.w_size);
  else if (z.S2 != 2 * z.F)
    hipLaunchKernelGGL(k_zero16, dim3(grid_for(z.n * z.S2)), dim3(256), 0, s, w.dgu, z.n * z.S2);
  if (keeps_codes(desc)) {
    kp.g = w.g;
    kp.u = w.u;
    // h goes where w h will be.
    product_by_rows<T, kIn>(in_args(z, kp.d, xr, w1, w.hw, w.g, w.u), z, s);
  }
  ProductArgs a = base_args(z, kp.d);
  a.a = gr.p;
  a.lda = gr.ld;
  a.b = w2.p;
  a.ldb = w2.ld;
  a.b_expert = z.D * w2.ld;
  a.N = a.Npad = (int)z.Fp;
  a.K = (int)z.D;
  a.Kpad = (int)z.Dp;
  a.c = kScaled<T> ? (void*)w.dgu32 : w.dgu;
  a.size = w.w_size;
  a.ldc = z.S2;
  a.g = kp.g;
  a.u = kp.u;
  a.hw = w.hw;
  a.dval_part = w.part;
  a.parts = dval_parts(z, tile_rows(z) == 128 && narrow_tiles(z, z.Fp, false) ? 64 : 128);
  const int parts = a.parts;
  product_by_rows<T, kGradH>(a, z, s);
  const void* dgu_w = w.dgu;  // as dW_in sums it
  if constexpr (kScaled<T>) {
    dgu_w = w.dgu32;
    hipLaunchKernelGGL(k_scale_rows, dim3(grid_for(z.n * kWave)), dim3(256), 0, s,
                       kp.d.row_ptr + z.E, (int)(2 * z.F), (int)z.S2, w.dgu32, (_Float16*)w.dgu,
                       w.row_unit);
    hipLaunchKernelGGL(k_expert_size, dim3((unsigned)z.E), dim3(1024), 0, s, kp.d.row_ptr,
                       w.row_unit, 0, w.dgu_size);
    hipLaunchKernelGGL(k_unit_rows, dim3(grid_for(z.n * kWave)), dim3(256), 0, s, kp.d.row_ptr,
                       (int)z.E, (int)z.S2, (const _Float16*)w.dgu, w.row_unit, w.dgu_size,
                       (_Float16*)dgu_w);
  }
  a = base_args(z, kp.d);
  a.a = w.dgu;
  a.lda = z.S2;
  a.b = w1.p;
  a.ldb = w1.ld;
  a.b_expert = 2 * z.F * w1.ld;
  a.N = (int)z.D;
  a.Npad = (int)z.Dp;
  a.K = (int)(2 * z.F);
  a.Kpad = (int)z.S2;
  a.c = w.rows;
  a.ldc = z.Dp;
  product_by_rows<T, kGradX>(a, z, s);
  combine<T>(z, w.rows, kp.d.pos, nullptr, w.row_unit, dx, s);
  hipLaunchKernelGGL(k_dval, dim3((unsigned)((z.n + 255) / 256)), dim3(256), 0, s, z.n,
                     parts, kp.d.pos, w.part, dval);
  a = base_args(z, kp.d);
  a.a = gr.p;
  a.lda = gr.ld;
  a.b = w.hw;
  a.ldb = z.Fp;
  a.M = (int)z.D;
  a.Mpad = (int)z.Dp;
  a.N = (int)z.F;
  a.Npad = (int)z.Fp;
  a.size = w.w_size;
  a.c = dw_out;
  a.ldc = z.F;
  a.c_expert = z.D * z.F;
  weight_gradient<T, kGradWOut>(a, z, s);
  a = base_args(z, kp.d);
  a.a = dgu_w;
  a.lda = z.S2;
  a.b = xr.p;
  a.ldb = xr.ld;
  a.M = (int)(2 * z.F);
  a.Mpad = (int)z.S2;
  a.N = (int)z.D;
  a.Npad = (int)z.Dp;
  a.size = w.dgu_size;
  a.c = dw_in;
  a.ldc = z.D;
  a.c_expert = 2 * z.F * z.D;
  weight_gradient<T, kGradWIn>(a, z, s);
}

// ---- checks ----

spgemm_status refuse(spgemm_status st, const char* msg) {
  set_thread_error(msg);
  return st;
}

spgemm_status check_desc(const spgemm_experts_desc* d) {
  if (!d) return refuse(SPGEMM_ERR_INVALID_ARG, "experts: null description");
  if (d->dtype != SPGEMM_BF16 && d->dtype != SPGEMM_F16)
    return refuse(SPGEMM_ERR_INVALID_ARG, "experts: tensors must be bf16 or fp16");
  if (d->tokens < 0 || d->experts < 1 || d->experts > kMaxExperts || d->k < 1 || d->k > 64)
    return refuse(SPGEMM_ERR_INVALID_ARG,
                  "experts: tokens < 0, experts outside [1, 1024] or k outside [1, 64]");
  if (d->width < 1 || d->hidden < 1 || d->x_ld < d->width)
    return refuse(SPGEMM_ERR_INVALID_ARG, "experts: empty width, or a row stride below it");
  if (d->x_ld >= 1 << 30 || d->grad_ld >= 1 << 30)
    return refuse(SPGEMM_ERR_INDEX_OVERFLOW, "experts: a row stride of 2^30 elements or more");
  if (d->width > (1 << 22) || d->hidden > (1 << 22) ||
      2 * round8(d->hidden) * round8(d->width) >= (int64_t)1 << 31 ||
      d->tokens > INT32_MAX / d->k ||
      d->tokens * d->k / 128 + d->experts > INT32_MAX / ((d->width + d->hidden) / 128 + 1) / 2 ||
      !launchable((d->tokens * (round8(d->width) / 8) + 255) / 256, 256) ||
      d->experts * ((d->width + 255) / 256 + 1) * ((2 * d->hidden + 255) / 256 + 1) >
          INT32_MAX / 2)
    return refuse(SPGEMM_ERR_INDEX_OVERFLOW, "experts: too many entries or tiles");
  return SPGEMM_OK;
}

spgemm_status launched() {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return SPGEMM_OK;
  return refuse(SPGEMM_ERR_HIP, hipGetErrorString(e));
}

}  // namespace
}  // namespace sg

using namespace sg;

extern "C" spgemm_status spgemm_experts_sizes(const spgemm_experts_desc* desc, int64_t* kept,
                                              int64_t* forward_work, int64_t* backward_work) {
  const spgemm_status st = check_desc(desc);
  if (st != SPGEMM_OK) return st;
  const Sizes z = sizes_of(*desc);
  // A base that is not 16-byte aligned is only known at the call: room for
  // the copies is always counted when a size makes them needed, and else
  // when the caller says so.
  const bool padded = desc->unaligned || needs_padding(*desc, nullptr, nullptr, nullptr, nullptr) ||
                      desc->grad_ld % 8;
  if (kept) {
    Carver c(nullptr);
    take_kept(c, z, keeps_codes(*desc));
    *kept = c.used;
  }
  if (forward_work) {
    Carver c(nullptr);
    take_forward(c, z, false, padded);
    *forward_work = c.used;
  }
  if (backward_work) {
    Carver c(nullptr);
    take_backward(c, z, desc->dtype == SPGEMM_F16, keeps_codes(*desc), padded);
    *backward_work = c.used;
  }
  return SPGEMM_OK;
}

extern "C" spgemm_status spgemm_experts_forward(const spgemm_experts_desc* desc, const void* dX,
                                                const void* dWIn, const void* dWOut,
                                                const int32_t* dCol, const float* dVal, void* dY,
                                                void* dKept, void* dWork, int64_t work_bytes,
                                                void* stream) {
  const spgemm_status st = check_desc(desc);
  if (st != SPGEMM_OK || desc->tokens == 0) return st;
  if (!dX || !dWIn || !dWOut || !dCol || !dVal || !dY || !dWork)
    return refuse(SPGEMM_ERR_INVALID_ARG, "experts: null array");
  const Sizes z = sizes_of(*desc);
  Carver c(dWork);
  const ForwardWork w =
      take_forward(c, z, dKept != nullptr, needs_padding(*desc, dX, dWIn, dWOut, nullptr));
  if (work_bytes < c.used) return refuse(SPGEMM_ERR_INVALID_ARG, "experts: workspace too small");
  (void)hipGetLastError();  // an error that earlier calls left is not this one's
  const hipStream_t s = (hipStream_t)stream;
  if (desc->dtype == SPGEMM_BF16)
    forward<__bf16>(*desc, dX, dWIn, dWOut, dCol, dVal, dY, dKept, w, s);
  else
    forward<_Float16>(*desc, dX, dWIn, dWOut, dCol, dVal, dY, dKept, w, s);
  return launched();
}

extern "C" spgemm_status spgemm_experts_backward(
    const spgemm_experts_desc* desc, const void* dX, const void* dWIn, const void* dWOut,
    const void* dGradY, const void* dKept, void* dGradX, void* dGradWIn,
    void* dGradWOut, float* dGradVal, void* dWork, int64_t work_bytes, void* stream) {
  const spgemm_status st = check_desc(desc);
  if (st != SPGEMM_OK) return st;
  if (!dGradWIn || !dGradWOut || !dWork ||
      (desc->tokens > 0 &&
       ((!dX && !keeps_codes(*desc)) || !dWIn || !dWOut || !dGradY || !dKept || !dGradX ||
        !dGradVal)))
    return refuse(SPGEMM_ERR_INVALID_ARG, "experts: null array");
  if (desc->grad_ld < desc->width)
    return refuse(SPGEMM_ERR_INVALID_ARG, "experts: a row stride below the width");
  const Sizes z = sizes_of(*desc);
  (void)hipGetLastError();  // an error that earlier calls left is not this one's
  const hipStream_t s = (hipStream_t)stream;
  if (desc->tokens == 0) {
    const int64_t n1 = z.E * 2 * z.F * z.D, n2 = z.E * z.D * z.F;
    hipLaunchKernelGGL(k_zero16, dim3(grid_for(n1)), dim3(256), 0, s, (uint16_t*)dGradWIn, n1);
    hipLaunchKernelGGL(k_zero16, dim3(grid_for(n2)), dim3(256), 0, s, (uint16_t*)dGradWOut, n2);
    return launched();
  }
  Carver c(dWork);
  const BackwardWork w =
      take_backward(c, z, desc->dtype == SPGEMM_F16, keeps_codes(*desc),
                    needs_padding(*desc, keeps_codes(*desc) ? nullptr : dX, dWIn, dWOut, dGradY));
  if (work_bytes < c.used) return refuse(SPGEMM_ERR_INVALID_ARG, "experts: workspace too small");
  if (desc->dtype == SPGEMM_BF16)
    backward<__bf16>(*desc, dX, dWIn, dWOut, dGradY, dKept, dGradX, dGradWIn, dGradWOut,
                     dGradVal, w, s);
  else
    backward<_Float16>(*desc, dX, dWIn, dWOut, dGradY, dKept, dGradX, dGradWIn, dGradWOut,
                       dGradVal, w, s);
  return launched();
}
