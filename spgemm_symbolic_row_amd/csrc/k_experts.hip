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
// from K-slices of 64 staged in LDS (two stages), its waves multiply 16x16x32
// MFMA blocks with fp32 accumulators.  An operand tile lies in LDS in one of
// two forms, both filled by 16-byte global-to-LDS loads whose lane-linear
// destination is permuted by choosing the source address:
//   row form (K contiguous in memory): [row][64 k], 16-byte chunk c of row r
//     at slot c ^ (r & 7); fragments are ds_read_b128.
//   column form (K strided): [k][column], the 32-byte segment s of row k at
//     segment s ^ f(k), f(k) = (k & 3) | (k >> 3 & 1) << 2; fragments are two
//     transposing 8-byte reads.  The xor spreads the 16 k-rows that one read
//     touches over the banks.
// Rows that a tile has not, and K beyond its end, are read from a block of
// zeros, so no tile ever multiplies foreign data.
#include <algorithm>

#include "expert_common.hpp"

namespace sg {
namespace {

constexpr int kBK = 64;  // K of one stage

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
template <typename T>
struct Vec8 { typedef T type __attribute__((ext_vector_type(8))); };

__device__ __forceinline__ f32x4 mfma(__bf16, s16x8 a, s16x8 b, f32x4 c) {
  typedef __bf16 v8 __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a),
                                                 __builtin_bit_cast(v8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(_Float16, s16x8 a, s16x8 b, f32x4 c) {
  typedef _Float16 v8 __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a),
                                                __builtin_bit_cast(v8, b), c, 0, 0, 0);
}

static __device__ __align__(16) const uint32_t zeros16[4] = {0, 0, 0, 0};

// 64 lanes x 16 bytes from each lane's address to LDS, lane-linear from
// `lds` (uniform).  Nothing waits for it but wait_stage(): the compiler, which
// would wait before the next LDS read, does not see it.  A load to LDS must
// not follow a write of M0 at once, hence the s_nop.
__device__ __forceinline__ void load_to_lds(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds),
               "v"(p)
               : "memory");
}
// The wave's loads to LDS and its LDS reads are done, then all waves' are.
__device__ __forceinline__ void wait_stage() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ s16x8 lds_read8(uint32_t a) {
  return *(const __attribute__((address_space(3))) s16x8*)a;
}
__device__ __forceinline__ s16x4 lds_read_tr(uint32_t a) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)a);
}

// ---- operand tiles ----

// Row form: ROWS rows of K, loaded by NW waves.
template <int ROWS, int NW>
struct RowTile {
  static constexpr int kBytes = ROWS * kBK * 2;
  static constexpr int kLoads = kBytes / (NW * 1024);
  static_assert(kLoads * NW * 1024 == kBytes, "tile must divide over the waves");
  const char* p[kLoads];  // the lane's chunk of row i in the current slice
  int k;                  // its first k there
  __device__ static int row(int i) {
    return (i * NW + (int)threadIdx.x / kWave) * 8 + lane_id() / 8;
  }
  __device__ static int chunk() { return (lane_id() & 7) ^ (lane_id() >> 3); }
  __device__ void start() { k = chunk() * 8; }
  // `src` is row i's first element, null for a row that is not there.
  __device__ void set_row(int i, const void* src) {
    p[i] = src ? (const char*)src + chunk() * 16 : nullptr;
  }
  __device__ void load(uint32_t lds, int wave, int K) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const bool ok = p[i] && k < K;
      load_to_lds(ok ? p[i] : (const char*)zeros16, lds + (i * NW + wave) * 1024);
      if (p[i]) p[i] += kBK * 2;
    }
    k += kBK;
  }
  // Fragment addresses: rows row0 + 16 m + lane % 16, K step kk of 32.
  uint32_t base;
  uint32_t swz;
  __device__ void frag_init(int row0) {
    const int l = lane_id();
    base = (row0 + (l & 15)) * (kBK * 2);
    swz = ((l >> 4) ^ (l & 7)) * 16;
  }
  __device__ s16x8 frag(uint32_t lds, int m, int kk) const {
    return lds_read8(lds + base + m * 16 * kBK * 2 + (swz ^ (kk * 64)));
  }
};

// Column form: 64 k-rows of COLS columns.
template <int COLS, int NW>
struct ColTile {
  static constexpr int kBytes = COLS * kBK * 2;
  static constexpr int kLoads = kBytes / (NW * 1024);
  static constexpr int kRowBytes = COLS * 2;
  static constexpr int kRowsPerLoad = 1024 / kRowBytes;
  static_assert(kLoads * NW * 1024 == kBytes && kRowsPerLoad >= 1, "tile over the waves");
  __device__ static int f(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }
  // k-row of load i within the slice.
  __device__ static int row(int i) {
    return (i * NW + (int)threadIdx.x / kWave) * kRowsPerLoad + lane_id() * 16 / kRowBytes;
  }
  // First column of the lane's chunk in load i (the same for every slice).
  __device__ static int col(int i) {
    const int c = lane_id() % (kRowBytes / 16);
    const int seg = c >> 1;
    return (((seg & ~7) | ((seg ^ f(row(i))) & 7)) * 2 + (c & 1)) * 8;
  }
  __device__ static void load(uint32_t lds, int wave, int i, const void* src) {
    load_to_lds(src ? src : (const void*)zeros16, lds + (i * NW + wave) * 1024);
  }
  uint32_t base;
  int seg0, fk;
  __device__ void frag_init(int col0) {
    const int l = lane_id(), k = (l >> 4) * 8 + ((l & 15) >> 2);
    fk = f(k);
    seg0 = col0 / 16;
    base = k * kRowBytes + (l & 3) * 8;
  }
  __device__ s16x8 frag(uint32_t lds, int m, int kk) const {
    const int s = seg0 + m;
    const uint32_t a =
        lds + base + ((s & ~7) | ((s ^ fk) & 7)) * 32 + kk * 32 * kRowBytes;
    const s16x4 lo = lds_read_tr(a), hi = lds_read_tr(a + 4 * kRowBytes);
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
  const float* val;
  float* dval_part;  // per entry: one partial sum of each 64 columns
  int parts;
};

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

// Work group -> tile.  Work groups go round-robin to the XCDs, so XCD x takes
// a contiguous share of the tiles; inside it they come as groups of 8 row
// tiles by all column tiles, which keeps a group's rows and weights in its L2.
__device__ __forceinline__ bool tile_of(int rows, int cols, int& tr, int& tc) {
  const int total = rows * cols, share = (total + kXcds - 1) / kXcds;
  const int b = blockIdx.x, at = b / kXcds;
  const int lin = (b % kXcds) * share + at;
  if (at >= share || lin >= total) return false;
  const int group = lin / (8 * cols), r = lin % (8 * cols);
  const int gr = min(8, rows - group * 8);
  tr = group * 8 + r % gr;
  tc = r / gr;
  return true;
}

template <typename T, int KIND, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * kWave) void k_product(ProductArgs a) {
  constexpr int NW = WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
  constexpr bool kWGrad = KIND == kGradWOut || KIND == kGradWIn;
  constexpr bool kACol = kWGrad, kBCol = kWGrad || KIND == kGradH || KIND == kGradX;
  constexpr int kStage = (BM + BN) * kBK * 2;
  extern __shared__ char smem[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN, l = lane_id();

  // Which tile: expert, its rows, first row and column of the result.
  int expert, row0, rows, n0;  // row0: first sorted position, rows: how many
  int m0 = 0;                  // weight gradients: first row of the result
  constexpr int kNStep = KIND == kIn ? BN / 2 : BN;
  const int cols = (a.N + kNStep - 1) / kNStep;
  int tr, tc;
  if constexpr (kWGrad) {
    const int mts = (a.M + BM - 1) / BM;
    if (!tile_of(a.E * mts, cols, tr, tc)) return;
    expert = tr / mts;
    m0 = tr % mts * BM;
    row0 = a.d.row_ptr[expert];
    rows = a.d.row_ptr[expert + 1] - row0;
  } else {
    if (!tile_of(*a.d.ntiles, cols, tr, tc)) return;
    expert = a.d.tiles[2 * tr];
    row0 = a.d.tiles[2 * tr + 1];
    rows = min(BM, a.d.row_ptr[expert + 1] - row0);
  }
  n0 = tc * kNStep;
  const int K = kWGrad ? rows : a.K;
  const int slices = (K + kBK - 1) / kBK;

  const T* A = (const T*)a.a;
  const T* B = (const T*)a.b + (kWGrad ? 0 : expert * a.b_expert);

  RowTile<BM, NW> ar;
  RowTile<BN, NW> br;
  ColTile<BM, NW> ac;
  ColTile<BN, NW> bc;
  // Sorted tokens of the next slice's rows (weight gradients).
  constexpr int AL = ColTile<BM, NW>::kLoads, BL = ColTile<BN, NW>::kLoads;
  int ai[AL], bi[BL];

  if constexpr (!kACol) {
    ar.start();
#pragma unroll
    for (int i = 0; i < RowTile<BM, NW>::kLoads; ++i) {
      const int r = ar.row(i);
      const T* src = nullptr;
      if (r < rows) {
        const int64_t at = KIND == kIn || KIND == kGradH ? a.d.tok[row0 + r] : row0 + r;
        src = A + at * a.lda;
      }
      ar.set_row(i, src);
    }
    ar.frag_init(wm * (BM / WM));
  } else {
    ac.frag_init(wm * (BM / WM));
  }
  if constexpr (!kBCol) {
    br.start();
#pragma unroll
    for (int i = 0; i < RowTile<BN, NW>::kLoads; ++i) {
      const int r = br.row(i);
      int64_t n;
      if constexpr (KIND == kIn) {
        // Each wave's columns: half gate rows, then the same rows of up.
        constexpr int H = BN / WN / 2;
        const int f = n0 + r / (2 * H) * H + r % H;
        n = f < a.N ? (r % (2 * H) < H ? f : a.N + f) : -1;
      } else {
        n = n0 + r < a.N ? n0 + r : -1;
      }
      br.set_row(i, n >= 0 ? B + n * a.ldb : nullptr);
    }
    br.frag_init(wn * (BN / WN));
  } else {
    bc.frag_init(wn * (BN / WN));
  }

  // Where the rows of slice s of a column-form operand are: the sorted
  // position itself, or its token.
  auto fetch_rows = [&](int s) {
    if constexpr (kWGrad) {
#pragma unroll
      for (int i = 0; i < AL; ++i) {
        const int r = s * kBK + ac.row(i);
        ai[i] = r < rows ? (KIND == kGradWOut ? a.d.tok[row0 + r] : row0 + r) : -1;
      }
#pragma unroll
      for (int i = 0; i < BL; ++i) {
        const int r = s * kBK + bc.row(i);
        bi[i] = r < rows ? (KIND == kGradWIn ? a.d.tok[row0 + r] : row0 + r) : -1;
      }
    }
  };
  auto load_slice = [&](int s) {
    const uint32_t lds = lds0 + (s & 1) * kStage;
    if constexpr (!kACol) {
      ar.load(lds, wave, a.Kpad);
    } else {
#pragma unroll
      for (int i = 0; i < AL; ++i) {
        const int c = m0 + ac.col(i);
        ac.load(lds, wave, i, ai[i] >= 0 && c < a.Mpad ? A + ai[i] * a.lda + c : nullptr);
      }
    }
    const uint32_t ldsb = lds + BM * kBK * 2;
    if constexpr (!kBCol) {
      br.load(ldsb, wave, a.Kpad);
    } else {
#pragma unroll
      for (int i = 0; i < BL; ++i) {
        const int c = n0 + bc.col(i);
        int64_t r;
        if constexpr (kWGrad) {
          r = bi[i];
        } else {
          r = s * kBK + bc.row(i);
          if (r >= K) r = -1;
        }
        bc.load(ldsb, wave, i, r >= 0 && c < a.Npad ? B + r * a.ldb + c : nullptr);
      }
    }
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0, 0, 0, 0};

  if (slices > 0) {
    fetch_rows(0);
    load_slice(0);
    fetch_rows(1);
    wait_stage();
  }
  for (int s = 0; s < slices; ++s) {
    if (s + 1 < slices) {
      load_slice(s + 1);
      fetch_rows(s + 2);
    }
    const uint32_t lds = lds0 + (s & 1) * kStage, ldsb = lds + BM * kBK * 2;
#pragma unroll
    for (int kk = 0; kk < kBK / 32; ++kk) {
      s16x8 fa[MT], fb[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) fb[n] = kBCol ? bc.frag(ldsb, n, kk) : br.frag(ldsb, n, kk);
#pragma unroll
      for (int m = 0; m < MT; ++m) fa[m] = kACol ? ac.frag(lds, m, kk) : ar.frag(lds, m, kk);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = mfma(T{}, fb[n], fa[m], acc[m][n]);
    }
    wait_stage();
  }

  // acc[m][n][j]: row wm*(BM/WM) + 16 m + l % 16, column 16 n + l / 16 * 4 + j
  // of the wave's part.
  if constexpr (KIND == kIn) {
    T* h = (T*)a.c;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = wm * (BM / WM) + m * 16 + (l & 15);
      if (r >= rows) continue;
#pragma unroll
      for (int n = 0; n < NT / 2; ++n) {
        const int f = n0 + wn * (BN / WN / 2) + n * 16 + (l >> 4) * 4;
        if (f >= a.Fpad) continue;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = acc[m][n][j];
          v[j] = x / (1.0f + expf(-x)) * acc[m][n + NT / 2][j];
        }
        const int64_t at = (int64_t)(row0 + r) * a.Fpad + f;
        store4(h + at, true, 4, v);
        if (a.g) {
          *(f32x4*)(a.g + at) = acc[m][n];
          *(f32x4*)(a.u + at) = acc[m][n + NT / 2];
        }
      }
    }
  } else if constexpr (KIND == kOut || KIND == kGradX) {
    float* c = (float*)a.c;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = wm * (BM / WM) + m * 16 + (l & 15);
      if (r >= rows) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int x = n0 + wn * (BN / WN) + n * 16 + (l >> 4) * 4;
        if (x < a.ldc) *(f32x4*)(c + (int64_t)(row0 + r) * a.ldc + x) = acc[m][n];
      }
    }
  } else if constexpr (KIND == kGradH) {
    T* dgu = (T*)a.c;
    T* hw = (T*)a.hw;
    const bool vec = a.F % 4 == 0;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = wm * (BM / WM) + m * 16 + (l & 15);
      float dot = 0.0f;
      if (r < rows) {
        const int64_t row = row0 + r;
        const float w = a.val[a.d.ent[row]];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int f = n0 + wn * (BN / WN) + n * 16 + (l >> 4) * 4;
          if (f >= a.Fpad) continue;
          const f32x4 g = *(const f32x4*)(a.g + row * a.Fpad + f);
          const f32x4 u = *(const f32x4*)(a.u + row * a.Fpad + f);
          float dg[4], du[4], hv[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float q = acc[m][n][j];
            const float s = 1.0f / (1.0f + expf(-g[j]));
            const float silu = g[j] * s, h = silu * u[j], dh = w * q;
            dot += h * q;
            dg[j] = dh * u[j] * s * (1.0f + g[j] * (1.0f - s));
            du[j] = dh * silu;
            hv[j] = w * h;
          }
          store4(hw + row * a.Fpad + f, true, 4, hv);
          T* o = dgu + row * a.ldc + f;
          store4(o, vec, a.F - f, dg);
          store4(o + a.F, vec, a.F - f, du);
        }
      }
      dot += __shfl_xor(dot, 16);
      dot += __shfl_xor(dot, 32);
      const int part = n0 / (BN / WN) + wn;
      if (l < 16 && r < rows && part < a.parts)
        a.dval_part[(int64_t)(row0 + r) * a.parts + part] = dot;
    }
  } else {
    T* c = (T*)a.c + expert * a.c_expert;
    const bool vec = a.ldc % 4 == 0 && (uintptr_t)a.c % 8 == 0;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = m0 + wm * (BM / WM) + m * 16 + (l & 15);
      if (r >= a.M) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int x = n0 + wn * (BN / WN) + n * 16 + (l >> 4) * 4;
        if (x >= a.N) continue;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = acc[m][n][j];
        store4(c + (int64_t)r * a.ldc + x, vec, a.N - x, v);
      }
    }
  }
}

template <typename T, int KIND, int BM, int BN, int WM, int WN>
void launch_product(const ProductArgs& a, int64_t row_tiles, hipStream_t s) {
  auto kernel = k_product<T, KIND, BM, BN, WM, WN>;
  static const bool once = (allow_max_dynamic_lds((const void*)kernel), true);
  (void)once;
  const int64_t step = KIND == kIn ? BN / 2 : BN;
  const int64_t tiles = row_tiles * ((a.N + step - 1) / step);
  const int64_t grid = (tiles + kXcds - 1) / kXcds * kXcds;
  if (grid == 0) return;
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(WM * WN * kWave),
                     2 * (BM + BN) * kBK * 2, s, a);
}

// ---- sums over a token's entries ----

// out[t] = sum over its entries of w * rows[pos] (w = 1 without val), in the
// entries' order, in fp32, rounded once.  One work group per token and 1024
// columns, 4 columns to a thread.
template <typename T>
__global__ __launch_bounds__(256) void k_combine(int64_t Tn, int k, int D, int Dpad,
                                                 const float* __restrict__ rows,
                                                 const int32_t* __restrict__ pos,
                                                 const float* __restrict__ val,
                                                 T* __restrict__ out) {
  const int blocks = (Dpad + 1023) / 1024;
  const int64_t t = blockIdx.x / blocks;
  const int x = (blockIdx.x % blocks) * 1024 + (int)threadIdx.x * 4;
  if (x >= D) return;
  float s[4] = {0, 0, 0, 0};
  for (int i = 0; i < k; ++i) {
    const int p = pos[t * k + i];
    if (p < 0) continue;
    const float w = val ? val[t * k + i] : 1.0f;
    const f32x4 v = *(const f32x4*)(rows + (int64_t)p * Dpad + x);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] += w * v[j];
  }
  store4(out + t * D + x, D % 4 == 0 && (uintptr_t)out % 8 == 0, D - x, s);
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

// Rows of a tile: 256 when the experts' rows fill such tiles to more than
// about half on average, else 128.
int tile_rows(const Sizes& z) { return z.n > 256 * z.E ? 256 : 128; }

// What the forward pass leaves for the backward pass.
struct Kept {
  Dispatch d;
  float* g;
  float* u;
};

void take_dispatch(Carver& c, const Sizes& z, Dispatch& d) {
  d.row_ptr = c.take<int32_t>(z.E + 1);
  d.ent = c.take<int32_t>(z.n);
  d.tok = c.take<int32_t>(z.n);
  d.pos = c.take<int32_t>(z.n);
  d.tiles = c.take<int32_t>(2 * dispatch_max_tiles(z.n, z.E, tile_rows(z)));
  d.ntiles = c.take<int32_t>(1);
}

Kept take_kept(Carver& c, const Sizes& z) {
  Kept k{};
  take_dispatch(c, z, k.d);
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
  float* part;
  Padded pad;
};

int dval_parts(const Sizes& z) { return (int)((z.Fp + 63) / 64); }

BackwardWork take_backward(Carver& c, const Sizes& z, bool padded) {
  BackwardWork w{};
  w.dgu = c.take<uint16_t>(z.n * z.S2);
  w.hw = c.take<uint16_t>(z.n * z.Fp);
  w.rows = c.take<float>(z.n * z.Dp);
  w.part = c.take<float>(z.n * dval_parts(z));
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

template <typename T, int KIND>
void product_by_rows(const ProductArgs& a, const Sizes& z, hipStream_t s) {
  const int bm = tile_rows(z);
  const int64_t tiles = dispatch_max_tiles(z.n, z.E, bm);
  if (bm == 256) launch_product<T, KIND, 256, 256, 2, 4>(a, tiles, s);
  else launch_product<T, KIND, 128, 256, 2, 4>(a, tiles, s);
}

ProductArgs base_args(const Sizes& z, const Dispatch& d) {
  ProductArgs a{};
  a.d = d;
  a.E = (int)z.E;
  a.F = (int)z.F;
  a.Fpad = (int)z.Fp;
  return a;
}

template <typename T>
void combine(const Sizes& z, const float* rows, const int32_t* pos, const float* val, void* out,
             hipStream_t s) {
  const int64_t blocks = (z.Dp + 1023) / 1024;
  hipLaunchKernelGGL((k_combine<T>), dim3((unsigned)(z.T * blocks)), dim3(256), 0, s, z.T, z.k,
                     (int)z.D, (int)z.Dp, rows, pos, val, (T*)out);
}

template <typename T>
void forward(const spgemm_experts_desc& desc, const void* x, const void* w_in, const void* w_out,
             const int32_t* col, const float* val, void* y, void* kept, const ForwardWork& w,
             hipStream_t s) {
  const Sizes z = sizes_of(desc);
  Kept kp{};
  if (kept) {
    Carver c(kept);
    kp = take_kept(c, z);
  } else {
    kp.d = w.d;
  }
  launch_dispatch(col, z.n, z.k, z.E, tile_rows(z), kp.d, w.tmp, s);
  const Rows xr = padded_rows(x, desc.x_ld, z.T, z.D, w.pad.x, s);
  const Rows w1 = padded_rows(w_in, z.D, z.E * 2 * z.F, z.D, w.pad.w_in, s);
  const Rows w2 = padded_rows(w_out, z.F, z.E * z.D, z.F, w.pad.w_out, s);
  ProductArgs a = base_args(z, kp.d);
  a.a = xr.p;
  a.lda = xr.ld;
  a.b = w1.p;
  a.ldb = w1.ld;
  a.b_expert = 2 * z.F * w1.ld;
  a.N = (int)z.F;
  a.K = (int)z.D;
  a.Kpad = (int)z.Dp;
  a.c = w.h;
  a.g = kp.g;
  a.u = kp.u;
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
  product_by_rows<T, kOut>(a, z, s);
  combine<T>(z, w.rows, kp.d.pos, val, y, s);
}

template <typename T>
void backward(const spgemm_experts_desc& desc, const void* x, const void* w_in,
              const void* w_out, const float* val, const void* dy, const void* kept, void* dx,
              void* dw_in, void* dw_out, float* dval, const BackwardWork& w, hipStream_t s) {
  const Sizes z = sizes_of(desc);
  Carver kc((void*)kept);
  const Kept kp = take_kept(kc, z);
  const Rows xr = padded_rows(x, desc.x_ld, z.T, z.D, w.pad.x, s);
  const Rows gr = padded_rows(dy, desc.grad_ld, z.T, z.D, w.pad.dy, s);
  const Rows w1 = padded_rows(w_in, z.D, z.E * 2 * z.F, z.D, w.pad.w_in, s);
  const Rows w2 = padded_rows(w_out, z.F, z.E * z.D, z.F, w.pad.w_out, s);
  if (z.S2 != 2 * z.F)
    hipLaunchKernelGGL(k_zero16, dim3(grid_for(z.n * z.S2)), dim3(256), 0, s, w.dgu, z.n * z.S2);
  ProductArgs a = base_args(z, kp.d);
  a.a = gr.p;
  a.lda = gr.ld;
  a.b = w2.p;
  a.ldb = w2.ld;
  a.b_expert = z.D * w2.ld;
  a.N = a.Npad = (int)z.Fp;
  a.K = (int)z.D;
  a.Kpad = (int)z.Dp;
  a.c = w.dgu;
  a.ldc = z.S2;
  a.g = kp.g;
  a.u = kp.u;
  a.hw = w.hw;
  a.val = val;
  a.dval_part = w.part;
  a.parts = dval_parts(z);
  product_by_rows<T, kGradH>(a, z, s);
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
  combine<T>(z, w.rows, kp.d.pos, nullptr, dx, s);
  hipLaunchKernelGGL(k_dval, dim3((unsigned)((z.n + 255) / 256)), dim3(256), 0, s, z.n,
                     dval_parts(z), kp.d.pos, w.part, dval);
  a = base_args(z, kp.d);
  a.a = gr.p;
  a.lda = gr.ld;
  a.b = w.hw;
  a.ldb = z.Fp;
  a.M = (int)z.D;
  a.Mpad = (int)z.Dp;
  a.N = (int)z.F;
  a.Npad = (int)z.Fp;
  a.c = dw_out;
  a.ldc = z.F;
  a.c_expert = z.D * z.F;
  launch_product<T, kGradWOut, 256, 256, 2, 4>(a, z.E * ((z.D + 255) / 256), s);
  a = base_args(z, kp.d);
  a.a = w.dgu;
  a.lda = z.S2;
  a.b = xr.p;
  a.ldb = xr.ld;
  a.M = (int)(2 * z.F);
  a.Mpad = (int)z.S2;
  a.N = (int)z.D;
  a.Npad = (int)z.Dp;
  a.c = dw_in;
  a.ldc = z.D;
  a.c_expert = 2 * z.F * z.D;
  launch_product<T, kGradWIn, 256, 256, 2, 4>(a, z.E * ((2 * z.F + 255) / 256), s);
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
  if (d->width > (1 << 24) || d->hidden > (1 << 24) ||
      d->tokens > INT32_MAX / d->k ||
      d->tokens * d->k / 128 + d->experts > INT32_MAX / ((d->width + d->hidden) / 128 + 1) / 2 ||
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
    take_kept(c, z);
    *kept = c.used;
  }
  if (forward_work) {
    Carver c(nullptr);
    take_forward(c, z, false, padded);
    *forward_work = c.used;
  }
  if (backward_work) {
    Carver c(nullptr);
    take_backward(c, z, padded);
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
  const hipStream_t s = (hipStream_t)stream;
  if (desc->dtype == SPGEMM_BF16)
    forward<__bf16>(*desc, dX, dWIn, dWOut, dCol, dVal, dY, dKept, w, s);
  else
    forward<_Float16>(*desc, dX, dWIn, dWOut, dCol, dVal, dY, dKept, w, s);
  return launched();
}

extern "C" spgemm_status spgemm_experts_backward(
    const spgemm_experts_desc* desc, const void* dX, const void* dWIn, const void* dWOut,
    const float* dVal, const void* dGradY, const void* dKept, void* dGradX, void* dGradWIn,
    void* dGradWOut, float* dGradVal, void* dWork, int64_t work_bytes, void* stream) {
  const spgemm_status st = check_desc(desc);
  if (st != SPGEMM_OK) return st;
  if (!dGradWIn || !dGradWOut || !dWork ||
      (desc->tokens > 0 &&
       (!dX || !dWIn || !dWOut || !dVal || !dGradY || !dKept || !dGradX || !dGradVal)))
    return refuse(SPGEMM_ERR_INVALID_ARG, "experts: null array");
  if (desc->grad_ld < desc->width)
    return refuse(SPGEMM_ERR_INVALID_ARG, "experts: a row stride below the width");
  const Sizes z = sizes_of(*desc);
  const hipStream_t s = (hipStream_t)stream;
  if (desc->tokens == 0) {
    const int64_t n1 = z.E * 2 * z.F * z.D, n2 = z.E * z.D * z.F;
    hipLaunchKernelGGL(k_zero16, dim3(grid_for(n1)), dim3(256), 0, s, (uint16_t*)dGradWIn, n1);
    hipLaunchKernelGGL(k_zero16, dim3(grid_for(n2)), dim3(256), 0, s, (uint16_t*)dGradWOut, n2);
    return launched();
  }
  Carver c(dWork);
  const BackwardWork w = take_backward(c, z, needs_padding(*desc, dX, dWIn, dWOut, dGradY));
  if (work_bytes < c.used) return refuse(SPGEMM_ERR_INVALID_ARG, "experts: workspace too small");
  if (desc->dtype == SPGEMM_BF16)
    backward<__bf16>(*desc, dX, dWIn, dWOut, dVal, dGradY, dKept, dGradX, dGradWIn, dGradWOut,
                     dGradVal, w, s);
  else
    backward<_Float16>(*desc, dX, dWIn, dWOut, dVal, dGradY, dKept, dGradX, dGradWIn, dGradWOut,
                       dGradVal, w, s);
  return launched();
}
