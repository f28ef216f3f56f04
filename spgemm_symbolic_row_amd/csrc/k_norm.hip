// Layer norm and its gradient.  A row x of D columns:
//   m = sum x / D,  r = 1 / sqrt(sum (x - m)^2 / D + eps),  n = (x - m) r,
//   y = n w + b;
// and for the gradient dy, with a = dy w:
//   dx = r (a - sum a / D - n sum (a n) / D),  dw = sum over rows of dy n,
//   db = sum over rows of dy.
//
// L lanes take a row, 8 columns to a lane, so a row is read once and stays in
// registers; the sum of squares is taken about the mean, which loses nothing in
// rows whose mean is large.  The gradient from rows in 8 bits does: it takes n at the
// rounded row, which is 2^-4 |x| off, a whole deviation where the mean is 16 of them.
// R rows at once keep enough loads in flight.  The gradient's work groups take rows in
// turn and keep their share of dw and db in registers; one partial row of each work
// group is then summed by a second kernel, in an order that the sizes alone fix.  Sums
// are in 32 bits.
//
// Both passes are bound by their bytes: 16384 x 2048 bfloat16 forward 24 us (5.6
// TB/s; a large copy runs at 4.9), 6000 x 4096 fp32 forward 39 and backward 54 us (5.1
// and 5.5 TB/s), 32768 x 2048 bfloat16 kept in 8 bits forward 65 and backward 70 us (5.2
// and 4.8 TB/s), the sum of the partial rows 4 to 6 more.  Work groups of L = NT threads
// hold a row of up to 8192 columns at 8 to a lane; rows of up to 128 columns go
// four to a wave, which at 64 lanes to a row would leave three quarters idle.
#include <algorithm>

#include "rows8.hpp"

namespace sg {
namespace {

enum Form { kPlain, kStats, kCodes };  // what is kept: nothing, m and r, and the rows in 8 bits

struct NormArgs {
  const void* x;
  int64_t x_ld;
  const void* weight;
  const void* bias;
  void* y;
  const void* dy;
  int64_t dy_ld;
  void* dx;
  float* mean;
  float* rstd;
  uint8_t* code;
  uint8_t* scale;
  float* part;  // by work group: D sums of dy n, then D of dy
  int64_t T;
  int D;
  bool w32;     // weight and bias are fp32
  float eps, inv_D;
};

template <typename T>
__device__ __forceinline__ void load_weight(const void* w, bool w32, int c, int n, float v[8]) {
  if (w32) load8_any((const float*)w + c, n, v);
  else load8_any((const T*)w + c, n, v);
}

// Sums of N values over the L lanes of a row, in all of them.  `red` is LDS for
// N * (waves of the work group) values, not the one of the call before.
template <int L, int NT, int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float* red) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (L == 16) {
      s[i] = dpp_add<0x128, 0xf>(s[i]);
      s[i] = dpp_add<0x124, 0xf>(s[i]);
      s[i] = dpp_add<0x122, 0xf>(s[i]);
      s[i] = dpp_add<0x121, 0xf>(s[i]);
    } else {
      s[i] = wave_sum_f32(s[i]);
    }
  }
  if constexpr (L > kWave) {
    constexpr int kOf = L / kWave;  // waves of a row
    const int wave = threadIdx.x / kWave;
    if (lane_id() == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[i * (NT / kWave) + wave] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float* p = red + i * (NT / kWave) + wave / kOf * kOf;
      float t = 0.0f;
#pragma unroll
      for (int j = 0; j < kOf; ++j) t += p[j];
      s[i] = t;
    }
  }
}

template <typename T, int L, int NT, int V, int R, int FORM>
__global__ __launch_bounds__(NT) void k_norm(NormArgs a) {
  __shared__ float red[2][R * NT / kWave];
  constexpr int kGroups = NT / L;
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int64_t t0 = ((int64_t)blockIdx.x * kGroups + group) * R;
  float x[R][V][8];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * L + lane) * 8;
      load8_any((const T*)a.x + (t0 + r) * a.x_ld + c, t0 + r < a.T ? a.D - c : 0, x[r][v]);
    }
  float w[V][8], b[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * L + lane) * 8;
    load_weight<T>(a.weight, a.w32, c, a.D - c, w[v]);
    if (a.bias) {
      load_weight<T>(a.bias, a.w32, c, a.D - c, b[v]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) b[v][j] = 0.0f;
    }
  }
  if constexpr (FORM == kCodes) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * L + lane) * 8;
        uint32_t scale;
        const uint2 q = kept_encode<T>(x[r][v], scale);
        if (t0 + r < a.T && c < a.D) {
          *(uint2*)(a.code + (t0 + r) * kept_pitch(a.D) + c) = q;
          if (c % kKeptBlock == 0)
            a.scale[(t0 + r) * kept_blocks(a.D) + c / kKeptBlock] = (uint8_t)scale;
        }
      }
  }
  float mean[R], var[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    mean[r] = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) mean[r] += x[r][v][j];
  }
  row_sums<L, NT, R>(mean, red[0]);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    mean[r] *= a.inv_D;
    var[r] = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = x[r][v][j] - mean[r];
        x[r][v][j] = d;
        if ((v * L + lane) * 8 + j < a.D) var[r] += d * d;
      }
  }
  row_sums<L, NT, R>(var, red[1]);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (t0 + r >= a.T) break;
    const float rstd = 1.0f / sqrtf(var[r] * a.inv_D + a.eps);
    if (FORM != kPlain && lane == 0) {
      a.mean[t0 + r] = mean[r];
      a.rstd[t0 + r] = rstd;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * L + lane) * 8;
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = x[r][v][j] * rstd * w[v][j] + b[v][j];
      store8_any((T*)a.y + (t0 + r) * a.D + c, a.D - c, y);
    }
  }
}

// A lane's part of a row of the gradient as it lies in memory.
template <typename T, int V, int FORM>
struct RawRow {
  typedef T V8 __attribute__((ext_vector_type(8)));
  V8 dy[V], x[V];
  uint2 code[V];
  uint32_t scale[V];
  float mean, rstd;
};

template <typename T, typename V8>
__device__ __forceinline__ V8 load_raw(const T* p, int n) {
  typedef V8 Any __attribute__((aligned(1)));
  if (n >= 8) return *(const Any*)p;
  V8 v;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < n ? p[j] : (T)0.0f;
  return v;
}

template <typename T, int L, int NT, int V, int R, int FORM>
__global__ __launch_bounds__(NT) void k_norm_grad(NormArgs a) {
  constexpr int kGroups = NT / L;
  __shared__ float red[2][2 * R * NT / kWave];
  __shared__ float sums[kGroups > 1 ? 2 * NT * 8 : 1];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  typedef RawRow<T, V, FORM> Raw;
  auto fetch = [&](Raw (&raw)[R], int64_t t0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t t = t0 + r;
      const bool inside = t < a.T;
      raw[r].mean = inside ? a.mean[t] : 0.0f;
      raw[r].rstd = inside ? a.rstd[t] : 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * L + lane) * 8, left = inside ? a.D - c : 0;
        raw[r].dy[v] = load_raw<T, typename Raw::V8>((const T*)a.dy + t * a.dy_ld + c, left);
        if constexpr (FORM == kCodes) {
          raw[r].code[v] = uint2{0, 0};
          raw[r].scale[v] = 0;
          if (left > 0) {
            raw[r].code[v] = *(const uint2*)(a.code + t * kept_pitch(a.D) + c);
            raw[r].scale[v] = a.scale[t * kept_blocks(a.D) + c / kKeptBlock];
          }
        } else {
          raw[r].x[v] = load_raw<T, typename Raw::V8>((const T*)a.x + t * a.x_ld + c, left);
        }
      }
    }
  };
  // Every work group takes the same number of turns, so that all lanes of a row meet.
  // The rows of the next turn are loaded ahead, but not those of two chunks, which do not fit
  // the registers (2000 x 16384 fp32 152 us, without 95).
  constexpr bool kAhead = V == 1;
  const int64_t step = (int64_t)gridDim.x * kGroups * R;
  Raw raw[R];
  if (kAhead) fetch(raw, (int64_t)blockIdx.x * kGroups * R + group * R);
  float w[V][8], dw[V][8], db[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * L + lane) * 8;
    load_weight<T>(a.weight, a.w32, c, a.D - c, w[v]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[v][j] = db[v][j] = 0.0f;
  }
  int turn = 0;
#pragma unroll 1
  for (int64_t base = (int64_t)blockIdx.x * kGroups * R; base < a.T; base += step, ++turn) {
    const int64_t t0 = base + group * R;
    float n[R][V][8], g[R][V][8], rstd[R], s[2 * R];
    auto work = [&](const Raw (&raw)[R]) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s[2 * r] = s[2 * r + 1] = 0.0f;
        rstd[r] = raw[r].rstd;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if constexpr (FORM == kCodes) {
            kept_decode(raw[r].code[v], raw[r].scale[v], n[r][v]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) n[r][v][j] = to_f32(raw[r].x[v][j]);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) n[r][v][j] = (n[r][v][j] - raw[r].mean) * rstd[r];
          // Columns beyond the row have no dy; their -m r may be infinite where n is not.
          const int left = a.D - (v * L + lane) * 8;
          if (left < 8)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j >= left) n[r][v][j] = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float gj = to_f32(raw[r].dy[v][j]), aj = gj * w[v][j], nj = n[r][v][j];
            g[r][v][j] = gj;
            db[v][j] += gj;
            dw[v][j] += gj * nj;
            s[2 * r] += aj;
            s[2 * r + 1] += aj * nj;
          }
        }
      }
    };
    if (!kAhead) fetch(raw, t0);
    work(raw);
    if (kAhead) {
      __builtin_amdgcn_sched_barrier(0);
      fetch(raw, t0 + step);
      __builtin_amdgcn_sched_barrier(0);
    }
    row_sums<L, NT, 2 * R>(s, red[turn & 1]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (t0 + r >= a.T) break;
      const float s1 = s[2 * r] * a.inv_D, s2 = s[2 * r + 1] * a.inv_D;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * L + lane) * 8;
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          d[j] = rstd[r] * (g[r][v][j] * w[v][j] - s1 - n[r][v][j] * s2);
        store8_any((T*)a.dx + (t0 + r) * a.D + c, a.D - c, d);
      }
    }
  }
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.D;
  if constexpr (kGroups > 1) {
    static_assert(V == 1, "rows of one work group side by side");
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sums[threadIdx.x * 8 + j] = dw[0][j];
      sums[NT * 8 + threadIdx.x * 8 + j] = db[0][j];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * L * 8; c += NT) {
      const int which = c / (L * 8), col = c % (L * 8);
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) t += sums[which * NT * 8 + i * L * 8 + col];
      if (col < a.D) out[which * a.D + col] = t;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * L + lane) * 8;
      store8_any(out + c, a.D - c, dw[v]);
      store8_any(out + a.D + c, a.D - c, db[v]);
    }
  }
}

// dw and db from the work groups' partial rows: 64 columns to a work group, 16
// shares of the rows.
__global__ __launch_bounds__(1024) void k_norm_sum(const float* __restrict__ part, int rows, int D,
                                                   void* __restrict__ dw, void* __restrict__ db,
                                                   spgemm_dtype type) {
  __shared__ float sums[16][64];
  const int c = blockIdx.x * 64 + threadIdx.x % 64, share = threadIdx.x / 64;
  const int all = db ? 2 * D : D;
  float s = 0.0f;
  if (c < all) {
#pragma unroll 8
    for (int r = share; r < rows; r += 16) s += part[(int64_t)r * 2 * D + c];
  }
  sums[share][threadIdx.x % 64] = s;
  __syncthreads();
  if (share || c >= all) return;
  for (int i = 1; i < 16; ++i) s += sums[i][threadIdx.x];
  void* out = c < D ? dw : db;
  const int at = c < D ? c : c - D;
  if (type == SPGEMM_F32) ((float*)out)[at] = s;
  else if (type == SPGEMM_BF16) ((__bf16*)out)[at] = from_f32<__bf16>(s);
  else ((_Float16*)out)[at] = from_f32<_Float16>(s);
}

constexpr int64_t kMostColumns = 16384;

// Work groups of a gradient, each of which leaves a partial row: three of 256 threads
// to a compute unit, else one.  More run at a time, but leave more partial rows.  us of the
// backward pass:
//   256 threads, work groups        512   768  1024  1536
//     32768 x 2048 bf16              83    82    96    89
//     the same kept in 8 bits        80    73    84    77
//     65536 x 256 bf16               45    36    34    40
//     4099 x 1001 fp16               17    18    22    21
//   512 and 1024 threads            128   192   256   384   512
//     6000 x 4096 fp32               66    56    54    62    62
//     2000 x 4096 bf16               20    18    17    20    22
//     8192 x 8192 bf16              105    84    84    91    89
//     2000 x 16384 fp32             120   100    96   107   109
int64_t grad_groups(int64_t T, int64_t rows, int threads) {
  const int64_t most = threads == 256 ? 768 : 256;
  return std::max<int64_t>(1, std::min((T + rows - 1) / rows, most));
}

template <typename T, int L, int NT, int V, int R, int RG>
struct Shape {
  static void forward(const NormArgs& a, int form, hipStream_t s) {
    constexpr int64_t rows = NT / L * R;
    const dim3 grid((unsigned)((a.T + rows - 1) / rows));
    if (form == kPlain)
      hipLaunchKernelGGL((k_norm<T, L, NT, V, R, kPlain>), grid, dim3(NT), 0, s, a);
    else if (form == kStats)
      hipLaunchKernelGGL((k_norm<T, L, NT, V, R, kStats>), grid, dim3(NT), 0, s, a);
    else
      hipLaunchKernelGGL((k_norm<T, L, NT, V, R, kCodes>), grid, dim3(NT), 0, s, a);
  }
  // Work items of a forward launch.
  static int64_t items(int64_t T_) { return (T_ + NT / L * R - 1) / (NT / L * R) * NT; }
  static int64_t groups(int64_t T_) { return grad_groups(T_, NT / L * RG, NT); }
  static void backward(const NormArgs& a, int form, hipStream_t s) {
    const dim3 grid((unsigned)groups(a.T));
    if (form == kStats)
      hipLaunchKernelGGL((k_norm_grad<T, L, NT, V, RG, kStats>), grid, dim3(NT), 0, s, a);
    else
      hipLaunchKernelGGL((k_norm_grad<T, L, NT, V, RG, kCodes>), grid, dim3(NT), 0, s, a);
  }
};

// Calls f with the shape for rows of D columns.
template <typename T, typename F>
auto by_width(int64_t D, F f) {
  if (D <= 128) return f(Shape<T, 16, 256, 1, 4, 2>{});
  if (D <= 512) return f(Shape<T, 64, 256, 1, 4, 2>{});
  if (D <= 1024) return f(Shape<T, 128, 256, 1, 4, 2>{});
  if (D <= 2048) return f(Shape<T, 256, 256, 1, 4, 2>{});
  if (D <= 4096) return f(Shape<T, 512, 512, 1, 2, 2>{});
  if (D <= 8192) return f(Shape<T, 1024, 1024, 1, 1, 1>{});
  return f(Shape<T, 1024, 1024, 2, 1, 1>{});
}

template <typename F>
auto by_type(spgemm_dtype t, F f) {
  if (t == SPGEMM_F32) return f(float{});
  if (t == SPGEMM_BF16) return f(__bf16{});
  return f(_Float16{});
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

spgemm_status check_desc(const spgemm_layer_norm_desc* d) {
  if (!d) return refuse(SPGEMM_ERR_INVALID_ARG, "layer_norm: null description");
  if (d->dtype != SPGEMM_F32 && d->dtype != SPGEMM_BF16 && d->dtype != SPGEMM_F16)
    return refuse(SPGEMM_ERR_INVALID_ARG, "layer_norm: rows must be fp32, bf16 or fp16");
  if (d->weight_dtype != SPGEMM_F32 && d->weight_dtype != d->dtype)
    return refuse(SPGEMM_ERR_INVALID_ARG, "layer_norm: weights must be fp32 or of the rows' type");
  if (d->rows < 0 || d->width < 1 || d->width > kMostColumns)
    return refuse(SPGEMM_ERR_INVALID_ARG, "layer_norm: rows < 0, or a width outside [1, 16384]");
  if (d->x_ld < d->width || d->grad_ld < d->width)
    return refuse(SPGEMM_ERR_INVALID_ARG, "layer_norm: a row stride below the width");
  if (!(d->eps >= 0.0f) || d->eps > 3.4e38f)
    return refuse(SPGEMM_ERR_INVALID_ARG, "layer_norm: eps must be finite and not negative");
  if (d->kept_form < 0 || d->kept_form > 2)
    return refuse(SPGEMM_ERR_INVALID_ARG, "layer_norm: kept_form outside [0, 2]");
  if (d->rows > INT32_MAX || d->x_ld >= 1 << 30 || d->grad_ld >= 1 << 30)
    return refuse(SPGEMM_ERR_INDEX_OVERFLOW, "layer_norm: 2^31 rows, or a stride of 2^30, or more");
  // A launch takes fewer than 2^32 work items.
  if (by_type(d->dtype, [&](auto t) {
        return by_width<decltype(t)>(d->width, [&](auto shape) { return shape.items(d->rows); });
      }) >= (int64_t)1 << 32)
    return refuse(SPGEMM_ERR_INDEX_OVERFLOW, "layer_norm: more rows than one launch takes");
  return SPGEMM_OK;
}

void take_kept(Carver& c, const spgemm_layer_norm_desc& d, NormArgs& a) {
  if (d.kept_form == kPlain) return;
  a.mean = c.take<float>(d.rows);
  a.rstd = c.take<float>(d.rows);
  if (d.kept_form != kCodes) return;
  a.code = c.take<uint8_t>(d.rows * kept_pitch(d.width));
  a.scale = c.take<uint8_t>(d.rows * kept_blocks(d.width));
}

int64_t work_groups(const spgemm_layer_norm_desc& d) {
  return by_type(d.dtype, [&](auto t) {
    return by_width<decltype(t)>(d.width, [&](auto shape) { return shape.groups(d.rows); });
  });
}

NormArgs args_of(const spgemm_layer_norm_desc& d, const void* x, const void* weight) {
  NormArgs a{};
  a.x = x;
  a.x_ld = d.x_ld;
  a.weight = weight;
  a.T = d.rows;
  a.D = (int)d.width;
  a.w32 = d.weight_dtype == SPGEMM_F32;
  a.eps = d.eps;
  a.inv_D = 1.0f / (float)d.width;
  return a;
}

}  // namespace
}  // namespace sg

using namespace sg;

extern "C" spgemm_status spgemm_layer_norm_sizes(const spgemm_layer_norm_desc* desc, int64_t* kept,
                                                 int64_t* backward_work) {
  const spgemm_status st = check_desc(desc);
  if (st != SPGEMM_OK) return st;
  if (kept) {
    Carver c(nullptr);
    NormArgs a{};
    take_kept(c, *desc, a);
    *kept = c.used;
  }
  if (backward_work) {
    Carver c(nullptr);
    c.take<float>(work_groups(*desc) * 2 * desc->width);
    *backward_work = c.used;
  }
  return SPGEMM_OK;
}

extern "C" spgemm_status spgemm_layer_norm_forward(const spgemm_layer_norm_desc* desc,
                                                   const void* dX, const void* dWeight,
                                                   const void* dBias, void* dY, void* dKept,
                                                   void* stream) {
  const spgemm_status st = check_desc(desc);
  if (st != SPGEMM_OK || desc->rows == 0) return st;
  if (!dX || !dWeight || !dY || (desc->kept_form != kPlain && !dKept))
    return refuse(SPGEMM_ERR_INVALID_ARG, "layer_norm: null array");
  NormArgs a = args_of(*desc, dX, dWeight);
  a.bias = dBias;
  a.y = dY;
  Carver c(dKept);
  take_kept(c, *desc, a);
  (void)hipGetLastError();  // an error that earlier calls left is not this one's
  by_type(desc->dtype, [&](auto t) {
    by_width<decltype(t)>(desc->width, [&](auto shape) {
      shape.forward(a, desc->kept_form, (hipStream_t)stream);
    });
  });
  return launched();
}

extern "C" spgemm_status spgemm_layer_norm_backward(const spgemm_layer_norm_desc* desc,
                                                    const void* dX, const void* dWeight,
                                                    const void* dGradY, const void* dKept,
                                                    void* dGradX, void* dGradWeight,
                                                    void* dGradBias, void* dWork,
                                                    int64_t work_bytes, void* stream) {
  const spgemm_status st = check_desc(desc);
  if (st != SPGEMM_OK) return st;
  if (desc->kept_form == kPlain)
    return refuse(SPGEMM_ERR_INVALID_ARG, "layer_norm: a backward pass needs what a forward kept");
  // Without rows the kernel that writes zeros reads the weight all the same.
  if (!dWeight || !dGradWeight || !dWork ||
      (desc->rows > 0 &&
       ((!dX && desc->kept_form == kStats) || !dGradY || !dKept || !dGradX)))
    return refuse(SPGEMM_ERR_INVALID_ARG, "layer_norm: null array");
  NormArgs a = args_of(*desc, dX, dWeight);
  a.dy = dGradY;
  a.dy_ld = desc->grad_ld;
  a.dx = dGradX;
  Carver kc((void*)dKept);
  take_kept(kc, *desc, a);
  const int64_t groups = work_groups(*desc);
  Carver c(dWork);
  a.part = c.take<float>(groups * 2 * desc->width);
  if (work_bytes < c.used) return refuse(SPGEMM_ERR_INVALID_ARG, "layer_norm: workspace too small");
  (void)hipGetLastError();  // an error that earlier calls left is not this one's
  const hipStream_t s = (hipStream_t)stream;
  // Without rows one work group leaves a partial row of zeros.
  by_type(desc->dtype, [&](auto t) {
    by_width<decltype(t)>(desc->width, [&](auto shape) { shape.backward(a, desc->kept_form, s); });
  });
  const int64_t cols = desc->width * (dGradBias ? 2 : 1);
  hipLaunchKernelGGL(k_norm_sum, dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, s, a.part,
                     (int)groups, (int)desc->width, dGradWeight, dGradBias, desc->weight_dtype);
  return launched();
}
