// The 2-norm over many tensors and the scaling that clips it:
//   norm = sqrt(sum of g^2),  out = g * min(1, max_norm / (norm + 1e-6)).
// Squares are summed in fp64, which no finite value overflows, in an order
// that only the sizes fix.  The first kernel leaves one partial sum per work
// group; each work group of the second adds them up again (at most 16 KB from
// L2, which costs less than a launch between) and scales its share.  Tables
// that do not fit one launch's arguments take several of each, and one work
// group between that adds all partial sums up.  Every element is read twice and
// written once; the bytes bound it (8 10^8 elements of two types, 2.1 GB: 1.27 ms,
// 5.0 TB/s, the rate of a device copy).  The scaling goes backwards, so that it
// begins with what the memory-side cache still holds.
#include <algorithm>

#include "expert_common.hpp"

namespace sg {
namespace {

constexpr int kGnNT = 256;
constexpr int kGnTable = 96;       // tensors of one launch (2.8 KB of kernel arguments)
constexpr int kGnParts = 2048;     // partial sums, and work groups, of one launch
constexpr int64_t kGnChunk = 16384;  // elements of one work item

struct GradTable {
  const void* in[kGnTable];
  void* out[kGnTable];
  int64_t n[kGnTable];
  int32_t first[kGnTable + 1];  // first work item of each tensor
  uint8_t type[kGnTable];       // spgemm_dtype of input (low 4 bits) and output
  int32_t count;
};

// The tensor that holds work item i.
__device__ __forceinline__ int tensor_of(const GradTable& t, int i) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ double sum_squares(const T* p, int64_t n) {
  constexpr int V = 16 / sizeof(T);
  double s = 0.0;
  int64_t at = 0;
  if ((uintptr_t)p % 16 == 0) {
    struct alignas(16) Pack { T v[V]; };
    const int64_t packs = n / V;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < packs; i += kGnNT) {
      const Pack q = ((const Pack*)p)[i];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const double x = (double)to_f32(q.v[j]);
        s = fma(x, x, s);
      }
    }
    at = packs * V;
  }
  for (int64_t i = at + threadIdx.x; i < n; i += kGnNT) {
    const double x = (double)to_f32(p[i]);
    s = fma(x, x, s);
  }
  return s;
}

// Sum over the work group, in every thread.
__device__ __forceinline__ double group_sum(double s) {
  __shared__ double part[kGnNT / kWave];
  s = wave_sum(s);
  if (lane_id() == 0) part[threadIdx.x / kWave] = s;
  __syncthreads();
  s = part[0];
  for (int w = 1; w < kGnNT / kWave; ++w) s += part[w];
  return s;
}

__global__ __launch_bounds__(kGnNT) void k_grad_squares(GradTable t, double* __restrict__ parts) {
  double s = 0.0;
  for (int i = blockIdx.x; i < t.first[t.count]; i += gridDim.x) {
    const int x = tensor_of(t, i);
    const int64_t off = (int64_t)(i - t.first[x]) * kGnChunk;
    const int64_t n = min(kGnChunk, t.n[x] - off);
    const int in = t.type[x] & 15;
    if (in == SPGEMM_F32) s += sum_squares((const float*)t.in[x] + off, n);
    else if (in == SPGEMM_BF16) s += sum_squares((const __bf16*)t.in[x] + off, n);
    else s += sum_squares((const _Float16*)t.in[x] + off, n);
  }
  s = group_sum(s);
  if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

template <typename T, typename U>
__device__ __forceinline__ void scale_into(const T* p, U* o, int64_t n, double c) {
  constexpr int V = 16 / (sizeof(T) > sizeof(U) ? sizeof(T) : sizeof(U));
  int64_t at = 0;
  if ((uintptr_t)p % (V * sizeof(T)) == 0 && (uintptr_t)o % (V * sizeof(U)) == 0) {
    struct alignas(V * sizeof(T)) Pi { T v[V]; };
    struct alignas(V * sizeof(U)) Po { U v[V]; };
    const int64_t packs = n / V;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < packs; i += kGnNT) {
      const Pi q = ((const Pi*)p)[i];
      Po r;
#pragma unroll
      for (int j = 0; j < V; ++j) r.v[j] = from_f32<U>((float)(to_f32(q.v[j]) * c));
      ((Po*)o)[i] = r;
    }
    at = packs * V;
  }
  for (int64_t i = at + threadIdx.x; i < n; i += kGnNT) o[i] = from_f32<U>((float)(to_f32(p[i]) * c));
}

template <typename T>
__device__ __forceinline__ void scale_from(const T* p, void* o, int out, int64_t off, int64_t n,
                                           double c) {
  if (out == SPGEMM_F32) scale_into(p, (float*)o + off, n, c);
  else if (out == SPGEMM_BF16) scale_into(p, (__bf16*)o + off, n, c);
  else scale_into(p, (_Float16*)o + off, n, c);
}

// total = the sum of all partial sums.
__global__ __launch_bounds__(kGnNT) void k_grad_total(const double* __restrict__ parts, int nparts,
                                                      double* __restrict__ total) {
  double s = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < nparts; i += kGnNT) s += parts[i];
  s = group_sum(s);
  if (threadIdx.x == 0) *total = s;
}

__global__ __launch_bounds__(kGnNT) void k_grad_scale(GradTable t,
                                                      const double* __restrict__ parts,
                                                      int nparts, double max_norm,
                                                      float* __restrict__ norm_out) {
  double s = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kGnNT) s += parts[i];
  const double norm = sqrt(group_sum(s));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  const double q = max_norm / (norm + 1e-6);
  // In fp64: as the norm passes 2^126 the factor leaves fp32's normal numbers, and
  // the products need not.  NaN stays NaN.
  const double c = q > 1.0 ? 1.0 : q;
  for (int i = blockIdx.x; i < t.first[t.count]; i += gridDim.x) {
    const int x = tensor_of(t, i);
    const int64_t off = (int64_t)(i - t.first[x]) * kGnChunk;
    const int64_t n = min(kGnChunk, t.n[x] - off);
    const int in = t.type[x] & 15, out = t.type[x] >> 4;
    if (in == SPGEMM_F32) scale_from((const float*)t.in[x] + off, t.out[x], out, off, n, c);
    else if (in == SPGEMM_BF16) scale_from((const __bf16*)t.in[x] + off, t.out[x], out, off, n, c);
    else scale_from((const _Float16*)t.in[x] + off, t.out[x], out, off, n, c);
  }
}

bool is_grad_type(int32_t t) { return t == SPGEMM_F32 || t == SPGEMM_BF16 || t == SPGEMM_F16; }

int64_t items_of(int64_t n) { return (n + kGnChunk - 1) / kGnChunk; }

int grid_of(int64_t items) { return (int)std::min<int64_t>(std::max<int64_t>(items, 1), kGnParts); }

int64_t launches_of(int64_t count) { return std::max<int64_t>(count, 0) / kGnTable + 1; }

}  // namespace
}  // namespace sg

using namespace sg;

extern "C" int64_t spgemm_clip_grad_norm_workspace(int64_t count) {
  return (launches_of(count) * kGnParts + 1) * (int64_t)sizeof(double);
}

extern "C" spgemm_status spgemm_clip_grad_norm(int64_t count, const void* const* dGrads,
                                               void* const* dOut, const int64_t* sizes,
                                               const int32_t* grad_types,
                                               const int32_t* out_types, double max_norm,
                                               float* dNorm, void* dWork, int64_t work_bytes,
                                               void* stream) {
  auto refuse = [](spgemm_status st, const char* msg) {
    set_thread_error(msg);
    return st;
  };
  if (count < 0 || !dNorm || (count && (!dGrads || !dOut || !sizes || !grad_types || !out_types)))
    return refuse(SPGEMM_ERR_INVALID_ARG, "clip_grad_norm: null array or negative count");
  if (!(max_norm >= 0.0))
    return refuse(SPGEMM_ERR_INVALID_ARG, "clip_grad_norm: max_norm must not be negative");
  if (!dWork || work_bytes < spgemm_clip_grad_norm_workspace(count))
    return refuse(SPGEMM_ERR_INVALID_ARG, "clip_grad_norm: workspace too small");
  int64_t all = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (sizes[i] < 0 || (sizes[i] > 0 && (!dGrads[i] || !dOut[i])))
      return refuse(SPGEMM_ERR_INVALID_ARG, "clip_grad_norm: null tensor or negative size");
    if (!is_grad_type(grad_types[i]) || !is_grad_type(out_types[i]))
      return refuse(SPGEMM_ERR_INVALID_ARG, "clip_grad_norm: tensors must be fp32, bf16 or fp16");
    all += items_of(sizes[i]);
  }
  if (all > INT32_MAX)
    return refuse(SPGEMM_ERR_INDEX_OVERFLOW, "clip_grad_norm: too many elements");
  (void)hipGetLastError();  // an error that earlier calls left is not this one's
  const hipStream_t s = (hipStream_t)stream;
  double* parts = (double*)dWork;
  auto add = [&](GradTable& t, int64_t i) {
    if (!sizes[i]) return;
    t.in[t.count] = dGrads[i];
    t.out[t.count] = dOut[i];
    t.n[t.count] = sizes[i];
    t.type[t.count] = (uint8_t)(grad_types[i] | out_types[i] << 4);
    t.first[t.count + 1] = t.first[t.count] + (int32_t)items_of(sizes[i]);
    ++t.count;
  };
  int nparts = 0, launches = 0;
  int64_t i = 0;
  do {
    GradTable t{};
    for (; i < count && t.count < kGnTable; ++i) add(t, i);
    const int grid = grid_of(t.first[t.count]);
    hipLaunchKernelGGL(k_grad_squares, dim3(grid), dim3(kGnNT), 0, s, t, parts + nparts);
    nparts += grid;
    ++launches;
  } while (i < count);
  const double* sums = parts;
  if (launches > 1) {
    double* total = parts + launches * kGnParts;
    hipLaunchKernelGGL(k_grad_total, dim3(1), dim3(kGnNT), 0, s, sums, nparts, total);
    sums = total;
    nparts = 1;
  }
  do {
    GradTable t{};
    for (; i > 0 && t.count < kGnTable; --i) add(t, i - 1);
    hipLaunchKernelGGL(k_grad_scale, dim3(grid_of(t.first[t.count])), dim3(kGnNT), 0, s, t, sums,
                       nparts, max_norm, dNorm);
  } while (i > 0);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SPGEMM_OK : refuse(SPGEMM_ERR_HIP, hipGetErrorString(e));
}
