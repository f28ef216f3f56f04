// Dispatch: the transpose of a routing matrix whose rows hold k entries each
// (column -1 where there is none).  The entries are counted per expert,
// scanned, and placed stably, so that an expert's tokens rise and every sum
// over them has one order.  Moves 4 bytes in and 16 bytes out per entry; at
// the sizes it meets (up to some 10^5 entries) it is bound by its launches and
// their chains of dependent reads, so up to 8192 entries take one launch of one
// work group (384 entries 4.7 us, 5331 entries 10 us, where three launches took
// 13), and more take three (131,072 entries 27 us).
#include <algorithm>

#include "expert_common.hpp"

namespace sg {
namespace {

constexpr int kDispNT = 1024;
constexpr int kDispNW = kDispNT / kWave;
constexpr int kDispBlock = 4096;  // entries of one work group of several
constexpr int kDispOne = 8192;    // entries that one launch of one work group takes

// A wave's range is kIt rounds of 64 entries, held in registers: each lane's
// expert, -1 where there is none.
template <int kIt>
__device__ __forceinline__ void load_experts(const int32_t* col, int64_t n, int E, int64_t first,
                                             int (&c)[kIt]) {
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    const int64_t e = first + i * kWave + lane_id();
    const int x = e < n ? col[e] : -1;
    c[i] = (uint32_t)x < (uint32_t)E ? x : -1;
  }
}

// Entries per expert of each wave's range: wc[w * E + x].
template <int kIt>
__device__ __forceinline__ void count_waves(const int (&c)[kIt], int E, int32_t* wc) {
  for (int i = threadIdx.x; i < kDispNW * E; i += kDispNT) wc[i] = 0;
  __syncthreads();
  int32_t* my = wc + threadIdx.x / kWave * E;
#pragma unroll
  for (int i = 0; i < kIt; ++i)
    if (c[i] >= 0) atomicAdd(&my[c[i]], 1);
  __syncthreads();
}

// Turns each wave's counts of expert x into its first positions, from `at`.
__device__ __forceinline__ void count_to_start(int E, int x, int at, int32_t* wc) {
#pragma unroll
  for (int w = 0; w < kDispNW; ++w) {
    const int c = wc[w * E + x];
    wc[w * E + x] = at;
    at += c;
  }
}

// Places the work group's entries.  wc holds each wave's first position per
// expert and is advanced.
template <int kIt>
__device__ __forceinline__ void place(const int (&c)[kIt], const float* val, int64_t n, int k,
                                      int E, int bits, int64_t first, int32_t* wc,
                                      const Dispatch& d) {
  int32_t* my = wc + threadIdx.x / kWave * E;
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    const int64_t e = first + i * kWave + lane_id();
    const uint64_t peers = match_key((uint32_t)c[i], bits, c[i] >= 0);
    int p = -1;
    if (c[i] >= 0) {
      // The lanes of one expert read its position before the last of them
      // advances it; one wave's LDS accesses are performed in order.
      p = my[c[i]] + (int)__popcll(peers & lanemask_lt());
      if (lane_id() == last_set64(peers)) my[c[i]] = p + 1;
      d.ent[p] = (int32_t)e;
      d.tok[p] = (int32_t)((uint32_t)e / (uint32_t)k);
      if (val) d.w[p] = val[e];
    }
    if (e < n) d.pos[e] = p;
  }
}

// First position of expert x = threadIdx.x (< E) from its total: an exclusive
// scan over the work group of the totals and of the experts' row tiles.
// Writes the row pointers and the tiles.
__device__ __forceinline__ int scan_experts(int E, int tile_rows, int total, const Dispatch& d) {
  __shared__ int64_t wave_total[kDispNW];
  const int x = threadIdx.x, w = x / kWave;
  const int tiles = (total + tile_rows - 1) / tile_rows;
  const int64_t own = (int64_t)tiles << 32 | (uint32_t)total;  // no total reaches 2^31
  const int64_t incl = wave_incl_scan(own);
  if (lane_id() == kWave - 1) wave_total[w] = incl;
  __syncthreads();
  int64_t before = incl - own;
  for (int i = 0; i < w; ++i) before += wave_total[i];
  const int start = (int)(uint32_t)before;
  int t = (int)(before >> 32);
  if (x < E) d.row_ptr[x] = start;
  for (int i = 0; i < total; i += tile_rows, ++t) {
    d.tiles[2 * t] = x;
    d.tiles[2 * t + 1] = start + i;
  }
  if (x == E - 1) {
    d.row_ptr[E] = start + total;
    *d.ntiles = t;
  }
  return start;
}

template <int kIt>
__global__ __launch_bounds__(kDispNT) void k_dispatch_one(const int32_t* __restrict__ col,
                                                          const float* __restrict__ val,
                                                          int64_t n, int k, int E, int bits,
                                                          int tile_rows, Dispatch d) {
  extern __shared__ int32_t wc[];  // kDispNW * E
  const int64_t first = (int64_t)(threadIdx.x / kWave) * kIt * kWave;
  int c[kIt];
  load_experts(col, n, E, first, c);
  count_waves(c, E, wc);
  const int x = threadIdx.x;
  int total = 0;
  if (x < E)
#pragma unroll
    for (int w = 0; w < kDispNW; ++w) total += wc[w * E + x];
  const int start = scan_experts(E, tile_rows, total, d);
  if (x < E) count_to_start(E, x, start, wc);
  __syncthreads();
  place(c, val, n, k, E, bits, first, wc, d);
}

// hist[b * E + x]: entries of expert x in work group b's range.
__global__ __launch_bounds__(kDispNT) void k_dispatch_count(const int32_t* __restrict__ col,
                                                            int64_t n, int E,
                                                            int32_t* __restrict__ hist) {
  extern __shared__ int32_t h[];  // E
  for (int i = threadIdx.x; i < E; i += kDispNT) h[i] = 0;
  __syncthreads();
  const int64_t e0 = (int64_t)blockIdx.x * kDispBlock;
#pragma unroll
  for (int i = 0; i < kDispBlock; i += kDispNT) {
    const int64_t e = e0 + i + threadIdx.x;
    const int c = e < n ? col[e] : -1;
    if ((uint32_t)c < (uint32_t)E) atomicAdd(&h[c], 1);
  }
  __syncthreads();
  for (int x = threadIdx.x; x < E; x += kDispNT) hist[(int64_t)blockIdx.x * E + x] = h[x];
}

// Turns hist into every range's first position per expert, and writes the row
// pointers and the tiles.  One work group; thread x walks expert x's column.
__global__ __launch_bounds__(kDispNT) void k_dispatch_scan(int64_t nb, int E, int tile_rows,
                                                           int32_t* __restrict__ hist,
                                                           Dispatch d) {
  const int x = threadIdx.x;
  int total = 0;
  if (x < E)
#pragma unroll 8
    for (int64_t b = 0; b < nb; ++b) total += hist[b * E + x];
  int at = scan_experts(E, tile_rows, total, d);
  if (x < E)
#pragma unroll 8
    for (int64_t b = 0; b < nb; ++b) {
      const int c = hist[b * E + x];
      hist[b * E + x] = at;
      at += c;
    }
}

__global__ __launch_bounds__(kDispNT) void k_dispatch_place(const int32_t* __restrict__ col,
                                                            const float* __restrict__ val,
                                                            int64_t n, int k, int E, int bits,
                                                            const int32_t* __restrict__ hist,
                                                            Dispatch d) {
  extern __shared__ int32_t wc[];
  constexpr int kIt = kDispBlock / kDispNT;
  const int64_t first =
      (int64_t)blockIdx.x * kDispBlock + (int64_t)(threadIdx.x / kWave) * kIt * kWave;
  int c[kIt];
  load_experts(col, n, E, first, c);
  count_waves(c, E, wc);
  for (int x = threadIdx.x; x < E; x += kDispNT)
    count_to_start(E, x, hist[(int64_t)blockIdx.x * E + x], wc);
  __syncthreads();
  place(c, val, n, k, E, bits, first, wc, d);
}

}  // namespace

int64_t dispatch_tmp_elems(int64_t n, int64_t E) {
  return (n + kDispBlock - 1) / kDispBlock * E;
}

int64_t dispatch_max_tiles(int64_t n, int64_t E, int tile_rows) {
  return n / tile_rows + std::min(n, E);
}

void launch_dispatch(const int32_t* col, const float* val, int64_t n, int k, int64_t E, int tile_rows,
                     const Dispatch& d, int32_t* tmp, hipStream_t s) {
  int bits = 0;
  while (((int64_t)1 << bits) < E) ++bits;
  const int64_t nb = (n + kDispBlock - 1) / kDispBlock;
  const size_t wcb = (size_t)kDispNW * E * sizeof(int32_t);
  if (n <= kDispOne) {
    auto one = n <= kDispNT       ? k_dispatch_one<1>
               : n <= 2 * kDispNT ? k_dispatch_one<2>
               : n <= 4 * kDispNT ? k_dispatch_one<4>
                                  : k_dispatch_one<8>;
    hipLaunchKernelGGL(one, dim3(1), dim3(kDispNT), wcb, s, col, val, n, k, (int)E, bits,
                       tile_rows, d);
    return;
  }
  hipLaunchKernelGGL(k_dispatch_count, dim3((unsigned)nb), dim3(kDispNT), E * sizeof(int32_t), s,
                     col, n, (int)E, tmp);
  hipLaunchKernelGGL(k_dispatch_scan, dim3(1), dim3(kDispNT), 0, s, nb, (int)E, tile_rows, tmp, d);
  hipLaunchKernelGGL(k_dispatch_place, dim3((unsigned)nb), dim3(kDispNT), wcb, s, col, val, n, k,
                     (int)E, bits, (const int32_t*)tmp, d);
}

namespace {

struct DispatchWork {
  int32_t *tok, *pos, *tiles, *ntiles, *tmp;
};

DispatchWork take_work(Carver& c, int64_t n, int64_t E) {
  DispatchWork w{};
  w.tok = c.take<int32_t>(n);
  w.pos = c.take<int32_t>(n);
  w.tiles = c.take<int32_t>(2 * dispatch_max_tiles(n, E, 256));
  w.ntiles = c.take<int32_t>(1);
  w.tmp = c.take<int32_t>(dispatch_tmp_elems(n, E));
  return w;
}

}  // namespace
}  // namespace sg

using namespace sg;

extern "C" int64_t spgemm_dispatch_workspace(int64_t T, int32_t k, int64_t E) {
  if (T < 0 || k < 1 || E < 1 || E > kMaxExperts || T > INT32_MAX / k) return 0;
  Carver c(nullptr);
  take_work(c, T * k, E);
  return c.used;
}

extern "C" spgemm_status spgemm_dispatch(int64_t T, int32_t k, int64_t E, const int32_t* dCol,
                                         int32_t* dRowPtr, int32_t* dEntry, void* dWork,
                                         int64_t work_bytes, void* stream) {
  if (T < 0 || k < 1 || k > 64 || E < 1 || E > kMaxExperts) {
    set_thread_error("dispatch: tokens < 0, k outside [1, 64] or experts outside [1, 1024]");
    return SPGEMM_ERR_INVALID_ARG;
  }
  if (T > INT32_MAX / k) {
    set_thread_error("dispatch: more than 2^31 - 1 entries");
    return SPGEMM_ERR_INDEX_OVERFLOW;
  }
  const int64_t n = T * k;
  Carver c(dWork);
  const DispatchWork w = take_work(c, n, E);
  if (!dRowPtr || !dWork || work_bytes < c.used || (n > 0 && (!dCol || !dEntry))) {
    set_thread_error("dispatch: null array or workspace too small");
    return SPGEMM_ERR_INVALID_ARG;
  }
  Dispatch d{};
  d.row_ptr = dRowPtr;
  d.ent = dEntry;
  d.tok = w.tok;
  d.pos = w.pos;
  d.tiles = w.tiles;
  d.ntiles = w.ntiles;
  (void)hipGetLastError();  // an error that earlier calls left is not this one's
  launch_dispatch(dCol, nullptr, n, k, E, 256, d, w.tmp, (hipStream_t)stream);
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return SPGEMM_OK;
  set_thread_error(hipGetErrorString(e));
  return SPGEMM_ERR_HIP;
}
