// Dispatch: the transpose of a routing matrix whose rows hold k entries each
// (column -1 where there is none).  The entries are counted per expert,
// scanned, and placed stably, so that an expert's tokens rise and every sum
// over them has one order.  Moves 4 bytes in and 16 bytes out per entry; at
// the sizes it meets (up to some 10^5 entries) it is bound by its launches,
// so up to kDispBlock entries take one launch of one work group, and more
// take three.
#include <algorithm>

#include "expert_common.hpp"

namespace sg {
namespace {

constexpr int kDispNT = 256;
constexpr int kDispNW = kDispNT / kWave;
constexpr int kDispBlock = 4096;                 // entries of one work group
constexpr int kDispWave = kDispBlock / kDispNW;  // consecutive entries of one wave

__device__ __forceinline__ int expert_of(const int32_t* col, int64_t e, int64_t n, int E) {
  const int c = e < n ? col[e] : -1;
  return (uint32_t)c < (uint32_t)E ? c : -1;
}

// Entries per expert of each wave's range: wc[w * E + x].
__device__ __forceinline__ void count_waves(const int32_t* col, int64_t n, int E, int64_t e0,
                                            int32_t* wc) {
  for (int i = threadIdx.x; i < kDispNW * E; i += kDispNT) wc[i] = 0;
  __syncthreads();
  const int w = threadIdx.x / kWave;
  const int64_t first = e0 + (int64_t)w * kDispWave;
  for (int i = lane_id(); i < kDispWave && first + i < n; i += kWave) {
    const int c = expert_of(col, first + i, n, E);
    if (c >= 0) atomicAdd(&wc[w * E + c], 1);
  }
  __syncthreads();
}

// Places the work group's entries.  wc holds each wave's first position per
// expert and is advanced.
__device__ __forceinline__ void place(const int32_t* col, const float* val, int64_t n, int k, int E, int bits,
                                      int64_t e0, int32_t* wc, const Dispatch& d) {
  const int w = threadIdx.x / kWave;
  int32_t* my = wc + w * E;
  const int64_t first = e0 + (int64_t)w * kDispWave;
  for (int i = 0; i < kDispWave && first + i < n; i += kWave) {
    const int64_t e = first + i + lane_id();
    const int c = expert_of(col, e, n, E);
    const uint64_t peers = match_key((uint32_t)c, bits, c >= 0);
    int p = -1;
    if (c >= 0) {
      // The lanes of one expert read its position before the last of them
      // advances it; one wave's LDS accesses are performed in order.
      p = my[c] + (int)__popcll(peers & lanemask_lt());
      if (lane_id() == last_set64(peers)) my[c] = p + 1;
      d.ent[p] = (int32_t)e;
      d.tok[p] = (int32_t)(e / k);
      if (val) d.w[p] = val[e];
    }
    if (e < n) d.pos[e] = p;
  }
}

// Exclusive scan over the experts of their totals and of their row tiles by
// the first wave; every lane takes consecutive experts.
__device__ __forceinline__ void scan_experts(int E, int tile_rows, const int32_t* total,
                                             int32_t* start, const Dispatch& d) {
  const int per = (E + kWave - 1) / kWave;
  const int a = min(E, lane_id() * per), b = min(E, a + per);
  int rows = 0, tiles = 0;
  for (int x = a; x < b; ++x) {
    rows += total[x];
    tiles += (total[x] + tile_rows - 1) / tile_rows;
  }
  int r = wave_incl_scan(rows) - rows, t = wave_incl_scan(tiles) - tiles;
  for (int x = a; x < b; ++x) {
    d.row_ptr[x] = start[x] = r;
    for (int i = 0; i < total[x]; i += tile_rows, ++t) {
      d.tiles[2 * t] = x;
      d.tiles[2 * t + 1] = r + i;
    }
    r += total[x];
  }
  if (lane_id() == kWave - 1) {
    d.row_ptr[E] = r;
    *d.ntiles = t;
  }
}

__global__ __launch_bounds__(kDispNT) void k_dispatch_one(const int32_t* __restrict__ col,
                                                          const float* __restrict__ val, int64_t n, int k, int E, int bits,
                                                          int tile_rows, Dispatch d) {
  extern __shared__ int32_t lds[];
  int32_t* wc = lds;                  // kDispNW * E
  int32_t* total = wc + kDispNW * E;  // E
  int32_t* start = total + E;         // E
  count_waves(col, n, E, 0, wc);
  for (int x = threadIdx.x; x < E; x += kDispNT) {
    int sum = 0;
    for (int w = 0; w < kDispNW; ++w) sum += wc[w * E + x];
    total[x] = sum;
  }
  __syncthreads();
  if (threadIdx.x < kWave) scan_experts(E, tile_rows, total, start, d);
  __syncthreads();
  for (int x = threadIdx.x; x < E; x += kDispNT) {
    int at = start[x];
    for (int w = 0; w < kDispNW; ++w) {
      const int c = wc[w * E + x];
      wc[w * E + x] = at;
      at += c;
    }
  }
  __syncthreads();
  place(col, val, n, k, E, bits, 0, wc, d);
}

// hist[b * E + x]: entries of expert x in work group b's range.
__global__ __launch_bounds__(kDispNT) void k_dispatch_count(const int32_t* __restrict__ col,
                                                            int64_t n, int E,
                                                            int32_t* __restrict__ hist) {
  extern __shared__ int32_t lds[];
  count_waves(col, n, E, (int64_t)blockIdx.x * kDispBlock, lds);
  for (int x = threadIdx.x; x < E; x += kDispNT) {
    int sum = 0;
    for (int w = 0; w < kDispNW; ++w) sum += lds[w * E + x];
    hist[(int64_t)blockIdx.x * E + x] = sum;
  }
}

// Turns hist into every range's first position per expert, and writes the row
// pointers and the tiles.  One work group; thread x walks expert x's column.
__global__ __launch_bounds__(1024) void k_dispatch_scan(int64_t nb, int E, int tile_rows,
                                                        int32_t* __restrict__ hist, Dispatch d) {
  __shared__ int32_t total[kMaxExperts], start[kMaxExperts];
  const int x = threadIdx.x;
  if (x < E) {
    int sum = 0;
#pragma unroll 8
    for (int64_t b = 0; b < nb; ++b) sum += hist[b * E + x];
    total[x] = sum;
  }
  __syncthreads();
  if (threadIdx.x < kWave) scan_experts(E, tile_rows, total, start, d);
  __syncthreads();
  if (x < E) {
    int at = start[x];
#pragma unroll 8
    for (int64_t b = 0; b < nb; ++b) {
      const int c = hist[b * E + x];
      hist[b * E + x] = at;
      at += c;
    }
  }
}

__global__ __launch_bounds__(kDispNT) void k_dispatch_place(const int32_t* __restrict__ col,
                                                            const float* __restrict__ val,
                                                            int64_t n, int k, int E, int bits,
                                                            const int32_t* __restrict__ hist,
                                                            Dispatch d) {
  extern __shared__ int32_t wc[];
  const int64_t e0 = (int64_t)blockIdx.x * kDispBlock;
  count_waves(col, n, E, e0, wc);
  for (int x = threadIdx.x; x < E; x += kDispNT) {
    int at = hist[(int64_t)blockIdx.x * E + x];
    for (int w = 0; w < kDispNW; ++w) {
      const int c = wc[w * E + x];
      wc[w * E + x] = at;
      at += c;
    }
  }
  __syncthreads();
  place(col, val, n, k, E, bits, e0, wc, d);
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
  if (nb <= 1) {
    hipLaunchKernelGGL(k_dispatch_one, dim3(1), dim3(kDispNT), wcb + 2 * E * sizeof(int32_t), s,
                       col, val, n, k, (int)E, bits, tile_rows, d);
    return;
  }
  hipLaunchKernelGGL(k_dispatch_count, dim3((unsigned)nb), dim3(kDispNT), wcb, s, col, n, (int)E,
                     tmp);
  hipLaunchKernelGGL(k_dispatch_scan, dim3(1), dim3(1024), 0, s, nb, (int)E, tile_rows, tmp, d);
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
  launch_dispatch(dCol, nullptr, n, k, E, 256, d, w.tmp, (hipStream_t)stream);
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return SPGEMM_OK;
  set_thread_error(hipGetErrorString(e));
  return SPGEMM_ERR_HIP;
}
