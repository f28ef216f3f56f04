// Shared by the expert-layer translation units (routing, dispatch, the
// experts' products, gradient clipping): 16-bit types, DPP reductions over a
// wave, the workspace carver and the launchers' declarations.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace sg {

// ---- element types ----

template <typename T>
__device__ __forceinline__ float to_f32(T x) { return (float)x; }
template <typename T>
__device__ __forceinline__ T from_f32(float x) { return (T)x; }

// ---- reductions over a wave by DPP ----
// Rows of 16 lanes are reduced by shifts, then joined by two broadcasts;
// lane 63 ends with the result, which every lane gets through an SGPR.

template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t dpp_or_zero(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kCtrl, kRows, 0xf, false);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t x) {
  x = max(x, dpp_or_zero<0x111, 0xf>(x));  // row_shr:1
  x = max(x, dpp_or_zero<0x112, 0xf>(x));
  x = max(x, dpp_or_zero<0x114, 0xf>(x));
  x = max(x, dpp_or_zero<0x118, 0xf>(x));
  x = max(x, dpp_or_zero<0x142, 0xa>(x));  // row_bcast:15
  x = max(x, dpp_or_zero<0x143, 0xc>(x));  // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

template <int kCtrl, int kRows>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __uint_as_float(dpp_or_zero<kCtrl, kRows>(__float_as_uint(x)));
}

__device__ __forceinline__ float wave_sum_f32(float x) {
  x = dpp_add<0x111, 0xf>(x);
  x = dpp_add<0x112, 0xf>(x);
  x = dpp_add<0x114, 0xf>(x);
  x = dpp_add<0x118, 0xf>(x);
  x = dpp_add<0x142, 0xa>(x);
  x = dpp_add<0x143, 0xc>(x);
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), 63));
}

// Order-preserving bits of a float that is not NaN, both zeros alike; 0 is
// below every value.
__device__ __forceinline__ uint32_t ordered_bits(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}

// ---- workspace ----

// Takes 256-byte aligned pieces from a block; with a null block it only adds
// their sizes up.
struct Carver {
  char* base;
  int64_t used = 0;
  explicit Carver(void* b) : base((char*)b) {}
  template <typename T>
  T* take(int64_t count) {
    T* p = base ? (T*)(base + used) : nullptr;
    used += (count * (int64_t)sizeof(T) + 255) / 256 * 256;
    return p;
  }
};

// ---- dispatch: the transposed routing matrix ----

constexpr int64_t kMaxExperts = 1024;

// Entries of the routing matrix sorted by expert, in rising order inside each.
struct Dispatch {
  int32_t* row_ptr;  // E + 1
  int32_t* ent;      // sorted position -> entry t * k + i
  int32_t* tok;      // sorted position -> token t
  float* w;          // sorted position -> value, where values are given
  int32_t* pos;      // entry -> sorted position, -1 where there is none
  int32_t* tiles;    // (expert, first sorted position) of every row tile
  int32_t* ntiles;   // row tiles
};

int64_t dispatch_tmp_elems(int64_t n, int64_t E);
int64_t dispatch_max_tiles(int64_t n, int64_t E, int tile_rows);
void launch_dispatch(const int32_t* col, const float* val, int64_t n, int k, int64_t E, int tile_rows,
                     const Dispatch& d, int32_t* tmp, hipStream_t s);

}  // namespace sg
