// Rows of 16-bit values to their 8-bit form and back, for what a pass keeps until
// its gradients.  Both are bound by their bytes, 3 + 1/128 for every value: 8192 x
// 2048 in 15 and 11 us (3.4 and 4.6 TB/s), 0.7% of the training step that they are
// part of, so they stay kernels of their own beside the products.
#include <algorithm>

#include "rows8.hpp"

namespace sg {
namespace {

constexpr int kNT = 256;

// 16 lanes to a block of 128 columns.
template <typename T>
__global__ __launch_bounds__(kNT) void k_rows_encode(int64_t rows, int D, int64_t ld,
                                                     const T* __restrict__ x,
                                                     uint8_t* __restrict__ code,
                                                     uint8_t* __restrict__ scale) {
  const int64_t blocks = kept_blocks(D), pitch = kept_pitch(D);
  const int64_t step = (int64_t)gridDim.x * (kNT / 16), all = rows * blocks;
  for (int64_t i = (int64_t)blockIdx.x * (kNT / 16) + threadIdx.x / 16; i < all; i += step) {
    const int64_t t = i / blocks;
    const int b = (int)(i - t * blocks), c = b * kKeptBlock + (int)threadIdx.x % 16 * 8;
    float v[8];
    load8_any(x + t * ld + c, D - c, v);
    uint32_t e;
    const uint2 q = kept_encode<T>(v, e);
    if (c < D) *(uint2*)(code + t * pitch + c) = q;
    if (threadIdx.x % 16 == 0) scale[i] = (uint8_t)e;
  }
}

// Rows of the pitch of the codes, zeros beyond D.
template <typename T>
__global__ __launch_bounds__(kNT) void k_rows_decode(int64_t rows, int D,
                                                     const uint8_t* __restrict__ code,
                                                     const uint8_t* __restrict__ scale,
                                                     T* __restrict__ x) {
  const int64_t blocks = kept_blocks(D), per = kept_pitch(D) / 8;
  const int64_t step = (int64_t)gridDim.x * kNT, all = rows * per;
  for (int64_t i = (int64_t)blockIdx.x * kNT + threadIdx.x; i < all; i += step) {
    const int64_t t = i / per;
    const int c = (int)(i - t * per) * 8;
    float v[8];
    kept_decode(((const uint2*)code)[i], scale[t * blocks + c / kKeptBlock], v);
    store8_any(x + i * 8, 8, v);
  }
}

unsigned grid_for(int64_t threads) {
  return (unsigned)std::min<int64_t>((threads + kNT - 1) / kNT, 8192);
}

}  // namespace

void launch_rows_encode(spgemm_dtype type, int64_t rows, int64_t D, int64_t ld, const void* x,
                        uint8_t* code, uint8_t* scale, hipStream_t s) {
  const dim3 grid(grid_for(rows * kept_blocks(D) * 16));
  if (type == SPGEMM_BF16)
    hipLaunchKernelGGL((k_rows_encode<__bf16>), grid, dim3(kNT), 0, s, rows, (int)D, ld,
                       (const __bf16*)x, code, scale);
  else
    hipLaunchKernelGGL((k_rows_encode<_Float16>), grid, dim3(kNT), 0, s, rows, (int)D, ld,
                       (const _Float16*)x, code, scale);
}

void launch_rows_decode(spgemm_dtype type, int64_t rows, int64_t D, const uint8_t* code,
                        const uint8_t* scale, void* x, hipStream_t s) {
  const dim3 grid(grid_for(rows * kept_pitch(D) / 8));
  if (type == SPGEMM_BF16)
    hipLaunchKernelGGL((k_rows_decode<__bf16>), grid, dim3(kNT), 0, s, rows, (int)D, code, scale,
                       (__bf16*)x);
  else
    hipLaunchKernelGGL((k_rows_decode<_Float16>), grid, dim3(kNT), 0, s, rows, (int)D, code, scale,
                       (_Float16*)x);
}

}  // namespace sg
