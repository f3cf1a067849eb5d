// Rows of any width and alignment: 16-byte vectors of a row whose last vector
// may be partial.  Global vector accesses take any address on gfx950 (the
// target runs in unaligned-access mode), so odd widths and odd strides use
// the same vectors; only the row's last, partial vector goes by elements.
#pragma once

#include "m3_common.hpp"

namespace m3 {

typedef u32x4 u32x4_any __attribute__((aligned(2)));

// The same as loaded, for a row whose values are unpacked later.
template <typename T>
__device__ __forceinline__ u32x4 row_raw(const void* row, int64_t i, int64_t width) {
  constexpr int V = io<T>::VEC;
  if (i + V <= width) return *(const u32x4_any*)((const char*)row + i * io<T>::BYTES);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (i + j < width) {
      if constexpr (io<T>::BYTES == 2) v[j >> 1] |= (uint32_t)((const u16*)row)[i + j] << (16 * (j & 1));
      else v[j] = ((const uint32_t*)row)[i + j];
    }
  return v;
}
template <typename T>
__device__ __forceinline__ void unpack_raw(const u32x4& v, float* f) {
  io<T>::unpack(__builtin_bit_cast(typename io<T>::vec, v), f);
}

// Elements [i, i + VEC) of a row of `width` elements; those past its end read 0.
template <typename T>
__device__ __forceinline__ void row_load(const void* row, int64_t i, int64_t width, float* f) {
  constexpr int V = io<T>::VEC;
  if (i + V <= width) {
    const u32x4 v = *(const u32x4_any*)((const char*)row + i * io<T>::BYTES);
    io<T>::unpack(__builtin_bit_cast(typename io<T>::vec, v), f);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = i + j < width ? io<T>::load1(row, i + j) : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void row_store(void* row, int64_t i, int64_t width, const float* f) {
  constexpr int V = io<T>::VEC;
  if (i + V <= width) {
    *(u32x4_any*)((char*)row + i * io<T>::BYTES) = __builtin_bit_cast(u32x4, io<T>::pack(f));
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (i + j < width) io<T>::store1(row, i + j, f[j]);
  }
}
// Streamed past the caches: for what the kernel does not read again.
template <typename T>
__device__ __forceinline__ void row_stream(void* row, int64_t i, int64_t width, const float* f) {
  if (i + io<T>::VEC <= width)
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, io<T>::pack(f)), (u32x4_any*)((char*)row + i * io<T>::BYTES));
  else
    row_store<T>(row, i, width, f);
}
// The same for VEC consecutive fp32 values of a per-column vector; `missing`
// where the pointer is null.
template <int V>
__device__ __forceinline__ void col_load(const float* p, int64_t i, int64_t width, float missing, float* f) {
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = missing;
  if (!p) return;
  if (i + V <= width) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      typedef f32x4 f32x4_any __attribute__((aligned(4)));
      const f32x4 v = *(const f32x4_any*)(p + i + j);
      f[j] = v[0]; f[j + 1] = v[1]; f[j + 2] = v[2]; f[j + 3] = v[3];
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (i + j < width) f[j] = p[i + j];
  }
}

}  // namespace m3
