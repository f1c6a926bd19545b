// Loads and stores of 8 consecutive elements at any element-aligned address,
// converted to and from fp32, and sums across lanes: shared by the row-wise
// and elementwise kernels (layer norm, AdamW, the linear layer's gradients).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace vn {

// 16 bytes at any address: global memory takes unaligned 16-byte accesses, so
// rows of an odd width need no other path than their ragged end.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// A run of 8 elements as they lie in memory.
template <typename T> struct Run8;
template <> struct Run8<float> { u32x4_any a, b; };
template <> struct Run8<__bf16> { u32x4_any a; };

__device__ __forceinline__ void run_values(const Run8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __builtin_bit_cast(float, static_cast<uint32_t>(r.a[i]));
    v[i + 4] = __builtin_bit_cast(float, static_cast<uint32_t>(r.b[i]));
  }
}
__device__ __forceinline__ void run_values(const Run8<__bf16>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __builtin_bit_cast(float, static_cast<uint32_t>(r.a[i]) << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, static_cast<uint32_t>(r.a[i]) & 0xFFFF0000u);
  }
}

typedef float vn_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 vn_bf16x2 __attribute__((ext_vector_type(2)));
// Two values to bf16, nearest even (one v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((vn_f32x2){a, b}, vn_bf16x2));
}

__device__ __forceinline__ Run8<float> make_run(const float (&v)[8], const float*) {
  Run8<float> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.a[i] = __builtin_bit_cast(uint32_t, v[i]);
    r.b[i] = __builtin_bit_cast(uint32_t, v[i + 4]);
  }
  return r;
}
__device__ __forceinline__ Run8<__bf16> make_run(const float (&v)[8], const __bf16*) {
  Run8<__bf16> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.a[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  return r;
}

// Elements [c, c + 8) of a row of n, zeros past its end.  (A run past the end is a
// case of its own: the waves that hold such runs, but none that the end cuts, skip
// the single elements; 131072 rows of 1000 in bf16 take 187 us of gradients, not 202.)
template <typename T, typename I>
__device__ __forceinline__ Run8<T> load_run(const T* row, I c, I n) {
  Run8<T> r;
  if (c + 8 <= n) {
    __builtin_memcpy(&r, row + c, sizeof(r));
  } else if (c < n) {
    T e[8];
    e[0] = row[c];
#pragma unroll
    for (int i = 1; i < 8; ++i) e[i] = c + i < n ? row[c + i] : static_cast<T>(0.0f);
    __builtin_memcpy(&r, e, sizeof(r));
  } else {
    __builtin_memset(&r, 0, sizeof(r));
  }
  return r;
}

template <typename T, typename I>
__device__ __forceinline__ void store_run(T* row, I c, I n, const float (&v)[8]) {
  const Run8<T> r = make_run(v, row);
  if (c + 8 <= n) {
    __builtin_memcpy(row + c, &r, sizeof(r));
  } else {
    T e[8];
    __builtin_memcpy(e, &r, sizeof(r));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = e[i];
  }
}

// The same past the caches (PAST; runs that are whole): for tensors that the
// caches cannot hold until they are read again.
template <bool PAST, typename T, typename I>
__device__ __forceinline__ void store_run(T* row, I c, I n, const float (&v)[8]) {
  if (PAST && c + 8 <= n) {
    const Run8<T> r = make_run(v, row);
    u32x4_any part[sizeof(r) / 16];
    __builtin_memcpy(part, &r, sizeof(r));
#pragma unroll
    for (unsigned i = 0; i < sizeof(r) / 16; ++i)
      __builtin_nontemporal_store(part[i], reinterpret_cast<u32x4_any*>(row + c) + i);
  } else {
    store_run(row, c, n, v);
  }
}
template <bool PAST, typename T, typename I>
__device__ __forceinline__ Run8<T> load_run(const T* row, I c, I n) {
  if (PAST && c + 8 <= n) {
    Run8<T> r;
    u32x4_any part[sizeof(r) / 16];
#pragma unroll
    for (unsigned i = 0; i < sizeof(r) / 16; ++i)
      part[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(row + c) + i);
    __builtin_memcpy(&r, part, sizeof(r));
    return r;
  }
  return load_run(row, c, n);
}

// Sum over the aligned group of G lanes that holds this lane (G a power of
// two, at most 64), in every lane of the group, in a fixed order.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = 1; o < G; o *= 2) v += __shfl_xor(v, o, 64);
  return v;
}

}  // namespace vn
