// Device helpers of the attention kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "vqmm_device.h"
#include "vqmm_internal.h"

namespace vqmm {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint2_t __attribute__((ext_vector_type(2)));
typedef short short4_t __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Two floats to two 16-bit values, nearest even (low half: a).
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  const float2_t v = {a, b};
  if (F16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, half2_t));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// Smallest / largest, NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) { return __builtin_elementwise_minimum(a, b); }
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Largest value of the lanes l, l ^ 32.
__device__ __forceinline__ float max_xor32(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_xor32(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// The same over the lanes l, l ^ 16.
__device__ __forceinline__ float max_xor16(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_xor16(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sequence bounds of the packed rows, clamped to them.
struct Rows {
  int begin, n;
};
__device__ __forceinline__ Rows seq_rows(const int32_t *cu, int b, int total) {
  const int lo = min(max(cu[b], 0), total);
  const int hi = min(max(cu[b + 1], lo), total);
  return {lo, hi - lo};
}

// Tiles of `rows` packed rows without a host-side plan: sequence b gets the
// tile numbers from cu[b] / rows + extra * b up to those of b + 1, which are
// at least the ceil(n / rows) (extra = 1) it needs, whatever the lengths;
// the spare ones have nothing to do.  Returns the sequence of tile number t
// (-1: none) and its first tile number.  cu is clamped and taken as its own
// running maximum by the search, so any contents end the search in range.
__device__ __forceinline__ int find_tile(const int32_t *cu, int nseq, int total, int rows, int extra, int t, int *first) {
  int lo = 0, hi = nseq - 1;  // the last b with start(b) <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    const int s = min(max(cu[mid], 0), total) / rows + extra * mid;
    if (s <= t) lo = mid;
    else hi = mid - 1;
  }
  *first = min(max(cu[lo], 0), total) / rows + extra * lo;
  return t >= *first ? lo : -1;
}

// The page that holds slot group `i` (slot / page size) of sequence b.
__device__ __forceinline__ int64_t page_of(const KvView &c, int b, int i) {
  const int p = c.table[(int64_t)b * c.mp + i];
  return (int64_t)min(max(p, 0), c.np - 1);
}

}  // namespace vqmm
