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
// (-1: none) and its first tile number.  cu is clamped to the rows and the
// search ends in range whatever it holds; offsets that fall give wrong rows,
// never rows outside.
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

template <bool F16>
__device__ __forceinline__ float16_t mfma32(uint4_t a, uint4_t b, float16_t c) {
  if (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// LDS by byte address.
typedef __attribute__((address_space(3))) uint4_t lds_uint4;
__device__ __forceinline__ uint4_t lds_read(uint32_t at) { return *(lds_uint4 *)(uintptr_t)at; }

// Tiles of BN rows go from global memory straight into LDS, 16 bytes a lane, a
// wave's 64 pieces next to one another: no registers, no LDS writes to issue.
// Rows are not padded; instead the 16-byte pieces of a row are permuted by an
// XOR with bits of the row, in the address each lane loads from:
//   keys (and queries): piece ^ (row & 15) (D = 64: row / 2 & 7): 16 rows of one piece,
//            a quarter of a b128 read
//   values : piece ^ 4 (row & 3) (D = 64: 4 (row / 2 & 1)): the 64-byte spans
//            that the transposing reads take from 4 rows
// fall on different banks (64 of 4 bytes).  For workgroups of four waves.
template <int D>
__device__ __forceinline__ int key_swizzle(int row) {
  return D == 64 ? (row >> 1) & 7 : row & 15;
}
template <int D>
__device__ __forceinline__ int value_swizzle(int row) {
  return D == 64 ? (row & 2) << 1 : (row & 3) << 2;
}

__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

// 16 bytes a lane from base + off to LDS at `lds` + 16 lane (in m0).  Not waited
// for: wait_loads() before the barrier that publishes the tile.
__device__ __forceinline__ void load_to_lds(uint32_t lds, const char *base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <int D, int BN>
struct Stage {
  static constexpr int kRowsPerLoad = 512 / D;                    // rows of a wave's 1024 bytes
  static constexpr int kLoads = BN / (4 * kRowsPerLoad);          // of a wave and tile
  // the lane's row of the tile for the wave's first load, and its piece in the
  // even and in the odd loads (4 kRowsPerLoad rows apart)
  uint32_t row, piece[2];
  __device__ __forceinline__ Stage(int wave, int lane, bool value) {
    row = kRowsPerLoad * wave + lane / (D / 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = row + i * 4 * kRowsPerLoad;
      piece[i] = (lane % (D / 8)) ^ (value ? value_swizzle<D>(r) : key_swizzle<D>(r));
    }
  }
  // rows row0 .. row0 + BN - 1 of n (those past the end repeat the last one)
  __device__ __forceinline__ void load(uint32_t lds, const uint16_t *base, int64_t ts, int row0, int n, int wave) const {
    lds += wave * 1024;
    const char *p = reinterpret_cast<const char *>(base + row0 * ts);
    if (row0 + BN <= n) {
      const uint32_t off = row * (uint32_t)ts * 2u;
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        load_to_lds(lds + i * 4096, p + (int64_t)i * (4 * kRowsPerLoad) * ts * 2, off + piece[i & 1] * 16u);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        load_to_lds(lds + i * 4096, p, (uint32_t)min((int)row + i * 4 * kRowsPerLoad, n - 1 - row0) * (uint32_t)ts * 2u + piece[i & 1] * 16u);
    }
  }
};

}  // namespace vqmm
