// kv4_append and kv4_read: packed rows into the 4-bit cache and back.
//
// A group of 32 channels of one token and head is held as m = f16(min), s =
// f16((max - min) / 15) and 4-bit codes of (x - m) / s.  Both kernels only
// move data: append reads 2 or 4 bytes a value and writes 5 bits, read the
// reverse, so HBM traffic bounds them.
//
// One thread takes an octet of channels of four consecutive slots that share
// a quad of the cache (slots 4i .. 4i+3): four 16-byte pieces of the packed
// rows, and in the cache one 32-bit word a slot of the keys, one 16-byte
// piece of the values and (one thread of four) one 16-byte piece of steps and
// minima.  Quads that the rows only partly cover are written by bytes and
// halves, never read back, so neighbouring slots keep what they hold and no
// two threads write the same byte.  The four threads of a group exchange
// minimum and maximum through DPP.  8192 rows of 8 heads of 128 in bf16: append
// 13.6 us (3.3 TB/s of rows and cache), read 9.6 us (4.6 TB/s).
#include "attn_device.h"

namespace vqmm {

namespace {

constexpr int kThreads = 256;

// The lane's neighbours in its four: lane ^ 1, lane ^ 2.
__device__ __forceinline__ float quad_xor1(float v) {
  const int u = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(u, u, 0xB1, 0xF, 0xF, false));  // quad_perm 1,0,3,2
}
__device__ __forceinline__ float quad_xor2(float v) {
  const int u = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(u, u, 0x4E, 0xF, 0xF, false));  // quad_perm 2,3,0,1
}

template <int DT>
__device__ __forceinline__ void load8(const void *base, int64_t at, float *x) {
  if (DT == VQ_F32) {
    const float4_t *p = reinterpret_cast<const float4_t *>(static_cast<const float *>(base) + at);
    const float4_t a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
  } else {
    const uint4_t a = *reinterpret_cast<const uint4_t *>(static_cast<const uint16_t *>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == VQ_BF16) {
        x[2 * i] = bf2f(a[i] & 0xffffu);
        x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
      } else {
        const half2_t h = as_h2(a[i]);
        x[2 * i] = (float)h[0];
        x[2 * i + 1] = (float)h[1];
      }
    }
  }
}

template <int DT>
__device__ __forceinline__ void store8(void *base, int64_t at, const float *x) {
  if (DT == VQ_F32) {
    float4_t *p = reinterpret_cast<float4_t *>(static_cast<float *>(base) + at);
    p[0] = float4_t{x[0], x[1], x[2], x[3]};
    p[1] = float4_t{x[4], x[5], x[6], x[7]};
  } else {
    uint4_t a;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = pack16<DT == VQ_F16>(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4_t *>(static_cast<uint16_t *>(base) + at) = a;
  }
}

// Where a thread's octet of a quad lives: the sequence's rows, its slots and
// the addresses in the pool.
struct Place {
  bool any;          // some of the four slots are wanted
  int lo, hi;        // wanted slots of the quad: lo <= i < hi
  int64_t row;       // packed row of slot 0 of the quad (may be outside)
  int seq, slot;     // sequence, first slot of the quad
  bool stored;       // the block table reaches this quad
  int64_t page;
  int off;           // first slot of the quad within its page
  int kind, head, oct;
};

template <int D>
__device__ __forceinline__ Place place_of(const KvView &c, const int32_t *cu, int total, int vq, int item) {
  constexpr int NO = D / 8;  // octets
  Place p{};
  p.oct = item % NO;
  const int rest = item / NO;
  p.head = rest % c.hkv;
  p.kind = rest / c.hkv;
  if (p.kind > 1) return p;
  int first;
  const int b = find_tile(cu, c.nseq, total, 4, 2, vq, &first);
  if (b < 0) return p;
  const Rows r = seq_rows(cu, b, total);
  const int start = c.lens ? max(c.lens[b], 0) : 0;
  const int64_t quad = (int64_t)(start >> 2) + (vq - first);
  const int64_t s0 = quad * 4;                 // first slot of the quad
  const int64_t i0 = s0 - start;               // its row within the sequence
  if (i0 >= r.n) return p;
  p.any = true;
  p.lo = i0 < 0 ? (int)-i0 : 0;
  p.hi = (int)min((int64_t)4, r.n - i0);
  p.row = r.begin + i0;
  p.seq = b;
  p.slot = (int)min(s0, (int64_t)0x7ffffffc);
  p.stored = s0 < (int64_t)c.mp * c.ps;
  if (p.stored) {
    const int pi = p.slot / c.ps;
    p.off = p.slot - pi * c.ps;
    p.page = page_of(c, b, pi);
  }
  return p;
}

// Byte offsets in the pool.
template <int D>
__device__ __forceinline__ uint8_t *codes_at(const KvView &c, const Place &p) {
  return c.codes + ((p.page * 2 + p.kind) * c.hkv + p.head) * ((int64_t)c.ps * (D / 2));
}
template <int D>
__device__ __forceinline__ uint16_t *scales_at(const KvView &c, const Place &p) {
  return c.scales + (((p.page * 2 + p.kind) * c.hkv + p.head) * (int64_t)(c.ps / 4) + p.off / 4) * (D / 32 * 8) +
         p.oct / 4 * 8;
}
// Word of the keys' row that holds octet o: a * DG + j with o = 4 j + a.
template <int D>
__device__ __forceinline__ int key_word(int o) {
  return (o & 3) * (D / 32) + (o >> 2);
}
// Byte position of slot i of a quad within a value word, and the reverse
// (the exchange of 1 and 2 is its own inverse).
__device__ __forceinline__ int value_byte(int i) { return i == 1 ? 2 : i == 2 ? 1 : i; }

template <int D, int DT>
__global__ __launch_bounds__(kThreads) void k_kv4_append(KvView c, const void *__restrict__ k,
                                                         const void *__restrict__ v, int64_t k_ts, int64_t k_hs,
                                                         int64_t v_ts, int64_t v_hs, int total,
                                                         const int32_t *__restrict__ cu,
                                                         const int32_t *__restrict__ pos,
                                                         const float *__restrict__ weights, int per) {
  const int vq = blockIdx.x / per;
  const int item = (blockIdx.x - vq * per) * kThreads + threadIdx.x;
  const Place p = place_of<D>(c, cu, total, vq, item);
  if (!p.any || !p.stored) return;  // the same for the four lanes of a group

  const void *src = p.kind ? v : k;
  const int64_t ts = p.kind ? v_ts : k_ts, hs = p.kind ? v_hs : k_hs;
  uint32_t word[4];  // a slot's eight codes, channel i in bits 4 i
  uint16_t s16[4], m16[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[8];
    if (i >= p.lo && i < p.hi) {
      load8<DT>(src, (p.row + i) * ts + p.head * hs + p.oct * 8, x);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    }
    float lo = min_nan(min_nan(min_nan(x[0], x[1]), min_nan(x[2], x[3])), min_nan(min_nan(x[4], x[5]), min_nan(x[6], x[7])));
    float hi = max_nan(max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3])), max_nan(max_nan(x[4], x[5]), max_nan(x[6], x[7])));
    lo = min_nan(lo, quad_xor1(lo));
    hi = max_nan(hi, quad_xor1(hi));
    lo = max_nan(min_nan(min_nan(lo, quad_xor2(lo)), 32768.0f), -32768.0f);
    hi = max_nan(min_nan(max_nan(hi, quad_xor2(hi)), 32768.0f), -32768.0f);
    float step = (hi - lo) * (1.0f / 15.0f);
    asm("" : "+v"(step));  // rounded to fp32 first: a fused multiply and conversion would round once
    const _Float16 m = (_Float16)lo, s = (_Float16)step;
    const float mf = (float)m, sf = (float)s;
    const float r = sf > 0.0f ? 1.0f / sf : 0.0f;
    // Saturating the ends saturates every value: one beyond them gets the code of the end.  At the lower one that is 0,
    // at the upper one 15, unless m was rounded up almost to it (fp32 only: 16-bit values are exact in m there).
    const float most = DT == VQ_F32 ? __builtin_amdgcn_fmed3f((hi - mf) * r, 0.0f, 15.0f) : 15.0f;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = (x[j] - mf) * r;  // NaN: the median is the smaller bound
      w |= (uint32_t)__builtin_rintf(__builtin_amdgcn_fmed3f(t, 0.0f, most)) << (4 * j);
    }
    word[i] = w;
    s16[i] = __builtin_bit_cast(uint16_t, s);
    m16[i] = __builtin_bit_cast(uint16_t, m);
  }

  uint8_t *cb = codes_at<D>(c, p);
  const bool full = p.lo == 0 && p.hi == 4;
  if (p.kind == 0) {
    uint32_t *rows = reinterpret_cast<uint32_t *>(cb) + (int64_t)p.off * (D / 8) + key_word<D>(p.oct);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i >= p.lo && i < p.hi) rows[i * (D / 8)] = word[i];
  } else {
    uint8_t *qb = cb + (int64_t)p.off * (D / 2) + p.oct * 16;
    if (full) {
      uint4_t o;
#pragma unroll
      for (int g = 0; g < 4; ++g)  // channel pair g: slots 0, 2, 1, 3 from the low byte
        o[g] = ((word[0] >> (8 * g)) & 0xffu) | ((word[2] >> (8 * g)) & 0xffu) << 8 |
               ((word[1] >> (8 * g)) & 0xffu) << 16 | ((word[3] >> (8 * g)) & 0xffu) << 24;
      *reinterpret_cast<uint4_t *>(qb) = o;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i >= p.lo && i < p.hi) {
#pragma unroll
          for (int g = 0; g < 4; ++g) qb[g * 4 + value_byte(i)] = (uint8_t)(word[i] >> (8 * g));
        }
    }
  }
  if ((p.oct & 3) == 0) {
    uint16_t *sp = scales_at<D>(c, p);
    if (full) {
      const uint4_t o = {(uint32_t)s16[0] | (uint32_t)s16[1] << 16, (uint32_t)s16[2] | (uint32_t)s16[3] << 16,
                         (uint32_t)m16[0] | (uint32_t)m16[1] << 16, (uint32_t)m16[2] | (uint32_t)m16[3] << 16};
      *reinterpret_cast<uint4_t *>(sp) = o;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i >= p.lo && i < p.hi) sp[i] = s16[i], sp[4 + i] = m16[i];
    }
  }
  if (p.kind == 0 && p.oct < 4) {  // slot p.oct of the quad: its weight and position
    const int i = p.oct;
    if (i >= p.lo && i < p.hi) {
      const int64_t at = (p.page * c.hkv + p.head) * c.ps + p.off + i;
      const int start = c.lens ? max(c.lens[p.seq], 0) : 0;
      c.weights[at] = weights ? weights[(int64_t)p.head * total + p.row + i] : 0.0f;
      c.pos[at] = (pos ? pos[p.seq] : start) + (p.slot + i - start);
    }
  }
}

template <int D, int DT>
__global__ __launch_bounds__(kThreads) void k_kv4_read(KvView c, int total, const int32_t *__restrict__ cu,
                                                       void *__restrict__ k_out, void *__restrict__ v_out, int per) {
  const int vq = blockIdx.x / per;
  const int item = (blockIdx.x - vq * per) * kThreads + threadIdx.x;
  const Place p = place_of<D>(c, cu, total, vq, item);
  if (!p.any) return;
  uint32_t word[4] = {0, 0, 0, 0};
  uint4_t sm = {0, 0, 0, 0};
  if (p.stored) {
    const uint8_t *cb = codes_at<D>(c, p);
    if (p.kind == 0) {
      const uint32_t *rows = reinterpret_cast<const uint32_t *>(cb) + (int64_t)p.off * (D / 8) + key_word<D>(p.oct);
#pragma unroll
      for (int i = 0; i < 4; ++i) word[i] = rows[i * (D / 8)];
    } else {
      const uint4_t o = *reinterpret_cast<const uint4_t *>(cb + (int64_t)p.off * (D / 2) + p.oct * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int sh = 8 * value_byte(i);
#pragma unroll
        for (int g = 0; g < 4; ++g) word[i] |= ((o[g] >> sh) & 0xffu) << (8 * g);
      }
    }
    sm = *reinterpret_cast<const uint4_t *>(scales_at<D>(c, p));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < p.lo || i >= p.hi) continue;
    const half2_t sp = as_h2(sm[i / 2]), mp = as_h2(sm[2 + i / 2]);
    const float s = (float)sp[i & 1], m = (float)mp[i & 1];
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(__fmul_rn((float)((word[i] >> (4 * j)) & 15u), s), m);
    store8<DT>(p.kind ? v_out : k_out, ((p.row + i) * c.hkv + p.head) * D + p.oct * 8, x);
  }
}

// Workgroups: `per` of them cover a quad's keys and values of every head.
int groups_per_quad(const KvView &c) { return (2 * c.hkv * (c.d / 8) + kThreads - 1) / kThreads; }

template <int D>
hipError_t append_d(const KvView &c, const void *k, const void *v, int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs,
                    int dtype, int total, const int32_t *cu, const int32_t *pos, const float *weights, hipStream_t s) {
  const int per = groups_per_quad(c);
  const dim3 grid((unsigned)((total / 4 + 2 * (int64_t)c.nseq) * per));
  auto go = [&](auto kernel) {
    kernel<<<grid, kThreads, 0, s>>>(c, k, v, k_ts, k_hs, v_ts, v_hs, total, cu, pos, weights, per);
    return hipGetLastError();
  };
  if (dtype == VQ_F32) return go(k_kv4_append<D, VQ_F32>);
  if (dtype == VQ_BF16) return go(k_kv4_append<D, VQ_BF16>);
  return go(k_kv4_append<D, VQ_F16>);
}

template <int D>
hipError_t read_d(const KvView &c, const int32_t *cu, int total, int dtype, void *k_out, void *v_out, hipStream_t s) {
  const int per = groups_per_quad(c);
  const dim3 grid((unsigned)((total / 4 + 2 * (int64_t)c.nseq) * per));
  auto go = [&](auto kernel) {
    kernel<<<grid, kThreads, 0, s>>>(c, total, cu, k_out, v_out, per);
    return hipGetLastError();
  };
  if (dtype == VQ_F32) return go(k_kv4_read<D, VQ_F32>);
  if (dtype == VQ_BF16) return go(k_kv4_read<D, VQ_BF16>);
  return go(k_kv4_read<D, VQ_F16>);
}

}  // namespace

hipError_t launch_kv4_append(const KvView &c, const void *k, const void *v, int64_t k_ts, int64_t k_hs, int64_t v_ts,
                             int64_t v_hs, int dtype, int total, const int32_t *cu, const int32_t *pos,
                             const float *weights, hipStream_t s) {
  if (c.d == 64) return append_d<64>(c, k, v, k_ts, k_hs, v_ts, v_hs, dtype, total, cu, pos, weights, s);
  if (c.d == 128) return append_d<128>(c, k, v, k_ts, k_hs, v_ts, v_hs, dtype, total, cu, pos, weights, s);
  return append_d<256>(c, k, v, k_ts, k_hs, v_ts, v_hs, dtype, total, cu, pos, weights, s);
}

hipError_t launch_kv4_read(const KvView &c, const int32_t *cu, int total, int dtype, void *k_out, void *v_out,
                           hipStream_t s) {
  if (c.d == 64) return read_d<64>(c, cu, total, dtype, k_out, v_out, s);
  if (c.d == 128) return read_d<128>(c, cu, total, dtype, k_out, v_out, s);
  return read_d<256>(c, cu, total, dtype, k_out, v_out, s);
}

}  // namespace vqmm
