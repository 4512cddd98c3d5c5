// attn_prompt: softmax(scale Q K^T) V over packed sequences, grouped heads.
//
// One pass over the keys with a running maximum and sum.  A workgroup of four
// waves takes 128 queries of one head, 32 a wave, and walks the keys BN at a
// time through double-buffered LDS (the next tile goes from global memory
// straight into LDS during the products).  Both products are taken transposed
// on 32x32x16 MFMA:
//   S^T = K Q^T   the operand of a query column stays in registers, and a lane
//                 ends up with half the keys of one query, so maximum and sum
//                 take one exchange between lane halves;
//   O^T = V^T P^T the reduction order is free, so the keys a lane holds are
//                 taken as its eight of the reduction and P never leaves its
//                 registers; V^T comes out of row-major LDS by the transposing
//                 reads (4 keys x 16 channels a group of 16 lanes).
// The reference maximum may lag the running one by 2^8, so most tiles skip the
// rescale of O.  P takes v's 16-bit type, as the product's other operand: its
// rounding leaves results 1.25 times the error of a 16-bit result of the fp32 form
// (relative 2.0e-3 and 1.6e-3 in bf16).  A second product with P's remainder ends
// that and was not taken: half as many matrix instructions again, 729 -> 967 us for
// the prompts below.
//
// Bound: the matrix cores and, sharing each SIMD's issue with them, the vector
// work of the softmax (about 100 instructions a lane for 32 keys, 16 of
// them exponentials, against 16 products of 32 cycles; matrix cores 60% busy).
// Waves overlap the two, so
// tiles are as small as it takes to hold three waves a SIMD for heads of 128
// (BN = 32), four for 64 (BN = 64) and two for 256 (BN = 32): 64 keys and two
// waves took 751 us where 32 and three took 731.  Under this load the clock falls to
// about 1.8 GHz (a library product of 8192^3 with its matrix cores 93% busy runs at
// 1.4), so instructions saved count twice.  Measured: 14,919 tokens in five prompts,
// 32/8 heads of 128, bf16, causal: 729 us a pass, 1.0 PFLOP/s (a bf16 library product
// reached 1.35 to 1.41; 776 us is the median of 30 traced ones, at a lower clock);
// 4096 + 2000 tokens of 16/4 heads of 256: 190 us, 0.90 PFLOP/s.
#include "attn_device.h"

#include <algorithm>

namespace vqmm {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 128;  // queries of a workgroup
constexpr float kSlack = 8.0f;
// fp16 probabilities are taken 2^7 larger, by a reference that much below the maximum it was taken from: up to 2^15 with
// the lag, and with 11 bits down to 2^-21 of the largest.  Without it that ends at 2^-14, and below 2^-25 they are lost:
// where one key of 32 has a score 17 above the others', the others' part of the result was off by 4 %, at 18.5 by 95 %.
// bf16 has fp32's exponents.
template <bool F16>
constexpr float kRoom = F16 ? 7.0f : 0.0f;
template <bool F16>
constexpr float kUnroom = F16 ? 0.0078125f : 1.0f;
// Beyond this reference (log2 domain) one fused multiply-add no longer does: the reference is a rounded product and its
// rounding, 2^-24 of itself, is then many powers of two, which exp2 would send to infinity.
constexpr float kLargeRef = 1048576.0f;

typedef __attribute__((address_space(3))) short4_t lds_short4;
// Four 16-bit values of one column, rows 0..3 of a 4 x 16 block in LDS whose
// row r, columns 4 j .. 4 j + 3 the lane 4 r + j of the 16 points at.
__device__ __forceinline__ uint2_t lds_column(uint32_t at) {
  return __builtin_bit_cast(uint2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(uintptr_t)at));
}

// Infinities and NaN among the eight values of a 16-byte piece become zeros;
// returns whether there were any.
template <bool F16>
__device__ __forceinline__ bool clear_nonfinite(uint4_t &w) {
  constexpr uint32_t kExp = F16 ? 0x7c007c00u : 0x7f807f80u, kOne = F16 ? 0x04000400u : 0x00800080u;
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t full = ((w[i] & kExp) + kOne) & 0x80008000u;  // a full exponent carries into the sign's place
    any |= full;
    w[i] &= ~((full >> 15) * 0xffffu);
  }
  return any != 0;
}
template <bool F16>
__device__ __forceinline__ float nonfinite_of(uint32_t h) {
  const float f = F16 ? h2f(h) : bf2f(h);
  return __builtin_isfinite(f) ? 0.0f : f;
}

// The pieces of a row block's keys: `piece` of them takes tiles from *lo to
// *hi of nt, none of fewer than kMinKeys keys but the last.
constexpr int kMinKeys = 256;
__device__ __forceinline__ void piece_tiles(int nt, int pieces, int piece, int bn, int *lo, int *hi) {
  const int per = max((nt + pieces - 1) / pieces, kMinKeys / bn);
  *lo = min(piece * per, nt);
  *hi = min(*lo + per, nt);
}

struct PromptOut {
  uint16_t *out;
  float *lse;
  float *part;  // [piece][row][head][D], sums of p v
  float *stat;  // [piece][row][head][2]: reference (log2 domain), sum of p
};

// SPLIT: the workgroup takes one piece of its keys and leaves its sums in the
// workspace for k_attn_join.
template <int D, int BN, bool F16, bool CAUSAL, bool SPLIT>
__global__ __launch_bounds__(kThreads, D <= 128 ? 3 : 2) void k_attn_prompt(AttnView a, PromptOut o, int tiles,
                                                                            int pieces) {
  constexpr int NS = BN / 32, ND = D / 32, NK = D / 16;
  __shared__ __attribute__((aligned(1024))) uint16_t s_k[2][BN * D];
  __shared__ __attribute__((aligned(1024))) uint16_t s_v[2][BN * D];
  __shared__ int s_cleared;

  // heads of a group share keys and values: they come next to one another,
  // key/value heads fastest (workgroups are dealt to the XCDs in turn, so with
  // 8 of them an XCD's L2 serves one); late tiles, the long ones, first
  int id = blockIdx.x;
  const int kvh = id % a.hkv;
  id /= a.hkv;
  int piece = 0;
  if (SPLIT) {
    piece = id % pieces;
    id /= pieces;
  }
  const int group = a.hq / a.hkv;
  const int head = kvh * group + id % group;
  const int vt = tiles - 1 - id / group;
  int first;
  const int b = find_tile(a.cu_q, a.nseq, a.tq, kRows, 1, vt, &first);
  if (b < 0) return;
  const Rows rq = seq_rows(a.cu_q, b, a.tq), rk = seq_rows(a.cu_k, b, a.tk);
  const int q0 = (vt - first) * kRows;
  if (q0 >= rq.n) return;
  const int off = rk.n - rq.n;  // query i sees keys j <= i + off

  const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int qw = q0 + wave * 32;  // the wave's first query
  const int qi = qw + col;
  const int lim = CAUSAL ? min(qi + off, rk.n - 1) : rk.n - 1;  // last key this lane's query sees
  const int lim_first = CAUSAL ? min(qw + off, rk.n - 1) : rk.n - 1;  // the same of the wave's first and last
  const int lim_last = CAUSAL ? min(qw + 31 + off, rk.n - 1) : rk.n - 1;
  const int seen = CAUSAL ? min(q0 + kRows + off, rk.n) : rk.n;  // keys the workgroup needs
  const int all_see = CAUSAL ? min(q0 + off, rk.n - 1) : rk.n - 1;  // the last key that every query of it sees
  int t_lo = 0, nt = seen > 0 ? (seen + BN - 1) / BN : 0;
  if (SPLIT) {
    piece_tiles(nt, pieces, piece, BN, &t_lo, &nt);
    if (t_lo >= nt) return;  // an empty piece: k_attn_join knows
  }

  const uint16_t *kb = a.k + rk.begin * a.k_ts + kvh * a.k_hs;
  const uint16_t *vb = a.v + rk.begin * a.v_ts + kvh * a.v_hs;

  uint4_t qf[NK];
  {
    const uint16_t *qp = a.q + (rq.begin + (int64_t)min(qi, rq.n - 1)) * a.q_ts + head * a.q_hs + 8 * h;
#pragma unroll
    for (int i = 0; i < NK; ++i) qf[i] = *reinterpret_cast<const uint4_t *>(qp + 16 * i);
  }
  float16_t acc[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.0f;
  float mref = -INFINITY, m0 = 0.0f, lsum = 0.0f;  // the reference in units of scores and in the log2 domain
  const float cs = a.scale * kLog2e;
  const float room = kRoom<F16> / cs, slack = (kSlack + kRoom<F16>) / cs;
  bool large = false;  // some query's reference is beyond kLargeRef

  const Stage<D, BN> sk(wave, lane, false), sv(wave, lane, true);
  const uint32_t lk = lds_address(s_k), lv = lds_address(s_v);
  auto fetch = [&](int t) {
    sk.load(lk + (t & 1) * (BN * D * 2), kb, a.k_ts, t * BN, seen, wave);
    sv.load(lv + (t & 1) * (BN * D * 2), vb, a.v_ts, t * BN, seen, wave);
  };
  // Where the lane reads: piece 2 i + h of its key row, at ka ^ 32 i (256 bytes on from i = 8); of the value rows
  // 4 h + (i16 / 4) the channels 16 (lane / 16 % 2) + 4 (i16 % 4) of 32-channel block d, at va ^ 64 d (256 bytes on
  // from d = 4).  The swizzles are XORs too, and rows and tiles begin at multiples of 128 or 256 bytes, so one base a
  // tile does.
  const uint32_t ka = lk + col * (2 * D) + (h ^ key_swizzle<D>(col)) * 16;
  const int vrow = 4 * h + ((lane & 15) >> 2);
  const uint32_t va = lv + vrow * (2 * D) + ((2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ value_swizzle<D>(vrow)) * 16 + (lane & 1) * 8;
  if (threadIdx.x == 0) s_cleared = 0;
  if (t_lo < nt) fetch(t_lo);
  wait_loads();
  __syncthreads();
  for (int t = t_lo; t < nt; ++t) {
    const int k0 = t * BN;
    if (t + 1 < nt) fetch(t + 1);
    if (k0 + BN - 1 > all_see) {
      // Some query does not see some key of this tile: its probability is 0, but 0 times an infinity would be NaN.
      // What is not finite leaves the tile and comes back at the end, for the queries that do see it.
#pragma unroll
      for (int i = threadIdx.x; i < BN * D / 8; i += kThreads) {
        uint4_t *p = reinterpret_cast<uint4_t *>(s_v[t & 1]) + i;
        uint4_t w = *p;
        if (clear_nonfinite<F16>(w)) {
          *p = w;
          s_cleared = 1;
        }
      }
      __syncthreads();
    }
    if (k0 <= lim_last) {
      const uint32_t ks = ka + (t & 1) * (BN * D * 2), vs = va + (t & 1) * (BN * D * 2);
      float16_t S[NS];
      // the keys' pieces in the order of their products, kAhead of them read ahead
      constexpr int kAhead = D == 256 ? 4 : NK < 8 ? NK : 8, kAll = NS * NK;
      uint4_t kf[kAhead];
      auto read_k = [&](int x) {
        const int n = x / NK, i = x % NK;
        return lds_read((ks ^ (i & 7) * 32) + n * 64 * D + (i >> 3) * 256);
      };
#pragma unroll
      for (int x = 0; x < kAhead; ++x) kf[x] = read_k(x);
      sched_fence();
#pragma unroll
      for (int n = 0; n < NS; ++n) {
#pragma unroll
        for (int r = 0; r < 16; ++r) S[n][r] = 0.0f;
      }
#pragma unroll
      for (int x = 0; x < kAll; ++x) {
        S[x / NK] = mfma32<F16>(kf[x % kAhead], qf[x % NK], S[x / NK]);
        if (x + kAhead < kAll) kf[x % kAhead] = read_k(x + kAhead);
      }
#pragma unroll
      for (int x = 0; x < kAll; ++x) {
        sched_group<0x008, 1>();
        if (x + kAhead < kAll) sched_group<0x100, 1>();
      }
      sched_fence();
      if (k0 + BN - 1 > lim_first) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int key = k0 + 32 * n + 8 * (r / 4) + 4 * h + (r & 3);
            S[n][r] = key <= lim ? S[n][r] : -INFINITY;
          }
      }
      float top = S[0][0];
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, S[n][r]);
      top = max_xor32(top);
      if (__any(top - mref > slack) | large) {
        const float mnew = fmaxf(mref, F16 ? top - room : top);
        const float f = mnew == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((mref - mnew) * cs);
        lsum *= f;
#pragma unroll
        for (int i = 0; i < ND; ++i) acc[i] *= f;
        mref = mnew;
        m0 = mref == -INFINITY ? 0.0f : mref * cs;
        large = __any(fabsf(m0) > kLargeRef);
        if (large) {  // the difference first: exact near the top
          asm volatile("");
          const float m = mref == -INFINITY ? 0.0f : mref;
#pragma unroll
          for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r) S[n][r] -= m;
          m0 = 0.0f;
        }
      }
      float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          S[n][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[n][r], cs, -m0));
          part[r & 3] += S[n][r];
        }
      lsum += (part[0] + part[1]) + (part[2] + part[3]);
      constexpr int kVAhead = (ND < 4 ? ND : 4), kVAll = 2 * NS * ND;
      uint4_t vf[kVAhead];
      auto read_v = [&](int x) {
        const int st = x / ND, d = x % ND;
        const uint32_t p = (vs ^ (d & 3) * 64) + 32 * st * D + (d >> 2) * 256;
        const uint2_t v0 = lds_column(p), v1 = lds_column(p + 16 * D);
        return uint4_t{v0[0], v0[1], v1[0], v1[1]};
      };
#pragma unroll
      for (int x = 0; x < kVAhead; ++x) vf[x] = read_v(x);
      uint4_t pf[2 * NS];
#pragma unroll
      for (int st = 0; st < 2 * NS; ++st)
#pragma unroll
        for (int i = 0; i < 4; ++i) pf[st][i] = pack16<F16>(S[st / 2][8 * (st & 1) + 2 * i], S[st / 2][8 * (st & 1) + 2 * i + 1]);
      sched_fence();
#pragma unroll
      for (int x = 0; x < kVAll; ++x) {
        acc[x % ND] = mfma32<F16>(vf[x % kVAhead], pf[x / ND], acc[x % ND]);
        if (x + kVAhead < kVAll) vf[x % kVAhead] = read_v(x + kVAhead);
      }
#pragma unroll
      for (int x = 0; x < kVAll; ++x) {
        sched_group<0x008, 1>();
        if (x + kVAhead < kVAll) sched_group<0x100, 2>();
      }
      sched_fence();
    }
    wait_loads();
    __syncthreads();
  }

  if (s_cleared) {
#pragma unroll 1
    for (int key = max((all_see + 1) / BN * BN, t_lo * BN); key < min(seen, nt * BN); ++key) {
      const uint16_t *vp_key = vb + key * a.v_ts + 4 * h;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint2_t w = *reinterpret_cast<const uint2_t *>(vp_key + 32 * d + 8 * x);
          if (key <= lim) {
            acc[d][4 * x] += nonfinite_of<F16>(w[0] & 0xffffu);
            acc[d][4 * x + 1] += nonfinite_of<F16>(w[0] >> 16);
            acc[d][4 * x + 2] += nonfinite_of<F16>(w[1] & 0xffffu);
            acc[d][4 * x + 3] += nonfinite_of<F16>(w[1] >> 16);
          }
        }
    }
  }

  lsum = sum_xor32(lsum);
  if (qi >= rq.n) return;
  const int64_t row = rq.begin + (int64_t)qi;
  if (SPLIT) {
    const int64_t at = ((int64_t)piece * a.tq + row) * a.hq + head;
    float *pp = o.part + at * D + 4 * h;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        *reinterpret_cast<float4_t *>(pp + 32 * d + 8 * x) =
            float4_t{acc[d][4 * x], acc[d][4 * x + 1], acc[d][4 * x + 2], acc[d][4 * x + 3]};
    if (h == 0) *reinterpret_cast<float2_t *>(o.stat + at * 2) = float2_t{mref * cs, lsum};
    return;
  }
  const float r = lsum == 0.0f ? 0.0f : 1.0f / lsum;
  uint16_t *op = o.out + (row * a.hq + head) * D + 4 * h;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint2_t w = {pack16<F16>(acc[d][4 * x] * r, acc[d][4 * x + 1] * r),
                         pack16<F16>(acc[d][4 * x + 2] * r, acc[d][4 * x + 3] * r)};
      *reinterpret_cast<uint2_t *>(op + 32 * d + 8 * x) = w;
    }
  if (o.lse && h == 0) {
    const float ref = mref == -INFINITY ? 0.0f : mref * cs, l2 = __builtin_amdgcn_logf(lsum * kUnroom<F16>);
    o.lse[(int64_t)head * a.tq + row] =
        fabsf(ref) > kLargeRef ? mref * a.scale + l2 * kLn2 : ((ref + kRoom<F16>)+l2) * kLn2;
  }
}

// The pieces meet: D / 4 lanes take one row of one head, in piece order.
template <int D, int BN, bool F16>
__global__ __launch_bounds__(kThreads) void k_attn_join(AttnView a, PromptOut o, int pieces) {
  constexpr int kLanes = D / 4;
  const int64_t at = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int d = threadIdx.x % kLanes * 4;
  if (at >= (int64_t)a.tq * a.hq) return;
  const int row = (int)(at / a.hq), head = (int)(at % a.hq);
  // the row's sequence: the last whose rows begin at or before it
  int lo = 0, hi = a.nseq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_rows(a.cu_q, mid, a.tq).begin <= row) lo = mid;
    else hi = mid - 1;
  }
  const Rows rq = seq_rows(a.cu_q, lo, a.tq), rk = seq_rows(a.cu_k, lo, a.tk);
  if (row < rq.begin || row >= rq.begin + rq.n) return;
  const int q0 = (row - rq.begin) / kRows * kRows;
  const int seen = a.causal ? min(q0 + kRows + rk.n - rq.n, rk.n) : rk.n;
  const int nt = seen > 0 ? (seen + BN - 1) / BN : 0;
  const int64_t step = (int64_t)a.tq * a.hq;
  const int per = max((nt + pieces - 1) / pieces, kMinKeys / BN), np = (nt + per - 1) / per;  // as piece_tiles
  float top = -INFINITY;
#pragma unroll 4
  for (int p = 0; p < np; ++p) top = fmaxf(top, o.stat[(p * step + at) * 2]);
  const float m0 = top == -INFINITY ? 0.0f : top;
  float4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
  float l = 0.0f;
#pragma unroll 4
  for (int p = 0; p < np; ++p) {
    const float2_t st = *reinterpret_cast<const float2_t *>(o.stat + (p * step + at) * 2);
    const float4_t v = *reinterpret_cast<const float4_t *>(o.part + (p * step + at) * D + d);
    const float f = __builtin_amdgcn_exp2f(st[0] - m0);
    l = __builtin_fmaf(st[1], f, l);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = __builtin_fmaf(v[i], f, sum[i]);
  }
  const float r = l == 0.0f ? 0.0f : 1.0f / l;
  *reinterpret_cast<uint2_t *>(o.out + at * D + d) =
      uint2_t{pack16<F16>(sum[0] * r, sum[1] * r), pack16<F16>(sum[2] * r, sum[3] * r)};
  if (o.lse && d == 0)
    o.lse[(int64_t)head * a.tq + row] = ((m0 + kRoom<F16>)+__builtin_amdgcn_logf(l * kUnroom<F16>)) * kLn2;
}

template <int D, int BN, bool F16>
hipError_t prompt_d(const AttnView &a, const PromptPlan &p, const PromptOut &o, hipStream_t s) {
  const int tiles = a.tq / kRows + a.nseq;
  const unsigned grid = (unsigned)((int64_t)tiles * a.hq * p.pieces);
  if (p.pieces == 1) {
    if (a.causal) k_attn_prompt<D, BN, F16, true, false><<<grid, kThreads, 0, s>>>(a, o, tiles, 1);
    else k_attn_prompt<D, BN, F16, false, false><<<grid, kThreads, 0, s>>>(a, o, tiles, 1);
    return hipGetLastError();
  }
  if (a.causal) k_attn_prompt<D, BN, F16, true, true><<<grid, kThreads, 0, s>>>(a, o, tiles, p.pieces);
  else k_attn_prompt<D, BN, F16, false, true><<<grid, kThreads, 0, s>>>(a, o, tiles, p.pieces);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int kRowsPerBlock = kThreads / (D / 4);
  const int64_t rows = (int64_t)a.tq * a.hq;
  k_attn_join<D, BN, F16><<<(unsigned)((rows + kRowsPerBlock - 1) / kRowsPerBlock), kThreads, 0, s>>>(a, o, p.pieces);
  return hipGetLastError();
}

}  // namespace

// Few row blocks (less than two a CU) are cut along the keys, into about 768
// workgroups of at most 8 pieces a row block, where there are keys enough (1024 a
// piece) to pay for the second launch; a short row block of such a call still
// keeps to pieces of 256.  Over ten shapes of chunks (1 to 1024 queries of one to
// eight sequences on 1,000 to 16,400 keys) with five head layouts, the mean time
// against 768 workgroups was 3.0 times in one piece, 1.25 with 256, 1.04 with 512,
// 1.00 with 1024 and with 1536, within 3 % the same for each head size but for 512
// (64: 1.03, 128: 1.09, 256: 1.00).
PromptPlan attn_prompt_plan(const AttnView &a) {
  PromptPlan p{1, 0, 0};
  const int64_t blocks = ((int64_t)a.tq / kRows + a.nseq) * a.hq;
  const int64_t most = a.tk / 1024;
  if (blocks > 0 && blocks < 512) p.pieces = (int)std::max<int64_t>(1, std::min<int64_t>({768 / blocks, most, 8}));
  if (p.pieces > 1) {
    const size_t rows = (size_t)p.pieces * a.tq * a.hq;
    p.stat_off = rows * a.d * 4;
    p.bytes = p.stat_off + rows * 8;
  }
  return p;
}

hipError_t launch_attn_prompt(const AttnView &a, const PromptPlan &p, uint16_t *out, float *lse, void *ws, hipStream_t s) {
  char *w = static_cast<char *>(ws);
  const PromptOut o{out, lse, reinterpret_cast<float *>(w), reinterpret_cast<float *>(w + p.stat_off)};
  if (a.d == 64) return a.f16 ? prompt_d<64, 64, true>(a, p, o, s) : prompt_d<64, 64, false>(a, p, o, s);
  if (a.d == 128) return a.f16 ? prompt_d<128, 32, true>(a, p, o, s) : prompt_d<128, 32, false>(a, p, o, s);
  return a.f16 ? prompt_d<256, 32, true>(a, p, o, s) : prompt_d<256, 32, false>(a, p, o, s);
}

}  // namespace vqmm
