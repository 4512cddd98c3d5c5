// attn_prompt_weights: the weight each key gathers, the column sums of
// exp(scale q.k - lse) over a group's heads and a run of queries.
//
// A workgroup owns 128 keys of one key/value head, 32 a wave, held in registers
// as one operand of 32x32x16 MFMA; the queries of the group's heads pass through
// double-buffered LDS, straight from global memory.  S = Q K^T puts a key in a lane's column and 16 queries in
// its registers, so the sum over queries needs no exchange until the end, and
// one workgroup sees all the queries of its keys (or a piece of them, where key
// blocks are few; pieces meet in a second launch): no atomics, a fixed order.
//
// Bound: vector issue (an exponential, a fused multiply-add and an add a pair)
// next to 2 head_dim flops on the matrix cores.  Every query of 8191 + 2000
// tokens, 32/8 heads of 128: 324 + 5 us, 0.89 PFLOP/s.  7620 keys of three prompts
// against their last 64 queries: 13.1 us, mostly the latency of four rounds;
// every query of 2048 + 701, 9/3 heads of 64: 11.4 + 3.9 us.
#include "attn_device.h"

#include <algorithm>

namespace vqmm {

namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 128;
// Beyond this |lse| exp(s - lse) cannot be taken as exp2(s c - lse log2 e): the two
// roundings, 2^-24 of their size, are then many powers of two.
constexpr float kLargeLse = 1048576.0f;

template <int D, int BQ, bool F16, bool CAUSAL>
__global__ __launch_bounds__(kThreads) void k_attn_weights(AttnView a, const float *__restrict__ lse, int last,
                                                           int accumulate, float *__restrict__ weights, int pieces) {
  constexpr int NK = D / 16, NQ = BQ / 32;
  __shared__ __attribute__((aligned(1024))) uint16_t s_q[2][BQ * D];
  __shared__ __attribute__((aligned(16))) float s_lse[2][BQ];
  __shared__ __attribute__((aligned(16))) float s_raw[2][BQ];  // the lse as they came, for tiles with one beyond kLargeLse
  __shared__ int s_large[2];

  const int kvh = blockIdx.x % a.hkv;
  const int piece = blockIdx.x / a.hkv % pieces, vt = blockIdx.x / a.hkv / pieces;
  int first;
  const int b = find_tile(a.cu_k, a.nseq, a.tk, kKeys, 1, vt, &first);
  if (b < 0) return;
  const Rows rq = seq_rows(a.cu_q, b, a.tq), rk = seq_rows(a.cu_k, b, a.tk);
  const int k0 = (vt - first) * kKeys;
  if (k0 >= rk.n) return;
  const int off = rk.n - rq.n;
  const int group = a.hq / a.hkv;

  const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = k0 + wave * 32, ki = kw + col;
  uint4_t kf[NK];
  {
    const uint16_t *kp = a.k + (rk.begin + (int64_t)min(ki, rk.n - 1)) * a.k_ts + kvh * a.k_hs + 8 * h;
#pragma unroll
    for (int i = 0; i < NK; ++i) kf[i] = *reinterpret_cast<const uint4_t *>(kp + 16 * i);
  }

  // queries from `low` on: the last ones, and of those the ones that see the first key
  int low = last > 0 ? max(0, rq.n - last) : 0;
  if (CAUSAL) low = max(low, k0 - off);
  const int ni = low < rq.n ? (rq.n - low + BQ - 1) / BQ : 0;
  const int items = ni * group;
  const int it0 = (int)((int64_t)items * piece / pieces), it1 = (int)((int64_t)items * (piece + 1) / pieces);
  const float cs = a.scale * kLog2e;

  const Stage<D, BQ> sq(wave, lane, false);
  const uint32_t lq = lds_address(s_q);
  // piece 2 i + h of the lane's query row, at qa ^ 32 i (256 bytes on from i = 8)
  const uint32_t qa = lq + col * (2 * D) + (h ^ key_swizzle<D>(col)) * 16;
  float next_lse = 0.0f;
  auto fetch = [&](int it) {
    const int head = kvh * group + it / ni, r0 = low + it % ni * BQ;
    if (threadIdx.x < BQ) {
      const int row = r0 + threadIdx.x;
      next_lse = row < rq.n ? lse[(int64_t)head * a.tq + rq.begin + row] : -INFINITY;
    }
    sq.load(lq + (it & 1) * (BQ * D * 2), a.q + rq.begin * a.q_ts + head * a.q_hs, a.q_ts, r0, rq.n, wave);
  };
  auto publish = [&](int it) {
    // rows past the end, and rows of nothing but -inf, give exp2(-inf) = 0
    if (threadIdx.x < BQ) {
      s_lse[it & 1][threadIdx.x] = next_lse == -INFINITY ? INFINITY : next_lse * kLog2e;
      const bool large = __any(fabsf(next_lse) > kLargeLse && next_lse != -INFINITY);
      if (large) s_raw[it & 1][threadIdx.x] = next_lse == -INFINITY ? INFINITY : next_lse;
      if (threadIdx.x == 0) s_large[it & 1] = large;
    }
    wait_loads();
    __syncthreads();
  };
  float sum = 0.0f;
  if (it0 < it1) {
    fetch(it0);
    publish(it0);
  }
  for (int it = it0; it < it1; ++it) {
    if (it + 1 < it1) fetch(it + 1);
    const int r0 = low + it % ni * BQ;
    const uint32_t qs = qa + (it & 1) * (BQ * D * 2);
    const int large = s_large[it & 1];
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int rw = r0 + 32 * n;
      if (rw >= rq.n || (CAUSAL && rw + 31 + off < kw)) continue;  // none of these queries sees a key of the wave
      const bool mask = rw + 32 > rq.n || (CAUSAL && rw + off < kw + 31);
      float16_t S;
      auto scores = [&] {
#pragma unroll
        for (int r = 0; r < 16; ++r) S[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < NK; ++i) S = mfma32<F16>(lds_read((qs ^ (i & 7) * 32) + n * 64 * D + (i >> 3) * 256), kf[i], S);
      };
      scores();
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float4_t l4 = *reinterpret_cast<const float4_t *>(&s_lse[it & 1][32 * n + 8 * x + 4 * h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) S[4 * x + i] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[4 * x + i], cs, -l4[i]));
      }
      if (mask | __builtin_amdgcn_readfirstlane(large)) {
        asm volatile("");  // a branch, not selects in every tile
        if (large) {  // anew, the difference first: the common tiles pay nothing for these
          scores();
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const float l = s_raw[it & 1][32 * n + 8 * (r / 4) + 4 * h + (r & 3)];
            S[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[r], a.scale, -l) * kLog2e);
          }
        }
        const int from = max(CAUSAL ? ki - off : 0, 0) - rw - 4 * h, to = rq.n - rw - 4 * h;  // the queries that count
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int q = 8 * (r / 4) + (r & 3);
          S[r] = q >= from && q < to ? S[r] : 0.0f;
        }
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) part[r & 3] += S[r];
    }
    sum += (part[0] + part[1]) + (part[2] + part[3]);
    if (it + 1 < it1) publish(it + 1);
  }
  sum = sum_xor32(sum);
  if (h == 0 && ki < rk.n) {
    float *w = weights + ((int64_t)piece * a.hkv + kvh) * a.tk + rk.begin + ki;
    *w = accumulate ? *w + sum : sum;
  }
}

// Pieces of the queries meet, in order.  Keys before the first sequence or past
// the last have no pieces and keep what they hold, as they do without pieces.
__global__ __launch_bounds__(kThreads) void k_attn_weights_join(const float *__restrict__ part, int64_t n, int tk, int nseq,
                                                                const int32_t *__restrict__ cu_k, int pieces,
                                                                int accumulate, float *__restrict__ weights) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  const int key = (int)(i % tk);
  if (key < cu_k[0] || key >= cu_k[nseq]) return;
  float sum = 0.0f;
#pragma unroll 8
  for (int p = 0; p < pieces; ++p) sum += part[p * n + i];
  weights[i] = accumulate ? weights[i] + sum : sum;
}

template <int D, int BQ, bool F16>
hipError_t weights_d(const AttnView &a, const PromptPlan &p, const float *lse, int last, bool accumulate, float *weights,
                     float *ws, hipStream_t s) {
  const unsigned grid = (unsigned)((int64_t)(a.tk / kKeys + a.nseq) * a.hkv * p.pieces);
  const int64_t n = (int64_t)a.hkv * a.tk;
  float *to = p.pieces > 1 ? ws : weights;
  const int add = p.pieces == 1 && accumulate;
  if (a.causal) k_attn_weights<D, BQ, F16, true><<<grid, kThreads, 0, s>>>(a, lse, last, add, to, p.pieces);
  else k_attn_weights<D, BQ, F16, false><<<grid, kThreads, 0, s>>>(a, lse, last, add, to, p.pieces);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.pieces == 1) return e;
  k_attn_weights_join<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(ws, n, a.tk, a.nseq, a.cu_k, p.pieces,
                                                                                      accumulate, weights);
  return hipGetLastError();
}

}  // namespace

// Few key blocks (less than one and a half a CU) are cut along the queries,
// into about 1536 workgroups of at least one tile, and long runs of queries
// into pieces of about 64 tiles: under a causal mask the first keys have the
// most queries, so pieces also even the work out (8191 + 2000 tokens of 32/8
// heads, 648 key blocks: one piece took 841 us, five 447 us).
PromptPlan attn_weights_plan(const AttnView &a, int last) {
  PromptPlan p{1, 0, 0};
  const int64_t blocks = ((int64_t)a.tk / kKeys + a.nseq) * a.hkv, group = a.hq / a.hkv;
  const int64_t mean = a.nseq > 0 ? ((int64_t)a.tq + a.nseq - 1) / a.nseq : 0;
  const int64_t most = ((last > 0 ? std::min(last, a.tq) : a.tq) + 63) / 64 * group;
  const int64_t run = ((last > 0 ? std::min<int64_t>(last, mean) : mean) + 63) / 64 * group;
  const int64_t want = std::max<int64_t>(blocks > 0 && blocks < 384 ? 1536 / blocks : 1, (run + 63) / 64);
  p.pieces = (int)std::max<int64_t>(1, std::min<int64_t>({want, most, 32, blocks > 0 ? kMaxBlocks / blocks : 1}));
  if (p.pieces > 1) p.bytes = (size_t)p.pieces * a.hkv * a.tk * 4;
  return p;
}

hipError_t launch_attn_weights(const AttnView &a, const PromptPlan &p, const float *lse, int last, bool accumulate,
                               float *weights, void *ws, hipStream_t s) {
  float *w = static_cast<float *>(ws);
  if (a.d == 64)
    return a.f16 ? weights_d<64, 64, true>(a, p, lse, last, accumulate, weights, w, s)
                 : weights_d<64, 64, false>(a, p, lse, last, accumulate, weights, w, s);
  if (a.d == 128)
    return a.f16 ? weights_d<128, 64, true>(a, p, lse, last, accumulate, weights, w, s)
                 : weights_d<128, 64, false>(a, p, lse, last, accumulate, weights, w, s);
  return a.f16 ? weights_d<256, 32, true>(a, p, lse, last, accumulate, weights, w, s)
               : weights_d<256, 32, false>(a, p, lse, last, accumulate, weights, w, s);
}

}  // namespace vqmm
