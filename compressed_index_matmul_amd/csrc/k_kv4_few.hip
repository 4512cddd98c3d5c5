// kv4_attend_chunk for sequences of few rows (queries times heads of a group):
// single tokens under a window, drafted tokens to verify, short ends of chunks.
//
// A row tile is 32 rows of one sequence and key/value head: the columns of 32x32x16
// fp16 MFMA.  A wave walks tiles of 32 slots on its own and decodes them straight into
// its matrix operands; nothing of keys or values goes through LDS:
//   S^T = K Q^T   a lane takes one slot and half its words, the octets 4 j + 2 h + x, and
//                 the queries' registers follow that order;
//   O^T = V^T P^T a lane takes D / 32 neighbouring channels, one in each 32-channel block
//                 of the product, so that a word's two channels are both its own, and of
//                 the slots the quads that it holds of S^T.
// The tiles of all sequences, heads and row tiles form one line that a fixed number of
// workgroups cuts into equal shares, as kv4_attend does; parts of a row tile meet in a
// second launch.  Where no sequence has many slots a workgroup takes a row tile whole.
//
// Bound: HBM, 2 (D / 2 + D / 8) bytes a slot and head, next to vector issue (about 320
// instructions a tile of 32 slots and 128 channels, 216 of them decoding); in small
// calls the latency of the share that ends last and of the second launch.  Measured:
// 64 sequences of four queries on 1500 to 7200 slots, 32/8 heads of 128, bf16: 108 us,
// 3.3 TB/s; 512 single tokens on 1400 to 2900 slots 385 us, 3.7 TB/s (a torch maximum
// over as many bytes reads 3.85).
//
// Queries lie in LDS, the same for every wave.  Two tiles in flight a wave gained
// nothing (64 sequences on 8000 slots: 172 and 173 us), nor three waves a SIMD for heads
// of 128 (the same on long lengths, 5 to 10 % slower on short ones).  Heads of 256 in shares
// spill 2 registers, for fp16 results 8.
#include <algorithm>

#include "kv4_chunk.h"

namespace vqmm {

namespace {

constexpr int kTile = kFewTile, kRowTile = kFewRowTile;
constexpr int kJoinThreads = 256;
int shares_of(int d) { return 256 * (d == 64 ? kFewPerCu<64> : d == 128 ? kFewPerCu<128> : kFewPerCu<256>); }

template <int N>
struct Words {
  uint32_t w[N];
  __device__ __forceinline__ void load(const void *p) {
    if (N == 1) {
      w[0] = *static_cast<const uint32_t *>(p);
    } else if (N == 2) {
      const uint2_t v = *static_cast<const uint2_t *>(p);
      w[0] = v[0], w[N - 1] = v[1];
    } else {
#pragma unroll
      for (int i = 0; i + 3 < N; i += 4) {
        const uint4_t v = static_cast<const uint4_t *>(p)[i / 4];
        w[i] = v[0], w[i + 1] = v[1], w[i + 2] = v[2], w[i + 3] = v[3];
      }
    }
  }
};

template <int D, bool F16, int NW, bool LONE>
__global__ __launch_bounds__(NW *kWave, LONE ? 2 : kFewPerCu<D>) void k_kv4_few(KvView c, ChunkPlan p, ChunkArgs a) {
  constexpr int DG = D / 32, ND = D / 32, NK = D / 16;
  constexpr int kPitch = D + 4;  // floats of a row in LDS: 16-byte pieces of 16 rows fall on different banks
  typedef float Sums[16][kPitch];
  // the queries as the lanes want them, the same for every wave: in registers they would cost a third wave a SIMD (heads
  // of 128) or spill (256); then the waves' sums
  __shared__ __attribute__((aligned(16))) uint8_t s_buf[NW * sizeof(Sums)];
  static_assert(NW * sizeof(Sums) >= NK * kWave * 16, "");
  Sums *const s_o = reinterpret_cast<Sums *>(s_buf);
  __shared__ float s_m[NW][kRowTile], s_l[NW][kRowTile];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  typename FewCuts<D>::Line line{};
  int pos = 0, pos_end = 1;
  if (!LONE) line = FewCuts<D>::line_of(c, p, a, blockIdx.x, &pos, &pos_end);
  const int pos0 = pos;
  while (pos < pos_end) {
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // anew for each row tile: what follows from it would else be kept in registers throughout
    const int lane = tid & 63, col = lane & 31, h = lane >> 5;
    int b, kvh, rt, t_begin, t_end, side = 0;
    Extent e;
    if (LONE) {
      kvh = blockIdx.x % c.hkv;
      e = FewCuts<D>::row_tile(c, p, a, blockIdx.x / c.hkv, &b, &rt);
      if (rt < 0 || rt >= e.rtiles) return;
      t_begin = 0;
      t_end = e.tiles;
      pos = pos_end;
    } else {
      const auto seg = FewCuts<D>::segment(c, p, a, line, pos, pos_end);
      b = seg.b, kvh = seg.kvh, rt = seg.rt, t_begin = seg.begin, t_end = seg.end, e = seg.e;
      side = pos == pos0 && t_begin > 0 ? 0 : 1;  // 0: the row tile began in an earlier share
      pos += seg.steps;
      if (t_begin >= t_end) continue;  // only the end's allowance
    }
    const Rows rq = e.rq;
    const int len = e.len, off = len - rq.n, nrows = rq.n * p.group, r0 = rt * kRowTile;
    const int row = max(min(r0 + col, nrows - 1), 0), qi = row / p.group, head = kvh * p.group + row - qi * p.group;
    auto newest_of = [&](int r) { return max(min(r, nrows - 1) / p.group + off, -1); };
    const int lim = max(qi + off, -1), lim_first = newest_of(r0), lim_last = newest_of(r0 + kRowTile - 1);
    // some row does not see some slot of the tile
    auto partly = [&](int k0) { return k0 + kTile - 1 > lim_first || (k0 <= lim_last - p.window && k0 + kTile > p.sinks); };
    auto sees = [&](int slot) { return slot <= lim && (slot > lim - p.window || slot < p.sinks); };
    const Walk<kTile> walk(p, len, max(off, -1));

    const int64_t code_head = (int64_t)c.ps * (D / 2), scale_head = (int64_t)c.ps * (DG * 4);  // bytes
    const int last_block = max(len - 1, 0) >> 5;
    const uint32_t ko = col * (D / 2) + h * (D / 4), kso = (col >> 2) * (DG * 16) + (col & 2) * 2;
    const uint32_t vo = h * (2 * D) + col * (2 * DG), vso = h * (DG * 16) + (col * DG / 32) * 16;
    const uint32_t half_of = col & 1 ? 0x03020302u : 0x01000100u;  // the slot's half of a pair, twice
    Words<2 * DG> kw;
    uint32_t ks[DG], km[DG];
    Words<DG / 2> vw[4];
    uint4_t vs[4];
    const uint8_t *next_v, *next_vs;
    // Every tile's loads are followed by those of the wave's next tile, the last one's by its own again: no branch.  The
    // page of a tile is looked up while the one before it is fetched.
    int block, entry;
    auto look_up = [&](int t) {
      block = min(walk.tile(t), last_block);
      entry = table_entry(c, b, page_index(p, block));
    };
    auto fetch_keys = [&](int next) {
      const int64_t hd = (int64_t)page_in_pool(c, entry) * 2 * c.hkv + kvh;
      const int at = (block - page_index(p, block) * p.page_blocks) * 32;
      look_up(next);
      const uint8_t *kb = c.codes + hd * code_head + (int64_t)at * (D / 2);
      const uint8_t *sb = reinterpret_cast<const uint8_t *>(c.scales) + hd * scale_head + (int64_t)at * (DG * 4);
      kw.load(kb + ko);
#pragma unroll
      for (int j = 0; j < DG; ++j) {
        ks[j] = *reinterpret_cast<const uint32_t *>(sb + kso + 16 * j);
        km[j] = *reinterpret_cast<const uint32_t *>(sb + kso + 16 * j + 8);
      }
      next_v = kb + c.hkv * code_head;
      next_vs = sb + c.hkv * scale_head;
    };
    auto fetch_values = [&] {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        vw[i].load(next_v + vo + i * (4 * D));
        vs[i] = *reinterpret_cast<const uint4_t *>(next_vs + vso + i * (DG * 32));
      }
    };
    const Unpack unpack;
    int tile = t_begin + wave;
    auto after = [&](int t) { return t + NW < t_end ? t + NW : t; };
    if (tile < t_end) {
      look_up(tile);
      fetch_keys(after(tile));
      fetch_values();
    }

    // queries as fp16 after a power-of-two rescale per row, in the order of the unpacked codes
    float cs;  // scores -> log2 domain
    uint4_t qmid;
    {
      const uint16_t *qp = a.q + min(rq.begin + (int64_t)qi, (int64_t)a.tq - 1) * a.q_ts + head * a.q_hs;
      uint4_t qf[NK];
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        qf[i] = *reinterpret_cast<const uint4_t *>(qp + 8 * (4 * (i % DG) + 2 * h + i / DG));
        top = fmaxf(top, largest16<F16>(qf[i]));
      }
      top = max_xor32(top);
      const int lift = lift_of<F16>(top);
      cs = a.scale * kLog2e * __uint_as_float((uint32_t)(127 - lift) << 23);
#pragma unroll
      for (int i = 0; i < NK; ++i) qf[i] = lift16<F16>(qf[i], lift);
      if (F16) {
        float sums[DG];
#pragma unroll
        for (int g = 0; g < DG; ++g) sums[g] = sum_xor32(sum8(qf[g]) + sum8(qf[g + DG]));
        qmid = sums_operand<DG>(sums, h);
      }
      if (wave == 0)
#pragma unroll
        for (int i = 0; i < NK; ++i) *reinterpret_cast<uint4_t *>(s_buf + (i * kWave + lane) * 16) = qf[i];
      __syncthreads();
    }
    const uint32_t sq = lds_address(s_buf) + lane * 16;

    float16_t acc[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][r] = 0.0f;
    float mref = -INFINITY, m0 = 0.0f, lsum = 0.0f;  // the reference in units of scores and in the log2 domain
    const float room = kRoom / cs, slack = (kSlack + kRoom) / cs;
    bool large = false, cleared = false;
    for (; tile < t_end; tile += NW) {
#pragma unroll
      for (int i = 0; i < ND; ++i) asm volatile("" : "+v"(acc[i]));  // else a copy of them is kept for the rescale
      const int k0 = walk.tile(tile) * kTile;
      float16_t S;
#pragma unroll
      for (int r = 0; r < 16; ++r) S[r] = 0.0f;
      if (F16) {
        uint32_t mid[DG];  // pairs of minima, then of steps times 8
#pragma unroll
        for (int g = 0; g < DG; g += 2) {
          const uint32_t pair = col & 1 ? 0x07060302u : 0x05040100u;
          const half2_t eight = {(_Float16)8.0f, (_Float16)8.0f};
          mid[g / 2] = __builtin_amdgcn_perm(km[g + 1], km[g], pair);
          mid[DG / 2 + g / 2] = __builtin_bit_cast(uint32_t, as_h2(__builtin_amdgcn_perm(ks[g + 1], ks[g], pair)) * eight);
        }
        if (DG == 2) S = mfma32<true>(uint4_t{mid[0], mid[1], 0, 0}, qmid, S);
        else S = mfma32<true>(uint4_t{mid[0], mid[1], mid[2 % DG], mid[3 % DG]}, qmid, S);
        if (DG == 8) S = mfma32<true>(uint4_t{mid[4 % DG], mid[5 % DG], mid[6 % DG], mid[7 % DG]}, qmid, S);
        sched_fence();
      }
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const uint32_t sw = __builtin_amdgcn_perm(ks[i % DG], ks[i % DG], half_of);
        const uint4_t q = lds_read(sq + i * (kWave * 16));
        if (F16) {
          uint4_t upper, lower;
          split8(unpack, kw.w[i], as_h2(sw), &upper, &lower);
          S = mfma32<true>(upper, q, S);
          S = mfma32<true>(lower, q, S);
        } else {
          const uint32_t mw = __builtin_amdgcn_perm(km[i % DG], km[i % DG], half_of);
          S = mfma32<true>(values8(unpack, kw.w[i], as_h2(sw), as_h2(mw)), q, S);
        }
        if (i & 1) sched_fence();  // two words' values in registers at a time, not all of them
      }
      fetch_keys(after(after(tile)));

      if (partly(k0)) {
        asm volatile("");  // a branch, not selects in every tile
        // relative to the lane's first slot, so that the others are constants
        const int base = k0 + 4 * h, past = lim - base, low = past - p.window, sunk = p.sinks - base;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int x = 8 * (r / 4) + (r & 3);
          S[r] = (x <= past) & ((x > low) | (x < sunk)) ? S[r] : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) {  // see k_kv4_chunk
            const uint32_t shift = 16 * (x & 1), keep = ~(0xffffu << shift);
            const uint32_t s = vs[i][x / 2] >> shift, m = vs[i][2 + x / 2] >> shift;
            const bool out = k0 + 8 * i + 4 * h + x >= len, bad = (s & 0x7c00u) == 0x7c00u || (m & 0x7c00u) == 0x7c00u;
            if (out || bad) vs[i][x / 2] &= keep, vs[i][2 + x / 2] &= keep;
            cleared |= !out && bad;
          }
      }
      float top = S[0];
#pragma unroll
      for (int r = 1; r < 16; ++r) top = fmaxf(top, S[r]);
      top = max_xor32(top);
      if (__any(top - mref > slack) | large) {
        const float mnew = fmaxf(mref, top - room);
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
          for (int r = 0; r < 16; ++r) S[r] -= m;
          m0 = 0.0f;
        }
      }
      float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        S[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[r], cs, -m0));
        part[r & 3] += S[r];
      }
      lsum += (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        uint4_t pf, rest;  // rest: what the rounding left
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p0 = S[8 * st + 2 * i], p1 = S[8 * st + 2 * i + 1];
          pf[i] = pack16<true>(p0, p1);
          if (F16) rest[i] = pack16<true>(p0 - (float)as_h2(pf[i])[0], p1 - (float)as_h2(pf[i])[1]);
        }
#pragma unroll
        for (int i = 0; i < DG / 2; ++i) {
          uint4_t even, odd;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint4_t &sm = vs[2 * st + x];
            const uint32_t w = vw[2 * st + x].w[i];
            const half2_t s01 = as_h2(sm[0]), s23 = as_h2(sm[1]), m01 = as_h2(sm[2]), m23 = as_h2(sm[3]);
            even[2 * x] = __builtin_bit_cast(uint32_t, value(code_lo(unpack, w), s01, m01));
            even[2 * x + 1] = __builtin_bit_cast(uint32_t, value(code_lo(unpack, w >> 8), s23, m23));
            odd[2 * x] = __builtin_bit_cast(uint32_t, value(code_hi(unpack, w), s01, m01));
            odd[2 * x + 1] = __builtin_bit_cast(uint32_t, value(code_hi(unpack, w >> 8), s23, m23));
          }
          acc[2 * i] = mfma32<true>(even, pf, acc[2 * i]);
          acc[2 * i + 1] = mfma32<true>(odd, pf, acc[2 * i + 1]);
          if (F16) {
            acc[2 * i] = mfma32<true>(even, rest, acc[2 * i]);
            acc[2 * i + 1] = mfma32<true>(odd, rest, acc[2 * i + 1]);
          }
          sched_fence();
        }
      }
      fetch_values();
    }

    if (__any(cleared)) {  // what is not finite comes back for the rows that see it
#pragma unroll 1
      for (int t = t_begin + wave; t < t_end; t += NW) {
        const int k0 = walk.tile(t) * kTile;
        if (!partly(k0)) continue;
#pragma unroll 1
        for (int slot = k0; slot < min(k0 + kTile, len); ++slot) {
          const int pi = page_index(p, slot >> 5), at = slot - pi * c.ps;
          const int64_t hd = (page_of(c, b, pi) * 2 + 1) * c.hkv + kvh;
          const uint16_t *sb = c.scales + hd * (scale_head / 2) + (int64_t)(at / 4) * (DG * 8) + (at & 3);
          const bool seen = sees(slot);
#pragma unroll
          for (int r = 0; r < 16; ++r) {  // channels DG (8 (r / 4) + 4 h + (r & 3)) ..
            const int g = D == 256 ? 2 * (r / 4) + h : D == 128 ? r / 4 : r / 8;
            const uint32_t s = sb[8 * g], m = sb[8 * g + 4];
            const bool bad = (s & 0x7c00u) == 0x7c00u || (m & 0x7c00u) == 0x7c00u;
            if (bad && seen)
#pragma unroll
              for (int d = 0; d < ND; ++d) acc[d][r] = __builtin_nanf("");
          }
        }
      }
    }

    // the waves meet, 16 rows at a time
    const bool whole = LONE || (t_begin == 0 && t_end == e.tiles);
    lsum = sum_xor32(lsum);
    __syncthreads();  // every wave is done with the queries
    if (h == 0) s_m[wave][col] = mref == -INFINITY ? -INFINITY : mref * cs, s_l[wave][col] = lsum;
#pragma unroll 1
    for (int row0 = 0; row0 < kRowTile && r0 + row0 < nrows; row0 += 16) {
      if ((col & 16) == row0) {
#pragma unroll
        for (int x = 0; x < 16; ++x)
#pragma unroll
          for (int d = 0; d < ND; d += 2)
            *reinterpret_cast<float2_t *>(&s_o[wave][col & 15][DG * (8 * (x / 4) + 4 * h + (x & 3)) + d]) =
                float2_t{acc[d][x], acc[d + 1][x]};
      }
      __syncthreads();
      for (int e = tid * 4; e < min(nrows - r0 - row0, 16) * D; e += NW * kWave * 4) {
        const int in = e / D, r = r0 + row0 + in, d = e % D;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, s_m[w][row0 + in]);
        const float m = top == -INFINITY ? 0.0f : top;
        float4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
        float l = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float f = __builtin_amdgcn_exp2f(s_m[w][row0 + in] - m);
          l = __builtin_fmaf(s_l[w][row0 + in], f, l);
          const float4_t ow = *reinterpret_cast<const float4_t *>(&s_o[w][in][d]);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(ow[i], f, o[i]);
        }
        if (whole) {
          const int qr = r / p.group, hr = kvh * p.group + r - qr * p.group;
          const int64_t query = rq.begin + (int64_t)qr;
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
          *reinterpret_cast<uint2_t *>(a.out + (query * a.hq + hr) * D + d) =
              uint2_t{pack16<F16>(o[0] * inv, o[1] * inv), pack16<F16>(o[2] * inv, o[3] * inv)};
          if (d == 0 && a.lse) a.lse[(int64_t)hr * a.tq + query] = ((m + kRoom) + __builtin_amdgcn_logf(l * kUnroom)) * kLn2;
        } else {
          const int64_t place = ((int64_t)blockIdx.x * 2 + side) * kRowTile + row0 + in;
          *reinterpret_cast<float4_t *>(a.part + place * D + d) = o;
          if (d == 0) *reinterpret_cast<float2_t *>(a.stat + place * 2) = float2_t{top, l};
        }
      }
      __syncthreads();  // free for the next rows, or row tile
    }
  }
}

// The parts of one row: a workgroup takes one query and head, for few rows that may have many parts each.  (Many rows:
// join_rows.)
template <int D, bool F16>
__global__ __launch_bounds__(kJoinThreads) void k_kv4_few_join(KvView c, ChunkPlan p, ChunkArgs a) {
  constexpr int kSub = kJoinThreads / (D / 4);  // parts summed side by side, four channels a thread
  __shared__ float s_part[kSub][D];
  const int64_t at = blockIdx.x;
  const int query = (int)(at / a.hq), head = (int)(at - (int64_t)query * a.hq);
  int lo = 0, hi = c.nseq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (query_rows(a, mid).begin <= query) lo = mid;
    else hi = mid - 1;
  }
  const Rows rq = query_rows(a, lo);
  if (query < rq.begin || query >= rq.begin + rq.n || !few_rows(p, rq.n)) return;
  const int rtiles = (rq.n * p.group + kRowTile - 1) / kRowTile;
  const int row = (query - rq.begin) * p.group + head % p.group, rt = row / kRowTile, col = row % kRowTile;
  const Parts parts = FewCuts<D>::parts_of(c, a, lo, head / p.group * rtiles + rt, rtiles);
  if (parts.n == 1) return;  // whole
  const int n = parts.n;
  auto place = [&](int i) { return parts.place(i) * kRowTile + col; };
  const int lane = threadIdx.x & 63;
  float top = -INFINITY, sum = 0.0f;
  for (int i = lane; i < n; i += kWave) top = fmaxf(top, a.stat[place(i) * 2]);
#pragma unroll
  for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  const float m0 = top == -INFINITY ? 0.0f : top;
  for (int i = lane; i < n; i += kWave) {
    const float *st = a.stat + place(i) * 2;
    sum = __builtin_fmaf(st[1], __builtin_amdgcn_exp2f(st[0] - m0), sum);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
  const int d = threadIdx.x % (D / 4) * 4, sub = threadIdx.x / (D / 4);
  float4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int i = sub; i < n; i += kSub) {
    const float f = __builtin_amdgcn_exp2f(a.stat[place(i) * 2] - m0);
    const float4_t v = *reinterpret_cast<const float4_t *>(a.part + place(i) * D + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = __builtin_fmaf(v[j], f, o[j]);
  }
  *reinterpret_cast<float4_t *>(&s_part[sub][d]) = o;
  __syncthreads();
  const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
  for (int x = threadIdx.x * 2; x < D; x += kJoinThreads * 2) {
    float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
    for (int i = 0; i < kSub; ++i) y0 += s_part[i][x], y1 += s_part[i][x + 1];
    *reinterpret_cast<uint32_t *>(a.out + at * D + x) = pack16<F16>(y0 * r, y1 * r);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[(int64_t)head * a.tq + query] = ((m0 + kRoom) + __builtin_amdgcn_logf(sum * kUnroom)) * kLn2;
}

template <int D, bool F16>
hipError_t few_d(const KvView &c, const ChunkPlan &p, const ChunkArgs &a, hipStream_t s) {
  if (p.lone) {
    const int rtiles = (int)((int64_t)a.tq * p.group / kRowTile) + c.nseq;
    const unsigned grid = (unsigned)(rtiles * c.hkv);
    if (D < 256 && p.lone == 8) k_kv4_few<D, F16, (D < 256 ? 8 : 4), true><<<grid, 8 * kWave, 0, s>>>(c, p, a);
    else k_kv4_few<D, F16, 4, true><<<grid, 4 * kWave, 0, s>>>(c, p, a);
    return hipGetLastError();
  }
  k_kv4_few<D, F16, kFewWaves, false><<<256 * kFewPerCu<D>, kFewWaves * kWave, 0, s>>>(c, p, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.join_few) return e;
  k_kv4_few_join<D, F16><<<(unsigned)((int64_t)a.tq * a.hq), kJoinThreads, 0, s>>>(c, p, a);
  return hipGetLastError();
}

}  // namespace

size_t kv4_few_sums(const KvView &c) { return (size_t)shares_of(c.d) * 2 * kRowTile * c.d * 4; }

// The line and the launches have to fit their counters.
bool kv4_few_takes(const KvView &c, const ChunkPlan &p, int total_q) {
  const int64_t rtiles = ((int64_t)total_q * p.group / kRowTile + c.nseq) * c.hkv;
  const int64_t tiles = std::min<int64_t>(p.len_cap, (int64_t)p.window + p.sinks + total_q + 2 * kTile) / kTile + 2;
  return rtiles * tiles < ((int64_t)1 << 30) && rtiles <= kMaxBlocks / 2 && (int64_t)total_q * p.group * c.hkv <= kMaxBlocks;
}

hipError_t launch_kv4_few(const KvView &c, const ChunkPlan &p, const ChunkCall &x, void *ws, hipStream_t s) {
  const ChunkArgs a = few_args(p, x, ws);
  if (c.d == 64) return x.f16 ? few_d<64, true>(c, p, a, s) : few_d<64, false>(c, p, a, s);
  if (c.d == 128) return x.f16 ? few_d<128, true>(c, p, a, s) : few_d<128, false>(c, p, a, s);
  return x.f16 ? few_d<256, true>(c, p, a, s) : few_d<256, false>(c, p, a, s);
}

}  // namespace vqmm
