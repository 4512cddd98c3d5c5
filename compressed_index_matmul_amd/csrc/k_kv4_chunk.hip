// kv4_attend_chunk: packed queries of several tokens a sequence against the
// 4-bit cache, causal, under a sliding window with sinks or not.
//
// A row is one query of one head; the rows of a key/value head's group, Lq *
// group of a sequence, share its keys.  A workgroup of eight waves takes 256
// rows, 32 a wave, and walks the cache BN = 8192 / D slots at a time: four waves
// turn the tile's keys into fp16, four its values, for the products of all eight
// (16 words of codes a thread and side would be 208 instructions in every wave;
// shared by eight they are 26 a 32 slots).  Tiles are double-buffered in LDS, codes
// of the tile after the next in registers, so a round has one barrier.  Waves of
// the first half decode first and multiply then, those of the second the other way
// round: the two that share a SIMD keep its vector unit and its matrix cores busy
// at different times.
//
//   S^T = K Q^T   32x32x16 fp16 MFMA.  A key's channels lie in LDS in the order in which
//                 the codes unpack (0 4 1 5 2 6 3 7 of an octet), the query's
//                 registers in the same.  Queries are held in fp16 after a
//                 power-of-two rescale per row.
//   O^T = V^T P^T the keys a lane holds of S^T are its eight of the reduction, and
//                 values lie in LDS by channel with the slots in that order:
//                 neighbouring slots, as the cache interleaves them, unpack to
//                 pairs.  P stays in its registers.
//
// For bf16 results keys, values and probabilities are rounded to fp16 (relative 2^-11), an eighth of the result's own
// rounding.  For fp16 results scores are exact but for their fp32 sums and the probabilities' remainders take part (see
// split8): twice as many products, errors of 2.8e-4 of the result where its own rounding leaves 2.1e-4, and 4.9e-4 without.
//
// The work is cut into 256 equal shares of a line of tiles (Cut) whose parts a second launch joins, or row tiles are
// taken whole (few_slots, many_even_tiles).  Sequences of up to 64 rows go to k_kv4_few.
//
// Bound: matrix cores and vector issue (matrix cores busy 43 % of the cycles; vector units 51 %, the issue of matrix
// instructions among it, so the two do not add up; some wave issuing in 92 %; clock 1.95 GHz), which is as far as two waves
// a SIMD overlapped them: opposite orders, priorities and products between the exponentials of one wave gained nothing
// more.  In calls of few tiles the latency of a share and of the second launch.  Heads of 256 hold all 256 registers and
// spill 17 more, for fp16 results 42, of which a tile's loop reads 4 and 34 back.  Measured, median: 1000 tokens after
// 30,011, 64/8 heads of 128, fp16: 1866 to 1980 us from card to card, 0.53 PFLOP/s of visible pairs (bf16, which rounds
// keys: 1012); 512 tokens after 16,001 of 32/8 heads of 128, bf16: 163 to 169 us, 0.83 PFLOP/s; of 16/4 heads of 256 186 to
// 205 (fp16 311 to 343).
#include <algorithm>
#include <climits>

#include "kv4_chunk.h"

namespace vqmm {

namespace {

constexpr int kWaves = 8, kThreads = kWaves * kWave;
constexpr int kRows = kWaves * 32;
// The 16-byte piece of a value row is permuted by an XOR with bits of its channel: reads of a piece of 16 neighbouring
// channels, and writes of one slot of every eighth, fall on different banks.  Rows are BN slots: 256, 128 or 64 bytes.
template <int D>
__device__ __forceinline__ int channel_swizzle(int c) {
  return D == 256 ? ((c >> 2) ^ (c >> 4)) & 3 : D == 128 ? (c ^ (c >> 3)) & 7 : (c ^ (c >> 3)) & 15;
}

// Sequences of up to so many rows go to the kernel whose waves decode for themselves.  With 4, 16, 32 and 64 rows a
// sequence it is the faster one for each head size and from 1 to 64 sequences; with 128 and more this one is.
constexpr int kFewRows = 64;
// Few-row calls of up to so many query heads join their parts with a workgroup each, which sums parts side by side: one
// sequence of eight queries on 16,000 slots takes 14.9 / 23.2 / 26.9 us (9/3 heads of 64, 32/8 of 128, 16/4 of 256), joined a
// row tile a workgroup 55 / 49 / 95.  Of more, 64 sequences of four on 7000 slots 36 / 117 / 112 against 34 / 108 / 107.
constexpr int kJoinSingly = 2048;

constexpr int kJoinThreads = 256, kJoinRows = 16;

// What a row tile's start and end cost, in tiles.  Four sequences of 300 queries on 500 to 4000 slots: 35.4 / 86.4 / 98.5 us
// (9/3 heads of 64, 32/8 of 128, 16/4 of 256), with none 39.0 / 88.5 / 105.7, with six 36.8 / 87.6 / 97.9.
constexpr int kRowTileCost = 2;
// Workgroups that 256 CUs hold at once; a share is 256 slots or more.
constexpr int kShares = 256;
template <int D>
using Cuts = Cut<8192 / D, kRows, false, kShares, 1, D / 32, kRowTileCost>;

// What a thread holds of the next tile: 32 codes and the steps and minima they
// need.  Keys: one word of each of four slots.  Values: 8 channels of four slots.
struct Codes {
  uint32_t w[4];
  uint4_t sm;
};

template <int D, bool F16>
__global__ __launch_bounds__(kThreads, 2) void k_kv4_chunk(KvView c, ChunkPlan p, ChunkArgs a, int tiles) {
  constexpr int BN = 8192 / D, NS = BN / 32, ND = D / 32, NK = D / 16, DG = D / 32;
  constexpr int kWords = D / 8, kQuads = kWave / kWords;  // words a slot; quads of slots a wave decodes
  constexpr int kTileBytes = BN * D * 2;
  constexpr int kParts = F16 ? 2 : 1;  // of a key: upper and lower bits of its steps (see split8)
  __shared__ __attribute__((aligned(1024))) uint8_t s_k[2][kParts * kTileBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t s_v[2][kTileBytes];
  // Heads of 256: part of the queries, which with 128 registers of sums do not fit; each wave's own.
  constexpr int kHeld = D < 256 ? NK : F16 ? NK - 6 : NK - 8, kLdsQ = NK - kHeld;
  __shared__ uint4_t s_q[kLdsQ ? kWaves : 1][kLdsQ ? kLdsQ : 1][kWave];
  __shared__ __attribute__((aligned(16))) _Float16 s_mid[2][F16 ? BN : 1][2 * DG];  // a slot's minima, and steps times 8
  __shared__ int s_cleared;

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  typename Cuts<D>::Line line{};
  int pos = 0, pos_end = 1;
  // workgroups are dealt to the 8 XCDs in turn: neighbouring shares, which read the same slots, go to one of them
  const int id = p.whole ? blockIdx.x : (blockIdx.x & 7) * (kShares / 8) + (blockIdx.x >> 3);
  if (!p.whole) line = Cuts<D>::line_of(c, p, a, id, &pos, &pos_end);
  const int pos0 = pos;
  while (pos < pos_end) {
    int b, kvh, rt, t_lo, nt, side = 0;
    Extent e;
    if (p.whole) {
      // heads of a group share slots, and with 8 of them an XCD's L2 serves one; late row tiles, the long ones, first
      kvh = id % c.hkv;
      e = Cuts<D>::row_tile(c, p, a, tiles - 1 - id / c.hkv, &b, &rt);
      if (rt < 0 || rt >= e.rtiles) return;
      t_lo = 0;
      nt = e.tiles;
      pos = pos_end;
    } else {
      const Segment seg = Cuts<D>::segment(c, p, a, line, pos, pos_end);
      b = seg.b, kvh = seg.kvh, rt = seg.rt, t_lo = seg.begin, nt = seg.end, e = seg.e;
      side = pos == pos0 && t_lo > 0 ? 0 : 1;  // 0: the row tile began in an earlier share
      pos += seg.steps;
      if (t_lo >= nt) continue;  // only the end's allowance
    }
    const Rows rq = e.rq;
    const int nrows = rq.n * p.group, r0 = rt * kRows;
    const int len = e.len, off = len - rq.n;  // query i sees slots <= i + off

    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // anew for each run: what follows from it would else be kept in registers throughout
    const int lane = tid & 63, col = lane & 31, h = lane >> 5;
    const int rw = r0 + wave * 32;
    const int row = max(min(rw + col, nrows - 1), 0), qi = row / p.group, head = kvh * p.group + row - qi * p.group;
    // the newest slot that a query sees (-1: none): this lane's, the wave's first and last, the workgroup's first and last
    auto newest_of = [&](int r) { return max(min(r, nrows - 1) / p.group + off, -1); };
    const int lim = max(qi + off, -1), lim_first = newest_of(rw), lim_last = newest_of(rw + 31);
    const int all_see = newest_of(r0), newest = newest_of(r0 + kRows - 1);
    const int seen = newest + 1;
    // some query of the workgroup does not see some slot of the tile
    auto partly = [&](int k0) { return k0 + BN - 1 > all_see || (k0 <= newest - p.window && k0 + BN > p.sinks); };
    auto sees = [&](int slot) { return slot <= lim && (slot > lim - p.window || slot < p.sinks); };
    // All row tiles of a sequence count the same tiles.  This one leaves out those before its first query's window and
    // those past its newest slot.
    const Walk<BN> walk(p, len, max(off, -1));
    const int low = max(max(all_see - p.window + 1, 0) / BN - walk.jump, 0), past = (newest + BN) / BN;
    auto from = [&](int t) { return t >= walk.sink && t < low ? low : t; };
    const int t_end = min(nt, past <= walk.sink ? past : max(past - walk.jump, walk.sink));

    // decoding: quad `quad` of the tile, word `word` of its key rows (octet 4 j + a) or channels 8 word .. + 7 of its values
    const bool keys = wave < 4;
    const int unit = tid & 255, quad = unit / kWords, word = unit % kWords, in_wave = quad % kQuads;
    const int wave_slot = __builtin_amdgcn_readfirstlane((quad - in_wave) * 4);  // the wave's first slot in the tile
    const int group = keys ? word % DG : word / 4;
    const int64_t code_head = (int64_t)c.ps * (D / 2), scale_head = (int64_t)c.ps * (DG * 4);  // bytes of one head of a page
    const uint32_t code_lane = keys ? in_wave * (2 * D) + word * 4 : in_wave * (2 * D) + word * 16;
    const uint32_t scale_lane = (in_wave * DG + group) * 16;
    const int last_block = max(len - 1, 0) >> 5;
    const Unpack unpack;
    Codes codes;
    // The page of a tile is looked up while the one before it is fetched.  Slots past the sequence's last one: those of its
    // block again, in bounds and masked.
    int block, entry;
    auto look_up = [&](int t) {
      block = min((walk.tile(t) * BN + wave_slot) >> 5, last_block);
      entry = table_entry(c, b, page_index(p, block));
    };
    auto fetch = [&](int next) {
      const int at = (block - page_index(p, block) * p.page_blocks) * 32 + (wave_slot & 31);
      const int64_t hd = ((int64_t)page_in_pool(c, entry) * 2 + (keys ? 0 : 1)) * c.hkv + kvh;
      look_up(next);
      const uint8_t *cb = c.codes + hd * code_head + (int64_t)at * (D / 2) + code_lane;
      const uint8_t *sb = reinterpret_cast<const uint8_t *>(c.scales) + hd * scale_head + (int64_t)at * (DG * 4) + scale_lane;
      if (keys) {
#pragma unroll
        for (int i = 0; i < 4; ++i) codes.w[i] = *reinterpret_cast<const uint32_t *>(cb + i * (D / 2));
      } else {
        const uint4_t v = *reinterpret_cast<const uint4_t *>(cb);
#pragma unroll
        for (int i = 0; i < 4; ++i) codes.w[i] = v[i];
      }
      codes.sm = *reinterpret_cast<const uint4_t *>(sb);
    };
    int t = from(t_lo), buf = 0;
    if (t < t_end) {
      look_up(t);
      fetch(from(t + 1));
    }

    // the query in the order of the unpacked codes, its largest value in [2^14, 2^15)
    uint4_t q_held[kHeld];
    float cs;  // scores -> log2 domain
    uint4_t qmid;
    {
      const uint16_t *qp = a.q + min(rq.begin + (int64_t)qi, (int64_t)a.tq - 1) * a.q_ts + head * a.q_hs + 8 * h;
      uint4_t qf[NK];
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        qf[i] = *reinterpret_cast<const uint4_t *>(qp + 16 * i);
        top = fmaxf(top, largest16<F16>(qf[i]));
      }
      const int lift = lift_of<F16>(max_xor32(top));
      cs = a.scale * kLog2e * __uint_as_float((uint32_t)(127 - lift) << 23);
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        qf[i] = lift16<F16>(qf[i], lift);
        if (i < kHeld) q_held[i < kHeld ? i : 0] = qf[i];
        else s_q[wave % (kLdsQ ? kWaves : 1)][i < kHeld ? 0 : i - kHeld][lane] = qf[i];
      }
      if (F16) {
        float sums[DG];
#pragma unroll
        for (int g = 0; g < DG; ++g) sums[g] = sum_xor32(sum8(qf[2 * g]) + sum8(qf[2 * g + 1]));
        qmid = sums_operand<DG>(sums, h);
      }
    }
    const uint32_t sq = lds_address(s_q[wave % (kLdsQ ? kWaves : 1)][0]) + lane * 16;
    auto query = [&](int i) { return i < kHeld ? q_held[i < kHeld ? i : 0] : lds_read(sq + (i - kHeld) * (kWave * 16)); };

    float16_t acc[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][r] = 0.0f;
    float mref = -INFINITY, m0 = 0.0f, lsum = 0.0f;  // the reference in units of scores and in the log2 domain
    const float room = kRoom / cs, slack = (kSlack + kRoom) / cs;
    bool large = false;
    auto decode = [&](int t, int buf) {
      const Unpack &u = unpack;
      if (keys) {
        const int oct = 4 * group + word / DG;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const _Float16 sv = as_h2(codes.sm[i / 2])[i & 1], mv = as_h2(codes.sm[2 + i / 2])[i & 1];
          const half2_t s = {sv, sv}, m = {mv, mv};
          const int r = 4 * quad + i;
          if (F16) {
            uint4_t upper, lower;
            split8(u, codes.w[i], s, &upper, &lower);
            uint8_t *kp = s_k[buf] + r * (2 * D) + (oct ^ key_swizzle<D>(r)) * 16;
            *reinterpret_cast<uint4_t *>(kp) = upper;
            *reinterpret_cast<uint4_t *>(kp + kTileBytes) = lower;
            if (word < DG) s_mid[buf][r][group] = mv, s_mid[buf][r][DG + group] = sv * (_Float16)8.0f;
            continue;
          }
          *reinterpret_cast<uint4_t *>(s_k[buf] + r * (2 * D) + (oct ^ key_swizzle<D>(r)) * 16) = values8(u, codes.w[i], s, m);
        }
      } else {
        const int k0 = walk.tile(t) * BN;
        if (partly(k0)) {
          // 0 times NaN would be NaN for queries that do not see the slot: what is not finite, and what no query sees,
          // counts as zero here; the former comes back at the end for the queries that do see it
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t shift = 16 * (i & 1), keep = ~(0xffffu << shift);
            const uint32_t s = codes.sm[i / 2] >> shift, m = codes.sm[2 + i / 2] >> shift;
            const bool out = k0 + 4 * quad + i >= seen, bad = (s & 0x7c00u) == 0x7c00u || (m & 0x7c00u) == 0x7c00u;
            if (out || bad) codes.sm[i / 2] &= keep, codes.sm[2 + i / 2] &= keep;
            if (!out && bad) s_cleared = 1;
          }
        }
        const half2_t s01 = as_h2(codes.sm[0]), s23 = as_h2(codes.sm[1]), m01 = as_h2(codes.sm[2]), m23 = as_h2(codes.sm[3]);
        const int st = quad >> 2, q4 = quad & 3, piece16 = 2 * st + (q4 & 1), half = q4 >> 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = codes.w[i];
          const uint2_t even = {__builtin_bit_cast(uint32_t, value(code_lo(u, w), s01, m01)),
                                __builtin_bit_cast(uint32_t, value(code_lo(u, w >> 8), s23, m23))};
          const uint2_t odd = {__builtin_bit_cast(uint32_t, value(code_hi(u, w), s01, m01)),
                               __builtin_bit_cast(uint32_t, value(code_hi(u, w >> 8), s23, m23))};
          const int ch = 8 * word + 2 * i;
          uint8_t *vp = s_v[buf] + half * 8;
          *reinterpret_cast<uint2_t *>(vp + ch * (2 * BN) + (piece16 ^ channel_swizzle<D>(ch)) * 16) = even;
          *reinterpret_cast<uint2_t *>(vp + (ch + 1) * (2 * BN) + (piece16 ^ channel_swizzle<D>(ch + 1)) * 16) = odd;
        }
      }
    };

    const uint32_t ka = lds_address(s_k) + col * (2 * D) + (h ^ key_swizzle<D>(col)) * 16;
    const uint32_t va = lds_address(s_v) + col * (2 * BN) + (h ^ channel_swizzle<D>(col)) * 16;

    auto multiply = [&](int t, int buf) {
      const int k0 = walk.tile(t) * BN;
      if (rw >= nrows || k0 > lim_last || !(k0 + BN > lim_first - p.window + 1 || k0 < p.sinks)) return;
      const uint32_t ks = ka + buf * (kParts * kTileBytes), vs = va + buf * kTileBytes;
      float16_t S[NS];
      constexpr int kAhead = D == 256 ? (F16 ? 2 : 4) : NK < 8 ? NK : 8, kAll = NS * kParts * NK;
      uint4_t kf[kAhead];
      auto read_k = [&](int x) {
        const int n = x / (kParts * NK), part = x / NK % kParts, i = x % NK;
        return lds_read((ks ^ (i & 7) * 32) + part * kTileBytes + n * 64 * D + (i >> 3) * 256);
      };
#pragma unroll
      for (int x = 0; x < kAhead; ++x) kf[x] = read_k(x);
      sched_fence();
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[n][r] = 0.0f;
      if (F16) {
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const uint32_t at = lds_address(s_mid[buf][32 * n + col]);
          if (DG == 2) {
            const uint2_t x = *(lds_uint2 *)(uintptr_t)at;
            S[n] = mfma32<true>(uint4_t{x[0], x[1], 0, 0}, qmid, S[n]);
          } else {
            S[n] = mfma32<true>(lds_read(at), qmid, S[n]);
            if (DG == 8) S[n] = mfma32<true>(lds_read(at + 16), qmid, S[n]);
          }
        }
        sched_fence();
      }
#pragma unroll
      for (int x = 0; x < kAll; ++x) {
        S[x / (kParts * NK)] = mfma32<true>(kf[x % kAhead], query(x % NK), S[x / (kParts * NK)]);
        if (x + kAhead < kAll) kf[x % kAhead] = read_k(x + kAhead);
      }
#pragma unroll
      for (int x = 0; x < kAll; ++x) {
        sched_group<0x008, 1>();
        if (x + kAhead < kAll) sched_group<0x100, 1>();
        if (x + 1 < kAll && (x + 1) % NK >= kHeld) sched_group<0x100, 1>();
      }
      sched_fence();
      if (k0 + BN - 1 > lim_first || (k0 <= lim_last - p.window && k0 + BN > p.sinks)) {
        // relative to the lane's first slot, so that the others are constants
        const int base = k0 + 4 * h, past = lim - base, low = past - p.window, sunk = p.sinks - base;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int x = 32 * n + 8 * (r / 4) + (r & 3);
            S[n][r] = (x <= past) & ((x > low) | (x < sunk)) ? S[n][r] : -INFINITY;
          }
      }
      float top = S[0][0];
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, S[n][r]);
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
      constexpr int kVAhead = D == 256 && F16 ? 2 : ND < 4 ? ND : 4, kVAll = 2 * NS * ND;
      uint4_t vf[kVAhead];
      auto read_v = [&](int x) {
        const int st = x / ND, d = x % ND;
        constexpr int kTurn = D == 256 ? 2 : 4;  // channel_swizzle of 32 d, in the bits it has
        const int turn = (kTurn * d) & (BN / 8 - 1);
        return lds_read((vs ^ ((2 * st) ^ turn) * 16) + d * 64 * BN);
      };
#pragma unroll
      for (int part = 0; part < kParts; ++part) {  // probabilities, then what their rounding left
#pragma unroll
        for (int x = 0; x < kVAhead; ++x) vf[x] = read_v(x);
        uint4_t pf[2 * NS];
#pragma unroll
        for (int st = 0; st < 2 * NS; ++st)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * (st & 1) + 2 * i;
            pf[st][i] = pack16<true>(S[st / 2][r], S[st / 2][r + 1]);
            if (part + 1 < kParts) S[st / 2][r] -= (float)as_h2(pf[st][i])[0], S[st / 2][r + 1] -= (float)as_h2(pf[st][i])[1];
          }
        sched_fence();
#pragma unroll
        for (int x = 0; x < kVAll; ++x) {
          acc[x % ND] = mfma32<true>(vf[x % kVAhead], pf[x / ND], acc[x % ND]);
          if (x + kVAhead < kVAll) vf[x % kVAhead] = read_v(x + kVAhead);
        }
#pragma unroll
        for (int x = 0; x < kVAll; ++x) {
          sched_group<0x008, 1>();
          if (x + kVAhead < kVAll) sched_group<0x100, 1>();
        }
        sched_fence();
      }
    };

    __syncthreads();  // the run before is done with LDS
    if (tid == 0) s_cleared = 0;
    __syncthreads();
    if (t < t_end) {
      decode(t, 0);
      fetch(from(from(t + 1) + 1));
    }
    __syncthreads();
    while (t < t_end) {
      const int next = from(t + 1);
      if (!keys) multiply(t, buf);
      if (next < t_end) {
        decode(next, buf ^ 1);
        fetch(from(from(next + 1) + 1));  // of the tile after it, or of the last block
      }
      if (keys) multiply(t, buf);
      __syncthreads();
      t = next, buf ^= 1;
    }

    if (s_cleared) {
#pragma unroll 1
      for (int i = t_lo * BN; i < t_end * BN; ++i) {
        const int slot = walk.tile(i / BN) * BN + i % BN;
        if (slot >= seen || !partly(slot / BN * BN)) continue;
        const int pi = page_index(p, slot >> 5), at = slot - pi * c.ps;
        const int64_t hd = (page_of(c, b, pi) * 2 + 1) * c.hkv + kvh;
        const uint16_t *sb = c.scales + hd * (scale_head / 2) + (int64_t)(at / 4) * (DG * 8) + (at & 3);
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          const uint32_t s = sb[8 * d], m = sb[8 * d + 4];
          const bool bad = (s & 0x7c00u) == 0x7c00u || (m & 0x7c00u) == 0x7c00u;
          if (bad && sees(slot)) acc[d] += __builtin_nanf("");
        }
      }
    }

    const bool cut = t_lo > 0 || nt < e.tiles;
    lsum = sum_xor32(lsum);
    if (rw + col < nrows) {
      const int64_t query = rq.begin + (int64_t)qi;
      if (cut) {
        const int64_t at = ((int64_t)id * 2 + side) * kRows + wave * 32 + col;
        float *pp = a.part + at * D + 4 * h;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<float4_t *>(pp + 32 * d + 8 * x) =
                float4_t{acc[d][4 * x], acc[d][4 * x + 1], acc[d][4 * x + 2], acc[d][4 * x + 3]};
        if (h == 0) *reinterpret_cast<float2_t *>(a.stat + at * 2) = float2_t{mref * cs, lsum};
      } else {
        const float r = lsum == 0.0f ? 0.0f : 1.0f / lsum;
        uint16_t *op = a.out + (query * a.hq + head) * D + 4 * h;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint2_t w = {pack16<F16>(acc[d][4 * x] * r, acc[d][4 * x + 1] * r),
                               pack16<F16>(acc[d][4 * x + 2] * r, acc[d][4 * x + 3] * r)};
            *reinterpret_cast<uint2_t *>(op + 32 * d + 8 * x) = w;
          }
        if (a.lse && h == 0) {
          const float ref = mref == -INFINITY ? 0.0f : mref * cs;
          a.lse[(int64_t)head * a.tq + query] = ((ref + kRoom) + __builtin_amdgcn_logf(lsum * kUnroom)) * kLn2;
        }
      }
    }
  }
}

// The second launch, of both kernels' cut row tiles: the first `blocks` workgroups take kJoinRows rows each of
// k_kv4_chunk's (16: 46 us for two chunks beside 30 single tokens of 9/3 heads of 64, fp16, 86 with all 256), the others a row tile each of k_kv4_few's.
template <int D, bool F16>
__global__ __launch_bounds__(kJoinThreads) void k_kv4_chunk_join(KvView c, ChunkPlan p, ChunkArgs a, ChunkArgs few, int blocks) {
  int id = blockIdx.x;
  if (id < blocks) {
    const int from = id % (kRows / kJoinRows) * kJoinRows;
    id /= kRows / kJoinRows;
    join_rows<D, F16, kRows, Cuts<D>>(c, p, a, id / c.hkv, id % c.hkv, from, from + kJoinRows);
  } else {
    id -= blocks;
    join_rows<D, F16, kFewRowTile, FewCuts<D>>(c, p, few, id / c.hkv, id % c.hkv, 0, kFewRowTile);
  }
}

template <int D, bool F16>
hipError_t chunk_d(const KvView &c, const ChunkPlan &p, const ChunkCall &x, void *ws, hipStream_t s) {
  const ChunkArgs a = chunk_args(p, x, ws);
  const int64_t rows = (int64_t)x.tq * p.group;
  const int tiles = (int)(rows / kRows) + c.nseq;
  if (p.any_chunk) {
    k_kv4_chunk<D, F16><<<p.whole ? (unsigned)((int64_t)tiles * c.hkv) : kShares, kThreads, 0, s>>>(c, p, a, tiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t blocks = p.any_chunk && !p.whole ? (int64_t)tiles * c.hkv * (kRows / kJoinRows) : 0;
  const int64_t few = p.join_few ? (rows / kFewRowTile + c.nseq) * c.hkv : 0;
  if (blocks + few == 0) return hipSuccess;
  k_kv4_chunk_join<D, F16><<<(unsigned)(blocks + few), kJoinThreads, 0, s>>>(c, p, a, few_args(p, x, ws), (int)blocks);
  return hipGetLastError();
}

}  // namespace

// Whether a workgroup of k_kv4_few takes each of up to `tiles` row tiles whole, and of how many waves: where slots are few
// enough that shares and their second launch cost more.  In graphs, four queries a sequence of 512 / 1024 slots, shares
// against whole row tiles (us):
//   sequences             1                          8                          64                     256
//   9/3 heads of 64       10.3 / 8.5, 10.4 / 10.2    11.1 / 8.8, 11.6 / 10.7    17 / 13, 20 / 17       34 / 27, 40 / 34
//   32/8 heads of 128     12.1 / 11.2, 12.6 / 14.3   17.0 / 11.9, 18.4 / 15.3   34 / 20, 41 / 26       81 / 71, 121 / 108
//   16/4 heads of 256     16.0 / 17.7, 16.6 / 23.9   17.8 / 18.5, 24.3 / 24.8   39 / 28, 49 / 39       86 / 71, 124 / 111
// (heads of 128 with 64 sequences and more, and heads of 256: four waves, of which a CU holds two workgroups where it holds
// one of eight: 36 and 109 us at 512 slots).  At 2048 slots shares win but for heads of 64 (one sequence 10.7 / 14.5, eight
// 12.8 / 15.2, 64 24.5 / 25.4).
static int lone_waves(int d, int64_t slots, int64_t tiles) {
  if (d == 64) return slots <= 1280 ? 8 : 0;
  if (d == 128) return slots <= (tiles <= 16 ? 768 : 1280) ? (tiles <= 256 ? 8 : 4) : 0;
  return slots <= (tiles >= 128 ? 1280 : 512) ? 4 : 0;
}

// Row tiles of a call, at most.
int64_t kv4_chunk_blocks(const KvView &c, int n_q_heads, int total_q) {
  return ((int64_t)total_q * (n_q_heads / c.hkv) / kRows + c.nseq) * c.hkv;
}

// Slots that a row tile meets, at most.
static int64_t visible_slots(const ChunkPlan &p, int max_len) {
  return std::min<int64_t>(max_len, (int64_t)p.window + p.sinks + kRows);
}

// Whether k_kv4_chunk takes row tiles whole.
// So where slots are few (eight chunks of 300 tokens on 800 slots, shares / whole: 9/3 heads of 64 39 / 31 us, 32/8 of 128
// 87 / 79, 16/4 of 256 98 / 74; but 1000 tokens on 2000 slots 32 / 51, 62 / 73 and 82 / 141, and one chunk of 1024 on its
// own 25 / 30, 45 / 43 and 67 / 80).
static bool few_slots(int64_t slots, int64_t tiles) { return slots <= 512 || (slots <= 1024 && tiles >= 80); }
// And where row tiles are many, so that shares gain nothing and walk past the newest slots of a chunk's first rows (4096
// tokens on their own, 32/8 heads of 128: 260 / 176; two of 3000 on 5000 slots 492 / 409; six of 1000 on 1900 to 6000 414 /
// 376), unless a single one may walk much longer than all take together: the lengths are not on the host, and one long
// sequence beside short ones would go on alone (four of 1200 on their own and 30 tokens after 60,000: 206 / 1328; 16 of 512
// and one of 512 on 8000: 211 / 242, heads of 256 222 / 503).  What all take at least is counted by the queries' own tokens,
// one sequence of max_q and the others of equal length.  At five times that whole row tiles still win or tie (2000 tokens on
// 10,000 slots beside three of 2000 on their own, heads of 128, 2.6 times: 558 / 441; heads of 256, 5.1 times: 576 / 621),
// at seven times they lose in the unequal batches above (and a prompt of 4096 on its own whose bound says 32,000: 256 / 160).
static bool many_even_tiles(const KvView &c, const ChunkPlan &p, int64_t slots, int64_t tiles, int total_q, int max_q) {
  if (tiles < 384) return false;
  auto pairs = [&](double queries) { return queries * std::min<double>(queries, p.window) / 2; };
  const int longest = std::min(max_q, total_q), others = std::max(c.nseq - 1, 1);
  const double own = pairs(longest) + others * pairs((double)(total_q - longest) / others);
  return slots <= 5 * own * p.group * c.hkv / (kRows * (double)kShares);
}
// The second launch's limit leaves no choice.
static bool joins_past_grid(const KvView &c, const ChunkPlan &p, int total_q) {
  return kv4_chunk_blocks(c, p.group * c.hkv, total_q) * (kRows / kJoinRows) > kMaxBlocks / 2;
}
static int64_t row_tiles(const KvView &c, const ChunkPlan &p, int total_q) { return (int64_t)total_q * p.group / kRows * c.hkv; }

// The workspace's areas: sums of the parts with their references and sums of p, for either kernel, and where each sequence
// begins.
constexpr size_t kPlaces = (size_t)kShares * 2 * kRows;
static size_t chunk_area(const KvView &c) { return kPlaces * (c.d * 4 + 8); }
static size_t few_area(const KvView &c) { return kv4_few_sums(c) + kv4_few_sums(c) / c.d * 2; }
static size_t begins_area(const KvView &c) { return (((size_t)c.nseq + 1) * 4 + 255) & ~(size_t)255; }

ChunkPlan kv4_chunk_plan(const KvView &c, int n_q_heads, int total_q, int window, int sinks, int max_len, int max_q) {
  ChunkPlan p{};
  p.group = n_q_heads / c.hkv;
  p.len_cap = max_len;
  p.window = window == 0 || window > max_len ? std::max(max_len, 1) : window;
  p.sinks = std::min(sinks, max_len);
  p.page_blocks = c.ps / 32;
  p.page_mul = (uint32_t)((((uint64_t)1 << 32) + p.page_blocks - 1) / p.page_blocks);
  const int64_t visible = visible_slots(p, max_len), tiles = row_tiles(c, p, total_q);
  const bool all_few = (int64_t)max_q * p.group <= kFewRows;
  p.any_few = (all_few || c.nseq > 1) && kv4_few_takes(c, p, total_q);
  p.any_chunk = !(p.any_few && all_few);
  p.few = !p.any_few ? 0 : all_few ? INT_MAX : kFewRows;
  p.lone = lone_waves(c.d, visible, ((int64_t)total_q * p.group / kFewRowTile + c.nseq) * c.hkv);
  p.whole = few_slots(visible, tiles) || many_even_tiles(c, p, visible, tiles, total_q, max_q) || joins_past_grid(c, p, total_q);
  if (p.any_chunk && !p.whole) {
    p.stat_off = kPlaces * c.d * 4;
    p.begin_off = chunk_area(c);
    p.bytes = p.begin_off + begins_area(c);
  }
  if (p.any_few && !p.lone) {
    p.join_few = p.any_chunk || (int64_t)total_q * n_q_heads > kJoinSingly;
    p.few_off = p.bytes;
    p.few_stat_off = p.few_off + kv4_few_sums(c);
    p.few_begin_off = p.few_off + few_area(c);
    p.bytes = p.few_begin_off + begins_area(c);
  }
  return p;
}

// Enough for a call of these sizes and for every smaller one.  Which areas a plan has goes up and down with its sizes (row
// tiles are taken whole where they are many, and where slots are few), what an area takes does not: so these are the areas
// of any call with up to as many sequences, queries, slots and queries a sequence.  k_kv4_chunk has its area if it has with
// the fewest queries that go to it, k_kv4_few if it has with one sequence.  (Only sequences beyond the second launch's
// limit are counted as they are: theirs are whole.)
size_t kv4_chunk_bytes(const KvView &c, int n_q_heads, int total_q, int window, int sinks, int max_len, int max_q) {
  if (total_q == 0) return 0;
  const ChunkPlan p = kv4_chunk_plan(c, n_q_heads, total_q, window, sinks, max_len, max_q);
  const int fewest = std::min(total_q, kFewRows / p.group + 1);
  const int64_t visible = visible_slots(p, max_len);
  size_t n = 0;
  if (p.any_chunk && !few_slots(visible, row_tiles(c, p, fewest)) && !joins_past_grid(c, p, fewest)) n += chunk_area(c) + begins_area(c);
  if (!lone_waves(c.d, visible, c.hkv)) n += few_area(c) + begins_area(c);
  return n;
}

hipError_t launch_kv4_chunk(const KvView &c, const ChunkPlan &p, const ChunkCall &x, void *ws, hipStream_t s) {
  if (p.any_few) {
    const hipError_t e = launch_kv4_few(c, p, x, ws, s);
    if (e != hipSuccess) return e;
  }
  if (c.d == 64) return x.f16 ? chunk_d<64, true>(c, p, x, ws, s) : chunk_d<64, false>(c, p, x, ws, s);
  if (c.d == 128) return x.f16 ? chunk_d<128, true>(c, p, x, ws, s) : chunk_d<128, false>(c, p, x, ws, s);
  return x.f16 ? chunk_d<256, true>(c, p, x, ws, s) : chunk_d<256, false>(c, p, x, ws, s);
}

}  // namespace vqmm
