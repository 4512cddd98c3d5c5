// kv4_attend: one query a sequence against the 4-bit cache.
//
// For every sequence and key/value head the cache is read once, for up to 16
// query heads of the group at a time (they are the columns of the matrix
// products).  A wave walks tiles of 32 slots on its own, with the next tile's
// loads in flight, keeps a running maximum and sum, and meets the other waves
// of its workgroup in LDS.
//
// The tiles of all sequences and heads form one line, which a fixed number of
// workgroups (what the CUs hold at once) cuts into equal shares: lengths as
// unequal as may be end together, and one long sequence spreads over the whole
// chip.  A share covers the end of one row (sequence and head), whole rows, and
// the beginning of another; the parts of cut rows meet in a second launch, in
// the order of the line.  Every workgroup finds its place by a prefix sum over
// the lengths, 64 a step, so the host needs no lengths.
//
// Scores: S^T = K Q^T on 16x16x32 fp16 MFMA, a group of 32 channels a
// product.  Codes are integers, exact in fp16, so a product is exact up to its
// fp32 sum; step and minimum come in afterwards, in fp32:
//   q . k = sum_g s_g (q_g . c_g) + m_g sum(q_g).
// Output: O^T = V^T P^T.  A lane of the score product holds four slots of one
// head in each of two 16-slot halves, which is the operand the second product
// wants when its eight slots of the reduction are those same ones; the values
// are stored so that a word unpacks to pairs of neighbouring slots, so
// neither operand crosses lanes.
//
// Bound: HBM, 2 (head_dim / 2 + head_dim / 8) bytes a slot and head; next to it
// vector issue (330 instructions a tile of 32 slots and 128 channels: steps and
// minima of the keys, unpacking, steps and minima of the values).  Measured:
// four sequences of 300,000 slots in all, 64/8 heads of 128, fp16: 93 us, 4.1 TB/s,
// and 6 us for the join; with weights 106 us, 4.4 TB/s with the scores it
// writes, and 23 us for the join that reads them.  32 x 4096 slots of 32/8 heads:
// 34 us, 4.9 TB/s, and 5; 256 sequences of 200 to 1900 slots: 94 us, 3.6 TB/s, and
// 14.  One launch: one sequence of 1001 slots 10.5 us, 256 of up to 1000 68 us.
#include "attn_device.h"

#include <algorithm>

namespace vqmm {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kLoneWaves = 8;  // of a workgroup that takes a whole sequence and head
constexpr int kTile = 32;  // slots a wave takes at a time
// Where no weights are added, a workgroup takes a row whole up to this many slots.  Measured in graphs, one workgroup a
// row against shares and their join (us; 32/8 heads of 128, all lengths equal, then spread evenly up to the bound):
//   rows       8               256                          2048
//   512    6.9 /  8.5    7.5 / 15.5,  7.2 / 20.8     52 / 49,  45 / 80
//   1024  10.2 /  8.7   12.8 / 19.6, 10.7 / 31.4    101 / 86,  62 / 98
//   2048  16.5 /  9.0   20.8 / 26.1, 19.3 / 37.4    175 / 152, 114 / 114
// so it wins wherever rows are many and unequal, and loses where few rows are long: at 1024 slots 1.5 us, less than the
// 4 us that the second launch and its workspace cost a caller outside a graph.  Heads of 64 cross there too (8 rows: 7.4 /
// 7.9, 2048 slots 11.7 / 8.0); heads of 256 earlier (512 slots 10.5 / 10.0, 768 13.4 / 10.5, 1024 16.3 / 10.5).
constexpr int lone_slots(int d) { return d == 256 ? 768 : 1024; }
// Workgroups of four waves that 256 CUs hold at once, by their registers.
// Heads of 128: four workgroups a CU (128 registers, 8 bytes spilled) took 41 us where three took 45 for 32 x 4096
// slots of 32/8 heads; with weights, whose scores are written as well, four took 143 us and three 138 for the 300,000
// slots of 64/8 heads.
template <int D, bool WEIGH>
constexpr int kSharesPerCu = D == 64 ? 4 : D == 128 ? (WEIGH ? 3 : 4) : 2;
template <int D, bool WEIGH>
constexpr int kShares = 256 * kSharesPerCu<D, WEIGH>;
// The most of them, for the workspace.
int shares_of(int d) { return d == 64 ? kShares<64, false> : d == 128 ? kShares<128, false> : kShares<256, false>; }
constexpr float kSlack = 8.0f;  // the reference maximum may lag by up to 2^8
// Probabilities enter fp16 times 2^7, by a reference that much below the maximum it was taken from: up to 2^15 with the
// lag, and with 11 bits down to 2^-21 of the largest.  Without it that ends at 2^-14, and below 2^-25 they are lost: where
// one slot of 32 has a score 17 above the others', the others' part of the result was off by 4 %, at 18.5 by 95 %.
constexpr float kRoom = 7.0f, kUnroom = 0.0078125f;
// Beyond this reference (log2 domain) one fused multiply-add no longer does: the reference is a rounded product and its
// rounding, 2^-24 of itself, is then many powers of two, which exp2 would send to infinity.
constexpr float kLargeRef = 1048576.0f;

// dword N of the 16 lanes of a row, in all of them.
template <int N>
__device__ __forceinline__ uint32_t row_bcast(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x150 + N, 0xF, 0xF, true);
}

// Masks and bias of the unpacking, in registers: an instruction that takes
// all three operands holds no literals.
struct Unpack {
  uint32_t lo = 0x000f000fu, hi = 0x00f000f0u, bias = 0x64006400u;
  __device__ __forceinline__ Unpack() { asm("" : "+v"(lo), "+v"(hi), "+v"(bias)); }
};
// Eight 4-bit codes of a word as fp16 integers, in the order of the bits 0,
// 16, 4, 20, 8, 24, 12, 28.  1024 + n has the bits 0x6400 | n in fp16, 1024 +
// 16 n the bits 0x6400 | n << 4; one packed operation takes the 1024 off.
__device__ __forceinline__ half2_t code_lo(const Unpack &k, uint32_t w) {
  const half2_t bias = {(_Float16)1024.0f, (_Float16)1024.0f};
  return as_h2((w & k.lo) | k.bias) - bias;
}
__device__ __forceinline__ half2_t code_hi(const Unpack &k, uint32_t w) {
  const half2_t sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f}, bias = {(_Float16)64.0f, (_Float16)64.0f};
  return as_h2((w & k.hi) | k.bias) * sixteenth - bias;
}
// What codes stand for, rounded once: 15 times the largest step, 4368, is beyond fp16 before the minimum joins it.
__device__ __forceinline__ half2_t value(half2_t code, half2_t step, half2_t low) {
  return __builtin_elementwise_fma(code, step, low);
}
__device__ __forceinline__ half8_t join(half2_t a, half2_t b, half2_t c, half2_t d) {
  return half8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <int N>
struct Words {
  uint32_t w[N];
  __device__ __forceinline__ void load(const void *p) {
    if (N == 2) {
      const uint2_t v = *static_cast<const uint2_t *>(p);
      w[0] = v[0], w[1] = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint4_t v = static_cast<const uint4_t *>(p)[i / 4];
        w[i] = v[0], w[i + 1] = v[1], w[i + 2] = v[2], w[i + 3] = v[3];
      }
    }
  }
};

// What a lane loads of one tile.
template <int D>
struct Tile {
  static constexpr int DG = D / 32;
  static constexpr int SW = DG <= 4 ? 1 : DG / 4;  // dwords of key steps and minima a lane brings in
  Words<DG> k[2];        // two halves of 16 slots: a lane's DG words of its slot
  uint32_t ks[2][SW];
  Words<DG> v[2];        // two quads of slots: a lane's D / 16 channels
  uint4_t vs[2];

  // From the tile's first byte of keys or values and of their steps, the same
  // for every lane; the lane's offsets stay the same from tile to tile.
  __device__ __forceinline__ void load_keys(const uint8_t *kb, const uint8_t *sb, int lane) {
    const uint32_t c = lane & 15, h4 = lane >> 4;
    const uint32_t ko = c * (D / 2) + h4 * (DG * 4), so = h4 * (DG * 16) + (SW == 1 ? (c & (4 * DG - 1)) * 4 : c * 8);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      k[u].load(kb + u * (8 * D) + ko);
      if (SW == 1) ks[u][0] = *reinterpret_cast<const uint32_t *>(sb + u * (DG * 64) + so);
      else {
        const uint2_t x = *reinterpret_cast<const uint2_t *>(sb + u * (DG * 64) + so);
        ks[u][0] = x[0], ks[u][SW - 1] = x[1];
      }
    }
  }
  __device__ __forceinline__ void load_values(const uint8_t *vb, const uint8_t *sb, int lane) {
    const uint32_t c = lane & 15, h4 = lane >> 4;
    const uint32_t vo = h4 * (2 * D) + c * (D / 8), so = h4 * (DG * 16) + (c * DG / 16) * 16;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      v[u].load(vb + u * (8 * D) + vo);
      vs[u] = *reinterpret_cast<const uint4_t *>(sb + u * (DG * 64) + so);
    }
  }
};

// One group of the scores of a half: S[i] += s_i D[i] + m_i qsum.
template <int D, int J>
__device__ __forceinline__ void add_group(float *S, const Tile<D> &t, int u, half8_t qf, float qsum, const Unpack &k) {
  constexpr int SW = Tile<D>::SW;
  const uint32_t w = t.k[u].w[J];
  const half8_t kf = join(code_lo(k, w), code_hi(k, w), code_lo(k, w >> 8), code_hi(k, w >> 8));
  const float4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const float4_t dot = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf, zero, 0, 0, 0);
  const half2_t s01 = as_h2(row_bcast<(4 * J + 0) / SW>(t.ks[u][0]));
  const half2_t s23 = as_h2(row_bcast<(4 * J + 1) / SW>(t.ks[u][SW - 1]));
  const half2_t m01 = as_h2(row_bcast<(4 * J + 2) / SW>(t.ks[u][0]));
  const half2_t m23 = as_h2(row_bcast<(4 * J + 3) / SW>(t.ks[u][SW - 1]));
  S[0] = __builtin_fmaf((float)m01[0], qsum, __builtin_fmaf((float)s01[0], dot[0], S[0]));
  S[1] = __builtin_fmaf((float)m01[1], qsum, __builtin_fmaf((float)s01[1], dot[1], S[1]));
  S[2] = __builtin_fmaf((float)m23[0], qsum, __builtin_fmaf((float)s23[0], dot[2], S[2]));
  S[3] = __builtin_fmaf((float)m23[1], qsum, __builtin_fmaf((float)s23[1], dot[3], S[3]));
}

template <int D, int J>
struct AddGroups {
  static __device__ __forceinline__ void run(float *S, const Tile<D> &t, int u, const half8_t *qf, const float *qsum,
                                             const Unpack &k) {
    AddGroups<D, J - 1>::run(S, t, u, qf, qsum, k);
    add_group<D, J>(S, t, u, qf[J], qsum[J], k);
  }
};
template <int D>
struct AddGroups<D, -1> {
  static __device__ __forceinline__ void run(float *, const Tile<D> &, int, const half8_t *, const float *, const Unpack &) {}
};

struct AttendArgs {
  const void *q;
  int64_t q_ts, q_hs;
  float scale;
  int hq;
  void *out;
  float *lse;
  float *part;    // [share][2][16][D]: a share's part of the row it begins in, and of the one it ends in
  float *stat;    // [share][2][16][2]: reference (log2 domain), sum
  float *whole;   // [seq][head][2]: the same of rows that one share covers (add_weights)
  float *score;   // of each sequence after the other [head][its tiles][32], log2 domain (add_weights)
  int64_t *begins;  // [seq + 1]: tiles of one row before each sequence
};

__device__ __forceinline__ int tiles_of(const KvView &c, const AttendPlan &p, int b) {
  return (min(max(c.lens[b], 0), p.len_cap) + kTile - 1) / kTile;
}

// Where a sequence's scores begin, `before` tiles of one head after the first's.  Sequences that share pages, which
// weights must not be added to, can pass the end: their scores fall on others', not outside.
__device__ __forceinline__ float *scores_of(const AttendPlan &p, const AttendArgs &a, int64_t before, int tiles) {
  return a.score + min(before, p.score_tiles - tiles) * (kTile * (int64_t)a.hq);
}

__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)v) |
         (int64_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32;
}

// The line of tiles: sequence by sequence, in it head by head (`rows` of them).
struct Line {
  int64_t total, share;
  int rows;
  // the 64 sequences that the search has come to: the first of them, where it
  // begins, and of the lane's sequence the tiles and their sum up to it
  int b0;
  int64_t base, tiles;  // (tiles: of one row)
  uint32_t n, upto;
};
// Inclusive sum over the lanes of the wave.
__device__ __forceinline__ uint32_t prefix64(uint32_t v) {
#define VQMM_ADD_DPP(ctrl, rows) v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, false)
  VQMM_ADD_DPP(0x111, 0xF);  // row_shr 1, 2, 4, 8: within 16 lanes
  VQMM_ADD_DPP(0x112, 0xF);
  VQMM_ADD_DPP(0x114, 0xF);
  VQMM_ADD_DPP(0x118, 0xF);
  VQMM_ADD_DPP(0x142, 0xA);  // lane 15 of a row to the next one (rows 1 and 3)
  VQMM_ADD_DPP(0x143, 0xC);  // lane 31 to the upper half
#undef VQMM_ADD_DPP
  return v;
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); }
// Tiles of the 64 sequences from b0 on (64 of below 2^26: their sum is within 32 bits).
__device__ __forceinline__ uint32_t tiles64(const KvView &c, const AttendPlan &p, int b0) {
  const int b = b0 + (threadIdx.x & 63);
  return b < c.nseq ? (uint32_t)tiles_of(c, p, b) : 0u;
}
// Shares of equal size, in whole rounds of a workgroup's waves.
template <int D, bool WEIGH>
__device__ __forceinline__ int64_t share_of(int64_t total) {
  const int64_t even = (total + kShares<D, WEIGH> - 1) / kShares<D, WEIGH>;
  return max((even + kWaves - 1) / kWaves * kWaves, (int64_t)kWaves);
}
// The whole line; the first workgroup leaves where each sequence begins (in
// tiles of one row), and the end, for k_kv4_join.
template <int D, bool WEIGH>
__device__ __forceinline__ Line line_of(const KvView &c, const AttendPlan &p, int64_t *begins) {
  Line l;
  l.n = tiles64(c, p, 0);
  l.upto = prefix64(l.n);
  const bool leave = blockIdx.x == 0 && threadIdx.x < 64;
  if (leave && (int)threadIdx.x < c.nseq) begins[threadIdx.x] = l.upto - l.n;
  int64_t sum = lane_value(l.upto, 63);
  for (int b0 = 64; b0 < c.nseq; b0 += 64) {
    const uint32_t n = tiles64(c, p, b0), upto = prefix64(n);
    if (leave && b0 + (int)threadIdx.x < c.nseq) begins[b0 + threadIdx.x] = sum + (upto - n);
    sum += lane_value(upto, 63);
  }
  if (leave && threadIdx.x == 0) begins[c.nseq] = sum;
  l.rows = c.hkv * p.htiles;
  l.total = sum * l.rows;
  l.share = share_of<D, WEIGH>(l.total);
  l.b0 = 0;
  l.base = l.tiles = 0;
  return l;
}
// The sequence that holds position pos < total, no earlier than the last one
// found; where it begins, the tiles of one row before it and its own.
__device__ __forceinline__ int line_find(const KvView &c, const AttendPlan &p, Line &l, int64_t pos, int64_t *begin,
                                         int64_t *before, int *tiles) {
  for (;;) {
    const uint64_t past = __ballot(l.base + (int64_t)l.upto * l.rows > pos);
    if (past || l.b0 + 64 >= c.nseq) {
      const int at = past ? __builtin_ctzll(past) : 63;
      *tiles = (int)lane_value(l.n, at);
      const uint32_t in = lane_value(l.upto, at) - lane_value(l.n, at);
      *begin = l.base + (int64_t)in * l.rows;
      *before = l.tiles + in;
      return min(l.b0 + at, c.nseq - 1);
    }
    l.base += (int64_t)lane_value(l.upto, 63) * l.rows;
    l.tiles += lane_value(l.upto, 63);
    l.b0 += 64;
    l.n = tiles64(c, p, l.b0);
    l.upto = prefix64(l.n);
  }
}

// LONE: a workgroup of NW waves a row, all of it.
template <int D, bool F16, bool WEIGH, int NW, bool LONE>
__global__ __launch_bounds__(NW *kWave, (LONE ? 2 : kSharesPerCu<D, WEIGH>)) void k_kv4_attend(KvView c, AttendPlan p,
                                                                                              AttendArgs a) {
  constexpr int kThreads = NW * kWave, kWaves = NW;
  constexpr int DG = D / 32, CH = D / 16;
  constexpr int kPitch = D + 4;  // floats of a head's row in LDS: 16-byte pieces of 16 rows fall on different banks
  __shared__ float s_o[kWaves][16][kPitch];
  __shared__ float s_m[kWaves][16], s_l[kWaves][16];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Line line{};
  int64_t pos = 0, pos_end = 1;
  if (!LONE) {
    line = line_of<D, WEIGH>(c, p, a.begins);
    line.total = uniform(line.total);
    line.share = uniform(line.share);
    pos = blockIdx.x * line.share;
    pos_end = min(pos + line.share, line.total);
  }
  const int64_t pos0 = pos;
  while (pos < pos_end) {
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));  // anew for each row: what follows from it would else be kept in registers throughout
  const int lane = tid & 63, col = lane & 15, h4 = lane >> 4;
  int b, row, t_begin, t_end, ntiles;
  int64_t before = 0;
  if (LONE) {
    row = blockIdx.x % (c.hkv * p.htiles);
    b = blockIdx.x / (c.hkv * p.htiles);
    ntiles = tiles_of(c, p, b);
    t_begin = 0;
    t_end = ntiles;
    pos = pos_end;
  } else {
    int64_t begin;
    b = __builtin_amdgcn_readfirstlane(line_find(c, p, line, pos, &begin, &before, &ntiles));
    // Lengths that another stream shortens meanwhile are found shorter here than when the line was made: the bounds
    // keep such a row within the arrays, and the share moves on by a tile at least.
    ntiles = max(ntiles, 1);
    const int in = (int)min(pos - begin, (int64_t)ntiles * line.rows - 1);  // below 2^31
    row = __builtin_amdgcn_readfirstlane(in / ntiles);
    t_begin = __builtin_amdgcn_readfirstlane(in - row * ntiles);
    t_end = __builtin_amdgcn_readfirstlane((int)min((int64_t)ntiles, t_begin + (pos_end - pos)));
    pos += t_end - t_begin;
  }
  const int kvh = row / p.htiles, ht = row - kvh * p.htiles;
  const int len = min(max(c.lens[b], 0), p.len_cap);
  const int heads = min(16, p.group - ht * 16);   // of this row
  const int head0 = kvh * p.group + ht * 16;

  // the queries, in fp16 after a power-of-two rescale per head, in the order of the unpacked codes
  half8_t qf[DG];
  float qsum[DG];
  float cs;  // scores -> log2 domain
  {
    float x[DG][8];
    float top = 0.0f;
    const int h = head0 + min(col, heads - 1);
    const uint16_t *qp = static_cast<const uint16_t *>(a.q) + b * a.q_ts + h * a.q_hs;
#pragma unroll
    for (int j = 0; j < DG; ++j) {
      const uint4_t w = *reinterpret_cast<const uint4_t *>(qp + 8 * (4 * j + h4));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (F16) {
          const half2_t v = as_h2(w[i]);
          x[j][2 * i] = (float)v[0], x[j][2 * i + 1] = (float)v[1];
        } else {
          x[j][2 * i] = bf2f(w[i] & 0xffffu), x[j][2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[j][i]));
    }
    top = max_xor32(max_xor16(top));
    // largest |q| to [2^14, 2^15); zero, infinite and very small rows keep a finite factor
    int e = top > 0.0f && top <= 3.4e38f ? 14 - (int)((__float_as_uint(top) >> 23) - 127) : 0;
    e = min(max(e, -120), 100);
    const float up = __uint_as_float((uint32_t)(e + 127) << 23);
    cs = a.scale * kLog2e * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int j = 0; j < DG; ++j) {
      float sum = 0.0f;
      half8_t v;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const _Float16 y = (_Float16)(x[j][i] * up);
        v[(i & 3) * 2 + (i >> 2)] = y;  // channels 0 4 1 5 2 6 3 7
        sum += (float)y;
      }
      qf[j] = v;
      qsum[j] = sum_xor32(sum_xor16(sum));
    }
  }

  float4_t acc[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) acc[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  float mref = -INFINITY, lsum = 0.0f;
  bool large = false;  // some head's reference is beyond kLargeRef

  float *scores = nullptr;  // of the lane's head and slots, from the sequence's first tile on
  if (WEIGH) scores = scores_of(p, a, before, ntiles) + (int64_t)(head0 + col) * ntiles * kTile + 4 * h4;

  const int tpp = c.ps / kTile;  // tiles of a page
  const int64_t code_head = (int64_t)c.ps * (D / 2), scale_head = (int64_t)c.ps * (DG * 2);
  // Keys and values of the next tile go into the registers of this one as soon
  // as those are used up: half a round before they are wanted.
  Tile<D> cur;
  const uint8_t *next_v, *next_vs;
  auto fetch_keys = [&](int tile) {
    const int pi = tile / tpp;
    const int64_t page = page_of(c, b, pi);
    const int at = tile - pi * tpp;
    const uint8_t *kb = c.codes + (page * 2 * c.hkv + kvh) * code_head + at * (kTile * D / 2);
    const uint8_t *sb = reinterpret_cast<const uint8_t *>(c.scales + (page * 2 * c.hkv + kvh) * scale_head) + at * (kTile * DG * 4);
    cur.load_keys(kb, sb, lane);
    next_v = kb + c.hkv * code_head;
    next_vs = sb + 2 * c.hkv * scale_head;
  };
  const Unpack unpack;
  int tile = t_begin + wave;
  if (tile < t_end) {
    fetch_keys(tile);
    cur.load_values(next_v, next_vs, lane);
  }
  for (; tile < t_end; tile += kWaves) {
    float S[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      AddGroups<D, DG - 1>::run(S[u], cur, u, qf, qsum, unpack);
      // one half's products and broadcast steps in registers at a time, not both until after the loads below
      asm volatile("" : "+v"(S[u][0]), "+v"(S[u][1]), "+v"(S[u][2]), "+v"(S[u][3]));
    }
    const bool more = tile + kWaves < t_end;
    if (more) fetch_keys(tile + kWaves);

    const int left = len - tile * kTile;  // slots of the tile that exist
    if (left < kTile) {  // the last tile: slots past the end count for nothing, whatever they hold
      asm volatile("");  // a branch, not selects in every tile
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int in = left - 16 * u - 4 * h4;  // of the lane's four slots
#pragma unroll
        for (int i = 0; i < 4; ++i) S[u][i] = i < in ? S[u][i] : -INFINITY;
        const uint32_t m01 = in > 1 ? 0xffffffffu : in > 0 ? 0xffffu : 0u, m23 = in > 3 ? 0xffffffffu : in > 2 ? 0xffffu : 0u;
        cur.vs[u][0] &= m01, cur.vs[u][1] &= m23, cur.vs[u][2] &= m01, cur.vs[u][3] &= m23;
      }
    }
    if (WEIGH && col < heads) {
      float *sp = scores + (int64_t)tile * kTile;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        *reinterpret_cast<float4_t *>(sp + 16 * u) = float4_t{S[u][0] * cs, S[u][1] * cs, S[u][2] * cs, S[u][3] * cs};
    }

    // (a NaN spoils its own head's sum whatever the maximum is)
    float top = max_nan(max_nan(max_nan(S[0][0], S[0][1]), max_nan(S[0][2], S[0][3])),
                        max_nan(max_nan(S[1][0], S[1][1]), max_nan(S[1][2], S[1][3])));
    top = max_xor32(max_xor16(top)) * cs;
    if (__any(top - mref > kSlack + kRoom)) {
      const float mnew = fmaxf(mref, top - kRoom);
      const float f = mnew == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(mref - mnew);
      lsum *= f;
#pragma unroll
      for (int i = 0; i < CH; ++i) acc[i] *= f;
      mref = mnew;
      large = __any(fabsf(mref) > kLargeRef);
    }
    const float m0 = mref == -INFINITY ? 0.0f : mref;
    if (large) {  // the product rounded as the reference's was: their difference is exact near the top
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = S[u][i] * cs;
          asm volatile("" : "+v"(x));  // not fused with the subtraction
          S[u][i] = x - m0;
        }
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[u][i] = __builtin_fmaf(S[u][i], cs, -m0);
    }
    float P[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        P[u][i] = __builtin_amdgcn_exp2f(S[u][i]);
        lsum += P[u][i];
      }
    const uint4_t pw = {pack16<true>(P[0][0], P[0][1]), pack16<true>(P[0][2], P[0][3]),
                        pack16<true>(P[1][0], P[1][1]), pack16<true>(P[1][2], P[1][3])};
    const half8_t pf = __builtin_bit_cast(half8_t, pw);
    // fp16 results are as exact as the rounding of P: its remainder takes part too (bf16 results are not).
    half8_t pr;
    if (F16) {
      float R[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) R[i] = P[i / 4][i & 3] - (float)pf[i];
      pr = __builtin_bit_cast(half8_t, uint4_t{pack16<true>(R[0], R[1]), pack16<true>(R[2], R[3]),
                                               pack16<true>(R[4], R[5]), pack16<true>(R[6], R[7])});
    }

    half2_t sv[4], mv[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      sv[2 * u] = as_h2(cur.vs[u][0]), sv[2 * u + 1] = as_h2(cur.vs[u][1]);
      mv[2 * u] = as_h2(cur.vs[u][2]), mv[2 * u + 1] = as_h2(cur.vs[u][3]);
    }
#pragma unroll
    for (int i = 0; i < DG; ++i) {  // two pairs of channels a word: 2 i' = CH channels in all
      const uint32_t w0 = cur.v[0].w[i], w1 = cur.v[1].w[i];
      const Unpack &k = unpack;
      const half8_t lo = join(value(code_lo(k, w0), sv[0], mv[0]), value(code_lo(k, w0 >> 8), sv[1], mv[1]),
                              value(code_lo(k, w1), sv[2], mv[2]), value(code_lo(k, w1 >> 8), sv[3], mv[3]));
      const half8_t hi = join(value(code_hi(k, w0), sv[0], mv[0]), value(code_hi(k, w0 >> 8), sv[1], mv[1]),
                              value(code_hi(k, w1), sv[2], mv[2]), value(code_hi(k, w1 >> 8), sv[3], mv[3]));
      acc[2 * i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo, pf, acc[2 * i], 0, 0, 0);
      acc[2 * i + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, pf, acc[2 * i + 1], 0, 0, 0);
      if (F16) {
        acc[2 * i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo, pr, acc[2 * i], 0, 0, 0);
        acc[2 * i + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, pr, acc[2 * i + 1], 0, 0, 0);
      }
    }
    if (more) cur.load_values(next_v, next_vs, lane);
  }

  // the waves meet
  const bool whole = LONE || (t_begin == 0 && t_end == ntiles);
  const int side = pos - (t_end - t_begin) == pos0 && t_begin > 0 ? 0 : 1;  // 0: the row began in an earlier share
  lsum = sum_xor32(sum_xor16(lsum));
  if (col < heads) {
    if (h4 == 0) s_m[wave][col] = mref, s_l[wave][col] = lsum;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < CH; x += 4)
        *reinterpret_cast<float4_t *>(&s_o[wave][col][CH * (4 * h4 + i) + x]) =
            float4_t{acc[x][i], acc[x + 1][i], acc[x + 2][i], acc[x + 3][i]};
  }
  __syncthreads();
  for (int e = tid * 4; e < heads * D; e += kThreads * 4) {
    const int h = e / D, d = e % D;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_m[w][h]);
    const float m0 = top == -INFINITY ? 0.0f : top;
    float4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(s_m[w][h] - m0);
      l = __builtin_fmaf(s_l[w][h], f, l);
      const float4_t ow = *reinterpret_cast<const float4_t *>(&s_o[w][h][d]);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(ow[i], f, o[i]);
    }
    const int64_t at = (int64_t)b * a.hq + head0 + h;
    if (whole) {
      const float r = l == 0.0f ? 0.0f : 1.0f / l;
      const uint2_t w = {pack16<F16>(o[0] * r, o[1] * r), pack16<F16>(o[2] * r, o[3] * r)};
      *reinterpret_cast<uint2_t *>(static_cast<uint16_t *>(a.out) + at * D + d) = w;
      if (d == 0) {
        if (a.lse) a.lse[at] = (__builtin_amdgcn_logf(l * kUnroom) + (m0 + kRoom)) * kLn2;
        if (WEIGH) a.whole[at * 2] = top, a.whole[at * 2 + 1] = l;
      }
    } else {
      const int64_t piece = ((int64_t)blockIdx.x * 2 + side) * 16 + h;
      *reinterpret_cast<float4_t *>(a.part + piece * D + d) = o;
      if (d == 0) a.stat[piece * 2] = top, a.stat[piece * 2 + 1] = l;
    }
  }
  __syncthreads();  // the LDS is free for the next row
  }
}

// The parts of one row: the shares from `first` to `last` of the line, each at
// side 1 of the first and side 0 of the others.
struct Parts {
  int first, n;
  bool whole, empty;
};
__device__ __forceinline__ Parts parts_of(const AttendArgs &a, int64_t total, int64_t share, int rows, int b, int row) {
  const int nt = (int)(a.begins[b + 1] - a.begins[b]);
  const int64_t begin = a.begins[b] * rows + (int64_t)row * nt, end = begin + nt;
  Parts r;
  r.empty = nt == 0;
  if (total < ((int64_t)1 << 31)) {  // short divisions, nearly always
    r.first = (int)begin / (int)share;
    r.n = nt == 0 ? 0 : (int)(end - 1) / (int)share - r.first + 1;
  } else {
    r.first = (int)(begin / share);
    r.n = nt == 0 ? 0 : (int)((end - 1) / share) - r.first + 1;
  }
  r.whole = r.n == 1;
  return r;
}
__device__ __forceinline__ int64_t part_at(const Parts &r, int i, int h) {
  return ((int64_t)(r.first + i) * 2 + (i == 0 ? 1 : 0)) * 16 + h;
}
// Reference and sum of one head over its parts, by one wave.
__device__ __forceinline__ void head_stats(const AttendArgs &a, const Parts &r, int64_t at, int h, float *top, float *sum) {
  const int lane = threadIdx.x & 63;
  if (r.whole) {
    *top = a.whole[at * 2] == -INFINITY ? 0.0f : a.whole[at * 2];
    *sum = a.whole[at * 2 + 1];
    return;
  }
  float m = -INFINITY;
  for (int i = lane; i < r.n; i += kWave) m = fmaxf(m, a.stat[part_at(r, i, h) * 2]);
#pragma unroll
  for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  const float m0 = m == -INFINITY ? 0.0f : m;
  float l = 0.0f;
  for (int i = lane; i < r.n; i += kWave) {
    const float *st = a.stat + part_at(r, i, h) * 2;
    l = __builtin_fmaf(st[1], __builtin_amdgcn_exp2f(st[0] - m0), l);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) l += __shfl_xor(l, o);
  *top = m0;
  *sum = l;
}

constexpr int kWeighSlots = kThreads * 4;  // slots of a workgroup of the weights' part

// The first `out_blocks` workgroups take a head's output each, where its row
// was cut (or is empty); the others the weights of a run of slots of one
// sequence and key/value head.
template <int D, bool F16, bool WEIGH>
__global__ __launch_bounds__(kThreads) void k_kv4_join(KvView c, AttendPlan p, AttendArgs a, int out_blocks, int chunks) {
  const int rows = c.hkv * p.htiles;
  const int64_t total = a.begins[c.nseq] * rows, share = share_of<D, WEIGH>(total);
  if ((int)blockIdx.x < out_blocks) {
    constexpr int kSub = kThreads / (D / 4);  // parts summed side by side, four channels a thread
    __shared__ float s_part[kSub][D];
    const int b = (int)blockIdx.x / a.hq, head = (int)blockIdx.x - b * a.hq;
    const int64_t at = blockIdx.x;
    const int kvh = head / p.group, ht = (head - kvh * p.group) / 16, h = (head - kvh * p.group) % 16;
    const Parts parts = parts_of(a, total, share, rows, b, kvh * p.htiles + ht);
    if (parts.whole) return;
    float top, sum;
    head_stats(a, parts, at, h, &top, &sum);
    const int d = threadIdx.x % (D / 4) * 4, sub = threadIdx.x / (D / 4);
    float4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = sub; i < parts.n; i += kSub) {
      const int64_t piece = part_at(parts, i, h);
      const float f = __builtin_amdgcn_exp2f(a.stat[piece * 2] - top);
      const float4_t v = *reinterpret_cast<const float4_t *>(a.part + piece * D + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __builtin_fmaf(v[j], f, o[j]);
    }
    *reinterpret_cast<float4_t *>(&s_part[sub][d]) = o;
    __syncthreads();
    const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
    for (int x = threadIdx.x * 2; x < D; x += kThreads * 2) {
      float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
      for (int i = 0; i < kSub; ++i) y0 += s_part[i][x], y1 += s_part[i][x + 1];
      *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + at * D + x) = pack16<F16>(y0 * r, y1 * r);
    }
    if (threadIdx.x == 0 && a.lse) a.lse[at] = (__builtin_amdgcn_logf(sum * kUnroom) + (top + kRoom)) * kLn2;
    return;
  }
  __shared__ float s_top[16], s_inv[16];
  int id = blockIdx.x - out_blocks;
  const int chunk = id % chunks;
  id /= chunks;
  const int kvh = id % c.hkv, b = id / c.hkv;
  const int nt = (int)(a.begins[b + 1] - a.begins[b]);
  const int len = min(min(max(c.lens[b], 0), p.len_cap), nt * kTile);  // the scores there are
  if (chunk * kWeighSlots >= len) return;
  const int slot = chunk * kWeighSlots + threadIdx.x * 4;
  const float *scores = scores_of(p, a, a.begins[b], nt) + slot;
  float4_t w = {0.0f, 0.0f, 0.0f, 0.0f};
  const int wave = threadIdx.x >> 6;
  for (int ht = 0; ht < p.htiles; ++ht) {  // heads of the group, 16 at a time
    const int ng = min(16, p.group - ht * 16);
    const int head0 = kvh * p.group + ht * 16;
    const int64_t at0 = (int64_t)b * a.hq + head0;
    const Parts parts = parts_of(a, total, share, rows, b, kvh * p.htiles + ht);
    __syncthreads();
    for (int g = wave; g < ng; g += kWaves) {
      float top, sum;
      head_stats(a, parts, at0 + g, g, &top, &sum);
      if ((threadIdx.x & 63) == 0) s_top[g] = top, s_inv[g] = sum == 0.0f ? 0.0f : 1.0f / sum;
    }
    __syncthreads();
    if (slot < len)
#pragma unroll 8
      for (int g = 0; g < ng; ++g) {
        const float4_t x = *reinterpret_cast<const float4_t *>(scores + (int64_t)(head0 + g) * nt * kTile);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(x[i] - s_top[g]), s_inv[g], w[i]);
      }
  }
  if (slot >= len) return;
  const int pi = slot / c.ps;
  float *wp = c.weights + (page_of(c, b, pi) * c.hkv + kvh) * c.ps + (slot - pi * c.ps);
  if (slot + 4 <= len) {
    float4_t old = *reinterpret_cast<const float4_t *>(wp);
    *reinterpret_cast<float4_t *>(wp) = old + w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (slot + i < len) wp[i] += w[i];
  }
}

template <int D, bool F16, bool WEIGH>
hipError_t attend_shares(const KvView &c, const AttendPlan &p, const AttendArgs &a, hipStream_t s) {
  k_kv4_attend<D, F16, WEIGH, kWaves, false><<<kShares<D, WEIGH>, kThreads, 0, s>>>(c, p, a);
  return hipGetLastError();
}

template <int D, bool F16>
hipError_t attend_d(const KvView &c, const AttendPlan &p, const AttendArgs &a, bool weigh, hipStream_t s) {
  if (p.lone) {
    k_kv4_attend<D, F16, false, kLoneWaves, true><<<c.nseq * c.hkv * p.htiles, kLoneWaves * kWave, 0, s>>>(c, p, a);
    return hipGetLastError();
  }
  const int chunks = weigh ? (p.len_cap + kWeighSlots - 1) / kWeighSlots : 0;
  const int64_t grid = (int64_t)c.nseq * a.hq + (int64_t)chunks * c.nseq * c.hkv;
  const hipError_t e = weigh ? attend_shares<D, F16, true>(c, p, a, s) : attend_shares<D, F16, false>(c, p, a, s);
  if (e != hipSuccess) return e;
  if (weigh) k_kv4_join<D, F16, true><<<(unsigned)grid, kThreads, 0, s>>>(c, p, a, c.nseq * a.hq, chunks);
  else k_kv4_join<D, F16, false><<<(unsigned)grid, kThreads, 0, s>>>(c, p, a, c.nseq * a.hq, chunks);
  return hipGetLastError();
}

}  // namespace

AttendPlan kv4_attend_plan(const KvView &c, int n_q_heads, int max_len, bool add_weights) {
  AttendPlan p{};
  p.group = n_q_heads / c.hkv;
  p.htiles = (p.group + 15) / 16;
  p.len_cap = (int)std::min<int64_t>(max_len, (int64_t)c.mp * c.ps);
  // weights go to pages of one sequence each, so all sequences together hold no more than the pool
  const int64_t pool = (int64_t)c.np * c.ps;
  if (add_weights) p.len_cap = (int)std::min<int64_t>(p.len_cap, pool);
  p.lone = !add_weights && p.len_cap <= lone_slots(c.d);
  if (p.lone) return p;
  p.score_tiles = std::min((int64_t)c.nseq * ((p.len_cap + kTile - 1) / kTile), pool / kTile);
  auto round = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t pieces = (size_t)shares_of(c.d) * 2 * 16, heads = (size_t)c.nseq * n_q_heads;
  p.stat_off = round(pieces * c.d * 4);
  p.begin_off = p.stat_off + round(pieces * 8);
  p.whole_off = p.begin_off + round(((size_t)c.nseq + 1) * 8);
  p.score_off = p.whole_off + (add_weights ? round(heads * 8) : 0);
  p.bytes = p.score_off + (add_weights ? round((size_t)p.score_tiles * kTile * n_q_heads * 4) : 0);
  return p;
}

hipError_t launch_kv4_attend(const KvView &c, const AttendPlan &p, const void *q, int64_t q_ts, int64_t q_hs, bool f16,
                             int n_q_heads, float scale, bool add_weights, void *out, float *lse, void *ws,
                             hipStream_t s) {
  char *w = static_cast<char *>(ws);
  AttendArgs a{q,   q_ts, q_hs, scale, n_q_heads, out, lse, reinterpret_cast<float *>(w),
               reinterpret_cast<float *>(w + p.stat_off), reinterpret_cast<float *>(w + p.whole_off),
               reinterpret_cast<float *>(w + p.score_off), reinterpret_cast<int64_t *>(w + p.begin_off)};
  if (c.d == 64) return f16 ? attend_d<64, true>(c, p, a, add_weights, s) : attend_d<64, false>(c, p, a, add_weights, s);
  if (c.d == 128)
    return f16 ? attend_d<128, true>(c, p, a, add_weights, s) : attend_d<128, false>(c, p, a, add_weights, s);
  return f16 ? attend_d<256, true>(c, p, a, add_weights, s) : attend_d<256, false>(c, p, a, add_weights, s);
}

}  // namespace vqmm
