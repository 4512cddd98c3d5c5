// kv4_evict: cut each sequence and key/value head down to `keep` slots.
//
// k_kv4_select, one workgroup a sequence and head, finds the keep-th largest
// key by a radix search (four passes of 8 bits over keys that order as the
// weights do), splits its ties by slot, and lists the free slots below keep
// and the kept ones at or above it, both in ascending order; there are equally
// many.  k_kv4_move copies slot to slot, 16 lanes a move: sources lie at or above
// keep and targets below it, so no copy reads what another writes.  Counts are
// integers and every list position is a prefix sum, so nothing depends on the
// order in which waves run.
//
// Bound: 8 bytes (weight, position) of every slot, then the moved slots twice;
// a few microseconds at any size met in practice, so latency counts: a row's
// keys stay in registers through the search (two barriers a digit), loads go
// out in batches of eight, and where no more than 16 slots can move (a step's
// own eviction) the selecting workgroup moves them and the second launch is
// saved.  Eight sequences of up to 8191 slots of 8 heads of 128 down to 1024:
// 15.9 + 8.9 us; one slot over 1024 in 32 sequences: 7.8 us.
#include "attn_device.h"

#include <algorithm>

namespace vqmm {

namespace {

constexpr int kMoveThreads = 256;
constexpr int kMovesPerBlock = kMoveThreads / 16;
constexpr int kRegisterSlots = 32768;  // rows of more keep their keys in the workspace
constexpr int kFuseMoves = 16;  // one for each 16 lanes of the smallest selecting workgroup

// Keys in the order of the weights: NaN lowest, the protected slots on top.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix over the workgroup's waves of a count each wave holds.
__device__ __forceinline__ int wave_prefix(int *s, int wave, int count) {
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[wave] = count;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < wave; ++i) before += s[i];
  return before;
}

// Set bits of a wave's mask at the lanes below.
__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// Copies slot src to slot dst, by the 16 lanes l of one move: keys and values
// with their steps and minima, weight and position.
constexpr int kMoveLanes = 16;
template <int D>
__device__ __forceinline__ void move_slot(const KvView &c, int b, int kvh, int src, int dst, int l) {
  constexpr int DG = D / 32;
  const int64_t code_head = (int64_t)c.ps * (D / 2), scale_head = (int64_t)c.ps * (DG * 2);
  const int sp = src / c.ps, dp = dst / c.ps;
  const int so = src - sp * c.ps, d_o = dst - dp * c.ps;
  const int64_t spage = page_of(c, b, sp), dpage = page_of(c, b, dp);
  const uint8_t *sc = c.codes + (spage * 2 * c.hkv + kvh) * code_head;
  uint8_t *dc = c.codes + (dpage * 2 * c.hkv + kvh) * code_head;
  const uint16_t *ss = c.scales + (spage * 2 * c.hkv + kvh) * scale_head + (so >> 2) * (DG * 8) + (so & 3);
  uint16_t *ds = c.scales + (dpage * 2 * c.hkv + kvh) * scale_head + (d_o >> 2) * (DG * 8) + (d_o & 3);
  const int64_t sa = (spage * c.hkv + kvh) * c.ps + so, da = (dpage * c.hkv + kvh) * c.ps + d_o;
  const int sb = (so & 3) == 1 ? 2 : (so & 3) == 2 ? 1 : so & 3, db = (d_o & 3) == 1 ? 2 : (d_o & 3) == 2 ? 1 : d_o & 3;
  const uint32_t *sk = reinterpret_cast<const uint32_t *>(sc + so * (D / 2));
  uint32_t *dk = reinterpret_cast<uint32_t *>(dc + d_o * (D / 2));
  const uint8_t *sv = sc + c.hkv * code_head + (so >> 2) * (2 * D) + sb;
  uint8_t *dv = dc + c.hkv * code_head + (d_o >> 2) * (2 * D) + db;
  constexpr int NK = (D / 8 + kMoveLanes - 1) / kMoveLanes, NV = D / 2 / kMoveLanes, NS = (4 * DG + kMoveLanes - 1) / kMoveLanes;
  // every load first: their latencies overlap
  uint32_t key[NK] = {};
  uint16_t sm[NS] = {};
  uint8_t val[NV];
#pragma unroll
  for (int x = 0; x < NK; ++x)
    if (x * kMoveLanes + l < D / 8) key[x] = sk[x * kMoveLanes + l];
#pragma unroll
  for (int x = 0; x < NV; ++x) val[x] = sv[(x * kMoveLanes + l) * 4];
#pragma unroll
  for (int x = 0; x < NS; ++x) {  // (kind, group, step or minimum)
    const int i = x * kMoveLanes + l;
    if (i < 4 * DG) sm[x] = ss[i / (2 * DG) * (c.hkv * scale_head) + i % (2 * DG) * 4];
  }
  const float w = c.weights[sa];
  const int32_t at = c.pos[sa];
#pragma unroll
  for (int x = 0; x < NK; ++x)
    if (x * kMoveLanes + l < D / 8) dk[x * kMoveLanes + l] = key[x];
#pragma unroll
  for (int x = 0; x < NV; ++x) dv[(x * kMoveLanes + l) * 4] = val[x];
#pragma unroll
  for (int x = 0; x < NS; ++x) {
    const int i = x * kMoveLanes + l;
    if (i < 4 * DG) ds[i / (2 * DG) * (c.hkv * scale_head) + i % (2 * DG) * 4] = sm[x];
  }
  if (l == 0) c.weights[da] = w;
  if (l == 1) c.pos[da] = at;
}

// A wave's run of slots, 64 at a time, and where their keys are kept: in
// registers (R > 0: up to R a thread) or in the workspace (R = 0).
template <int R>
struct Keys {
  uint32_t r[R];
  __device__ __forceinline__ uint32_t get(int i, const uint32_t *, int) const { return r[i]; }
  __device__ __forceinline__ void set(int i, uint32_t *, int, uint32_t k) { r[i] = k; }
};
template <>
struct Keys<0> {
  __device__ __forceinline__ uint32_t get(int, const uint32_t *ws, int slot) const { return ws[slot]; }
  __device__ __forceinline__ void set(int, uint32_t *ws, int slot, uint32_t k) { ws[slot] = k; }
};

// f(i, slot) for the steps i of the wave's run; unrolled where the keys are registers.
template <int R, typename F>
__device__ __forceinline__ void each_step(int steps, int first, F f) {
  if (R > 0) {
#pragma unroll
    for (int i = 0; i < (R > 0 ? R : 1); ++i)
      if (i < steps) f(i, first + i * kWave);
  } else {
    for (int i = 0; i < steps; ++i) f(i, first + i * kWave);
  }
}

constexpr int kCopies = 4;  // histograms of a wave: equal digits of neighbouring lanes fall on different counters

// NT threads a row.  FUSE > 0: the workgroup moves its few slots itself,
// head_dim FUSE.
template <int NT, int R, int FUSE>
__global__ __launch_bounds__(NT) void k_kv4_select(KvView c, EvictPlan p, const int32_t *__restrict__ next_pos,
                                                            int keep, int recent, uint32_t *__restrict__ keys_all,
                                                            int32_t *__restrict__ moves, int32_t *__restrict__ counts) {
  constexpr int kSelThreads = NT, kSelWaves = NT / kWave;
  constexpr int kHist = kSelWaves / 4 * kCopies * 256;
  __shared__ int s_hist[2][kHist];  // one fills while the other is cleared
  __shared__ int s_sum[256];
  __shared__ int s_wave[kSelWaves], s_holes[kSelWaves];
  __shared__ int s_moved;
  __shared__ int s_to[FUSE ? kFuseMoves : 1], s_from[FUSE ? kFuseMoves : 1];

  const int row = blockIdx.x;
  const int b = row / c.hkv, kvh = row - b * c.hkv;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int len = min(max(c.lens[b], 0), p.len_cap);
  if (len <= keep) {
    if (!FUSE && tid == 0) counts[row] = 0;
    return;
  }
  uint32_t *ws = keys_all + (int64_t)row * p.len_cap;
  const int64_t oldest = (int64_t)next_pos[b] - recent;  // positions from here on are kept
  const int steps = (len + kSelThreads - 1) / kSelThreads;
  const int first = wave * steps * kWave + lane;  // (wave: uniform)

  // Keys in the order of the weights, protected slots on top; what lanes past
  // the end hold counts nowhere.
  Keys<R> keys;
  // 32-slot tile t is on page t / tiles: exact by one multiplication for t < 2^26 and tiles <= 32
  const uint32_t tiles = c.ps / 32, inverse = tiles > 1 ? 0xffffffffu / tiles + 1 : 0;
  constexpr int kBatch = 8;  // steps whose loads go out together
  auto load = [&](int i0) {
    int64_t at[kBatch];
    int32_t pos[kBatch];
    float w[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int slot = min(first + (i0 + j) * kWave, len - 1), pi = tiles > 1 ? (int)__umulhi(slot >> 5, inverse) : slot >> 5;
      at[j] = (page_of(c, b, pi) * c.hkv + kvh) * c.ps + (slot - pi * c.ps);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) pos[j] = c.pos[at[j]], w[j] = c.weights[at[j]];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int slot = first + (i0 + j) * kWave;
      const uint32_t key = pos[j] >= oldest ? 0xffffffffu : weight_key(w[j]);
      if (R > 0) {
        if (i0 + j < R) keys.set(i0 + j, ws, slot, key);
      } else if (i0 + j < steps && slot < len) {
        keys.set(i0 + j, ws, slot, key);
      }
    }
  };
  if (R > 0) {
#pragma unroll
    for (int i0 = 0; i0 < R; i0 += kBatch)
      if (i0 < steps) load(i0);
  } else {
    for (int i0 = 0; i0 < steps; i0 += kBatch) load(i0);
  }

  // Four digits of 8 bits from the top; `prefix` holds the digits found so far, `need` how many of the keys that have
  // them are kept.  Every wave reads the counts and finds the digit itself: two barriers a round.
  uint32_t prefix = 0;
  int need = keep;
  for (int i = tid; i < kHist; i += kSelThreads) s_hist[0][i] = 0;
  __syncthreads();
  bool all = false;  // every key with the digits so far is kept: the rest need not be known
#pragma unroll
  for (int round = 0; round < 4; ++round) {
    const int shift = 24 - 8 * round;
    if (all) continue;
    int *hist = &s_hist[round & 1][(wave / 4 * kCopies + lane % kCopies) * 256];
    each_step<R>(steps, first, [&](int i, int slot) {
      if (slot < len) {
        const uint32_t key = keys.get(i, ws, slot);
        if (round == 0 || (key >> (shift + 8 & 31)) == (prefix >> (shift + 8 & 31))) atomicAdd(&hist[(key >> shift) & 255u], 1);
      }
    });
    __syncthreads();
    if (tid < 256) {
      int n = 0;
#pragma unroll
      for (int w = 0; w < kSelWaves / 4 * kCopies; ++w) n += s_hist[round & 1][w * 256 + tid];
      s_sum[tid] = n;
    }
    if (round < 3)
      for (int i = tid; i < kHist; i += kSelThreads) s_hist[~round & 1][i] = 0;
    __syncthreads();
    int n[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = s_sum[255 - 4 * lane - i], mine += n[i];
    int upto = mine;  // inclusive prefix over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    int above = upto - mine, digit = -1, left = 0, count = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (above < need && need <= above + n[i]) digit = 255 - 4 * lane - i, left = need - above, count = n[i];
      above += n[i];
    }
    const int at = __builtin_ctzll(__ballot(digit >= 0));  // one lane holds it
    prefix |= (uint32_t)__builtin_amdgcn_readlane(digit, at) << shift;
    need = __builtin_amdgcn_readlane(left, at);
    all = need == __builtin_amdgcn_readlane(count, at);
    // s_sum is written again only after the next round's first barrier
  }
  // kept: keys above `limit`, and the first `need` of those equal to it (none where whole digits are kept; a prefix of
  // zero cannot be passed by one less, and keeps all its keys as ties)
  const uint32_t limit = all && prefix > 0 ? prefix - 1 : prefix;
  if (all) need = prefix > 0 ? 0 : len;

  // ties of the keep-th key by slot, then the two lists
  int ties_before = 0;
  if (need > 0) {
    int ties = 0;
    each_step<R>(steps, first, [&](int i, int slot) {
      ties += __popcll(__ballot(slot < len && keys.get(i, ws, min(slot, len - 1)) == limit));
    });
    ties_before = wave_prefix(s_wave, wave, ties);
  }
  int holes_at = 0, movers_at = 0;
  int32_t *to = moves + (int64_t)row * 2 * p.max_moves, *from = to + p.max_moves;
  uint32_t kept = 0;  // bit i: the lane's slot of step i stays (keys in registers)
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    int t = ties_before, h = holes_at, m = movers_at;
    each_step<R>(steps, first, [&](int i, int slot) {
      const int s0 = first - lane + i * kWave;  // the step's first slot, the same for the wave
      const bool in = slot < len;
      bool stays;
      if (R > 0 && pass == 1) {
        stays = (kept >> (i & 31)) & 1u;
      } else {
        const uint32_t key = keys.get(i, ws, min(slot, len - 1));
        stays = in && key > limit;
        if (need > 0) {
          const uint64_t tie = __ballot(in && key == limit);
          stays = stays || (in && key == limit && lanes_below(tie) + t < need);
          t += __popcll(tie);
        }
        if (R > 0) kept |= (uint32_t)stays << (i & 31);
      }
      if (s0 < keep) {
        const bool is = in && !stays && slot < keep;
        const uint64_t hole = __ballot(is);
        if (pass == 1 && is) (FUSE ? s_to : to)[h + lanes_below(hole)] = slot;
        h += __popcll(hole);
      }
      if (s0 + kWave > keep) {
        const bool is = stays && slot >= keep;
        const uint64_t mover = __ballot(is);
        if (pass == 1 && is) (FUSE ? s_from : from)[m + lanes_below(mover)] = slot;
        m += __popcll(mover);
      }
    });
    if (pass == 0) {
      if (lane == 0) s_holes[wave] = h;
      movers_at = wave_prefix(s_wave, wave, m);
      for (int i = 0; i < wave; ++i) holes_at += s_holes[i];
      if (wave == kSelWaves - 1 && lane == 0) {
        if (FUSE) s_moved = movers_at + m;
        else counts[row] = movers_at + m;
      }
    }
  }
  if (FUSE) {
    __syncthreads();
    const int i = tid / kMoveLanes;
    if (i < s_moved) move_slot<FUSE ? FUSE : 64>(c, b, kvh, s_from[i], s_to[i], lane % kMoveLanes);
  }
}

template <int D>
__global__ __launch_bounds__(kMoveThreads) void k_kv4_move(KvView c, EvictPlan p, const int32_t *__restrict__ moves,
                                                           const int32_t *__restrict__ counts, int chunks) {
  const int row = blockIdx.x / chunks, chunk = blockIdx.x - row * chunks;
  const int n = counts[row];
  const int32_t *to = moves + (int64_t)row * 2 * p.max_moves, *from = to + p.max_moves;
  for (int i = chunk * kMovesPerBlock + threadIdx.x / kMoveLanes; i < n; i += chunks * kMovesPerBlock)
    move_slot<D>(c, row / c.hkv, row % c.hkv, from[i], to[i], threadIdx.x % kMoveLanes);
}

template <int NT, int R, int FUSE>
hipError_t select_rows(const KvView &c, const EvictPlan &p, const int32_t *next_pos, int keep, int recent, uint32_t *keys,
                       int32_t *moves, int32_t *counts, hipStream_t s) {
  k_kv4_select<NT, R, FUSE><<<c.nseq * c.hkv, NT, 0, s>>>(c, p, next_pos, keep, recent, keys, moves, counts);
  return hipGetLastError();
}

// Rows of up to 2048 slots take four waves (barriers are cheaper there), up
// to 32768 sixteen; longer ones keep their keys in the workspace.
template <int D>
hipError_t evict_d(const KvView &c, const EvictPlan &p, const int32_t *next_pos, int keep, int recent, uint32_t *keys,
                   int32_t *moves, int32_t *counts, hipStream_t s) {
  const int rows = c.nseq * c.hkv;
  if (p.max_moves <= kFuseMoves) {
    if (p.len_cap <= 2048) return select_rows<256, 8, D>(c, p, next_pos, keep, recent, keys, moves, counts, s);
    if (p.len_cap <= 16384) return select_rows<1024, 16, D>(c, p, next_pos, keep, recent, keys, moves, counts, s);
  }
  hipError_t e = p.len_cap <= 2048    ? select_rows<256, 8, 0>(c, p, next_pos, keep, recent, keys, moves, counts, s)
                 : p.len_cap <= 16384 ? select_rows<1024, 16, 0>(c, p, next_pos, keep, recent, keys, moves, counts, s)
                 : p.len_cap <= kRegisterSlots ? select_rows<1024, 32, 0>(c, p, next_pos, keep, recent, keys, moves, counts, s)
                                      : select_rows<1024, 0, 0>(c, p, next_pos, keep, recent, keys, moves, counts, s);
  if (e != hipSuccess) return e;
  const int chunks = (int)std::min<int64_t>((p.max_moves + kMovesPerBlock - 1) / kMovesPerBlock, kMaxBlocks / rows);
  k_kv4_move<D><<<(unsigned)(rows * chunks), kMoveThreads, 0, s>>>(c, p, moves, counts, chunks);
  return hipGetLastError();
}

}  // namespace

EvictPlan kv4_evict_plan(const KvView &c, int keep, int max_len) {
  EvictPlan p{};
  p.len_cap = (int)std::min<int64_t>(max_len, (int64_t)c.mp * c.ps);
  p.max_moves = std::max(0, std::min(keep, p.len_cap - keep));
  const size_t rows = (size_t)c.nseq * c.hkv;
  auto round = [](size_t x) { return (x + 255) & ~(size_t)255; };
  p.key_off = 0;
  p.move_off = p.len_cap > kRegisterSlots ? round(rows * p.len_cap * 4) : 0;
  p.count_off = p.move_off + round(rows * 2 * p.max_moves * 4);
  p.bytes = p.max_moves > 0 ? p.count_off + round(rows * 4) : 0;
  return p;
}

hipError_t launch_kv4_evict(const KvView &c, const EvictPlan &p, const int32_t *next_pos, int keep, int recent,
                            void *ws, hipStream_t s) {
  char *w = static_cast<char *>(ws);
  uint32_t *keys = reinterpret_cast<uint32_t *>(w + p.key_off);
  int32_t *moves = reinterpret_cast<int32_t *>(w + p.move_off), *counts = reinterpret_cast<int32_t *>(w + p.count_off);
  if (c.d == 64) return evict_d<64>(c, p, next_pos, keep, recent, keys, moves, counts, s);
  if (c.d == 128) return evict_d<128>(c, p, next_pos, keep, recent, keys, moves, counts, s);
  return evict_d<256>(c, p, next_pos, keep, recent, keys, moves, counts, s);
}

}  // namespace vqmm
