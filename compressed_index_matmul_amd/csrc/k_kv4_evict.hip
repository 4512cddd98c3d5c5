// kv4_evict: cut each sequence and key/value head down to `keep` slots.
//
// k_kv4_select, one workgroup a sequence and head, finds the keep-th largest
// key by a radix search (four passes of 8 bits over keys that order as the
// weights do), splits its ties by slot, and lists the free slots below keep
// and the kept ones at or above it, both in ascending order; there are equally
// many.  k_kv4_move copies slot to slot, a wave a move: sources lie at or above
// keep and targets below it, so no copy reads what another writes.  Counts are
// integers and every list position is a prefix sum, so nothing depends on the
// order in which waves run.
//
// Bound: 8 bytes (weight, position) of every slot, then the moved slots twice.
#include "attn_device.h"

#include <algorithm>

namespace vqmm {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / kWave;
constexpr int kMoveThreads = 256;
constexpr int kMovesPerBlock = 16;

// Keys in the order of the weights: NaN lowest, the protected slots on top.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of a per-wave count over the workgroup's waves.
__device__ __forceinline__ int wave_prefix(int *s, int wave, int count) {
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[wave] = count;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < wave; ++i) before += s[i];
  return before;
}

__global__ __launch_bounds__(kSelThreads) void k_kv4_select(KvView c, EvictPlan p, const int32_t *__restrict__ next_pos,
                                                            int keep, int recent, uint32_t *__restrict__ keys_all,
                                                            int32_t *__restrict__ moves, int32_t *__restrict__ counts) {
  __shared__ int s_hist[kSelWaves][256];
  __shared__ int s_sum[256];
  __shared__ int s_wave[kSelWaves];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;

  const int row = blockIdx.x;
  const int b = row / c.hkv, kvh = row - b * c.hkv;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int len = min(max(c.lens[b], 0), p.len_cap);
  if (len <= keep) {
    if (tid == 0) counts[row] = 0;
    return;
  }
  uint32_t *keys = keys_all + (int64_t)row * p.len_cap;
  const int64_t oldest = (int64_t)next_pos[b] - recent;  // positions from here on are kept

  uint32_t prefix = 0;
  int need = keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < kSelWaves * 256; i += kSelThreads) (&s_hist[0][0])[i] = 0;
    __syncthreads();
    for (int slot = tid; slot < len; slot += kSelThreads) {
      uint32_t key;
      if (shift == 24) {
        const int pi = slot / c.ps;
        const int64_t at = (page_of(c, b, pi) * c.hkv + kvh) * c.ps + (slot - pi * c.ps);
        key = c.pos[at] >= oldest ? 0xffffffffu : weight_key(c.weights[at]);
        keys[slot] = key;
      } else {
        key = keys[slot];
      }
      if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&s_hist[wave][(key >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid < 256) {
      int n = 0;
#pragma unroll
      for (int w = 0; w < kSelWaves; ++w) n += s_hist[w][tid];
      s_sum[tid] = n;
    }
    __syncthreads();
    if (wave == 0) {  // digits from the top: the one that holds the need-th key
      int n[4], mine = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) n[i] = s_sum[255 - 4 * lane - i], mine += n[i];
      int upto = mine;  // inclusive prefix over the lanes
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(upto, o);
        if (lane >= o) upto += v;
      }
      int above = upto - mine;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (above < need && need <= above + n[i]) {
          s_prefix = prefix | (uint32_t)(255 - 4 * lane - i) << shift;
          s_need = need - above;
        }
        above += n[i];
      }
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    __syncthreads();
  }

  // a wave's run of slots: ties first, then the lists
  const int run = ((len + kSelWaves - 1) / kSelWaves + kWave - 1) / kWave * kWave;
  const int lo = min(wave * run, len), hi = min(lo + run, len);
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
  int ties = 0;
  for (int s0 = lo; s0 < hi; s0 += kWave) {
    const int slot = s0 + lane;
    ties += __popcll(__ballot(slot < hi && keys[slot] == prefix));
  }
  const int ties_before = wave_prefix(s_wave, wave, ties);
  int holes = 0, movers = 0, holes_at = 0, movers_at = 0;
  int32_t *to = moves + (int64_t)row * 2 * p.max_moves, *from = to + p.max_moves;
  for (int pass = 0; pass < 2; ++pass) {
    int t = ties_before, h = holes_at, m = movers_at;
    for (int s0 = lo; s0 < hi; s0 += kWave) {
      const int slot = s0 + lane;
      const bool in = slot < hi;
      const uint32_t key = in ? keys[slot] : 0u;
      const uint64_t tie = __ballot(in && key == prefix);
      const bool stays = in && (key > prefix || (key == prefix && t + __popcll(tie & below) < need));
      t += __popcll(tie);
      const uint64_t hole = __ballot(in && !stays && slot < keep), mover = __ballot(stays && slot >= keep);
      if (pass == 1) {
        if (in && !stays && slot < keep) to[h + __popcll(hole & below)] = slot;
        if (stays && slot >= keep) from[m + __popcll(mover & below)] = slot;
      }
      h += __popcll(hole);
      m += __popcll(mover);
    }
    if (pass == 0) {
      holes = h;
      movers = m;
      holes_at = wave_prefix(s_wave, wave, holes);
      movers_at = wave_prefix(s_wave, wave, movers);
      if (wave == kSelWaves - 1 && lane == 0) counts[row] = min(movers_at + movers, p.max_moves);
    }
  }
}

template <int D>
__global__ __launch_bounds__(kMoveThreads) void k_kv4_move(KvView c, EvictPlan p, const int32_t *__restrict__ moves,
                                                           const int32_t *__restrict__ counts, int chunks) {
  constexpr int DG = D / 32;
  const int row = blockIdx.x / chunks, chunk = blockIdx.x - row * chunks;
  const int b = row / c.hkv, kvh = row - b * c.hkv;
  const int n = counts[row], lane = threadIdx.x & 63;
  const int32_t *to = moves + (int64_t)row * 2 * p.max_moves, *from = to + p.max_moves;
  const int64_t code_head = (int64_t)c.ps * (D / 2), scale_head = (int64_t)c.ps * (DG * 2);
  for (int w = threadIdx.x >> 6; w < kMovesPerBlock; w += kMoveThreads / kWave) {
    const int i = chunk * kMovesPerBlock + w;
    if (i >= n) return;
    const int src = from[i], dst = to[i];
    const int sp = src / c.ps, dp = dst / c.ps;
    const int so = src - sp * c.ps, d_o = dst - dp * c.ps;
    const int64_t spage = page_of(c, b, sp), dpage = page_of(c, b, dp);
    uint8_t *sc = c.codes + (spage * 2 * c.hkv + kvh) * code_head, *dc = c.codes + (dpage * 2 * c.hkv + kvh) * code_head;
    uint16_t *ss = c.scales + (spage * 2 * c.hkv + kvh) * scale_head;
    uint16_t *ds = c.scales + (dpage * 2 * c.hkv + kvh) * scale_head;
    if (lane < D / 8)
      reinterpret_cast<uint32_t *>(dc + (int64_t)d_o * (D / 2))[lane] =
          reinterpret_cast<const uint32_t *>(sc + (int64_t)so * (D / 2))[lane];
    sc += c.hkv * code_head, dc += c.hkv * code_head;
    const int sb = (so & 3) == 1 ? 2 : (so & 3) == 2 ? 1 : so & 3, db = (d_o & 3) == 1 ? 2 : (d_o & 3) == 2 ? 1 : d_o & 3;
#pragma unroll
    for (int x = 0; x < D / 2; x += kWave)
      if (x + lane < D / 2)
        dc[(int64_t)(d_o >> 2) * (2 * D) + (x + lane) * 4 + db] = sc[(int64_t)(so >> 2) * (2 * D) + (x + lane) * 4 + sb];
    if (lane < 4 * DG) {  // (kind, group, step or minimum)
      const int kind = lane / (2 * DG), gs = lane % (2 * DG);
      const int64_t k0 = kind * c.hkv * scale_head;
      ds[k0 + (d_o >> 2) * (DG * 8) + gs * 4 + (d_o & 3)] = ss[k0 + (so >> 2) * (DG * 8) + gs * 4 + (so & 3)];
    }
    const int64_t sa = (spage * c.hkv + kvh) * c.ps + so, da = (dpage * c.hkv + kvh) * c.ps + d_o;
    if (lane == 62) c.weights[da] = c.weights[sa];
    if (lane == 63) c.pos[da] = c.pos[sa];
  }
}

}  // namespace

EvictPlan kv4_evict_plan(const KvView &c, int keep, int max_len) {
  EvictPlan p{};
  p.len_cap = (int)std::min<int64_t>(max_len, (int64_t)c.mp * c.ps);
  p.max_moves = std::max(0, std::min(keep, p.len_cap - keep));
  const size_t rows = (size_t)c.nseq * c.hkv;
  auto round = [](size_t x) { return (x + 255) & ~(size_t)255; };
  p.key_off = 0;
  p.move_off = round(rows * p.len_cap * 4);
  p.count_off = p.move_off + round(rows * 2 * p.max_moves * 4);
  p.bytes = p.max_moves > 0 ? p.count_off + round(rows * 4) : 0;
  return p;
}

hipError_t launch_kv4_evict(const KvView &c, const EvictPlan &p, const int32_t *next_pos, int keep, int recent,
                            void *ws, hipStream_t s) {
  char *w = static_cast<char *>(ws);
  uint32_t *keys = reinterpret_cast<uint32_t *>(w + p.key_off);
  int32_t *moves = reinterpret_cast<int32_t *>(w + p.move_off), *counts = reinterpret_cast<int32_t *>(w + p.count_off);
  const int rows = c.nseq * c.hkv;
  const int chunks = (p.max_moves + kMovesPerBlock - 1) / kMovesPerBlock;
  if ((int64_t)rows * chunks >= ((int64_t)1 << 31)) return hipErrorInvalidConfiguration;
  k_kv4_select<<<rows, kSelThreads, 0, s>>>(c, p, next_pos, keep, recent, keys, moves, counts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (c.d == 64) k_kv4_move<64><<<rows * chunks, kMoveThreads, 0, s>>>(c, p, moves, counts, chunks);
  else if (c.d == 128) k_kv4_move<128><<<rows * chunks, kMoveThreads, 0, s>>>(c, p, moves, counts, chunks);
  else k_kv4_move<256><<<rows * chunks, kMoveThreads, 0, s>>>(c, p, moves, counts, chunks);
  return hipGetLastError();
}

}  // namespace vqmm
