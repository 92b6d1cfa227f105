// Eviction from the paged cache by accumulated attention weight.
//
// The m best of n rows of a (sequence, key head) are those whose 33-bit key
// (protected, weight as an ordered integer) is above the m-th largest, and of
// those equal to it the lowest slots.  The m-th largest is found digit by digit
// (11 + 11 + 10 bits) with histograms in shared memory.  A cluster of blocks
// shares a head: each keeps the keys of its slots in shared memory, reads the
// weights once, adds up its share of the bins over all histograms by distributed
// shared memory, and reads the share that holds the rank from its owner, so the
// whole selection is one launch.
//
// Rows are not packed in their order: kept rows below slot m stay, and only
// those from m on move, into the slots given up below m.  Sources and targets are
// disjoint, so all moves run at once and as few bytes as possible are moved
// (about m (n - m) / n rows where the weights know no place, one row in a
// decoding step that evicts one).  With P(x) the number of kept rows below slot x,
// the target of rank x - P(x) is a given-up slot x, the source of rank P(x) -
// P(m) a kept slot x; both follow from counts of the rows above and at the
// threshold, so one scan writes both lists.
#include <cooperative_groups.h>

#include <algorithm>

#include "host.h"

namespace cg = cooperative_groups;

namespace lh {
namespace {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kBins = 2048;
constexpr int kAhead = 4;  // rows of 128 slots that a warp has in flight
constexpr int kMaxCluster = 8;
constexpr int kHists = 4;  // other and protected rows of the first digit, second, third
// Keys (4 bytes, and a byte for the protection of four) of a block's slots in
// shared memory; a block with more slots reads the weights again in every pass.
constexpr int kMaxKeys = 40960;
constexpr int kMoveThreads = 256;
// A head of one block whose moves are at most this many moves its rows itself.  The
// regular cut of a batch (64 heads of 2111 slots to 2048) takes 11.7 us in a graph,
// 0.2 more with a launch for the moves, and the call 18 us instead of 21.
constexpr int kFusedMoves = 256;

struct EvictCall {
  lh_cache c;
  int64_t budget, capacity, most;  // most: upper bound of the moves of a head
  const float* weights;
  const int32_t *positions, *protect;
  float* weights_out;
  int32_t *positions_out, *lengths_out;
  int32_t* count;               // [B * H] moves
  int32_t *from, *to;           // [B * H, most]
  float* moved_weight;          // [B * H, most]: the sources' weight and position,
  int32_t* moved_position;      // whose own entries are cleared; sources last first
  unsigned int* status;
  int page_shift;
  int keys;                     // slots whose keys fit the block's shared memory
  int row_chunks;               // 16-byte chunks of a row
  bool fused;                   // the selecting block moves the rows itself
};

// Larger weights have larger keys; a NaN has the smallest, -0 equals +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Moves the rows first, first + step, .. of a head's list: a group of row_chunks
// lanes a row, 16 bytes of key and value a lane.
// Neighbouring groups take neighbouring moves, so that DRAM pages stay open.  A
// move is a chain of three loads (slots, pages, rows): the first two of the next
// move are asked for while the rows of this one are on their way (98K cut to
// half, both launches in a graph: 74 us, 83 us without).  One move at a time and
// all the warps an SM holds do as well as two to four moves and fewer warps.
__device__ __forceinline__ void move_rows(const EvictCall& k, int64_t bh, int first, int step) {
  const int b = (int)(bh / k.c.H), h = (int)(bh % k.c.H);
  const int count = k.count[bh];
  const int32_t* const table = k.c.table + b * k.c.table_stride;
  const int32_t* const from = k.from + bh * k.most;
  const int32_t* const to = k.to + bh * k.most;
  const int mask = (1 << k.page_shift) - 1;
  const int lane = threadIdx.x & (k.row_chunks - 1);
  uint4* const keys = static_cast<uint4*>(k.c.k);
  uint4* const values = static_cast<uint4*>(k.c.v);
  int src = -1, dst = 0, ps = -1, pd = -1;
  auto ask = [&](int i) {  // moves are at most half the capacity: 32 bits hold their sums
    if (i >= count) return;
    src = from[count - 1 - i];
    dst = to[i];
    ps = table[src >> k.page_shift];
    pd = table[dst >> k.page_shift];
  };
  ask(first);
  for (int i = first; i < count; i += step) {
    uint4 kc, vc;
    int64_t ad = -1;
    if (ps >= 0 && ps < k.c.pages && pd >= 0 && pd < k.c.pages) {
      const int64_t as = ((((int64_t)ps * k.c.H + h) << k.page_shift) + (src & mask)) * k.row_chunks + lane;
      ad = ((((int64_t)pd * k.c.H + h) << k.page_shift) + (dst & mask)) * k.row_chunks + lane;
      kc = keys[as];
      vc = values[as];
    } else if (lane == 0) {
      atomicOr(k.status, kStatusPage);
    }
    if (lane == 0) {
      k.weights_out[bh * k.capacity + dst] = k.moved_weight[bh * k.most + count - 1 - i];
      if (k.positions_out) k.positions_out[bh * k.capacity + dst] = k.moved_position[bh * k.most + count - 1 - i];
    }
    ask(i + step);
    if (ad >= 0) {
      keys[ad] = kc;
      values[ad] = vc;
    }
  }
}

// A warp takes a run of its block's slots, 128 at a time, four neighbours a
// lane: wide loads and stores, and one scan by shuffles ranks 128 rows (ballots
// and population counts of single rows took longer).
// HELD: the block's keys are in shared memory; ANY: some rows are protected;
// POS: positions are given (template parameters, for a uniform branch in every
// row costs more than the row's arithmetic: 98K slots 43 us with branches).
template <bool HELD, bool ANY, bool POS>
__global__ void __launch_bounds__(kEvThreads, 2)
evict_select_kernel(const __grid_constant__ EvictCall k) {
  extern __shared__ __align__(16) uint32_t dyn[];
  uint32_t* const keys = dyn;                     // [k.keys]
  uint8_t* const prot = reinterpret_cast<uint8_t*>(dyn + k.keys);  // [k.keys / 4] bits of four slots
  __shared__ __align__(16) uint32_t hist[kHists][kBins];
  __shared__ __align__(16) uint32_t share[2][kBins / 2];  // this block's bins, summed over the cluster
  __shared__ uint32_t s_rows[2];            // rows of this block's share, by class
  __shared__ uint2 s_shares[kMaxCluster];   // and of each block's
  __shared__ uint2 s_counts[kMaxCluster];   // each block's rows above and at the threshold
  __shared__ uint2 s_warps[kEvWarps];       // each warp's
  __shared__ uint32_t s_tops[kEvWarps], s_digit, s_need;
  __shared__ uint32_t s_prot;               // this block's protected rows
  const cg::cluster_group cluster = cg::this_cluster();
  const int CS = cluster.num_blocks(), rank = cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t bh = blockIdx.x / CS;
  const int b = (int)(bh / k.c.H);
  const int raw = k.c.lengths[b];
  const int n = (int)max((int64_t)0, min((int64_t)raw, k.capacity));
  const int m = (int)min((int64_t)n, k.budget);
  const float* w = k.weights + bh * k.capacity;
  const int32_t* pos = k.positions + (POS ? bh * k.capacity : 0);
  float* wo = k.weights_out + bh * k.capacity;
  int32_t* po = k.positions_out + (POS ? bh * k.capacity : 0);
  const int from = ANY ? k.protect[b] : 0;
  cudaTriggerProgrammaticLaunchCompletion();
  if (tid == 0 && rank == 0) {
    if (bh % k.c.H == 0) {
      k.lengths_out[b] = m;
      if (raw != n) atomicOr(k.status, kStatusPage);
    }
    if (n == m) k.count[bh] = 0;
  }
  // Behind the rows there are.
  for (int64_t j = n + rank * kEvThreads + tid; j < k.capacity; j += CS * kEvThreads) {
    wo[j] = 0.f;
    if (POS) po[j] = -1;
  }
  // This block's slots lo .. hi - 1, and this warp's of them.
  const int chunk = (int)(((int64_t)n + CS * 128 - 1) / (CS * 128)) * 128;
  const int lo = (int)min((int64_t)n, (int64_t)rank * chunk), hi = min(n, lo + chunk);
  const int run = (chunk / 128 + kEvWarps - 1) / kEvWarps * 128;
  const int wlo = min(hi, lo + warp * run), whi = min(hi, wlo + run);
  if (n == m) {  // nothing to give up
    for (int j = wlo + lane; j < whi; j += 32) {
      wo[j] = w[j];
      if (POS) po[j] = pos[j];
    }
    return;
  }

  for (int x = 0; x < kHists; ++x) *reinterpret_cast<uint4*>(&hist[x][4 * tid]) = make_uint4(0, 0, 0, 0);
  if (tid < 2) s_rows[tid] = 0;
  if (tid == 2) s_prot = 0;
  __syncthreads();
  uint32_t mine = 0;  // protected rows of this thread
  // Weights and positions of this lane's four slots from j on.
  auto fetch = [&](int j, bool with_pos, float (&x)[4], int (&y)[4]) {
    if (j + 4 <= whi) {
      const float4 v = *reinterpret_cast<const float4*>(w + j);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
      if (POS && with_pos) {
        const int4 q = *reinterpret_cast<const int4*>(pos + j);
        y[0] = q.x; y[1] = q.y; y[2] = q.z; y[3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = j + i < whi ? w[j + i] : 0.f;
        if (POS && with_pos) y[i] = j + i < whi ? pos[j + i] : 0;
      }
    }
    if (!POS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = j + i;
    }
  };
  for (int base = wlo; base < whi; base += 128 * kAhead) {
    float x[kAhead][4];
    int y[kAhead][4];
#pragma unroll
    for (int r = 0; r < kAhead; ++r) fetch(base + 128 * r + 4 * lane, ANY, x[r], y[r]);
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
      if (base + 128 * r >= whi) break;
      const int j = base + 128 * r + 4 * lane;
      uint32_t key[4], bits = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        key[i] = weight_key(x[r][i]);
        if (ANY) bits |= (uint32_t)(y[r][i] >= from) << i;
      }
      if (j < whi) {
        if (HELD) {  // entries behind the last slot are never counted
          *reinterpret_cast<uint4*>(keys + j - lo) = make_uint4(key[0], key[1], key[2], key[3]);
          if (ANY) prot[(j - lo) >> 2] = (uint8_t)bits;
        }
        if (ANY) mine += __popc(bits & ((1u << min(4, whi - j)) - 1));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j + i < whi) atomicAdd(&hist[(bits >> i) & 1][key[i] >> 21], 1u);
      }
    }
  }
  if (ANY) {
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0 && mine) atomicAdd(&s_prot, mine);
  }
  // Keys and protection of the four slots from j on, in the passes behind.
  auto recall = [&](int j, uint32_t (&key)[4], uint32_t& bits) {
    if (HELD) {
      const uint4 v = *reinterpret_cast<const uint4*>(keys + j - lo);
      key[0] = v.x; key[1] = v.y; key[2] = v.z; key[3] = v.w;
      bits = ANY ? prot[(j - lo) >> 2] : 0;
    } else {
      float x[4];
      int y[4];
      fetch(j, ANY, x, y);
      bits = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        key[i] = weight_key(x[i]);
        if (ANY) bits |= (uint32_t)(y[i] >= from) << i;
      }
    }
  };
  // Digits of 11, 11 and 10 bits; need is the rank left inside the prefix.
  // Block r sums the r-th highest share of the bins; a thread takes four.
  uint32_t threshold = 0, mask = 0, need = m;
  bool active = false;  // the class (protected or not) that the threshold splits
  const int bins = CS == 1 ? kBins : (kBins + 4 * CS - 1) / (4 * CS) * 4;  // the lowest share may begin below bin 0
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    uint32_t* const level = pass == 0 ? hist[0] : hist[pass + 1];
    if (pass > 0) {
      for (int j = wlo + 4 * lane; j < whi; j += 128) {
        uint32_t key[4], right;  // bits of the class that is split
        recall(j, key, right);
        if (!active) right = ~right;
        right &= (1u << min(4, whi - j)) - 1;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((right >> i & 1) && (key[i] & mask) == threshold) atomicAdd(&level[(key[i] >> shift) & digits], 1u);
      }
    }
    if (CS > 1) cluster.sync();
    else __syncthreads();
    const int classes = pass == 0 && ANY ? 2 : 1;
    if (CS > 1 && tid < bins / 4) {
      const int at = kBins - bins * (rank + 1) + 4 * tid;
      for (int c = 0; c < classes; ++c) {
        uint32_t* const h = c == 1 ? hist[1] : level;
        uint4 v[kMaxCluster], all = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i)
          v[i] = i < CS && at >= 0 ? *reinterpret_cast<const uint4*>(cluster.map_shared_rank(h, i) + at) : all;
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i) {
          all.x += v[i].x;
          all.y += v[i].y;
          all.z += v[i].z;
          all.w += v[i].w;
        }
        *reinterpret_cast<uint4*>(&share[c][4 * tid]) = all;
        const int live = bins / 4 - (tid & ~31);  // threads of this warp with a part
        const uint32_t rows = __reduce_add_sync(live >= 32 ? ~0u : (1u << live) - 1, all.x + all.y + all.z + all.w);
        if (lane == 0) atomicAdd(&s_rows[c], rows);
      }
    }
    // The share that the rank lies in, and the rank in it.
    int owner = 0;
    if (CS > 1) {
      __syncthreads();
      if (tid < CS) cluster.map_shared_rank(s_shares, tid)[rank] = make_uint2(s_rows[0], s_rows[1]);
      cluster.sync();
      if (tid < 2) s_rows[tid] = 0;
      uint2 rows[kMaxCluster];
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) rows[i] = i < CS ? s_shares[i] : make_uint2(0, 0);
      if (ANY && pass == 0) {
        uint32_t all = 0;
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i) all += rows[i].y;
        active = all >= (uint32_t)m;
        need = active ? m : m - all;
      }
      bool found = false;
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) {
        const uint32_t here = ANY && pass == 0 && active ? rows[i].y : rows[i].x;
        found = found || need <= here || i >= CS - 1;
        if (!found) {
          need -= here;
          owner = i + 1;
        }
      }
    } else if (ANY && pass == 0) {
      active = s_prot >= (uint32_t)m;
      need = active ? m : m - s_prot;
    }
    const int cls = ANY && pass == 0 && active;
    const int top = bins - 4 - 4 * tid;  // the highest bins first
    uint4 v = make_uint4(0, 0, 0, 0);
    if (top >= 0) {
      uint32_t* const h = cls ? hist[1] : level;
      v = *reinterpret_cast<const uint4*>(CS > 1 ? cluster.map_shared_rank(share[cls], owner) + top : h + top);
    }
    const uint32_t four = v.x + v.y + v.z + v.w;
    uint32_t at = four;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    if (lane == 31) s_tops[warp] = at;
    __syncthreads();
    at -= four;
#pragma unroll
    for (int i = 0; i < kEvWarps; ++i) at += i < warp ? s_tops[i] : 0;
    const uint32_t a[4] = {v.w, v.z, v.y, v.x};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (at < need && need <= at + a[i]) {
        s_digit = kBins - bins * (owner + 1) + top + 3 - i;
        s_need = need - at;
      }
      at += a[i];
    }
    __syncthreads();
    threshold |= s_digit << shift;
    mask |= digits << shift;
    need = s_need;
  }
  // Kept are the rows above the threshold (all protected ones, where it splits
  // the others) and the first `need` of those at it.  Bits of the four slots.
  auto classify = [&](const uint32_t (&key)[4], uint32_t bits, int j, uint32_t& a, uint32_t& e) {
    const uint32_t valid = j < whi ? (1u << min(4, whi - j)) - 1 : 0;
    const uint32_t split = (active ? bits : ~bits) & valid;
    a = e = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a |= (uint32_t)(key[i] > threshold) << i;
      e |= (uint32_t)(key[i] == threshold) << i;
    }
    a = (a & split) | (active ? 0 : bits & valid);
    e &= split;
  };
  uint32_t above = 0, equal = 0;
#pragma unroll 2
  for (int j = wlo + 4 * lane; j < whi; j += 128) {
    uint32_t key[4], bits, a, e;
    recall(j, key, bits);
    classify(key, bits, j, a, e);
    above += __popc(a);
    equal += __popc(e);
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) s_warps[warp] = make_uint2(above, equal);
  __syncthreads();
  above = equal = 0;
  uint2 sum = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < kEvWarps; ++i) {
    const uint2 x = s_warps[i];
    above += i < warp ? x.x : 0;
    equal += i < warp ? x.y : 0;
    sum.x += x.x;
    sum.y += x.y;
  }
  if (CS > 1) {
    // Told to every block, so that none reads another's memory from here on.
    if (tid < CS) cluster.map_shared_rank(s_counts, tid)[rank] = sum;
    cluster.sync();
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i) {
      above += i < rank ? s_counts[i].x : 0;
      equal += i < rank ? s_counts[i].y : 0;
    }
  }
  int32_t* const to = k.to + bh * k.most;
  int32_t* const src = k.from + bh * k.most;
  float* const mw = k.moved_weight + bh * k.most;
  // 2 KB of the histograms, which no one reads any more, for each warp.
  static_assert(sizeof(hist) >= kEvWarps * 2048, "three lists of 128 entries a warp");
  int* const b_slot = reinterpret_cast<int*>(&hist[0][0]) + warp * 512;
  float* const b_weight = reinterpret_cast<float*>(b_slot + 128);
  int* const b_pos = b_slot + 256;
  int32_t* const mp = k.moved_position + bh * k.most;
  for (int base = wlo; base < whi; base += 128 * kAhead) {
    float x[kAhead][4];
    int y[kAhead][4];
#pragma unroll
    for (int r = 0; r < kAhead; ++r) fetch(base + 128 * r + 4 * lane, true, x[r], y[r]);
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
      if (base + 128 * r >= whi) break;  // a step's few rows: no more than there are
      const int j = base + 128 * r + 4 * lane;
      uint32_t key[4], bits = 0, a, e;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        key[i] = weight_key(x[r][i]);
        if (ANY) bits |= (uint32_t)(y[r][i] >= from) << i;
      }
      classify(key, bits, j, a, e);
      const uint32_t both = __popc(a) | __popc(e) << 16;
      uint32_t sum = both;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const uint32_t all = __shfl_sync(0xffffffffu, sum, 31);
      sum -= both;
      const uint32_t eq = equal + (sum >> 16);
      const int kept_before = (int)(above + (sum & 0xffff) + min(need, eq));
      const int row_kept = (int)(above + min(need, equal));  // rows kept before this row of 128
      above += all & 0xffff;
      equal += all >> 16;
      uint32_t kept = a;
      if (__any_sync(0xffffffffu, e != 0)) {  // rare: rows at the threshold
        uint32_t x = eq;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (e >> i & 1) {
            if (x < need) kept |= 1u << i;
            ++x;
          }
        }
      }
      const int row = base + 128 * r;
      if (row + 128 <= whi && (row + 128 <= m || row >= m)) {
        // A full row on one side of m.  Its entries are gathered in shared memory and
        // stored side by side: a lane's own 4-byte stores would touch each sector of
        // a list several times.
        const bool low = row < m;
        const uint32_t mine = low ? ~kept & 15u : kept;
        int at = low ? (j - row) - (kept_before - row_kept) : kept_before - row_kept;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (mine >> i & 1) {
            b_slot[at] = j + i;
            if (!low) {
              b_weight[at] = x[r][i];
              if (POS) b_pos[at] = y[r][i];
            }
            ++at;
          }
        }
        __syncwarp();
        const int moved = (int)(above + min(need, equal)) - row_kept;
        if (low) {
          for (int t = lane; t < 128 - moved; t += 32) to[row - row_kept + t] = b_slot[t];
          *reinterpret_cast<float4*>(wo + j) = make_float4(x[r][0], x[r][1], x[r][2], x[r][3]);
          if (POS) *reinterpret_cast<int4*>(po + j) = make_int4(y[r][0], y[r][1], y[r][2], y[r][3]);
        } else {
          if (row == m && lane == 0) k.count[bh] = m - row_kept;
          for (int t = lane; t < moved; t += 32) {
            const int to_last = m - 1 - row_kept - t;
            src[to_last] = b_slot[t];
            mw[to_last] = b_weight[t];
            if (POS) mp[to_last] = b_pos[t];
          }
          *reinterpret_cast<float4*>(wo + j) = make_float4(0.f, 0.f, 0.f, 0.f);
          if (POS) *reinterpret_cast<int4*>(po + j) = make_int4(-1, -1, -1, -1);
        }
        __syncwarp();
      } else if (j < whi) {
        const uint32_t valid = (1u << min(4, whi - j)) - 1;
        const uint32_t low = j + 4 <= m ? 15u : j >= m ? 0u : (1u << (m - j)) - 1;  // slots below m
        if (m >= j && m < j + 4 && m < whi) k.count[bh] = m - kept_before - __popc(kept & low);
        const uint32_t holes = ~kept & low & valid;  // their weights are written by the move
        if (holes) {
          int32_t* const p = to + (j - kept_before);
          if (holes & 1) p[0] = j;
          if (holes & 2) p[holes & 1] = j + 1;
          if (holes & 4) p[__popc(holes & 3)] = j + 2;
          if (holes & 8) p[__popc(holes & 7)] = j + 3;
        }
        const uint32_t moving = kept & ~low;
        if (moving) {
          const int last = m - 1 - kept_before - __popc(kept & low);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (moving >> i & 1) {
              const int at = last - __popc(moving & ((1u << i) - 1));
              src[at] = j + i;
              mw[at] = x[r][i];
              if (POS) mp[at] = y[r][i];
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[r][i] = (low >> i & 1) ? x[r][i] : 0.f;
          y[r][i] = (low >> i & 1) ? y[r][i] : -1;
        }
        if (j + 4 <= whi) {
          *reinterpret_cast<float4*>(wo + j) = make_float4(x[r][0], x[r][1], x[r][2], x[r][3]);
          if (POS) *reinterpret_cast<int4*>(po + j) = make_int4(y[r][0], y[r][1], y[r][2], y[r][3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (j + i < whi) {
              wo[j + i] = x[r][i];
              if (POS) po[j + i] = y[r][i];
            }
          }
        }
      }
    }
  }
  if (k.fused) {  // a cluster of one
    __syncthreads();
    move_rows(k, bh, tid / k.row_chunks, kEvThreads / k.row_chunks);
  }
}

// The moves of the other calls, each row by as many lanes as it has 16-byte chunks.
__global__ void __launch_bounds__(kMoveThreads, 7)
evict_move_kernel(const __grid_constant__ EvictCall k) {
  cudaGridDependencySynchronize();
  const int groups = kMoveThreads / k.row_chunks;
  move_rows(k, blockIdx.y, (int)blockIdx.x * groups + threadIdx.x / k.row_chunks, (int)gridDim.x * groups);
}

template <bool HELD>
auto select_kernel(const void* protect, const void* positions) {
  if (protect) return positions ? evict_select_kernel<HELD, true, true> : evict_select_kernel<HELD, true, false>;
  return positions ? evict_select_kernel<HELD, false, true> : evict_select_kernel<HELD, false, false>;
}

int64_t most_moves(const lh_cache& c, int64_t budget) {
  const int64_t capacity = (int64_t)c.width * c.page;
  return std::max<int64_t>(0, std::min(budget, capacity - budget));
}

}  // namespace

int64_t evict_ws_bytes(const lh_cache& c, int64_t budget) {
  const int64_t bh = (int64_t)c.B * c.H;
  return ((bh * 4 + 255) & ~int64_t(255)) + 4 * ((bh * most_moves(c, budget) * 4 + 255) & ~int64_t(255));
}

cudaError_t launch_evict(const lh_cache& c, int64_t budget, const float* weights,
                         const int32_t* positions, const int32_t* protect, float* weights_out,
                         int32_t* positions_out, int32_t* lengths_out, void* ws, cudaStream_t st) {
  const int64_t bh = (int64_t)c.B * c.H;
  EvictCall k{};
  k.c = c;
  k.budget = budget;
  k.capacity = (int64_t)c.width * c.page;
  k.most = most_moves(c, budget);
  k.weights = weights;
  k.positions = positions;
  k.protect = protect;
  k.weights_out = weights_out;
  k.positions_out = positions_out;
  k.lengths_out = lengths_out;
  char* p = static_cast<char*>(ws);
  const int64_t list = (bh * k.most * 4 + 255) & ~int64_t(255);
  k.count = reinterpret_cast<int32_t*>(p);
  p += (bh * 4 + 255) & ~int64_t(255);
  k.from = reinterpret_cast<int32_t*>(p);
  k.to = reinterpret_cast<int32_t*>(p + list);
  k.moved_weight = reinterpret_cast<float*>(p + 2 * list);
  k.moved_position = reinterpret_cast<int32_t*>(p + 3 * list);
  k.status = device_status_ptr();
  if (!k.status) return cudaErrorInvalidSymbol;
  k.page_shift = __builtin_ctz(c.page);
  k.row_chunks = c.d * (c.dtype == LH_BF16 ? 2 : 4) / 16;
  // Blocks of a head: one up to 4096 slots (8 heads of them: 12.6 us in a graph, 15.9 in
  // two), behind that one for each 2048, as many as leave every block an SM of its own
  // (kFit: clusters of one to eight that stand side by side, for none spans two parts of
  // the GPU).  16 heads of 98K slots, both launches in a graph: 71 us with six blocks a
  // head, 72 with four, 77 with eight and 84 with seven (two on some SMs); 32 heads of
  // 32K slots, few to move: 26 us with four, 33 with two.
  constexpr int kFit[kMaxCluster + 1] = {0, 148, 74, 45, 33, 26, 22, 15, 15};
  int cs = k.capacity > 4096 ? kMaxCluster : 1;
  while (cs > 1 && (bh > kFit[cs] || k.capacity <= (int64_t)(cs - 1) * 2048)) --cs;
  k.fused = cs == 1 && k.most <= kFusedMoves;
  const int64_t chunk = (k.capacity + cs * 128 - 1) / (cs * 128) * 128;
  k.keys = chunk <= kMaxKeys ? (int)chunk : 0;
  const size_t smem = (size_t)k.keys * 4 + k.keys / 4;
  auto select = k.keys ? select_kernel<true>(protect, positions) : select_kernel<false>(protect, positions);
  cudaError_t e = cudaSuccess;
  if (smem > 4096)  // beside the 41 KB of histograms, more than a block has without asking
    e = cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKeys * 4 + kMaxKeys / 4);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2]{};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(bh * cs));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, select, k);
  if (e != cudaSuccess || k.most == 0 || k.fused) return e;
  const int64_t groups = kMoveThreads / k.row_chunks;
  cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>((k.most + groups - 1) / groups, std::max<int64_t>(1, 148 * 16 / bh)),
                     (unsigned)bh);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = st;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr + 1;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, k);
}

}  // namespace lh
