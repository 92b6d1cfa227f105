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
#include "rotary.cuh"

namespace cg = cooperative_groups;

namespace lh {
namespace {

constexpr int kEvThreads = 512;
constexpr int kBins = 2048;
constexpr int kPerThread = 8;
constexpr int kSweep = kEvThreads * kPerThread;  // slots of one step of the scan
constexpr int kMaxCluster = 8;
constexpr int kHists = 4;  // other and protected rows of the first digit, second, third
// Keys (4 bytes) and protection bits of a block's slots in shared memory; a
// block with more slots reads the weights again in every pass.
constexpr int kMaxKeys = 40960;

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
  int32_t* moved_position;      // whose own entries the scan clears; sources last first
  unsigned int* status;
  int page_shift;
  int keys;                     // slots whose keys fit the block's shared memory
};

// Larger weights have larger keys; a NaN has the smallest, -0 equals +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sums of the values of the threads before this one, and of all.
template <typename V>
__device__ __forceinline__ V scan_excl(V v, V* warp_sums, V* total) {
  constexpr int NW = kEvThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  V w = lane < NW ? warp_sums[lane] : 0;  // every warp adds up the warps for itself
#pragma unroll
  for (int o = 1; o < NW; o <<= 1) {
    const V y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, NW - 1);
  const V before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  __syncthreads();
  return (warp == 0 ? 0 : before) + x - v;
}

__global__ void __launch_bounds__(kEvThreads, 2)
evict_select_kernel(const __grid_constant__ EvictCall k) {
  extern __shared__ __align__(16) uint32_t dyn[];
  uint32_t* const keys = dyn;                     // [k.keys]
  uint32_t* const bits = dyn + k.keys;            // [k.keys / 32] protected
  __shared__ __align__(16) uint32_t hist[kHists][kBins];
  __shared__ __align__(16) uint32_t share[2][kBins / 2];  // this block's bins, summed over the cluster
  __shared__ unsigned long long warp_sums[kEvThreads / 32];
  __shared__ unsigned long long s_shares[kMaxCluster];  // rows of each block's share, both classes
  __shared__ uint2 s_counts[kMaxCluster];  // each block's rows above and at the threshold
  __shared__ uint32_t s_digit, s_need;
  const cg::cluster_group cluster = cg::this_cluster();
  const int CS = cluster.num_blocks(), rank = cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t bh = blockIdx.x / CS;
  const int b = (int)(bh / k.c.H);
  const int raw = k.c.lengths[b];
  const int n = (int)max((int64_t)0, min((int64_t)raw, k.capacity));
  const int m = (int)min((int64_t)n, k.budget);
  const float* w = k.weights + bh * k.capacity;
  const int32_t* pos = k.positions ? k.positions + bh * k.capacity : nullptr;
  float* wo = k.weights_out + bh * k.capacity;
  int32_t* po = k.positions_out ? k.positions_out + bh * k.capacity : nullptr;
  const bool any = k.protect != nullptr;
  const int from = any ? k.protect[b] : 0;
  cudaTriggerProgrammaticLaunchCompletion();
  if (tid == 0 && rank == 0) {
    if (bh % k.c.H == 0) {
      k.lengths_out[b] = m;
      if (raw != n) atomicOr(k.status, kStatusPage);
    }
    if (n == m) k.count[bh] = 0;
  }
  // This block's slots lo .. hi - 1.
  const int chunk = (int)(((int64_t)n + CS * 32 - 1) / (CS * 32)) * 32;
  const int lo = (int)min((int64_t)n, (int64_t)rank * chunk), hi = min(n, lo + chunk);
  const bool held = chunk <= k.keys;

  // Weights and positions of the kPerThread slots from j on (j a multiple of it).
  // The loads of a step are asked for before the step before is worked on; a
  // block writes only slots that it has read.
  float wv[kPerThread];
  int32_t pv[kPerThread];
  auto fetch = [&](int j) {
#pragma unroll
    for (int q = 0; q < kPerThread; q += 4) {
      if (j + q + 4 <= hi) {
        const float4 x = *reinterpret_cast<const float4*>(w + j + q);
        wv[q] = x.x; wv[q + 1] = x.y; wv[q + 2] = x.z; wv[q + 3] = x.w;
        if (pos) {
          const int4 y = *reinterpret_cast<const int4*>(pos + j + q);
          pv[q] = y.x; pv[q + 1] = y.y; pv[q + 2] = y.z; pv[q + 3] = y.w;
        }
      } else {
#pragma unroll
        for (int i = q; i < q + 4; ++i) {
          wv[i] = j + i < hi ? w[j + i] : 0.f;
          pv[i] = pos && j + i < hi ? pos[j + i] : 0;
        }
      }
    }
    if (!pos) {
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) pv[i] = j + i;
    }
  };
  uint32_t threshold = 0, need = 0;
  bool active = false;  // the class (protected or not) that the threshold splits
  uint32_t above = 0, equal = 0;  // rows above and at the threshold before this block's
  if (n > m) {
    fetch(lo + tid * kPerThread);
    for (int x = 0; x < kHists; ++x)
      *reinterpret_cast<uint4*>(&hist[x][4 * tid]) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int base = lo; base < hi; base += kSweep) {
      const int j = base + tid * kPerThread;
      uint32_t key[kPerThread], mine = 0;
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) {
        key[i] = weight_key(wv[i]);
        mine |= (uint32_t)(any && pv[i] >= from) << i;
      }
      fetch(j + kSweep);
      if (j < hi) {
        if (held) {  // entries behind hi are never counted
#pragma unroll
          for (int q = 0; q < kPerThread; q += 4)
            *reinterpret_cast<uint4*>(keys + j - lo + q) = make_uint4(key[q], key[q + 1], key[q + 2], key[q + 3]);
        }
#pragma unroll
        for (int i = 0; i < kPerThread; ++i)
          if (j + i < hi) atomicAdd(&hist[(mine >> i) & 1][key[i] >> 21], 1u);
      }
      if (held && any) {  // four lanes' bits make a word
        uint32_t word = mine << (8 * (lane & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 1);
        word |= __shfl_xor_sync(0xffffffffu, word, 2);
        if ((lane & 3) == 0 && j < hi) bits[(j - lo) >> 5] = word;
      }
    }
    // Digits of 11, 11 and 10 bits; need is the rank left inside the prefix.
    // Block r sums the r-th highest share of the bins; a thread takes four.
    uint32_t mask = 0, mine_above = 0, mine_equal = 0;
    unsigned long long mine_total;
    const int bins = kBins / CS;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digits = pass == 2 ? 1023u : 2047u;
      if (pass > 0) {
        for (int base = lo; base < hi; base += kEvThreads * 4) {
          const int j = base + tid * 4;
          if (j < hi) {
            uint32_t key[4], prot;
            const int left = hi - j;
            if (held) {
              const uint4 x = *reinterpret_cast<const uint4*>(keys + j - lo);
              key[0] = x.x; key[1] = x.y; key[2] = x.z; key[3] = x.w;
              prot = any ? bits[(j - lo) >> 5] >> ((j - lo) & 31) : 0;
            } else {
              prot = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                key[i] = j + i < hi ? weight_key(w[j + i]) : 0;
                prot |= (uint32_t)(any && j + i < hi && (pos ? pos[j + i] : j + i) >= from) << i;
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((key[i] & mask) == threshold && i < left && ((prot >> i) & 1) == (uint32_t)active)
                atomicAdd(&hist[pass + 1][(key[i] >> shift) & digits], 1u);
          }
        }
      }
      cluster.sync();
      const int classes = pass == 0 && any ? 2 : 1;
      unsigned long long sum = 0, total;
      if (tid < bins / 4) {
        const int at = kBins - bins * (rank + 1) + 4 * tid;
        for (int c = 0; c < classes; ++c) {
          uint32_t* const h = pass == 0 ? hist[c] : hist[pass + 1];
          uint4 v[kMaxCluster], all = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < kMaxCluster; ++i)
            v[i] = i < CS ? *reinterpret_cast<const uint4*>(cluster.map_shared_rank(h, i) + at) : all;
#pragma unroll
          for (int i = 0; i < kMaxCluster; ++i) {
            all.x += v[i].x;
            all.y += v[i].y;
            all.z += v[i].z;
            all.w += v[i].w;
          }
          if (CS > 1) *reinterpret_cast<uint4*>(&share[c][4 * tid]) = all;
          sum += (unsigned long long)(all.x + all.y + all.z + all.w) << (32 * c);
        }
      }
      scan_excl(sum, warp_sums, &total);
      if (tid < CS) cluster.map_shared_rank(s_shares, tid)[rank] = total;
      cluster.sync();
      if (pass == 0) {
        uint32_t prot = 0;
        for (int i = 0; i < CS; ++i) prot += (uint32_t)(s_shares[i] >> 32);
        active = prot >= (uint32_t)m;
        need = active ? m : m - prot;
      }
      // The share that the rank lies in, and the bin in it.
      const int cls = pass == 0 && active;
      int owner = 0;
      for (; owner < CS - 1; ++owner) {
        const uint32_t rows = (uint32_t)(s_shares[owner] >> (32 * cls));
        if (need <= rows) break;
        need -= rows;
      }
      const int top = bins - 4 - 4 * tid;  // the highest bins first
      uint4 v = make_uint4(0, 0, 0, 0);
      uint32_t* const own = pass == 0 ? hist[cls] : hist[pass + 1];
      if (top >= 0)
        v = *reinterpret_cast<const uint4*>(CS > 1 ? cluster.map_shared_rank(share[cls], owner) + top : own + top);
      uint32_t at = (uint32_t)scan_excl((unsigned long long)(v.x + v.y + v.z + v.w), warp_sums, &total);
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
      const uint32_t digit = s_digit;
      need = s_need;
      threshold |= digit << shift;
      mask |= digits << shift;
      // This block's own rows above the digit.
      const uint4 o = *reinterpret_cast<const uint4*>(own + 4 * tid);
      const uint32_t ov[4] = {o.x, o.y, o.z, o.w};
      uint32_t more = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) more += 4 * tid + i > (int)digit ? ov[i] : 0;
      if (pass == 0 && any && !active) {  // the protected ones are above all others
        const uint4 q = *reinterpret_cast<const uint4*>(hist[1] + 4 * tid);
        more += q.x + q.y + q.z + q.w;
      }
      mine_above += more;
      if (pass == 2) mine_equal = own[digit];
    }
    scan_excl((unsigned long long)mine_above, warp_sums, &mine_total);
    // Told to every block, so that none reads another's memory from here on.
    if (tid < CS) cluster.map_shared_rank(s_counts, tid)[rank] = make_uint2((uint32_t)mine_total, mine_equal);
    cluster.sync();
    for (int i = 0; i < rank; ++i) {
      above += s_counts[i].x;
      equal += s_counts[i].y;
    }
  }
  // One scan in slot order over rows above the threshold (low half of a word)
  // and at it (high half); kept are the former and the first `need` of the
  // latter.
  fetch(lo + tid * kPerThread);
  for (int base = lo; base < hi; base += kSweep) {
    const int j0 = base + tid * kPerThread;
    // Bits of the thread's rows that are kept whatever the ties, and of those at
    // the threshold.
    uint32_t sure = 0, tied = 0;
    float x[kPerThread];
    int32_t y[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      x[i] = wv[i];
      y[i] = pv[i];
      const uint32_t key = weight_key(x[i]);
      const bool p = any && y[i] >= from;
      const bool split = p == active;
      sure |= (uint32_t)(split ? key > threshold : p) << i;
      tied |= (uint32_t)(split && key == threshold) << i;
    }
    const uint32_t valid = j0 >= hi ? 0u : (1u << min(kPerThread, hi - j0)) - 1;
    if (n == m) sure = valid, tied = 0;
    sure &= valid;
    tied &= valid;
    fetch(j0 + kSweep);
    unsigned long long total;
    const uint32_t run =
        (uint32_t)scan_excl((unsigned long long)(__popc(sure) | __popc(tied) << 16), warp_sums, &total);
    const uint32_t eq = equal + (run >> 16);
    uint32_t kept = sure;
    for (uint32_t t = tied, e = eq; t && e < need; t &= t - 1, ++e) kept |= t & -t;
    const int before = (int)(above + (run & 0xffff) + min(need, eq));  // rows kept below slot j0
    const uint32_t below = m <= j0 ? 0u : m - j0 >= kPerThread ? valid : (1u << (m - j0)) - 1;  // slots below m
    if (m >= j0 && m < j0 + kPerThread && m < hi) k.count[bh] = m - (before + __popc(kept & below));
    for (uint32_t t = valid & below & ~kept; t; t &= t - 1) {
      const int i = __ffs(t) - 1;
      k.to[bh * k.most + (j0 + i - before - __popc(kept & ((1u << i) - 1)))] = j0 + i;
    }
    if (kept & ~below) {
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) {
        if ((kept & ~below) >> i & 1) {
          const int64_t at = bh * k.most + (m - 1 - before - __popc(kept & ((1u << i) - 1)));
          k.from[at] = j0 + i;
          k.moved_weight[at] = x[i];
          if (po) k.moved_position[at] = y[i];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {  // a given-up slot below m is written by the move
      x[i] = (below >> i) & 1 ? x[i] : 0.f;
      y[i] = (below >> i) & 1 ? y[i] : -1;
    }
#pragma unroll
    for (int q = 0; q < kPerThread; q += 4) {
      if (j0 + q + 4 <= hi) {
        *reinterpret_cast<float4*>(wo + j0 + q) = make_float4(x[q], x[q + 1], x[q + 2], x[q + 3]);
        if (po) *reinterpret_cast<int4*>(po + j0 + q) = make_int4(y[q], y[q + 1], y[q + 2], y[q + 3]);
      } else {
#pragma unroll
        for (int i = q; i < q + 4; ++i) {
          if (j0 + i < hi) {
            wo[j0 + i] = x[i];
            if (po) po[j0 + i] = y[i];
          }
        }
      }
    }
    above += (uint32_t)total & 0xffff;
    equal += (uint32_t)total >> 16;
  }
  for (int64_t j = n + rank * kEvThreads + tid; j < k.capacity; j += CS * kEvThreads) {
    wo[j] = 0.f;
    if (po) po[j] = -1;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2)
evict_move_kernel(const __grid_constant__ EvictCall k) {
  constexpr int L = D / 8;  // lanes of a row
  const int64_t bh = blockIdx.y;
  const int b = (int)(bh / k.c.H), h = (int)(bh % k.c.H);
  cudaGridDependencySynchronize();
  const int count = k.count[bh];
  const int32_t* table = k.c.table + b * k.c.table_stride;
  const int mask = (1 << k.page_shift) - 1;
  const int lane = threadIdx.x % L;
  constexpr int R = 4;  // rows of a thread in flight
  const int64_t list = bh * k.most;
  const int64_t step = (int64_t)gridDim.x * (256 / L);
  for (int64_t i0 = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L; i0 < count; i0 += R * step) {
    Chunk<T> kc[R], vc[R];
    int64_t to[R];
    // Indexes, pages, rows: each kind is asked for R at a time, so that a chain of
    // three loads serves R rows.
    int src[R], dst[R];
#pragma unroll
    for (int x = 0; x < R; ++x) {
      const int64_t i = i0 + x * step;
      src[x] = i < count ? k.from[list + count - 1 - i] : -1;
      dst[x] = i < count ? k.to[list + i] : 0;
    }
    int ps[R], pd[R];
#pragma unroll
    for (int x = 0; x < R; ++x) {
      ps[x] = src[x] >= 0 ? table[src[x] >> k.page_shift] : -1;
      pd[x] = src[x] >= 0 ? table[dst[x] >> k.page_shift] : -1;
    }
#pragma unroll
    for (int x = 0; x < R; ++x) {
      const bool good = ps[x] >= 0 && ps[x] < k.c.pages && pd[x] >= 0 && pd[x] < k.c.pages;
      to[x] = -1;
      if (good) {
        const int64_t as = ((((int64_t)ps[x] * k.c.H + h) << k.page_shift) + (src[x] & mask)) * D + lane * 8;
        to[x] = ((((int64_t)pd[x] * k.c.H + h) << k.page_shift) + (dst[x] & mask)) * D + lane * 8;
        kc[x].load(static_cast<const T*>(k.c.k) + as);
        vc[x].load(static_cast<const T*>(k.c.v) + as);
      } else if (src[x] >= 0 && lane == 0) {
        atomicOr(k.status, kStatusPage);
      }
    }
    if (lane < R && i0 + lane * step < count) {  // lane x moves row x's weight and position
      const int64_t i = i0 + lane * step;
      const int slot = k.to[list + i];
      k.weights_out[bh * k.capacity + slot] = k.moved_weight[list + count - 1 - i];
      if (k.positions_out) k.positions_out[bh * k.capacity + slot] = k.moved_position[list + count - 1 - i];
    }
#pragma unroll
    for (int x = 0; x < R; ++x) {
      if (to[x] < 0) continue;
      kc[x].store(static_cast<T*>(k.c.k) + to[x]);
      vc[x].store(static_cast<T*>(k.c.v) + to[x]);
    }
  }
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
  // Blocks of a head: one for each 4096 slots, as long as the GPU has room for
  // all of them at once.
  int cs = 1;
  while (cs < kMaxCluster && k.capacity > (int64_t)cs * 4096 && bh * cs * 2 <= 148 * 2) cs *= 2;
  const int64_t chunk = (k.capacity + cs * 32 - 1) / (cs * 32) * 32;
  k.keys = chunk <= kMaxKeys ? (int)chunk : 0;
  const size_t smem = (size_t)k.keys * 4 + k.keys / 8;
  cudaError_t e = cudaSuccess;
  if (smem > 8192)  // beside the histograms' 32 KB, more than a block has without asking
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxKeys * 4 + kMaxKeys / 8);
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
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, k);
  if (e != cudaSuccess || k.most == 0) return e;
  with_type_dim(c.dtype, c.d, [&]<typename T, int D>() {
    const int64_t rows = 256 / (D / 8);
    cfg = cudaLaunchConfig_t{};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>((k.most + rows - 1) / rows, std::max<int64_t>(1, 148 * 16 / bh)),
                       (unsigned)bh);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr + 1;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, evict_move_kernel<T, D>, k);
  });
  return e;
}

}  // namespace lh
