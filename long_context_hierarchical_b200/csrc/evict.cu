// Eviction from the paged cache by accumulated attention weight.
//
// The m best of n rows of a (sequence, key head) are those whose 33-bit key
// (protected, weight as an ordered integer) is above the m-th largest, and of
// those equal to it the lowest slots.  The m-th largest is found digit by digit
// (11 + 11 + 10 bits) with histograms in shared memory.  A cluster of blocks
// shares a head: each keeps the keys of its slots in shared memory, reads the
// weights once, and adds up the others' histograms and counts over distributed
// shared memory, so the whole selection is one launch.
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

constexpr int kEvThreads = 1024;
constexpr int kBins = 2048;
constexpr int kPerThread = 4;
constexpr int kSweep = kEvThreads * kPerThread;  // slots of one step of the scan
constexpr int kMaxCluster = 8;
constexpr int kHists = 4;  // protected and other rows of the first digit, second, third
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
  int32_t* moved_position;      // whose own entries the scan clears
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

__device__ __forceinline__ uint32_t scan_excl(uint32_t v, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const uint32_t before = warp == 0 ? 0 : warp_sums[warp - 1];
  *total = warp_sums[31];
  __syncthreads();
  return before + x - v;
}

struct Counts {
  uint32_t above, equal, above_m, equal_m;  // of a block's slots, and of those below m
};

__global__ void __launch_bounds__(kEvThreads)
evict_select_kernel(const __grid_constant__ EvictCall k) {
  extern __shared__ uint32_t dyn[];
  uint32_t* const keys = dyn;                     // [k.keys]
  uint32_t* const bits = dyn + k.keys;            // [k.keys / 32] protected
  __shared__ uint32_t hist[kHists][kBins];
  __shared__ uint32_t warp_sums[32];
  __shared__ uint32_t s_digit, s_need;
  __shared__ Counts s_counts;
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
  const int lo = min(n, rank * chunk), hi = min(n, lo + chunk);
  const bool held = chunk <= k.keys;

  // Key and class of the four slots from j on (j a multiple of 4).
  auto fetch = [&](int j, float (&wv)[4], int32_t (&pv)[4]) {
    if (j + 4 <= hi) {
      const float4 x = *reinterpret_cast<const float4*>(w + j);
      wv[0] = x.x; wv[1] = x.y; wv[2] = x.z; wv[3] = x.w;
      if (pos) {
        const int4 y = *reinterpret_cast<const int4*>(pos + j);
        pv[0] = y.x; pv[1] = y.y; pv[2] = y.z; pv[3] = y.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wv[i] = j + i < hi ? w[j + i] : 0.f;
        if (pos) pv[i] = j + i < hi ? pos[j + i] : 0;
      }
    }
    if (!pos) {
#pragma unroll
      for (int i = 0; i < 4; ++i) pv[i] = j + i;
    }
  };
  uint32_t threshold = 0, need = 0;
  bool active = false;  // the class (protected or not) that the threshold splits
  if (n > m) {
    for (int x = 0; x < kHists; ++x)
      for (int i = tid; i < kBins; i += kEvThreads) hist[x][i] = 0;
    __syncthreads();
    for (int base = lo; base < hi; base += kSweep) {
      const int j = base + tid * 4;
      float wv[4];
      int32_t pv[4];
      uint32_t mine = 0;
      if (j < hi) {
        fetch(j, wv, pv);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t key = weight_key(wv[i]);
          const bool p = any && pv[i] >= from;
          mine |= (uint32_t)p << i;
          if (held) keys[j - lo + i] = key;  // entries behind hi are never read
          if (j + i < hi) atomicAdd(&hist[p ? 1 : 0][key >> 21], 1u);
        }
      }
      if (held && any) {  // eight lanes' bits make a word
        uint32_t word = mine << (4 * (lane & 7));
        word |= __shfl_xor_sync(0xffffffffu, word, 1);
        word |= __shfl_xor_sync(0xffffffffu, word, 2);
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        if ((lane & 7) == 0 && j < hi) bits[(j - lo) >> 5] = word;
      }
    }
    cluster.sync();
    // Digits of 11, 11 and 10 bits; need is the rank left inside the prefix.  A
    // thread takes two bins, the highest first.
    uint32_t mask = 0;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digits = pass == 2 ? 1023u : 2047u;
      if (pass > 0) {
        for (int base = lo; base < hi; base += kEvThreads) {
          const int j = base + tid;
          if (j < hi) {
            const uint32_t key = held ? keys[j - lo] : weight_key(w[j]);
            const bool p = any && (held ? (bits[(j - lo) >> 5] >> ((j - lo) & 31)) & 1 : (pos ? pos[j] : j) >= from);
            if (p == active && (key & mask) == threshold) atomicAdd(&hist[pass + 1][(key >> shift) & digits], 1u);
          }
        }
        cluster.sync();
      }
      const int top = kBins - 2 - 2 * tid;
      uint32_t h1 = 0, h0 = 0, above, total;
      if (pass == 0 && any) {
        for (int i = 0; i < CS; ++i) {
          const uint2 v = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&hist[1][0], i) + top);
          h0 += v.x;
          h1 += v.y;
        }
        above = scan_excl(h1 + h0, warp_sums, &total);
        active = total >= (uint32_t)m;
        need = active ? m : m - total;
      } else if (pass == 0) {
        need = m;
      }
      if (!(pass == 0 && active)) {
        h1 = h0 = 0;
        for (int i = 0; i < CS; ++i) {
          const uint2 v = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&hist[pass == 0 ? 0 : pass + 1][0], i) + top);
          h0 += v.x;
          h1 += v.y;
        }
        above = scan_excl(h1 + h0, warp_sums, &total);
      }
      if (above < need && need <= above + h1 + h0) {
        const bool upper = need <= above + h1;
        s_digit = top + (upper ? 1 : 0);
        s_need = need - above - (upper ? 0 : h1);
      }
      __syncthreads();
      threshold |= s_digit << shift;
      mask |= digits << shift;
      need = s_need;
      __syncthreads();
    }
  }
  // A row's class in the scan: above the threshold (low half of a word) or at it
  // (high half); kept are the former and the first `need` of the latter.
  auto classify = [&](uint32_t key, bool p) -> uint32_t {
    if (n == m) return 1u;
    if (p == active) return key > threshold ? 1u : key == threshold ? 0x10000u : 0u;
    return p ? 1u : 0u;
  };
  uint32_t above = 0, equal = 0, below_m = 0;  // before this block's slots; P(m)
  if (n > m) {
    Counts c{};
    for (int base = lo; base < hi; base += kEvThreads) {
      const int j = base + tid;
      if (j < hi) {
        const uint32_t key = held ? keys[j - lo] : weight_key(w[j]);
        const bool p = any && (held ? (bits[(j - lo) >> 5] >> ((j - lo) & 31)) & 1 : (pos ? pos[j] : j) >= from);
        const uint32_t cls = classify(key, p);
        c.above += cls & 0xffff;
        c.equal += cls >> 16;
        if (j < m) {
          c.above_m += cls & 0xffff;
          c.equal_m += cls >> 16;
        }
      }
    }
    if (tid == 0) s_counts = Counts{};
    __syncthreads();
    c.above = __reduce_add_sync(0xffffffffu, c.above);
    c.equal = __reduce_add_sync(0xffffffffu, c.equal);
    c.above_m = __reduce_add_sync(0xffffffffu, c.above_m);
    c.equal_m = __reduce_add_sync(0xffffffffu, c.equal_m);
    if (lane == 0) {
      atomicAdd(&s_counts.above, c.above);
      atomicAdd(&s_counts.equal, c.equal);
      atomicAdd(&s_counts.above_m, c.above_m);
      atomicAdd(&s_counts.equal_m, c.equal_m);
    }
    cluster.sync();
    uint32_t eq_m = 0;
    for (int i = 0; i < CS; ++i) {
      const Counts x = *cluster.map_shared_rank(&s_counts, i);
      if (i < rank) {
        above += x.above;
        equal += x.equal;
      }
      below_m += x.above_m;
      eq_m += x.equal_m;
    }
    below_m += min(need, eq_m);
    if (tid == 0 && rank == 0) k.count[bh] = m - (int)below_m;
  }
  for (int base = lo; base < hi; base += kSweep) {
    const int j0 = base + tid * 4;
    float wv[4];
    int32_t pv[4];
    uint32_t cls[4] = {0, 0, 0, 0}, sum = 0;
    if (j0 < hi) {
      fetch(j0, wv, pv);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (j0 + i < hi) cls[i] = classify(weight_key(wv[i]), any && pv[i] >= from);
        sum += cls[i];
      }
    }
    uint32_t total;
    uint32_t run = scan_excl(sum, warp_sums, &total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = j0 + i;
      if (j >= hi) continue;
      const uint32_t eq = equal + (run >> 16);
      const uint32_t kept_before = above + (run & 0xffff) + min(need, eq);
      const bool kept = cls[i] == 1u || (cls[i] == 0x10000u && eq < need);
      if (j < m) {
        if (kept) {
          wo[j] = wv[i];
          if (po) po[j] = pv[i];
        } else {
          k.to[bh * k.most + (j - kept_before)] = j;
        }
      } else {
        if (kept) {
          const int64_t at = bh * k.most + (kept_before - below_m);
          k.from[at] = j;
          k.moved_weight[at] = wv[i];
          if (po) k.moved_position[at] = pv[i];
        }
        wo[j] = 0.f;
        if (po) po[j] = -1;
      }
      run += cls[i];
    }
    above += total & 0xffff;
    equal += total >> 16;
  }
  for (int64_t j = n + rank * kEvThreads + tid; j < k.capacity; j += CS * kEvThreads) {
    wo[j] = 0.f;
    if (po) po[j] = -1;
  }
  cluster.sync();  // no block leaves while another reads its shared memory
}

template <typename T, int D>
__global__ void __launch_bounds__(256)
evict_move_kernel(const __grid_constant__ EvictCall k) {
  constexpr int L = D / 8;  // lanes of a row
  const int64_t bh = blockIdx.y;
  const int b = (int)(bh / k.c.H), h = (int)(bh % k.c.H);
  cudaGridDependencySynchronize();
  const int count = k.count[bh];
  const int32_t* table = k.c.table + b * k.c.table_stride;
  const int mask = (1 << k.page_shift) - 1;
  const int lane = threadIdx.x % L;
  for (int64_t i = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L; i < count; i += (int64_t)gridDim.x * (256 / L)) {
    const int src = k.from[bh * k.most + i], dst = k.to[bh * k.most + i];
    if (lane == 0) {
      k.weights_out[bh * k.capacity + dst] = k.moved_weight[bh * k.most + i];
      if (k.positions_out) k.positions_out[bh * k.capacity + dst] = k.moved_position[bh * k.most + i];
    }
    const int64_t ps = table[src >> k.page_shift], pd = table[dst >> k.page_shift];
    if (ps < 0 || ps >= k.c.pages || pd < 0 || pd >= k.c.pages) {
      if (lane == 0) atomicOr(k.status, kStatusPage);
      continue;
    }
    const int64_t as = (((ps * k.c.H + h) << k.page_shift) + (src & mask)) * D + lane * 8;
    const int64_t ad = (((pd * k.c.H + h) << k.page_shift) + (dst & mask)) * D + lane * 8;
    Chunk<T> kc, vc;
    kc.load(static_cast<const T*>(k.c.k) + as);
    vc.load(static_cast<const T*>(k.c.v) + as);
    kc.store(static_cast<T*>(k.c.k) + ad);
    vc.store(static_cast<T*>(k.c.v) + ad);
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
  // Blocks of a head: one for each 8192 slots, as long as the GPU has room for
  // all of them at once.
  int cs = 1;
  while (cs < kMaxCluster && k.capacity > (int64_t)cs * 8192 && bh * cs * 2 <= 148 * 2) cs *= 2;
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
