// Eviction from the paged cache by accumulated attention weight.
//
// The m best of n rows of a (sequence, key head) are those whose 33-bit key
// (protected, weight as an ordered integer) is above the m-th largest, and of
// those equal to it the lowest slots.  The m-th largest is found digit by digit
// (11 + 11 + 10 bits) with histograms in shared memory.
//
// Rows are not packed in their order: kept rows below slot m stay, and only
// those from m on move, into the slots given up below m.  Sources and targets are
// disjoint, so all moves run at once and as few bytes as possible are moved
// (about m (n - m) / n rows where the weights know no place, one row in a
// decoding step that evicts one).  With P(x) the number of kept rows below slot x,
// the target of rank x - P(x) is a given-up slot x, the source of rank P(x) -
// P(m) a kept slot x; both follow from counts of the rows above and at the
// threshold, so one scan writes both lists.
#include <algorithm>

#include "host.h"
#include "rotary.cuh"

namespace lh {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kBins = 2048;
constexpr int kPerThread = 4;
constexpr int kSweep = kEvThreads * kPerThread;  // slots of one step of the scan

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

__global__ void __launch_bounds__(kEvThreads)
evict_select_kernel(const __grid_constant__ EvictCall k) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_sums[32];
  __shared__ uint32_t s_digit, s_need;
  const int tid = threadIdx.x;
  const int64_t bh = blockIdx.x;
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
  if (tid == 0) {
    if (bh % k.c.H == 0) {
      k.lengths_out[b] = m;
      if (raw != n) atomicOr(k.status, kStatusPage);
    }
    if (n == m) k.count[bh] = 0;
  }
  uint32_t threshold = 0, need = 0;
  bool active = false;  // the class (protected or not) that the threshold splits
  if (n > m) {
    uint32_t mine = 0;
    for (int j = tid; j < n; j += kEvThreads) mine += any && (pos ? pos[j] : j) >= from;
    uint32_t prot;
    scan_excl(mine, warp_sums, &prot);
    active = prot >= (uint32_t)m;
    need = active ? m : m - prot;
    // Digits of 11, 11 and 10 bits; need is the rank left inside the prefix.
    uint32_t mask = 0;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digits = pass == 2 ? 1023u : 2047u;
      for (int i = tid; i < kBins; i += kEvThreads) hist[i] = 0;
      __syncthreads();
      for (int j = tid; j < n; j += kEvThreads) {
        const bool p = any && (pos ? pos[j] : j) >= from;
        const uint32_t key = weight_key(w[j]);
        if (p == active && (key & mask) == threshold) atomicAdd(&hist[(key >> shift) & digits], 1u);
      }
      __syncthreads();
      const uint32_t h1 = hist[kBins - 1 - 2 * tid], h0 = hist[kBins - 2 - 2 * tid];
      uint32_t total;
      const uint32_t above = scan_excl(h1 + h0, warp_sums, &total);
      if (above < need && need <= above + h1 + h0) {
        const bool upper = need <= above + h1;
        s_digit = kBins - (upper ? 1 : 2) - 2 * tid;
        s_need = need - above - (upper ? 0 : h1);
      }
      __syncthreads();
      threshold |= s_digit << shift;
      mask |= digits << shift;
      need = s_need;
      __syncthreads();
    }
  }
  // Scan in slot order: rows above the threshold (low half of a word) and at
  // it (high half); kept are the former and the first `need` of the latter.
  uint32_t above = 0, equal = 0;     // before this step's slots
  uint32_t below_m = 0;              // P(m)
  bool below_known = false;
  for (int base = 0; base < n; base += kSweep) {
    float wv[kPerThread];
    int32_t pv[kPerThread];
    uint32_t cls[kPerThread], sum = 0;
    const int j0 = base + tid * kPerThread;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int j = j0 + i;
      cls[i] = 0;
      wv[i] = 0.f;
      pv[i] = -1;
      if (j < n) {
        wv[i] = w[j];
        pv[i] = pos ? pos[j] : j;
        const bool p = any && pv[i] >= from;
        const uint32_t key = weight_key(wv[i]);
        if (n == m) cls[i] = 1;
        else if (p == active) cls[i] = key > threshold ? 1u : key == threshold ? 0x10000u : 0u;
        else cls[i] = p ? 1u : 0u;
      }
      sum += cls[i];
    }
    uint32_t total;
    uint32_t run = scan_excl(sum, warp_sums, &total);
    // P(m) when slot m lies in this step.
    if (!below_known && m < base + kSweep) {
      if (j0 <= m && m < j0 + kPerThread) {
        uint32_t at = run;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i)
          if (j0 + i < m) at += cls[i];
        s_need = above + (at & 0xffff) + min(need, equal + (at >> 16));
      }
      __syncthreads();
      below_m = s_need;
      below_known = true;
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int j = j0 + i;
      const uint32_t eq = equal + (run >> 16);
      const uint32_t kept_before = above + (run & 0xffff) + min(need, eq);
      const bool kept = cls[i] == 1u || (cls[i] == 0x10000u && eq < need);
      if (j < n) {
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
            k.moved_position[at] = pv[i];
          }
          wo[j] = 0.f;
          if (po) po[j] = -1;
        }
      }
      run += cls[i];
    }
    above += total & 0xffff;
    equal += total >> 16;
  }
  if (tid == 0 && n > m) k.count[bh] = m - (int)below_m;
  for (int64_t j = n + tid; j < k.capacity; j += kEvThreads) {
    wo[j] = 0.f;
    if (po) po[j] = -1;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(256)
evict_move_kernel(const __grid_constant__ EvictCall k) {
  constexpr int L = D / 8;  // lanes of a row
  const int64_t bh = blockIdx.y;
  const int b = (int)(bh / k.c.H), h = (int)(bh % k.c.H);
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
  evict_select_kernel<<<(unsigned)bh, kEvThreads, 0, st>>>(k);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || k.most == 0) return e;
  with_type_dim(c.dtype, c.d, [&]<typename T, int D>() {
    const int64_t rows = 256 / (D / 8);
    const dim3 grid((unsigned)std::min<int64_t>((k.most + rows - 1) / rows, std::max<int64_t>(1, 148 * 16 / bh)), (unsigned)bh);
    evict_move_kernel<T, D><<<grid, 256, 0, st>>>(k);
  });
  return cudaGetLastError();
}

}  // namespace lh
