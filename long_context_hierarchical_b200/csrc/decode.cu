// Attention of one new token over the paged cache.
//
//   s_j = scale q . k_j,  lse = log sum_j exp s_j,  O = sum_j exp(s_j - lse) v_j
//
// One pass over K and V with a running reference m and sum l (the scores in
// units of log 2): bound by HBM, 2 d elements read for 4 g d flops where g
// query heads share a key head.
//
// Split over the length.  All sequences' key tiles of 64 slots, (sequence, key
// head, tile) in this order, form one line of T tiles, cut into as many equal
// ranges as there are blocks.  The lengths are read on the device, so unequal
// batches are balanced, and a captured graph stays right as lengths grow.  A
// range that holds a whole (sequence, head) writes its output; the others
// leave (m, l, unnormalised O) and a second, overlapping launch joins them in
// the order of their ranges, so results do not depend on scheduling.  The
// ranges depend on lengths and grid alone: no atomics, no block waits for
// another.
//
// More than max_heads query heads on one key head are cut into parts of equal
// size that count as key heads of their own here.
#include <algorithm>

#include "host.h"
#include "rotary.cuh"

namespace lh {
namespace {

constexpr int kTile = 64;       // slots of a key tile: the unit of the split
constexpr int kWarps = 4;       // warps of a block
constexpr int kDecThreads = kWarps * 32;
constexpr int kJoinThreads = 128;
constexpr int kJoinSlots = 2048;  // slots whose weights one join block adds
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A warp keeps its running reference until a score passes it by this many
// powers of two: sums stay far inside fp32 and rescaling is rare.
constexpr float kSlack = 8.f;

struct DecodeCall {
  lh_cache c;
  RowsArg q;
  float scale;        // scale * log2(e)
  void* o;            // [B, Hq, d]
  float* lse;         // [B, Hq]
  float* part;        // [blocks][2][gv] rows of d + 2 floats: O, m, l
  float* scores;      // [B, Hq, capacity], or null
  const float* weights;
  float* weights_out;
  unsigned int* status;
  int page_shift, Hq, G;  // G = Hq / H
  int nv, gv;         // parts of a key head's group, query heads of a part
  int blocks;         // ranges of the split
};

__device__ __forceinline__ int seq_length(const DecodeCall& k, int b) {
  const int n = k.c.lengths[b];
  return max(0, min(n, k.c.width << k.page_shift));
}

__device__ __forceinline__ int tiles_of(int n) { return (n + kTile - 1) / kTile; }

// Sum over the block of one value per thread.
template <int NT>
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* warp_sums) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = v;
  __syncthreads();
  int64_t t = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) t += warp_sums[i];
  return t;
}

// Ranges in use and where a tile or a range lies: range c of W holds tiles
// [c T / W, (c + 1) T / W).
__device__ __forceinline__ int ranges(const DecodeCall& k, int64_t T) { return (int)min((int64_t)k.blocks, T); }
__device__ __forceinline__ int64_t range_begin(int64_t c, int64_t T, int W) { return c * T / W; }
__device__ __forceinline__ int range_of(int64_t tile, int64_t T, int W) { return (int)(((tile + 1) * W - 1) / T); }

// Keys handled by a quad of lanes: lane r*4 + c holds channels of key r (of
// the eight of a warp tile), in chunks of 16 bytes c, c + 4, ...; it keeps q and
// the running output of GT heads for those channels, so scores take two
// shuffles and the outputs none until the end of a segment.  GW warps share a
// tile where the heads are more than GT.
template <typename T, int D, int GT, int GW>
__global__ void __launch_bounds__(kDecThreads)
decode_kernel(const __grid_constant__ DecodeCall k) {
  constexpr int EPC = 16 / sizeof(T);     // elements of a 16-byte chunk
  constexpr int NC = D / 4 / EPC;         // chunks of a lane
  constexpr int NW = kWarps / GW;         // warps along the keys
  __shared__ float sm_o[NW][GT * GW][D + 2];
  __shared__ int64_t warp_sums[kWarps];
  __shared__ int s_b;
  __shared__ int64_t s_first;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c4 = lane & 3;
  const int kw = warp / GW, hg = warp % GW;
  const int Hv = k.c.H * k.nv;

  int64_t sum = 0;
  for (int b = tid; b < k.c.B; b += kDecThreads) sum += tiles_of(seq_length(k, b));
  const int64_t T_all = block_sum<kDecThreads>(sum, warp_sums) * Hv;
  const int W = ranges(k, T_all);
  if ((int)blockIdx.x >= W) return;
  int64_t u = range_begin(blockIdx.x, T_all, W);
  const int64_t u_end = range_begin(blockIdx.x + 1, T_all, W);

  // The sequence that tile u lies in.
  if (tid < 32) {
    int64_t base = 0;
    for (int b0 = 0; b0 < k.c.B; b0 += 32) {
      const int64_t mine = b0 + lane < k.c.B ? (int64_t)tiles_of(seq_length(k, b0 + lane)) * Hv : 0;
      int64_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const int64_t before = base + incl - mine;
      const bool hit = u >= before && u < before + mine;
      if (hit) {
        s_b = b0 + lane;
        s_first = before;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
      if (__any_sync(0xffffffffu, hit)) break;
    }
  }
  __syncthreads();
  int b = s_b;
  int64_t first = s_first;  // first tile of sequence b

  const int64_t capacity = (int64_t)k.c.width << k.page_shift;
  const T* const kp = static_cast<const T*>(k.c.k);
  const T* const vp = static_cast<const T*>(k.c.v);
  while (u < u_end) {
    const int n = seq_length(k, b);
    const int nt = tiles_of(n);
    if (u >= first + (int64_t)nt * Hv) {  // next sequence (empty ones have no tiles)
      first += (int64_t)nt * Hv;
      ++b;
      continue;
    }
    const int hv = (int)((u - first) / nt);
    const int64_t seg0 = first + (int64_t)hv * nt, seg1 = seg0 + nt;
    const int64_t stop = min(seg1, u_end);
    const int h = hv / k.nv, part = hv % k.nv;
    const int g0 = part * k.gv, gn = min(k.gv, k.G - g0);  // query heads g0 .. of the group
    const int head0 = h * k.G + g0;

    float q[GT][NC * EPC], o[GT][NC * EPC], m[GT], l[GT];
#pragma unroll
    for (int i = 0; i < GT; ++i) {
      const int g = hg * GT + i;
      m[i] = -INFINITY;
      l[i] = 0.f;
      const T* p = static_cast<const T*>(k.q.ptr) + b * k.q.sb + (int64_t)(head0 + min(g, gn - 1)) * k.q.sh;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
#pragma unroll
        for (int e = 0; e < EPC; ++e) {
          q[i][j * EPC + e] = (float)p[(c4 + 4 * j) * EPC + e] * k.scale;
          o[i][j * EPC + e] = 0.f;
        }
      }
    }
    const int j0 = (int)(u - seg0) * kTile, j1 = min(n, (int)(stop - seg0) * kTile);
    for (int t = j0 + kw * 8; t < j1; t += NW * 8) {
      const int j = t + r;
      bool live = j < j1;
      int64_t page = 0;
      if (live) {
        page = k.c.table[b * k.c.table_stride + (j >> k.page_shift)];
        if (page < 0 || page >= k.c.pages) {
          live = false;
          if (c4 == 0) atomicOr(k.status, kStatusPage);
        }
      }
      uint4 kc[NC], vc[NC];
      const int64_t at = (((page * k.c.H + h) << k.page_shift) + (j & ((1 << k.page_shift) - 1))) * D;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        kc[i] = vc[i] = make_uint4(0, 0, 0, 0);
        if (live) {
          kc[i] = __ldg(reinterpret_cast<const uint4*>(kp + at) + c4 + 4 * i);
          vc[i] = __ldg(reinterpret_cast<const uint4*>(vp + at) + c4 + 4 * i);
        }
      }
      float kf[NC * EPC], vf[NC * EPC];
      const uint32_t* kw_ = reinterpret_cast<const uint32_t*>(kc);
      const uint32_t* vw_ = reinterpret_cast<const uint32_t*>(vc);
#pragma unroll
      for (int i = 0; i < NC * 4; ++i) {
        if constexpr (sizeof(T) == 2) {
          kf[2 * i] = __uint_as_float(kw_[i] << 16);
          kf[2 * i + 1] = __uint_as_float(kw_[i] & 0xffff0000u);
          vf[2 * i] = __uint_as_float(vw_[i] << 16);
          vf[2 * i + 1] = __uint_as_float(vw_[i] & 0xffff0000u);
        } else {
          kf[i] = __uint_as_float(kw_[i]);
          vf[i] = __uint_as_float(vw_[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < GT; ++i) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < NC * EPC; ++e) s += q[i][e] * kf[e];
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        const int g = hg * GT + i;
        if (k.scores && c4 == 0 && g < gn && j < j1)
          k.scores[((int64_t)b * k.Hq + head0 + g) * capacity + j] = live ? s : -INFINITY;
        if (!live) continue;
        if (s > m[i] + kSlack) {  // also the first key: m is -inf
          const float f = exp2f(m[i] - s);
          m[i] = s;
          l[i] *= f;
#pragma unroll
          for (int e = 0; e < NC * EPC; ++e) o[i][e] *= f;
        }
        const float p = exp2f(s - m[i]);
        l[i] += p;
#pragma unroll
        for (int e = 0; e < NC * EPC; ++e) o[i][e] += p * vf[e];
      }
    }
    // Join the eight key rows of the warp, then the warps along the keys.
    __syncthreads();
#pragma unroll
    for (int i = 0; i < GT; ++i) {
      float top = m[i];
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float f = m[i] == -INFINITY ? 0.f : exp2f(m[i] - top);
      l[i] *= f;
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
      const int g = hg * GT + i;
#pragma unroll
      for (int e = 0; e < NC * EPC; ++e) {
        float v = o[i][e] * f;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
        if (r == 0) sm_o[kw][g][(c4 + 4 * (e / EPC)) * EPC + e % EPC] = v;
      }
      if (lane == 0) {
        sm_o[kw][g][D] = top;
        sm_o[kw][g][D + 1] = l[i];
      }
    }
    __syncthreads();
    const bool whole = u == seg0 && stop == seg1;
    // The segment that begins the range leaves its part in slot 0, one that
    // begins inside it and goes on behind it in slot 1.
    const int slot = u == range_begin(blockIdx.x, T_all, W) ? 0 : 1;
    float* part_out = k.part + ((int64_t)blockIdx.x * 2 + slot) * k.gv * (D + 2);
    for (int i = tid; i < gn * D; i += kDecThreads) {
      const int g = i / D, e = i % D;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) top = fmaxf(top, sm_o[w][g][D]);
      float acc = 0.f, tot = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float mw = sm_o[w][g][D];
        const float f = mw == -INFINITY ? 0.f : exp2f(mw - top);
        acc += f * sm_o[w][g][e];
        tot += f * sm_o[w][g][D + 1];
      }
      if (whole) {
        const int64_t row = (int64_t)b * k.Hq + head0 + g;
        static_cast<T*>(k.o)[row * D + e] = (T)(tot > 0.f ? acc / tot : 0.f);
        if (e == 0) k.lse[row] = tot > 0.f ? (top + log2f(tot)) * kLn2 : -INFINITY;
      } else {
        part_out[g * (D + 2) + e] = acc;
        if (e == 0) {
          part_out[g * (D + 2) + D] = top;
          part_out[g * (D + 2) + D + 1] = tot;
        }
      }
    }
    u = stop;
  }
}

// Joins the parts of one query head (blockIdx.y = 0 writes O and lse) and adds
// the probabilities of kJoinSlots slots to the weights of its key head.
// Without weights the grid is (B * Hq); with them (B * H, slot blocks) and the
// block goes over the group's heads.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
join_kernel(const __grid_constant__ DecodeCall k, bool with_weights) {
  __shared__ int64_t warp_sums[kJoinThreads / 32];
  const int tid = threadIdx.x;
  const int per_b = with_weights ? k.c.H : k.Hq;
  const int b = blockIdx.x / per_b;
  const int head_first = with_weights ? (blockIdx.x % per_b) * k.G : blockIdx.x % per_b;
  const int heads = with_weights ? k.G : 1;
  const int n = seq_length(k, b);
  const int slot0 = blockIdx.y * kJoinSlots;
  if (blockIdx.y > 0 && slot0 >= n) return;
  const int Hv = k.c.H * k.nv;
  const int64_t capacity = (int64_t)k.c.width << k.page_shift;

  int64_t all = 0, before = 0;
  for (int i = tid; i < k.c.B; i += kJoinThreads) {
    const int64_t t = tiles_of(seq_length(k, i));
    all += t;
    if (i < b) before += t;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      const int len = k.c.lengths[i];
      if (len < 0 || len > capacity) atomicOr(k.status, kStatusPage);
    }
  }
  const int64_t T_all = block_sum<kJoinThreads>(all, warp_sums) * Hv;
  const int64_t first = block_sum<kJoinThreads>(before, warp_sums) * Hv;
  const int nt = tiles_of(n);
  const int W = ranges(k, T_all);

  constexpr int kPer = kJoinSlots / kJoinThreads;
  float add[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) add[i] = 0.f;
  for (int i = 0; i < heads; ++i) {
    const int head = head_first + i;
    const int64_t row = (int64_t)b * k.Hq + head;
    if (n == 0) {
      for (int e = tid; e < D; e += kJoinThreads) static_cast<T*>(k.o)[row * D + e] = (T)0.f;
      if (tid == 0) k.lse[row] = -INFINITY;
      continue;
    }
    const int g = head % k.G;
    const int hv = head / k.G * k.nv + g / k.gv;
    const int64_t seg0 = first + (int64_t)hv * nt, seg1 = seg0 + nt;
    const int c0 = range_of(seg0, T_all, W), c1 = range_of(seg1 - 1, T_all, W);
    float lse2;
    if (c0 == c1) {
      lse2 = k.lse[row] * kLog2e;
    } else {
      const int64_t stride = (int64_t)k.gv * (D + 2);
      const int64_t base = (int64_t)(g % k.gv) * (D + 2);
      const int late = range_begin(c0, T_all, W) < seg0;  // range c0 holds another segment before
      float top = -INFINITY;
      for (int c = c0; c <= c1; ++c)
        top = fmaxf(top, k.part[(2 * (int64_t)c + (c == c0 ? late : 0)) * stride + base + D]);
      float tot = 0.f, acc = 0.f;
      for (int c = c0; c <= c1; ++c) {
        const float* p = k.part + (2 * (int64_t)c + (c == c0 ? late : 0)) * stride + base;
        const float f = p[D] == -INFINITY ? 0.f : exp2f(p[D] - top);
        tot += f * p[D + 1];
        if (blockIdx.y == 0 && tid < D) acc += f * p[tid];
      }
      lse2 = top + log2f(tot);
      if (blockIdx.y == 0) {
        if (tid < D) static_cast<T*>(k.o)[row * D + tid] = (T)(tot > 0.f ? acc / tot : 0.f);
        if (tid == 0) k.lse[row] = tot > 0.f ? lse2 * kLn2 : -INFINITY;
      }
    }
    if (with_weights) {
      const float* s = k.scores + row * capacity;
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        const int j = slot0 + x * kJoinThreads + tid;
        if (j < n) {
          const float v = s[j];
          add[x] += v == -INFINITY ? 0.f : exp2f(v - lse2);
        }
      }
    }
  }
  if (with_weights) {
    const int64_t row = ((int64_t)b * k.c.H + head_first / k.G) * capacity;
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int j = slot0 + x * kJoinThreads + tid;
      if (j < n) k.weights_out[row + j] = k.weights[row + j] + add[x];
    }
  }
}

// Query heads that one block serves: GT * GW of decode_kernel's widest form, as
// many as its registers hold.
constexpr int max_heads(int d) { return d == 64 ? 16 : 8; }

struct Sizes {
  int nv, gv, blocks;
  int64_t part, scores;
};

Sizes sizes(const lh_cache& c, int64_t Hq, bool with_weights) {
  Sizes s{};
  const int64_t G = Hq / c.H;
  const int most_heads = max_heads(c.d);
  s.nv = (int)((G + most_heads - 1) / most_heads);
  s.gv = (int)((G + s.nv - 1) / s.nv);
  s.nv = (int)((G + s.gv - 1) / s.gv);
  const int64_t capacity = (int64_t)c.width * c.page;
  const int64_t most = (int64_t)c.B * c.H * s.nv * ((capacity + kTile - 1) / kTile);
  s.blocks = (int)std::min<int64_t>(most, 148 * 4);
  s.part = ((int64_t)s.blocks * 2 * s.gv * (c.d + 2) * 4 + 255) & ~int64_t(255);
  s.scores = with_weights ? (int64_t)c.B * Hq * capacity * 4 : 0;
  return s;
}

template <typename T, int D, int GT, int GW>
void run(const DecodeCall& k, cudaStream_t st) {
  decode_kernel<T, D, GT, GW><<<k.blocks, kDecThreads, 0, st>>>(k);
}

}  // namespace

int64_t decode_ws_bytes(const lh_cache& c, int64_t Hq, bool with_weights) {
  const Sizes s = sizes(c, Hq, with_weights);
  return s.part + s.scores;
}

cudaError_t launch_decode(const lh_cache& c, const RowsArg& Q, float scale, void* O, float* lse,
                          const float* weights, float* weights_out, void* ws, cudaStream_t st) {
  const bool ww = weights != nullptr;
  const Sizes z = sizes(c, Q.H, ww);
  DecodeCall k{};
  k.c = c;
  k.q = Q;
  k.scale = scale * kLog2e;
  k.o = O;
  k.lse = lse;
  k.part = static_cast<float*>(ws);
  k.scores = ww ? reinterpret_cast<float*>(static_cast<char*>(ws) + z.part) : nullptr;
  k.weights = weights;
  k.weights_out = weights_out;
  k.status = device_status_ptr();
  if (!k.status) return cudaErrorInvalidSymbol;
  k.page_shift = __builtin_ctz(c.page);
  k.Hq = Q.H;
  k.G = Q.H / c.H;
  k.nv = z.nv;
  k.gv = z.gv;
  k.blocks = z.blocks;
  with_type_dim(c.dtype, c.d, [&]<typename T, int D>() {
    if (k.gv == 1) run<T, D, 1, 1>(k, st);
    else if (k.gv == 2) run<T, D, 2, 1>(k, st);
    else if (k.gv <= 4) run<T, D, 2, 2>(k, st);
    else if (k.gv <= 8) run<T, D, 2, 4>(k, st);
    else if constexpr (D == 64) run<T, D, 4, 4>(k, st);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return;
    const int64_t capacity = (int64_t)c.width * c.page;
    const dim3 grid(ww ? c.B * c.H : c.B * Q.H, ww ? (unsigned)((capacity + kJoinSlots - 1) / kJoinSlots) : 1);
    join_kernel<T, D><<<grid, kJoinThreads, 0, st>>>(k, ww);
  });
  return cudaGetLastError();
}

}  // namespace lh
