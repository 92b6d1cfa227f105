// Rotary positions on [B, H, N, d] tensors and the append of new rows to the
// paged cache.
//
// (a, b) -> m (a cos - b sin, b cos + a sin) for every channel pair, the angle
// being position * frequency; the transposed map (the gradient) turns the
// other way.  Bound by HBM: every row is read and written once, about six
// flops a pair.  The sines and cosines are formed in the kernel, once for a
// (position, eight pairs) and all heads of Q and K: a table of them would be
// read again for each call and cost a rounding of its own.
#include <algorithm>

#include "host.h"
#include "rotary.cuh"

namespace lh {
namespace {

constexpr int kRotThreads = 256;
// Heads of a thread in flight, 64 bytes of each, and blocks an SM that the registers
// are shared out for.  Measured in a graph (98,304 tokens of 8 + 2 heads of 128
// channels, bf16; 2 x 8191 of 8 + 8 of 64, fp32): 79 and 25 us; four heads and half
// the blocks 87 and 28 us, two heads in fp32 33 us (spills).
constexpr int kRotBlocks = 4;
template <typename T>
constexpr int kInFlight = sizeof(T) == 2 ? 2 : 1;

// A unit's chunks of the heads in flight.
template <typename T>
struct Batch {
  static constexpr int F = kInFlight<T>;
  Chunk<T> a[F], e[F];
  // From src, the first of n heads ss elements apart, the chunks `apart` elements apart.
  __device__ __forceinline__ void load(const T* src, int64_t ss, int apart, int n) {
#pragma unroll
    for (int i = 0; i < F; ++i) {
      if (i < n) {
        a[i].load(src + i * ss);
        e[i].load(src + i * ss + apart);
      }
    }
  }
};

// The unit's chunks of n heads, ss and ds elements apart, turned or copied; the first
// heads' are in x already.
template <typename T>
__device__ __forceinline__ void move_heads(Batch<T>& x, const T* src, int64_t ss, T* dst, int64_t ds, int n,
                                           const Unit& unit, bool half, const float (&c)[8], const float (&s)[8]) {
  constexpr int F = kInFlight<T>;
  const int apart = (unit.cb - unit.ca) * 8;
  while (true) {
#pragma unroll
    for (int i = 0; i < F; ++i) {
      if (i >= n) continue;
      T* const p = dst + i * ds;
      if (unit.turn) {
        float xa[8], xb[8];
        x.a[i].get(xa);
        x.e[i].get(xb);
        turn_unit(half, c, s, xa, xb);
        Vec8<T>::store(p, xa);
        Vec8<T>::store(p + apart, xb);
      } else {
        x.a[i].store(p);
        x.e[i].store(p + apart);
      }
    }
    n -= F;
    if (n <= 0) return;
    src += F * ss;
    dst += F * ds;
    x.load(src, ss, apart, n);
  }
}

// Heads of a block at most, evenly shared out.  98,304 rows of 16 + 16 heads of 64
// channels, bf16, calls of fresh inputs: 123 us with eight, 123 with six, 127 with four
// (the angles are formed more often) and 126 with sixteen (a block's stores reach
// farther apart); 524,288 rows 648, 663, 680 and 660 us.  The append keeps more: a row
// costs it its page as well as its angles (four prompts: 48 us with twelve, 50 with six).
constexpr int kMostHeads = 8;

struct RotaryCall {
  RowsArg x[2], y[2];
  const int32_t* positions;
  int64_t positions_stride, start;
  int64_t N, rows;  // rows = B * N
  int heads, group; // heads of both tensors, heads of one block
  bool transpose;
};

template <typename T, int D>
__global__ void __launch_bounds__(kRotThreads, kRotBlocks)
rotary_kernel(const __grid_constant__ RotaryArg r, const __grid_constant__ RotaryCall k) {
  constexpr int U = D / 16;
  __shared__ __align__(16) uint64_t s_turns[LH_MAX_PAIRS];
  stage_turns(r, s_turns);
  const int64_t row = (int64_t)blockIdx.x * (kRotThreads / U) + threadIdx.x / U;
  const int u = threadIdx.x % U;
  if (row >= k.rows) return;
  const int64_t b = row / k.N, n = row - b * k.N;
  const Unit unit = make_unit(r, u);
  const int apart = (unit.cb - unit.ca) * 8;
  const int h0 = blockIdx.y * k.group;
  const int h1 = min(k.heads, h0 + k.group);
  // The first rows are asked for before the angles are worked out: the fp32 case above
  // 25.1 us, 25.8 with the angles first.
  Batch<T> ahead;
  int t = h0 >= k.x[0].H, off = t ? k.x[0].H : 0;
  int lo = h0 - off, hi = min(h1 - off, k.x[t].H);
  auto source = [&] { return static_cast<const T*>(k.x[t].ptr) + b * k.x[t].sb + lo * k.x[t].sh + n * k.x[t].sn + unit.ca * 8; };
  const T* src = source();
  ahead.load(src, k.x[t].sh, apart, hi - lo);
  float c[8], s[8];
  if (unit.turn) {
    const int64_t pos = k.positions ? (int64_t)k.positions[b * k.positions_stride + n] : k.start + n;
    unit_angles(r, s_turns, u, pos, k.transpose, c, s);
  }
#pragma unroll 1
  while (true) {
    const RowsArg& y = k.y[t];
    move_heads(ahead, src, k.x[t].sh, static_cast<T*>(y.ptr) + b * y.sb + lo * y.sh + n * y.sn + unit.ca * 8, y.sh, hi - lo,
               unit, r.half, c, s);
    off += k.x[t].H;
    if (t == 1 || off >= h1) return;
    t = 1;
    lo = 0;
    hi = h1 - off;
    src = source();
    ahead.load(src, k.x[t].sh, apart, hi);
  }
}

struct AppendCall {
  lh_cache c;
  RowsArg q, qo, k, v;
  const int32_t *positions, *counts;
  int64_t positions_stride;
  int32_t* slot_positions;
  int64_t T, rows;  // rows = B * T
  int group;        // heads of one block
  int page_shift;
  unsigned int* status;
};

template <typename T, int D>
__global__ void __launch_bounds__(kRotThreads, kRotBlocks)
append_kernel(const __grid_constant__ RotaryArg r, const __grid_constant__ AppendCall k) {
  constexpr int U = D / 16, kHeadsInFlight = kInFlight<T>;
  __shared__ __align__(16) uint64_t s_turns[LH_MAX_PAIRS];
  stage_turns(r, s_turns);
  const int64_t row = (int64_t)blockIdx.x * (kRotThreads / U) + threadIdx.x / U;
  const int u = threadIdx.x % U;
  if (row >= k.rows) return;
  const int64_t b = row / k.T, t = row - b * k.T;
  const int64_t count = k.counts ? (int64_t)k.counts[b] : k.T;
  const int64_t capacity = (int64_t)k.c.width << k.page_shift;
  const bool there = t < count;
  const Unit unit = make_unit(r, u);
  const int Hq = k.q.H, H = k.c.H;
  const int h0 = blockIdx.y * k.group;
  const int h1 = min(Hq + 2 * H, h0 + k.group);
  Chunk<T> a[kHeadsInFlight], e[kHeadsInFlight];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < kHeadsInFlight; ++i) {
      const int x = h + i;
      a[i].zero();
      e[i].zero();
      if (x >= h1 || !there) continue;
      const RowsArg& rows = x < Hq ? k.q : x < Hq + H ? k.k : k.v;
      const int head = x < Hq ? x : x < Hq + H ? x - Hq : x - Hq - H;
      const T* p = static_cast<const T*>(rows.ptr) + b * rows.sb + head * rows.sh + t * rows.sn;
      a[i].load(p + unit.ca * 8);
      e[i].load(p + unit.cb * 8);
    }
  };
  load(h0);  // on their way while the slot's page and the angles are found (four ragged
  // prompts of up to 8192 rows, 16 + 4 heads: 49.6 -> 48.2 us)
  const int64_t slot = (int64_t)k.c.lengths[b] - count + t;
  // A row outside the cache is left out, and so is one of a batch whose count
  // is more than the T rows that were given.
  int64_t page = -1;
  if (there && slot >= 0 && slot < capacity && count <= k.T) {
    page = k.c.table[b * k.c.table_stride + (slot >> k.page_shift)];
    if (page >= k.c.pages) page = -1;
  }
  const bool bad = there && page < 0;
  if (u == 0 && blockIdx.y == 0 && (bad || (t == 0 && count < 0))) atomicOr(k.status, kStatusPage);
  const int64_t pos = k.positions && there ? (int64_t)k.positions[b * k.positions_stride + t] : slot;
  float c[8], s[8];
  if (unit.turn && h0 < Hq + H) unit_angles(r, s_turns, u, pos, false, c, s);

  const int64_t in_page = slot & ((1 << k.page_shift) - 1);
  // One loop over the heads of Q, K and V: a step of one row has them all in
  // flight at once (3.2 us; in three loops 3.6).
  for (int h = h0;;) {
#pragma unroll
    for (int i = 0; i < kHeadsInFlight; ++i) {
      const int x = h + i;
      if (x >= h1 || (x >= Hq && page < 0)) continue;  // padding of Q becomes zero, of K and V is left out
      const bool is_q = x < Hq, is_v = x >= Hq + H;
      const int head = is_q ? x : is_v ? x - Hq - H : x - Hq;
      T* out = is_q ? static_cast<T*>(k.qo.ptr) + b * k.qo.sb + head * k.qo.sh + t * k.qo.sn
                    : static_cast<T*>(is_v ? k.c.v : k.c.k) + (((page * H + head) << k.page_shift) + in_page) * D;
      if (!is_q && !is_v && u == 0 && k.slot_positions)
        k.slot_positions[(b * H + head) * capacity + slot] = (int32_t)pos;
      if (unit.turn && !is_v && there) {
        float xa[8], xb[8];
        a[i].get(xa);
        e[i].get(xb);
        turn_unit(r.half, c, s, xa, xb);
        Vec8<T>::store(out + unit.ca * 8, xa);
        Vec8<T>::store(out + unit.cb * 8, xb);
      } else {
        a[i].store(out + unit.ca * 8);
        e[i].store(out + unit.cb * 8);
      }
    }
    h += kHeadsInFlight;
    if (h >= h1) return;
    load(h);
  }
}

// Heads that one block takes: all of them where the rows alone make twelve blocks
// for each SM (the sines and cosines are then formed once), fewer for few rows.
int head_group(int64_t blocks, int heads) {
  int g = heads;
  while (g > 1 && blocks * ((heads + g - 1) / g) < 148 * 12) g = (g + 1) / 2;
  return g;
}

}  // namespace

cudaError_t launch_rotary(const lh_rotary_plan& plan, int dtype, int64_t B, int64_t N, int count,
                          const RowsArg* X, const RowsArg* Y, const int32_t* positions,
                          int64_t positions_stride, int64_t start, bool transpose, cudaStream_t st) {
  RotaryCall k{};
  for (int i = 0; i < count; ++i) {
    k.x[i] = X[i];
    k.y[i] = Y[i];
  }
  k.positions = positions;
  k.positions_stride = positions_stride;
  k.start = start;
  k.N = N;
  k.rows = B * N;
  k.heads = k.x[0].H + k.x[1].H;
  k.transpose = transpose;
  const int64_t per = kRotThreads / (plan.c.d / 16);
  const int64_t blocks = (k.rows + per - 1) / per;
  const int parts = (k.heads + kMostHeads - 1) / kMostHeads;
  k.group = std::min(head_group(blocks, k.heads), (k.heads + parts - 1) / parts);
  const dim3 grid((unsigned)blocks, (k.heads + k.group - 1) / k.group);
  const RotaryArg r = make_rotary_arg(&plan);
  with_type_dim(dtype, plan.c.d, [&]<typename T, int D>() { rotary_kernel<T, D><<<grid, kRotThreads, 0, st>>>(r, k); });
  return cudaGetLastError();
}

cudaError_t launch_cache_append(const lh_cache& c, const lh_rotary_plan* rotary, int64_t T,
                                const RowsArg& K, const RowsArg& V, const RowsArg& Q, const RowsArg& Qo,
                                const int32_t* positions, int64_t positions_stride,
                                const int32_t* counts, int32_t* slot_positions, cudaStream_t st) {
  AppendCall k{};
  k.c = c;
  k.q = Q;
  k.qo = Qo;
  k.k = K;
  k.v = V;
  k.positions = positions;
  k.positions_stride = positions_stride;
  k.counts = counts;
  k.slot_positions = slot_positions;
  k.T = T;
  k.rows = (int64_t)c.B * T;
  k.page_shift = __builtin_ctz(c.page);
  k.status = device_status_ptr();
  if (!k.status) return cudaErrorInvalidSymbol;
  const int64_t per = kRotThreads / (c.d / 16);
  const int64_t blocks = (k.rows + per - 1) / per;
  const int heads = Q.H + 2 * c.H;
  k.group = head_group(blocks, heads);
  const dim3 grid((unsigned)blocks, (heads + k.group - 1) / k.group);
  const RotaryArg r = make_rotary_arg(rotary);
  with_type_dim(c.dtype, c.d, [&]<typename E, int D>() { append_kernel<E, D><<<grid, kRotThreads, 0, st>>>(r, k); });
  return cudaGetLastError();
}

}  // namespace lh
