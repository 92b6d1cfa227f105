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
// More query heads on one key head than a block serves are cut into parts of equal
// size that count as key heads of their own here.
#include <algorithm>

#include "host.h"

namespace lh {
namespace {

constexpr int kTile = 64;       // slots of a key tile: the unit of the split
constexpr int kWarps = 4;       // warps of a block
constexpr int kDecThreads = kWarps * 32;
constexpr int kJoinThreads = 128;
constexpr int kJoinSlots = 512;   // slots whose weights one join block adds, four a thread
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
  float* part;        // [blocks][2][gv] rows of d + 4 floats: O, m, l
  float* scores;      // [B, Hq, capacity], or null
  const float* weights;
  float* weights_out;
  unsigned int* status;
  int page_shift, Hq, G;  // G = Hq / H
  int nv, gv;         // parts of a key head's group, query heads of a part
  int blocks;         // ranges of the split
  int slot_blocks;    // join blocks of a key head's slots
};

__device__ __forceinline__ int seq_length(const DecodeCall& k, int b) {
  const int n = k.c.lengths[b];
  return max(0, min(n, k.c.width << k.page_shift));
}

__device__ __forceinline__ int tiles_of(int n) { return (n + kTile - 1) / kTile; }

// Sums over the block of two values per thread.
struct Pair {
  int64_t x, y;
};
template <int NT>
__device__ __forceinline__ Pair block_sum(Pair v, Pair* warp_sums) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = v;
  __syncthreads();
  Pair t{0, 0};
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    t.x += warp_sums[i].x;
    t.y += warp_sums[i].y;
  }
  return t;
}

// Sum of the values of the threads before this one, and of all.  A block's worth
// of tile counts (less than 2^25 each) fits 32 bits.
__device__ __forceinline__ uint32_t scan_tiles(uint32_t v, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  uint32_t before = 0;
  *total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    before += i < warp ? warp_sums[i] : 0;
    *total += warp_sums[i];
  }
  return before + incl - v;
}

// Ranges in use and where a tile or a range lies: range c of W holds tiles
// [c T / W, (c + 1) T / W).
__device__ __forceinline__ int ranges(const DecodeCall& k, int64_t T) { return (int)min((int64_t)k.blocks, T); }
__device__ __forceinline__ int64_t range_begin(int64_t c, int64_t T, int W) { return c * T / W; }
__device__ __forceinline__ int range_of(int64_t tile, int64_t T, int W) { return (int)(((tile + 1) * W - 1) / T); }

// Where a segment (the part of one sequence and key head that lies in a range)
// stands: its slots j0 .. j1 - 1 and the query heads it serves.
struct Segment {
  int b, h;          // sequence, key head
  int head0, gn;     // first query head, how many
  int j0, j1;
};

// A core runs one segment with a block's warps and leaves in shared memory, for
// each of kParts groups of keys and each head, the unnormalised output, the
// reference m and the sum l.

// Word i (a constant where it is called) of a 16-byte chunk.
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// fp32, on the CUDA cores: keys handled by a quad of lanes.  Lane r*4 + c holds
// channels of key r (of the eight of a warp tile), in chunks of 16 bytes c, c + 4,
// ...; it keeps q and the running output of GT heads for those channels, so scores
// take two shuffles and the outputs none until the end of a segment.  GW warps
// share a tile where the heads are more than GT.  At the copy rate on long caches
// (16 heads of 98,304 slots: 121 us), bound by the latency of its loads where a
// block has few tiles (2 sequences of 8191 slots, 8 heads, with weights: 17 us,
// where the bytes take 11); a ring of asynchronous copies in shared memory, four
// tiles deep, took 22.
template <int D_, int GT, int GW>
struct QuadCore {
  using T = float;
  static constexpr int D = D_, kParts = kWarps / GW, kHeads = GT * GW;
  static constexpr int kBlocks = D == 64 ? (GT == 1 ? 4 : GT == 2 ? 3 : 2) : (GT == 1 ? 3 : 2);
  static constexpr int EPC = 4;            // elements of a 16-byte chunk
  static constexpr int NC = D / 4 / EPC;  // chunks of a lane

  static __device__ __forceinline__ void run(const DecodeCall& k, const Segment& s, float (*sm)[kHeads][D + 4]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c4 = lane & 3;
    const int kw = warp / GW, hg = warp % GW;
    const int64_t capacity = (int64_t)k.c.width << k.page_shift;
    const T* const kp = static_cast<const T*>(k.c.k);
    const T* const vp = static_cast<const T*>(k.c.v);
    float q[GT][NC * EPC], o[GT][NC * EPC], m[GT], l[GT];
#pragma unroll
    for (int i = 0; i < GT; ++i) {
      const int g = hg * GT + i;
      m[i] = -INFINITY;
      l[i] = 0.f;
      const T* p = static_cast<const T*>(k.q.ptr) + s.b * k.q.sb + (int64_t)(s.head0 + min(g, s.gn - 1)) * k.q.sh;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
#pragma unroll
        for (int e = 0; e < EPC; ++e) {
          q[i][j * EPC + e] = p[(c4 + 4 * j) * EPC + e] * k.scale;
          o[i][j * EPC + e] = 0.f;
        }
      }
    }
    // First element of slot j's row, or -1 where there is none.
    const int32_t* const table = k.c.table + s.b * k.c.table_stride;
    const int in_page = (1 << k.page_shift) - 1;
    auto place = [&](int j) -> int64_t {
      if (j >= s.j1) return -1;
      const int64_t page = table[j >> k.page_shift];
      if (page < 0 || page >= k.c.pages) {
        if (c4 == 0) atomicOr(k.status, kStatusPage);
        return -1;
      }
      return (((page * k.c.H + s.h) << k.page_shift) + (j & in_page)) * D + c4 * EPC;
    };
    uint4 kc[NC], vc[NC];
    auto load = [&](uint4 (&c)[NC], const T* p, int64_t at) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        c[i] = make_uint4(0, 0, 0, 0);
        if (at >= 0) c[i] = __ldg(reinterpret_cast<const uint4*>(p + at) + 4 * i);
      }
    };
    auto element = [](const uint4 (&c)[NC], int e) { return __uint_as_float(word(c[e / 4], e % 4)); };
    // K of the next tile is asked for as soon as the scores are formed, V as soon
    // as it is used.
    int64_t at = place(s.j0 + kw * 8 + r);
    load(kc, kp, at);
    load(vc, vp, at);
    for (int t = s.j0 + kw * 8; t < s.j1; t += kParts * 8) {
      const int j = t + r;
      const bool live = at >= 0;
      const int64_t next = place(j + kParts * 8);
      float sc[GT];
#pragma unroll
      for (int i = 0; i < GT; ++i) {
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < NC * EPC; ++e) x += q[i][e] * element(kc, e);
        sc[i] = x;
      }
      load(kc, kp, next);
#pragma unroll
      for (int i = 0; i < GT; ++i) {
        sc[i] += __shfl_xor_sync(0xffffffffu, sc[i], 1);
        sc[i] += __shfl_xor_sync(0xffffffffu, sc[i], 2);
        const int g = hg * GT + i;
        if (k.scores && c4 == 0 && g < s.gn && j < s.j1)
          k.scores[((int64_t)s.b * k.Hq + s.head0 + g) * capacity + j] = live ? sc[i] : -INFINITY;
        if (sc[i] > m[i] + kSlack && live) {  // also the first key: m is -inf
          const float f = exp2f(m[i] - sc[i]);
          m[i] = sc[i];
          l[i] *= f;
#pragma unroll
          for (int e = 0; e < NC * EPC; ++e) o[i][e] *= f;
        }
        // No finite score yet: -inf less 0, not less itself.
        const float p = live ? exp2f(sc[i] - (m[i] == -INFINITY ? 0.f : m[i])) : 0.f;
        l[i] += p;
#pragma unroll
        for (int e = 0; e < NC * EPC; ++e) o[i][e] += p * element(vc, e);
      }
      load(vc, vp, next);
      at = next;
    }
    // Join the eight key rows of the warp.
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
        if (r == 0) sm[kw][g][(c4 + 4 * (e / EPC)) * EPC + e % EPC] = v;
      }
      if (lane == 0) {
        sm[kw][g][D] = top;
        sm[kw][g][D + 1] = l[i];
      }
    }
  }
};

// bf16 on the tensor cores: a warp takes 16 keys, Sᵀ = K Qᵀ and Oᵀ += Vᵀ Pᵀ with
// mma.m16n8k16, NT groups of eight query heads as the n dimension.  Which keys
// and channels stand at which index of a contraction is free, so every lane
// loads its fragments straight from memory, 16 bytes at a time and each byte
// once:
//   K  lane (r, c) holds 16-byte chunks c, c + 4, .. of keys r and r + 8: two of
//      a chunk's four words are an A fragment's k pairs; Q is read alike;
//   V  it holds chunk r (and r + 8) of keys 2c, 2c + 1, 2c + 8, 2c + 9; a byte
//      permute pairs two keys of one channel, channels 8r + 2w and + 1 being rows
//      r and r + 8 of m tile w;
//   P  the two 8 x 8 halves of Sᵀ, in two bf16 parts, become B fragments by movmatrix.
// No shared memory is touched until the end of a segment.  K of the next tile is
// asked for as soon as Sᵀ is formed, V as soon as it is used.  The work is 4 g d
// flops per 4 d bytes, far below what even this instruction reaches, so it is
// chosen over tcgen05, whose operands would have to pass through shared
// memory, for its register operands.  16 heads of 98,304 slots of 64 channels take
// 64 us in a graph, 0.98 of the copy rate; 64 ragged sequences on 4 key heads of
// 128 channels 167 us, 1.00 (on the CUDA cores 101 and 519 us).
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// What a probability cut off to bf16 leaves of it (exact), at least 2^-126 of a positive one.
__device__ __forceinline__ float remainder_of(float p) {
  return fmaxf(p - __uint_as_float(__float_as_uint(p) & 0xffff0000u), fminf(p, 0x1p-126f));
}
// Cache rows are read once: past L1.
__device__ __forceinline__ uint4 load_row(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int D_, int NT>
struct MmaCore {
  using T = __nv_bfloat16;
  static constexpr int D = D_, kParts = kWarps, kHeads = 8 * NT;
  static constexpr int kBlocks = D == 64 ? (NT == 1 ? 5 : 4) : (NT == 1 ? 3 : 2);
  static constexpr int KC = D / 32, VC = D / 64;

  static __device__ __forceinline__ void run(const DecodeCall& k, const Segment& s, float (*sm)[kHeads][D + 4]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c4 = lane & 3;
    const int64_t capacity = (int64_t)k.c.width << k.page_shift;
    const int in_page = (1 << k.page_shift) - 1;
    const int32_t* const table = k.c.table + s.b * k.c.table_stride;
    const T* const kp = static_cast<const T*>(k.c.k);
    const T* const vp = static_cast<const T*>(k.c.v);

    uint4 q[NT][KC];
    float o[NT][VC * 4][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int g = i * 8 + r;
      const T* p = static_cast<const T*>(k.q.ptr) + s.b * k.q.sb + (int64_t)(s.head0 + min(g, s.gn - 1)) * k.q.sh;
#pragma unroll
      for (int j = 0; j < KC; ++j) q[i][j] = __ldg(reinterpret_cast<const uint4*>(p) + c4 + 4 * j);
#pragma unroll
      for (int w = 0; w < VC * 4; ++w) o[i][w][0] = o[i][w][1] = o[i][w][2] = o[i][w][3] = 0.f;
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
    }

    // First element of the tile's rows, or -1 where its page is bad.  A tile of
    // 16 slots lies in one page.
    auto place = [&](int t) -> int64_t {
      const int64_t page = table[t >> k.page_shift];
      if (page < 0 || page >= k.c.pages) {
        if (lane == 0) atomicOr(k.status, kStatusPage);
        return -1;
      }
      return (((page * k.c.H + s.h) << k.page_shift) + (t & in_page)) * D;
    };
    uint4 kc[2][KC], vc[4][VC];
    auto load_k = [&](int64_t at, int t) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool live = at >= 0 && t + r + 8 * i < s.j1;
#pragma unroll
        for (int j = 0; j < KC; ++j)
          kc[i][j] = live ? load_row(kp + at + (r + 8 * i) * D + (c4 + 4 * j) * 8) : make_uint4(0, 0, 0, 0);
      }
    };
    auto load_v = [&](int64_t at, int t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 2 * c4 + (i & 1) + 8 * (i >> 1);
        const bool live = at >= 0 && t + row < s.j1;
#pragma unroll
        for (int j = 0; j < VC; ++j)
          vc[i][j] = live ? load_row(vp + at + row * D + (r + 8 * j) * 8) : make_uint4(0, 0, 0, 0);
      }
    };

    int t = s.j0 + warp * 16;
    int64_t at = -1;
    if (t < s.j1) {
      at = place(t);
      load_k(at, t);
      load_v(at, t);
    }
    while (t < s.j1) {
      const int next = t + kWarps * 16;
      int64_t at_next = -1;
      if (next < s.j1) at_next = place(next);
      float x[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
#pragma unroll
        for (int j = 0; j < KC; ++j) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {word(kc[0][j], 2 * h), word(kc[1][j], 2 * h), word(kc[0][j], 2 * h + 1),
                                   word(kc[1][j], 2 * h + 1)};
            mma16816(x[i], a, word(q[i][j], 2 * h), word(q[i][j], 2 * h + 1));
          }
        }
      }
      if (next < s.j1) load_k(at_next, next);
      const bool live0 = at >= 0 && t + r < s.j1, live1 = at >= 0 && t + r + 8 < s.j1;
      bool grows = false;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[i][e] = (e < 2 ? live0 : live1) ? x[i][e] * k.scale : -INFINITY;
          grows |= x[i][e] > m[i][e & 1] + kSlack;
        }
        if (k.scores) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int g = i * 8 + 2 * c4 + (e & 1), j = t + r + 8 * (e >> 1);
            if (g < s.gn && j < s.j1) k.scores[((int64_t)s.b * k.Hq + s.head0 + g) * capacity + j] = x[i][e];
          }
        }
      }
      if (__any_sync(0xffffffffu, grows)) {  // the first tile, and then rarely
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(x[i][e], x[i][e + 2]);
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
            top = fmaxf(top, m[i][e]);
            const float f = top == -INFINITY ? 1.f : exp2_approx(m[i][e] - top);
            m[i][e] = top;
            l[i][e] *= f;
#pragma unroll
            for (int w = 0; w < VC * 4; ++w) {
              o[i][w][e] *= f;
              o[i][w][e + 2] *= f;
            }
          }
        }
      }
      uint32_t hi[NT][2], lo[NT][2];  // B fragments
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        // A masked score is -inf; where no finite one has been met, so is m.
        const float ref[2] = {m[i][0] == -INFINITY ? 0.f : m[i][0], m[i][1] == -INFINITY ? 0.f : m[i][1]};
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = exp2_approx(x[i][e] - ref[e & 1]);
        l[i][0] += p[0] + p[2];
        l[i][1] += p[1] + p[3];
        // Two bf16 operands each, a probability cut off and what that leaves of it: within 2^-16,
        // where a single one would be off by 2^-8.  Both are positive where the probability is,
        // so that an infinite value stays one.  In a graph 64 ragged sequences on 4 key heads of
        // 128 take 167 us, with one operand too; 8 of 16,384 slots on 4 key heads of 64, 16 query
        // heads each, 32.7 us, 30.9 with one.
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t x0 = __float_as_uint(p[2 * e]), x1 = __float_as_uint(p[2 * e + 1]);
          const __nv_bfloat162 rest = __floats2bfloat162_rn(remainder_of(p[2 * e]), remainder_of(p[2 * e + 1]));
          hi[i][e] = transpose8x8(__byte_perm(x0, x1, 0x7632));
          lo[i][e] = transpose8x8(*reinterpret_cast<const uint32_t*>(&rest));
        }
      }
#pragma unroll
      for (int j = 0; j < VC; ++j) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a[4] = {__byte_perm(word(vc[0][j], w), word(vc[1][j], w), 0x5410),
                                 __byte_perm(word(vc[0][j], w), word(vc[1][j], w), 0x7632),
                                 __byte_perm(word(vc[2][j], w), word(vc[3][j], w), 0x5410),
                                 __byte_perm(word(vc[2][j], w), word(vc[3][j], w), 0x7632)};
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            mma16816(o[i][j * 4 + w], a, lo[i][0], lo[i][1]);
            mma16816(o[i][j * 4 + w], a, hi[i][0], hi[i][1]);
          }
        }
      }
      if (next < s.j1) load_v(at_next, next);
      t = next;
      at = at_next;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int g = i * 8 + 2 * c4 + e;
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], y);
#pragma unroll
        for (int j = 0; j < VC; ++j) {
          float* p = &sm[warp][g][j * 64 + r * 8];
#pragma unroll
          for (int w = 0; w < 4; w += 2)
            *reinterpret_cast<float4*>(p + 2 * w) =
                make_float4(o[i][j * 4 + w][e], o[i][j * 4 + w][e + 2], o[i][j * 4 + w + 1][e], o[i][j * 4 + w + 1][e + 2]);
        }
        if (r == 0) {
          sm[warp][g][D] = m[i][e];
          sm[warp][g][D + 1] = l[i][e];
        }
      }
    }
  }
};

// Walks a block's range of tiles, segment by segment.
template <class Core>
__global__ void __launch_bounds__(kDecThreads, Core::kBlocks)
decode_kernel(const __grid_constant__ DecodeCall k) {
  using T = typename Core::T;
  constexpr int D = Core::D, NP = Core::kParts;
  __shared__ __align__(16) float sm_o[NP][Core::kHeads][D + 4];
  __shared__ uint32_t warp_sums[kWarps];
  __shared__ int s_b;
  __shared__ int64_t s_first;
  const int tid = threadIdx.x;
  const int Hv = k.c.H * k.nv;
  cudaTriggerProgrammaticLaunchCompletion();

  // Empty sequences are answered by the blocks in turn, behind their own work.
  auto answer_empty = [&] {
    for (int b = blockIdx.x; b < k.c.B; b += gridDim.x) {
      const int len = k.c.lengths[b];
      if (tid == 0 && (len < 0 || len > k.c.width << k.page_shift)) atomicOr(k.status, kStatusPage);
      if (len > 0) continue;
      for (int64_t i = tid; i < (int64_t)k.Hq * D; i += kDecThreads)
        static_cast<T*>(k.o)[(int64_t)b * k.Hq * D + i] = (T)0.f;
      for (int i = tid; i < k.Hq; i += kDecThreads) k.lse[(int64_t)b * k.Hq + i] = -INFINITY;
    }
  };
  // Tiles of a key head in all sequences; those of the first 128 are kept, for most
  // batches are no larger.
  auto tiles = [&](int b) { return b < k.c.B ? (uint32_t)tiles_of(seq_length(k, b)) : 0u; };
  uint32_t mine = tiles(tid), here;
  uint32_t before = scan_tiles(mine, warp_sums, &here);
  int64_t sum = here;
  for (int b0 = kDecThreads; b0 < k.c.B; b0 += kDecThreads) {
    uint32_t more;
    scan_tiles(tiles(b0 + tid), warp_sums, &more);
    sum += more;
  }
  const int64_t T_all = sum * Hv;
  const int W = ranges(k, T_all);
  if ((int)blockIdx.x >= W) {
    answer_empty();
    return;
  }
  int64_t u = range_begin(blockIdx.x, T_all, W);
  const int64_t u_begin = u, u_end = range_begin(blockIdx.x + 1, T_all, W);

  // The sequence that tile u lies in: the one whose tiles, Hv times, enclose it.
  const int64_t x = u / Hv;
  int64_t base = 0;
  for (int b0 = 0;; b0 += kDecThreads) {
    if (b0 > 0) {
      mine = tiles(b0 + tid);
      before = scan_tiles(mine, warp_sums, &here);
    }
    if (x >= base + before && x < base + before + mine) {
      s_b = b0 + tid;
      s_first = (base + before) * Hv;
    }
    base += here;
    if (x < base) break;
  }
  __syncthreads();
  int b = s_b;
  int64_t first = s_first;  // first tile of sequence b

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
    Segment s;
    s.b = b;
    s.h = hv / k.nv;
    const int g0 = hv % k.nv * k.gv;
    s.gn = min(k.gv, k.G - g0);
    s.head0 = s.h * k.G + g0;
    s.j0 = (int)(u - seg0) * kTile;
    s.j1 = (int)min((int64_t)n, (stop - seg0) * kTile);
    Core::run(k, s, sm_o);
    __syncthreads();
    const bool whole = u == seg0 && stop == seg1;
    // The segment that begins the range leaves its part in slot 0, one that
    // begins inside it and goes on behind it in slot 1.
    const int slot = u == u_begin ? 0 : 1;
    float* part_out = k.part + ((int64_t)blockIdx.x * 2 + slot) * k.gv * (D + 4);
    for (int i = tid; i < s.gn * D; i += kDecThreads) {
      const int g = i / D, e = i % D;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < NP; ++w) top = fmaxf(top, sm_o[w][g][D]);
      float acc = 0.f, tot = 0.f;
#pragma unroll
      for (int w = 0; w < NP; ++w) {
        const float mw = sm_o[w][g][D];
        const float f = mw == -INFINITY ? 0.f : exp2f(mw - top);
        acc += f * sm_o[w][g][e];
        tot += f * sm_o[w][g][D + 1];
      }
      if (whole) {
        const int64_t row = (int64_t)b * k.Hq + s.head0 + g;
        static_cast<T*>(k.o)[row * D + e] = (T)(tot == 0.f ? 0.f : acc / tot);
        if (e == 0) k.lse[row] = tot == 0.f ? -INFINITY : (top + log2f(tot)) * kLn2;
      } else {
        part_out[g * (D + 4) + e] = acc;
        if (e == 0) {
          part_out[g * (D + 4) + D] = top;
          part_out[g * (D + 4) + D + 1] = tot;
        }
      }
    }
    __syncthreads();
    u = stop;
  }
  answer_empty();
}

// Where the parts of a query head are: part c is the row of `of(c)`, c < count;
// none (count 0) where one range held the whole sequence and wrote its answer.
template <int D>
struct Parts {
  const float* base;
  int64_t stride;
  int count, late;
  __device__ __forceinline__ const float* of(int c) const {
    return base + (2 * (int64_t)c + (c == 0 ? late : 0)) * stride;
  }
};

template <int D>
__device__ __forceinline__ Parts<D> parts_of(const DecodeCall& k, int head, int64_t first, int nt, int64_t T_all, int W) {
  const int g = head % k.G;
  const int hv = head / k.G * k.nv + g / k.gv;
  const int64_t seg0 = first + (int64_t)hv * nt, seg1 = seg0 + nt;
  const int c0 = range_of(seg0, T_all, W), c1 = range_of(seg1 - 1, T_all, W);
  Parts<D> p;
  p.stride = (int64_t)k.gv * (D + 4);
  p.base = k.part + (int64_t)c0 * 2 * p.stride + (int64_t)(g % k.gv) * (D + 4);
  p.late = range_begin(c0, T_all, W) < seg0;  // range c0 holds another segment before: slot 1
  p.count = c0 == c1 ? 0 : c1 - c0 + 1;
  return p;
}

// Adds (m, l) to a running pair; returns the factors of the two sides.
__device__ __forceinline__ float2 merge(float& m, float& l, float m2, float l2) {
  const float top = fmaxf(m, m2);
  const float2 f = make_float2(m == -INFINITY ? 0.f : exp2f(m - top), m2 == -INFINITY ? 0.f : exp2f(m2 - top));
  m = top;
  l = l * f.x + l2 * f.y;
  return f;
}

// Joins the parts of a query head and, with weights, adds the probabilities to
// the slots of a key head.  A block of the first kind answers one head: its
// parts fall in 16 classes, a warp's of one class in turn, so that one load
// latency serves them all, and the classes are joined in their order; NT threads
// do not show in the bits.  A block of the second kind works out the lse of its
// key head's queries, a warp each, and adds kJoinSlots slots.  Grid: per
// (sequence, key head), G blocks of the first kind, then those of the second.
// Launched while decode_kernel still runs: what it needs of lengths and ranges is
// worked out before the wait.  Every block waits, those without work too: the next
// launch of the stream waits for this one alone, and must find decode_kernel done.
template <typename T, int D, int NT, bool with_weights>
__global__ void __launch_bounds__(NT)
join_kernel(const __grid_constant__ DecodeCall k) {
  constexpr int NW = NT / 32, E = D / 32, kClasses = 16, kPer = kClasses / NW, kChunk = 32;
  __shared__ Pair warp_sums[NW];
  __shared__ float s_m[kClasses], s_l[kClasses], s_acc[kClasses][D], s_lse[kChunk];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t capacity = (int64_t)k.c.width << k.page_shift;
  const int per = k.G + (with_weights ? k.slot_blocks : 0);
  const int64_t bh = blockIdx.x / per;
  const int kind = (int)(blockIdx.x - bh * per);
  const int b = (int)(bh / k.c.H), h = (int)(bh % k.c.H);
  const int n = seq_length(k, b);
  const int slot0 = (kind - k.G) * kJoinSlots;
  if (n == 0 || slot0 >= n) {  // decode_kernel has answered an empty sequence
    cudaGridDependencySynchronize();
    return;
  }

  Pair sum{0, 0};  // tiles of a key head in all sequences, and in those before
  for (int i = tid; i < k.c.B; i += NT) {
    const int64_t t = tiles_of(seq_length(k, i));
    sum.x += t;
    if (i < b) sum.y += t;
  }
  const int Hv = k.c.H * k.nv;
  sum = block_sum<NT>(sum, warp_sums);
  const int64_t T_all = sum.x * Hv, first = sum.y * Hv;
  const int nt = tiles_of(n);
  const int W = ranges(k, T_all);

  if (kind < k.G) {
    const int head = h * k.G + kind;
    const int64_t row = (int64_t)b * k.Hq + head;
    const Parts<D> parts = parts_of<D>(k, head, first, nt, T_all, W);
    cudaGridDependencySynchronize();
    if (parts.count == 0) return;
    float acc[kPer][E], m[kPer], l[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[i][e] = 0.f;
    }
    // Many blocks (kPer > 1): few registers, so that many are resident.  Few blocks,
    // perhaps of hundreds of parts: four parts of a class in flight (one head of 524,288
    // slots 38 -> 30 us; with four in the other form as well, 32 ragged sequences 24 -> 28 us).
    constexpr int kBatch = kPer == 1 ? 4 : 1;
#pragma unroll(kPer == 1 ? 1 : 2)
    for (int c = 0; c < parts.count; c += kClasses * kBatch) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        float v[kBatch][E], pm[kBatch], pl[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          const int x = c + q * kClasses + warp + NW * i;
          if (kBatch == 1 && x >= parts.count) continue;
          const bool in = x < parts.count;
          const float* p = parts.of(in ? x : 0);
          pm[q] = in ? p[D] : -INFINITY;
          pl[q] = in ? p[D + 1] : 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) v[q][e] = in ? p[lane + 32 * e] : 0.f;
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          if (kBatch == 1 && c + warp + NW * i >= parts.count) continue;
          const float2 f = merge(m[i], l[i], pm[q], pl[q]);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[i][e] = acc[i][e] * f.x + v[q][e] * f.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
#pragma unroll
      for (int e = 0; e < E; ++e) s_acc[warp + NW * i][lane + 32 * e] = acc[i][e];
      if (lane == 0) {
        s_m[warp + NW * i] = m[i];
        s_l[warp + NW * i] = l[i];
      }
    }
    __syncthreads();
    for (int e = tid; e < D; e += NT) {
      float top = -INFINITY, tot = 0.f, v = 0.f;
#pragma unroll
      for (int w = 0; w < kClasses; ++w) top = fmaxf(top, s_m[w]);
#pragma unroll
      for (int w = 0; w < kClasses; ++w) {
        const float f = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - top);
        tot += f * s_l[w];
        v += f * s_acc[w][e];
      }
      static_cast<T*>(k.o)[row * D + e] = (T)(tot == 0.f ? 0.f : v / tot);
      if (e == 0) k.lse[row] = tot == 0.f ? -INFINITY : (top + log2f(tot)) * kLn2;
    }
    return;
  }

  static_assert(!with_weights || kJoinSlots == 4 * NT, "four slots a thread");
  const int j0 = slot0 + tid * 4;
  const int64_t slots = bh * capacity;
  float4 add = make_float4(0.f, 0.f, 0.f, 0.f);
  if (j0 < n) add = *reinterpret_cast<const float4*>(k.weights + slots + j0);
  cudaGridDependencySynchronize();
  for (int h0 = 0; h0 < k.G; h0 += kChunk) {
    const int heads = min(kChunk, k.G - h0);
    __syncthreads();
    for (int i = warp; i < heads; i += NW) {
      const int head = h * k.G + h0 + i;
      const Parts<D> parts = parts_of<D>(k, head, first, nt, T_all, W);
      float lse2;
      if (parts.count == 0) {
        lse2 = k.lse[(int64_t)b * k.Hq + head] * kLog2e;
      } else {
        float m = -INFINITY, l = 0.f;
        for (int c = lane; c < parts.count; c += 32) {
          const float* p = parts.of(c);
          merge(m, l, p[D], p[D + 1]);
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) {
          const float m2 = __shfl_xor_sync(0xffffffffu, m, x), l2 = __shfl_xor_sync(0xffffffffu, l, x);
          merge(m, l, m2, l2);
        }
        lse2 = m + log2f(l);
      }
      if (lane == 0) s_lse[i] = lse2;
    }
    __syncthreads();
    if (j0 >= n) continue;
    for (int i = 0; i < heads; ++i) {
      // Slots from n on hold nothing: their sums are not stored.
      const float4 s = *reinterpret_cast<const float4*>(
          k.scores + ((int64_t)b * k.Hq + h * k.G + h0 + i) * capacity + j0);
      add.x += s.x == -INFINITY ? 0.f : exp2f(s.x - s_lse[i]);
      add.y += s.y == -INFINITY ? 0.f : exp2f(s.y - s_lse[i]);
      add.z += s.z == -INFINITY ? 0.f : exp2f(s.z - s_lse[i]);
      add.w += s.w == -INFINITY ? 0.f : exp2f(s.w - s_lse[i]);
    }
  }
  if (j0 < n) {
    float* out = k.weights_out + slots + j0;
    if (j0 + 4 <= n) {
      *reinterpret_cast<float4*>(out) = add;
    } else {
      out[0] = add.x;
      if (j0 + 1 < n) out[1] = add.y;
      if (j0 + 2 < n) out[2] = add.z;
    }
  }
}

// Calls f.template operator()<Core>() for the core that serves gv query heads a
// key head.  Measured in a graph (us; 16,384 slots unless said otherwise):
//   bf16, 64 sequences on 4 key heads of 64: 8 heads 169 in one group of eight, 184 in two;
//     16 heads 192 in two groups, 331 as two parts of one group;
//   fp32, as heads of a warp x warps of a tile, channels 64 | 128:
//     1 (1 sequence of 98,304 slots, 1024 channels in all)   1x1 119 | 119, 2x1 128 | 123;
//     2 (4 sequences, 512 channels)      2x1 51 | 48, 1x2 60 | 56, 2x2 74 | 67;
//     3, 4 (32 sequences, 512 channels)  2x2 514 | 467, two parts in 2x1 646 | 636; 4x1 504,
//       but 2 sequences of 3000 slots on 2 key heads 8.8 in place of 8.1;
//     8 (the same)                       2x4 992 | 878, two parts of four 998 | 918;
//     16 (the same)                      4x4 1924, four parts of four 1984 | 1825, two of eight | 1744.
//   A core's time does not fall with the heads it lacks: 12 heads take 1921 | 1743, where three
//   parts of four would take 1490 | 1373.
template <typename F>
void with_core(int dtype, int d, int gv, F&& f) {
  if (dtype == LH_BF16) {
    if (d == 64) {
      if (gv <= 8) f.template operator()<MmaCore<64, 1>>();
      else f.template operator()<MmaCore<64, 2>>();
    } else {
      if (gv <= 8) f.template operator()<MmaCore<128, 1>>();
      else f.template operator()<MmaCore<128, 2>>();
    }
  } else if (d == 64) {
    if (gv == 1) f.template operator()<QuadCore<64, 1, 1>>();
    else if (gv == 2) f.template operator()<QuadCore<64, 2, 1>>();
    else if (gv <= 4) f.template operator()<QuadCore<64, 2, 2>>();
    else if (gv <= 8) f.template operator()<QuadCore<64, 2, 4>>();
    else f.template operator()<QuadCore<64, 4, 4>>();
  } else {
    if (gv == 1) f.template operator()<QuadCore<128, 1, 1>>();
    else if (gv == 2) f.template operator()<QuadCore<128, 2, 1>>();
    else if (gv <= 4) f.template operator()<QuadCore<128, 2, 2>>();
    else f.template operator()<QuadCore<128, 2, 4>>();
  }
}

struct Sizes {
  int nv, gv, blocks;
  int64_t part, scores;
};

Sizes sizes(const lh_cache& c, int64_t Hq, bool with_weights) {
  Sizes s{};
  const int64_t G = Hq / c.H;
  // Query heads that one block serves at most: 16, or 8 where an fp32 row of 128
  // channels leaves registers for no more.  More are cut into parts that each go through the
  // cache: 64 sequences of 16,384 slots on 4 key heads of 64 channels, bf16, take 192 us in a
  // graph with 16 heads a key head, 370 with 32 and 571 with 40.
  const int most_heads = c.dtype == LH_F32 && c.d == 128 ? 8 : 16;
  s.nv = (int)((G + most_heads - 1) / most_heads);
  s.gv = (int)((G + s.nv - 1) / s.nv);
  s.nv = (int)((G + s.gv - 1) / s.gv);
  const int64_t capacity = (int64_t)c.width * c.page;
  const int64_t most = (int64_t)c.B * c.H * s.nv * ((capacity + kTile - 1) / kTile);
  with_core(c.dtype, c.d, s.gv, [&]<typename Core>() { s.blocks = (int)std::min<int64_t>(most, 148 * Core::kBlocks); });
  s.part = ((int64_t)s.blocks * 2 * s.gv * (c.d + 4) * 4 + 255) & ~int64_t(255);
  s.scores = with_weights ? (int64_t)c.B * Hq * capacity * 4 : 0;
  return s;
}

}  // namespace

bool decode_fits(const lh_cache& c, int64_t Hq, bool with_weights) {
  const int64_t slots = with_weights ? ((int64_t)c.width * c.page + kJoinSlots - 1) / kJoinSlots : 0;
  return (int64_t)c.B * c.H * (Hq / c.H + slots) < (int64_t(1) << 31);
}

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
  k.slot_blocks = (int)(((int64_t)c.width * c.page + kJoinSlots - 1) / kJoinSlots);
  cudaError_t e = cudaSuccess;
  with_core(c.dtype, c.d, k.gv, [&]<typename Core>() {
    decode_kernel<Core><<<k.blocks, kDecThreads, 0, st>>>(k);
    e = cudaGetLastError();
    const int64_t capacity = (int64_t)c.width * c.page;
    if (e != cudaSuccess || (capacity <= kTile && !ww)) return;  // one tile a head: no range splits it
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((int64_t)c.B * c.H * (k.G + (ww ? k.slot_blocks : 0))));
    // One block an SM at most: many warps, for the parts are many; else few.
    const bool few = !ww && cfg.gridDim.x <= 148;
    cfg.blockDim = dim3(few ? 512 : kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute overlap{};
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &overlap;
    cfg.numAttrs = 1;
    using T = typename Core::T;
    constexpr int D = Core::D;
    e = cudaLaunchKernelEx(&cfg, ww ? join_kernel<T, D, kJoinThreads, true>
                                 : few ? join_kernel<T, D, 512, false> : join_kernel<T, D, kJoinThreads, false>, k);
  });
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace lh
