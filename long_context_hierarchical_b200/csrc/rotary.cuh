// Rotation of 16-channel units of a row, shared by the rotary and the cache
// append kernels.
//
// A thread owns one unit: the 8 + 8 channels of eight pairs (two 16-byte
// chunks in bf16).  In the half layout these are the chunks u and u + rot/16,
// in the interleaved one 2u and 2u + 1; units behind the turned channels are
// copied.  The eight sines and cosines of a (position, unit) serve every head.
#pragma once

#include "common.cuh"

namespace lh {

// lh_rotary_plan as a kernel argument.
struct RotaryArg {
  uint64_t turns[LH_MAX_PAIRS];
  float magnitude;
  int units;  // turned units of a row: rot / 16
  int half;   // LH_ROTARY_HALF
};

inline RotaryArg make_rotary_arg(const lh_rotary_plan* p) {
  RotaryArg r{};
  r.magnitude = 1.f;
  if (!p) return r;
  for (int i = 0; i < LH_MAX_PAIRS; ++i) r.turns[i] = p->turns[i];
  r.magnitude = (float)p->c.magnitude;
  r.units = p->c.rot / 16;
  r.half = p->c.layout == LH_ROTARY_HALF;
  return r;
}

struct Unit {
  int ca, cb;  // its two 8-channel chunks
  bool turn;
};

__device__ __forceinline__ Unit make_unit(const RotaryArg& r, int u) {
  Unit x;
  x.turn = u < r.units;
  const bool split = r.half && x.turn;
  x.ca = split ? u : 2 * u;
  x.cb = split ? u + r.units : 2 * u + 1;
  return x;
}

// The frequencies in shared memory: a thread reads eight of its own, which as an
// indexed kernel argument would be one access for each unit in the warp.
__device__ __forceinline__ void stage_turns(const RotaryArg& r, uint64_t* s_turns) {
  if (threadIdx.x < r.units * 8) s_turns[threadIdx.x] = r.turns[threadIdx.x];
  __syncthreads();
}

// Sines and cosines of the unit's eight pairs.  The angle is a 64-bit fraction
// of a turn: position * turns wraps modulo one turn exactly (negative
// positions too), so the reduction costs no digits at any position.  Its upper 32
// bits, in [-1/2, 1/2) turns and cut off by at most 2^-32 of one, are then
// converted to fp32, which rounds by up to 2^-25 of a half turn.
__device__ __forceinline__ void unit_angles(const RotaryArg& r, const uint64_t* s_turns, int u, int64_t pos,
                                            bool transpose, float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int phase = (int)((uint64_t)pos * s_turns[u * 8 + j] >> 32);
    const float half_turns = __int2float_rn(phase) * 0x1p-31f;
    sincospif(half_turns, &s[j], &c[j]);
    c[j] *= r.magnitude;
    s[j] *= transpose ? -r.magnitude : r.magnitude;
  }
}

__device__ __forceinline__ void turn_unit(bool half, const float (&c)[8], const float (&s)[8],
                                          float (&a)[8], float (&b)[8]) {
  if (half) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = a[j], y = b[j];
      a[j] = x * c[j] - y * s[j];
      b[j] = y * c[j] + x * s[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = a[2 * j], y = a[2 * j + 1];
      a[2 * j] = x * c[j] - y * s[j];
      a[2 * j + 1] = y * c[j] + x * s[j];
      const float z = b[2 * j], w = b[2 * j + 1];
      b[2 * j] = z * c[j + 4] - w * s[j + 4];
      b[2 * j + 1] = w * c[j + 4] + z * s[j + 4];
    }
  }
}

// Eight channels as they lie in memory.  Plain loads: an output row may be
// the input row itself.
template <typename T>
struct Chunk {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    }
  }
};

}  // namespace lh
