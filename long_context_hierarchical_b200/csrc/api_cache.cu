// C-ABI entry points of the rotary positions and the paged cache: validation
// of their arguments.  Nothing is enqueued for a call that is refused.
#include <math.h>
#include <stddef.h>
#include <string.h>

#include <algorithm>
#include <string>

#include "host.h"

using namespace lh;

namespace {

constexpr int64_t kMaxCapacity = (int64_t(1) << 31) - 65536;

bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

#define LH_CHECK_INDEX(ptr)                                                                     \
  do {                                                                                          \
    if (!aligned4(ptr)) return fail(LH_ERR_INVALID_ARG, #ptr " is null or not 4-byte aligned"); \
  } while (0)

lh_status check_type_dim(int32_t dtype, int32_t d) {
  if (dtype != LH_F32 && dtype != LH_BF16) return fail(LH_ERR_UNSUPPORTED, "dtype must be LH_F32 or LH_BF16");
  if (d != 64 && d != 128) return fail(LH_ERR_UNSUPPORTED, "only d in {64, 128} is built");
  return LH_OK;
}

bool positive(double x) { return isfinite(x) && x > 0; }

// A checksum of a rotary plan's config and frequencies: a plan is checked in every
// call, and working its frequencies out again would take longer than a small
// launch.
uint64_t plan_check(const lh_rotary_plan& p) {
  uint64_t words[(sizeof(lh_rotary_plan) - 8) / 8];
  static_assert(sizeof(words) == offsetof(lh_rotary_plan, check), "the checksum covers all before it");
  memcpy(words, &p, sizeof(words));
  uint64_t h = 0x243f6a8885a308d3ull;
  for (uint64_t w : words) h = (h ^ w ^ (h >> 29)) * 0x9e3779b97f4a7c15ull;
  return h;
}

lh_status check_rotary(const lh_rotary_plan* plan) {
  if (!plan) return fail(LH_ERR_INVALID_ARG, "null rotary plan");
  if (plan->check != plan_check(*plan))
    return fail(LH_ERR_INVALID_ARG, "rotary plan does not match its config (not from lh_rotary_init?)");
  return LH_OK;
}

// A [B, H, N, d] tensor: pointer, alignment of every row, sizes.
lh_status check_rows(const lh_rows* x, const char* name, int64_t B, int64_t N, int32_t dtype, bool output,
                     int32_t d) {
  const std::string at(name);
  if (!x) return fail(LH_ERR_INVALID_ARG, at + " is null");
  if (x->H < 1 || x->H > 65535) return fail(LH_ERR_INVALID_ARG, at + ": H must be in 1..65535");
  if (!aligned16(x->ptr)) return fail(LH_ERR_INVALID_ARG, at + " is null or not 16-byte aligned");
  const int64_t es = dtype == LH_BF16 ? 2 : 4;
  struct Dim { int64_t size, stride; } dim[3] = {{B, x->stride_b}, {x->H, x->stride_h}, {N, x->stride_n}};
  for (const Dim& v : dim) {
    if (v.size <= 1) continue;
    if (v.stride < 0) return fail(LH_ERR_INVALID_ARG, at + ": negative stride");
    if (v.stride * es % 16 != 0) return fail(LH_ERR_INVALID_ARG, at + ": rows must start on 16-byte boundaries");
    if (v.stride > (int64_t(1) << 58) / v.size) return fail(LH_ERR_INVALID_ARG, at + ": stride too large");
  }
  if (output) {  // no two rows may overlap
    std::sort(dim, dim + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    int64_t extent = d;
    for (const Dim& v : dim) {
      if (v.size <= 1) continue;
      if (v.stride < extent) return fail(LH_ERR_INVALID_ARG, at + ": rows of an output overlap");
      extent += v.stride * (v.size - 1);
    }
  }
  return LH_OK;
}

int64_t span_bytes(const lh_rows& x, int64_t B, int64_t N, int32_t dtype, int32_t d) {
  const int64_t last = (B - 1) * (B > 1 ? x.stride_b : 0) + (x.H - 1) * (x.H > 1 ? x.stride_h : 0) +
                       (N - 1) * (N > 1 ? x.stride_n : 0) + d;
  return last * (dtype == LH_BF16 ? 2 : 4);
}

// An output is its input itself or lies apart from it.
lh_status check_pair(const lh_rows& x, const lh_rows& y, const char* name, int64_t B, int64_t N, int32_t dtype,
                     int32_t d) {
  if (x.H != y.H) return fail(LH_ERR_INVALID_ARG, std::string(name) + ": input and output differ in H");
  const bool same = x.ptr == y.ptr && (B == 1 || x.stride_b == y.stride_b) &&
                    (x.H == 1 || x.stride_h == y.stride_h) && (N == 1 || x.stride_n == y.stride_n);
  if (same) return LH_OK;
  const char* a = static_cast<const char*>(x.ptr);
  const char* c = static_cast<const char*>(y.ptr);
  if (a < c + span_bytes(y, B, N, dtype, d) && c < a + span_bytes(x, B, N, dtype, d))
    return fail(LH_ERR_INVALID_ARG, std::string(name) + ": output overlaps its input without being the same rows");
  return LH_OK;
}

// An in-place array: the output is the input itself or lies apart from it.
bool same_or_apart(const void* in, const void* out, int64_t bytes) {
  const char *a = static_cast<const char*>(in), *c = static_cast<const char*>(out);
  return a == c || a + bytes <= c || c + bytes <= a;
}

RowsArg rows_arg(const lh_rows* x) {
  if (!x) return RowsArg{};
  return RowsArg{x->ptr, x->stride_b, x->stride_h, x->stride_n, (int)x->H};
}

lh_status check_cache(const lh_cache* c, bool pointers = true) {
  if (!c) return fail(LH_ERR_INVALID_ARG, "null cache");
  lh_status s = check_type_dim(c->dtype, c->d);
  if (s != LH_OK) return s;
  if (c->pages < 1 || c->H < 1 || c->B < 1 || c->width < 1)
    return fail(LH_ERR_INVALID_ARG, "pages, H, B and width must be >= 1");
  if (c->page < 16 || c->page > 65536 || (c->page & (c->page - 1)))
    return fail(LH_ERR_UNSUPPORTED, "only pages of a power of two, 16 to 65536 rows, are built");
  if (c->pages >= int64_t(1) << 31) return fail(LH_ERR_UNSUPPORTED, "pages must stay below 2^31");
  if (c->H > 65535 || (int64_t)c->B * c->H > 65535)
    return fail(LH_ERR_UNSUPPORTED, "B * H above 65535 is not built");
  if ((int64_t)c->width * c->page > kMaxCapacity)
    return fail(LH_ERR_UNSUPPORTED, "capacity (width * page) must stay below 2^31 - 2^16");
  if (!pointers) return LH_OK;
  if (c->table_stride < 0 || (c->B > 1 && c->table_stride > (int64_t(1) << 60) / c->B))
    return fail(LH_ERR_INVALID_ARG, "table_stride out of range");
  const void *k = c->k, *v = c->v, *table = c->table, *lengths = c->lengths;
  LH_CHECK_PTR(k); LH_CHECK_PTR(v);
  LH_CHECK_INDEX(table); LH_CHECK_INDEX(lengths);
  const int64_t page_bytes = (int64_t)c->H * c->page * c->d * (c->dtype == LH_BF16 ? 2 : 4);
  if (c->pages > (int64_t(1) << 60) / page_bytes) return fail(LH_ERR_INVALID_ARG, "a cache of more than 2^60 bytes");
  const int64_t bytes = c->pages * page_bytes;
  if (k == v || !same_or_apart(k, v, bytes)) return fail(LH_ERR_INVALID_ARG, "k and v overlap");
  return LH_OK;
}

lh_status check_heads(const lh_cache* c, int64_t Hq, bool with_weights) {
  if (Hq < 1 || Hq % c->H != 0) return fail(LH_ERR_INVALID_ARG, "Hq must be a multiple of the cache's H");
  if ((int64_t)c->B * Hq > (int64_t(1) << 22)) return fail(LH_ERR_UNSUPPORTED, "B * Hq above 2^22 is not built");
  if (!decode_fits(*c, Hq, with_weights))
    return fail(LH_ERR_UNSUPPORTED, "weights of more than about 2^40 slots are not built");
  return LH_OK;
}

int64_t slots_bytes(const lh_cache* c) { return (int64_t)c->B * c->H * c->width * c->page * 4; }

}  // namespace

extern "C" {

int64_t lh_rotary_plan_bytes(void) { return (int64_t)sizeof(lh_rotary_plan); }
int64_t lh_cache_bytes(void) { return (int64_t)sizeof(lh_cache); }

lh_status lh_rotary_init(const lh_rotary_config* cfg, lh_rotary_plan* out) {
  if (!cfg || !out) return fail(LH_ERR_INVALID_ARG, "null config or plan");
  const lh_rotary_config c = *cfg;
  if (c.rot < 1 || c.rot > c.d) return fail(LH_ERR_INVALID_ARG, "rot must be in 1..d");
  if (c.layout != LH_ROTARY_HALF && c.layout != LH_ROTARY_INTERLEAVED)
    return fail(LH_ERR_INVALID_ARG, "layout must be LH_ROTARY_HALF or LH_ROTARY_INTERLEAVED");
  if (c.scaling != LH_SCALE_NONE && c.scaling != LH_SCALE_LINEAR && c.scaling != LH_SCALE_BANDS)
    return fail(LH_ERR_INVALID_ARG, "scaling must be LH_SCALE_NONE, LH_SCALE_LINEAR or LH_SCALE_BANDS");
  if (!positive(c.base) || !positive(c.magnitude))
    return fail(LH_ERR_INVALID_ARG, "base and magnitude must be positive and finite");
  if (c.scaling != LH_SCALE_NONE && !positive(c.factor))
    return fail(LH_ERR_INVALID_ARG, "factor must be positive and finite");
  if (c.scaling == LH_SCALE_BANDS &&
      (!positive(c.original) || !isfinite(c.low) || !isfinite(c.high) || c.low < 0 || c.high <= c.low))
    return fail(LH_ERR_INVALID_ARG, "bands need original > 0 and 0 <= low < high");
  if (c.d != 64 && c.d != 128) return fail(LH_ERR_UNSUPPORTED, "only d in {64, 128} is built");
  if (c.rot % 16 != 0) return fail(LH_ERR_UNSUPPORTED, "only rot in multiples of 16 is built");
  lh_rotary_plan p{};
  p.c = c;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  for (int i = 0; i < c.rot / 2; ++i) {
    double f = pow(c.base, -2.0 * i / c.rot);
    if (c.scaling == LH_SCALE_LINEAR) f /= c.factor;
    if (c.scaling == LH_SCALE_BANDS) {
      const double g = std::min(1.0, std::max(0.0, (c.original * f / kTwoPi - c.low) / (c.high - c.low)));
      f = (1.0 - g) * f / c.factor + g * f;
    }
    const double turns = f / kTwoPi;
    if (!isfinite(turns)) return fail(LH_ERR_INVALID_ARG, "a frequency is not finite");
    const double frac = turns - floor(turns);  // in [0, 1]: whole turns are none
    p.turns[i] = frac < 1.0 ? (uint64_t)(frac * 0x1p64) : 0;
  }
  p.check = plan_check(p);
  *out = p;
  return ok();
}

lh_status lh_rotary(const lh_rotary_plan* plan, int32_t dtype, int64_t B, int64_t N, int32_t count,
                    const lh_rows* X, const lh_rows* Y, const int32_t* positions,
                    int64_t positions_stride, int64_t start, int32_t transpose,
                    lh_stream_t stream) {
  Range range("lh_rotary");
  LH_TRY(check_rotary(plan));
  LH_TRY(check_type_dim(dtype, plan->c.d));
  if (B < 0 || N < 0 || (N > 0 && B > (int64_t(1) << 31) / N))
    return fail(LH_ERR_INVALID_ARG, "B and N must be >= 0 and B * N at most 2^31");
  if (count != 1 && count != 2) return fail(LH_ERR_INVALID_ARG, "count must be 1 or 2");
  if (!X || !Y) return fail(LH_ERR_INVALID_ARG, "X or Y is null");
  if (B == 0 || N == 0) return ok();
  if (!positions && (start < -(int64_t(1) << 31) || start > (int64_t(1) << 31) - N))
    return fail(LH_ERR_INVALID_ARG, "positions must fit 32 bits");
  RowsArg x[2] = {}, y[2] = {};
  for (int i = 0; i < count; ++i) {
    LH_TRY(check_rows(X + i, "X", B, N, dtype, false, plan->c.d));
    LH_TRY(check_rows(Y + i, "Y", B, N, dtype, true, plan->c.d));
    LH_TRY(check_pair(X[i], Y[i], "X, Y", B, N, dtype, plan->c.d));
    x[i] = rows_arg(X + i);
    y[i] = rows_arg(Y + i);
  }
  if (count == 2 && (Y[0].ptr == Y[1].ptr || Y[0].ptr == X[1].ptr || Y[1].ptr == X[0].ptr))
    return fail(LH_ERR_INVALID_ARG, "Y: an output overlaps another tensor of the call");
  if (x[0].H + x[1].H > 65535) return fail(LH_ERR_UNSUPPORTED, "more than 65535 heads");
  if (positions) {
    LH_CHECK_INDEX(positions);
    if (positions_stride < 0) return fail(LH_ERR_INVALID_ARG, "positions_stride must be >= 0");
  }
  LH_TRY(cuda_status(launch_rotary(*plan, dtype, B, N, count, x, y, positions, positions_stride, start,
                                   transpose != 0, as_cuda(stream)), "lh_rotary"));
  return ok();
}

lh_status lh_cache_append(const lh_cache* cache, const lh_rotary_plan* rotary, int64_t T,
                          const lh_rows* K, const lh_rows* V, const lh_rows* Q, const lh_rows* Qo,
                          const int32_t* positions, int64_t positions_stride,
                          const int32_t* counts, int32_t* slot_positions, lh_stream_t stream) {
  Range range("lh_cache_append");
  LH_TRY(check_cache(cache));
  if (rotary) {
    LH_TRY(check_rotary(rotary));
    if (rotary->c.d != cache->d) return fail(LH_ERR_INVALID_ARG, "rotary plan and cache differ in d");
  }
  const int64_t B = cache->B;
  if (T < 0 || T > (int64_t(1) << 31) / B) return fail(LH_ERR_INVALID_ARG, "T must be >= 0 and B * T at most 2^31");
  if ((Q == nullptr) != (Qo == nullptr)) return fail(LH_ERR_INVALID_ARG, "Q and Qo: both or neither");
  if (T == 0) return ok();
  LH_TRY(check_rows(K, "K", B, T, cache->dtype, false, cache->d));
  LH_TRY(check_rows(V, "V", B, T, cache->dtype, false, cache->d));
  if (K->H != cache->H || V->H != cache->H)
    return fail(LH_ERR_INVALID_ARG, "K and V must have the cache's H");
  if (Q) {
    LH_TRY(check_rows(Q, "Q", B, T, cache->dtype, false, cache->d));
    LH_TRY(check_rows(Qo, "Qo", B, T, cache->dtype, true, cache->d));
    LH_TRY(check_pair(*Q, *Qo, "Q, Qo", B, T, cache->dtype, cache->d));
    if (Qo->ptr == K->ptr || Qo->ptr == V->ptr || Qo->ptr == cache->k || Qo->ptr == cache->v)
      return fail(LH_ERR_INVALID_ARG, "Qo: the output overlaps another tensor of the call");
    if (Q->H + 2 * cache->H > 65535) return fail(LH_ERR_UNSUPPORTED, "more than 65535 heads");
  }
  if (positions) {
    LH_CHECK_INDEX(positions);
    if (positions_stride < 0) return fail(LH_ERR_INVALID_ARG, "positions_stride must be >= 0");
  }
  if (counts) LH_CHECK_INDEX(counts);
  if (slot_positions) LH_CHECK_INDEX(slot_positions);
  LH_TRY(cuda_status(launch_cache_append(*cache, rotary, T, rows_arg(K), rows_arg(V), rows_arg(Q), rows_arg(Qo),
                                         positions, positions_stride, counts, slot_positions, as_cuda(stream)),
                     "lh_cache_append"));
  return ok();
}

int64_t lh_decode_ws_bytes(const lh_cache* cache, int64_t Hq, int32_t with_weights) {
  if (check_cache(cache, false) != LH_OK || check_heads(cache, Hq, with_weights != 0) != LH_OK) return -1;
  return decode_ws_bytes(*cache, Hq, with_weights != 0);
}

lh_status lh_decode(const lh_cache* cache, const lh_rows* Q, float scale, void* O, float* lse,
                    const float* weights, float* weights_out, void* ws, size_t ws_bytes,
                    lh_stream_t stream) {
  Range range("lh_decode");
  LH_TRY(check_cache(cache));
  LH_TRY(check_rows(Q, "Q", cache->B, 1, cache->dtype, false, cache->d));
  LH_TRY(check_heads(cache, Q->H, weights != nullptr));
  if (!isfinite(scale * 2.f)) return fail(LH_ERR_INVALID_ARG, "scale must be finite and below 2^127");
  LH_CHECK_PTR(O);
  LH_CHECK_INDEX(lse);
  if ((weights == nullptr) != (weights_out == nullptr))
    return fail(LH_ERR_INVALID_ARG, "weights and weights_out: both or neither");
  if (weights) { LH_CHECK_PTR(weights); LH_CHECK_PTR(weights_out); }
  if (weights && !same_or_apart(weights, weights_out, slots_bytes(cache)))
    return fail(LH_ERR_INVALID_ARG, "weights_out overlaps weights without being the same array");
  LH_CHECK_PTR(ws);
  if ((int64_t)ws_bytes < decode_ws_bytes(*cache, Q->H, weights != nullptr))
    return fail(LH_ERR_WORKSPACE, "lh_decode workspace smaller than lh_decode_ws_bytes()");
  LH_TRY(cuda_status(launch_decode(*cache, rows_arg(Q), scale, O, lse, weights, weights_out, ws, as_cuda(stream)),
                     "lh_decode"));
  return ok();
}

int64_t lh_evict_ws_bytes(const lh_cache* cache, int64_t budget) {
  if (check_cache(cache, false) != LH_OK) return -1;
  if (budget < 1) {
    fail(LH_ERR_INVALID_ARG, "budget must be >= 1");
    return -1;
  }
  return evict_ws_bytes(*cache, budget);
}

lh_status lh_evict(const lh_cache* cache, int64_t budget, const float* weights,
                   const int32_t* positions, const int32_t* protect, float* weights_out,
                   int32_t* positions_out, int32_t* lengths_out, void* ws, size_t ws_bytes,
                   lh_stream_t stream) {
  Range range("lh_evict");
  LH_TRY(check_cache(cache));
  if (budget < 1) return fail(LH_ERR_INVALID_ARG, "budget must be >= 1");
  LH_CHECK_PTR(weights); LH_CHECK_PTR(weights_out);
  if ((positions == nullptr) != (positions_out == nullptr))
    return fail(LH_ERR_INVALID_ARG, "positions and positions_out: both or neither");
  if (positions) { LH_CHECK_PTR(positions); LH_CHECK_PTR(positions_out); }
  if (!same_or_apart(weights, weights_out, slots_bytes(cache)) ||
      (positions && !same_or_apart(positions, positions_out, slots_bytes(cache))))
    return fail(LH_ERR_INVALID_ARG, "an output overlaps its input without being the same array");
  if (protect) LH_CHECK_INDEX(protect);
  LH_CHECK_INDEX(lengths_out);
  if (lengths_out < cache->lengths + cache->B && cache->lengths < lengths_out + cache->B)
    return fail(LH_ERR_INVALID_ARG, "lengths_out must not overlap the cache's lengths");
  LH_CHECK_PTR(ws);
  if ((int64_t)ws_bytes < evict_ws_bytes(*cache, budget))
    return fail(LH_ERR_WORKSPACE, "lh_evict workspace smaller than lh_evict_ws_bytes()");
  LH_TRY(cuda_status(launch_evict(*cache, budget, weights, positions, protect, weights_out, positions_out,
                                  lengths_out, ws, as_cuda(stream)), "lh_evict"));
  return ok();
}

}  // extern "C"
