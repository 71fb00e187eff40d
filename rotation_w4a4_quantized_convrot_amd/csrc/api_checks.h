// Host-side argument checks that the decoding entry points share (api_decode.hip, api_draft.hip).
#pragma once

#include "convrot.h"
#include "convrot_internal.h"

#include <initializer_list>

namespace {

constexpr int64_t kIntMax = 0x7FFFFFFF;
// A launch takes fewer than 2^32 threads along x; what would need more is refused here, before it
// becomes an error that the runtime keeps for a later call to find.
constexpr int64_t kMaxThreads = 0xFFFFFFFF;
constexpr int64_t kMaxStride = int64_t(1) << 46;   // elements; keeps every offset within 63 bits
constexpr int64_t kMaxBytes = int64_t(1) << 62;

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t elem_size(int32_t dtype) { return dtype == CONVROT_F32 ? 4 : dtype == CONVROT_BF16 ? 2 : 0; }
int status_of(hipError_t e) { return e == hipSuccess ? CONVROT_OK : CONVROT_ERR_HIP; }
bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

// A rotation window: 0 (none) or a power of 4 between 16 and `most`.
int check_window(int64_t g, int64_t most) {
  if (g == 0) return CONVROT_OK;
  if (convrot_is_power_of_4(g) == 0) return CONVROT_ERR_GROUP;
  return g >= 16 && g <= most ? CONVROT_OK : CONVROT_ERR_UNSUPPORTED;
}

bool launch_fits(int64_t workgroups, int64_t threads) { return workgroups <= kMaxThreads / threads; }

int check_cache(int64_t num_pages, int64_t page, int64_t H, int64_t D, int64_t g, int64_t B, int64_t T,
                int64_t max_pages, int64_t table_ld) {
  const int st = check_window(g, 256);
  if (st != CONVROT_OK) return st;
  if (num_pages < 1 || num_pages > kIntMax || H < 1 || D < 1 || B < 0 || T < 0 || T > kIntMax ||
      max_pages < 0 || max_pages > kIntMax || table_ld < max_pages || !stride_ok(table_ld))
    return CONVROT_ERR_SHAPE;
  if (page != 16 && page != 32 && page != 64 && page != 128) return CONVROT_ERR_UNSUPPORTED;
  if (D % 16 != 0 || D > 256 || (g != 0 && D % g != 0)) return CONVROT_ERR_UNSUPPORTED;
  if (H > 65535 || B > kMaxThreads / 256 / (2 * H)) return CONVROT_ERR_UNSUPPORTED;
  return CONVROT_OK;
}

int check_batch_pointers(const int32_t* cu, const int32_t* lens, const int32_t* table, int64_t max_pages,
                         const void* kc, const float* ks, const void* vc, const float* vs) {
  if (cu == nullptr || lens == nullptr || (table == nullptr && max_pages > 0) || kc == nullptr || ks == nullptr ||
      vc == nullptr || vs == nullptr)
    return CONVROT_ERR_NULL;
  if (!aligned(cu, 4) || !aligned(lens, 4) || !aligned(table, 4) || !aligned(kc, 16) || !aligned(vc, 16) ||
      !aligned(ks, 4) || !aligned(vs, 4))
    return CONVROT_ERR_ALIGN;
  return CONVROT_OK;
}

bool attention_shape_ok(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t max_new, int64_t max_len) {
  return T >= 0 && T <= kIntMax && B >= 0 && B <= kIntMax && H >= 1 && H <= 65535 && Hq >= 1 && Hq <= 65535 &&
         Hq % H == 0 && D >= 1 && max_new >= 0 && max_len >= 0 && max_new <= kIntMax && max_len <= kIntMax;
}

// Within these the plan's counts stay far inside 64 bits.
bool attention_plannable(int64_t T, int64_t B, int64_t Hq, int64_t H) {
  return T <= kIntMax / Hq && B <= kMaxThreads / 256 / (2 * H);
}

// The workspace of a plan; 0 for what the entry points refuse.
size_t attention_workspace(decltype(convrot::plan_kv8_attention)* plan_of, int64_t T, int64_t B, int64_t Hq, int64_t H,
                           int64_t D, int64_t max_new, int64_t max_len) {
  if (!attention_shape_ok(T, B, Hq, H, D, max_new, max_len) || !attention_plannable(T, B, Hq, H) || T == 0 ||
      B == 0 || D > 256 || D % 16 != 0)
    return 0;
  const convrot::Kv8Plan p = plan_of(B, T, Hq, H, D, max_new, max_len);
  return p.threads <= kMaxThreads ? p.bytes : 0;
}

// What the entry points for attention over the cache refuse, and the plan of a call; *nothing: there is nothing to do.
int check_attention(const void* q, int64_t q_t, int64_t q_h, int32_t dtype, int64_t T, int64_t Hq, const int32_t* cu,
                    const int32_t* lens, const int32_t* table, int64_t table_ld, int64_t B, int64_t max_pages,
                    const int8_t* kc, const float* ks, const int8_t* vc, const float* vs, int64_t num_pages,
                    int64_t page, int64_t H, int64_t D, int64_t g, int64_t max_new, int64_t max_len, const void* out,
                    const void* workspace, size_t ws_bytes, decltype(convrot::plan_kv8_attention)* plan_of,
                    convrot::Kv8Plan* p, bool* nothing) {
  int st = check_cache(num_pages, page, H, D, g, B, T, max_pages, table_ld);
  if (st != CONVROT_OK) return st;
  if (elem_size(dtype) == 0) return CONVROT_ERR_DTYPE;
  if (!attention_shape_ok(T, B, Hq, H, D, max_new, max_len) || !stride_ok(q_t) || !stride_ok(q_h))
    return CONVROT_ERR_SHAPE;
  *nothing = T == 0 || B == 0;
  if (*nothing) return CONVROT_OK;
  if (!attention_plannable(T, B, Hq, H)) return CONVROT_ERR_UNSUPPORTED;
  const convrot::Kv8Plan plan = *p = plan_of(B, T, Hq, H, D, max_new, max_len);
  if (plan.threads > kMaxThreads) return CONVROT_ERR_UNSUPPORTED;
  if (q == nullptr || out == nullptr || (plan.bytes > 0 && workspace == nullptr)) return CONVROT_ERR_NULL;
  st = check_batch_pointers(cu, lens, table, max_pages, kc, ks, vc, vs);
  if (st != CONVROT_OK) return st;
  if (!aligned(q, elem_size(dtype)) || !aligned(out, 16) || !aligned(workspace, 256)) return CONVROT_ERR_ALIGN;
  if (ws_bytes < plan.bytes) return CONVROT_ERR_WORKSPACE;
  return CONVROT_OK;
}

// Rows of D elements, one for each of T tokens and `heads` heads, as they stand in memory.
struct Rows {
  uintptr_t at;
  int64_t t, h, heads;
};

// Elements from the first row's first to behind the last row's last; -1 past what memory can hold.
int64_t span_of(const Rows& r, int64_t T, int64_t D) {
  const __int128 n = __int128(T - 1) * r.t + __int128(r.heads - 1) * r.h + D;
  return n < (int64_t(1) << 58) ? int64_t(n) : -1;
}

// Whether two rows (t, h) of a tensor meet, with head and token strides of at least D: some k heads' step is
// within D of some number of tokens' steps.
bool rows_meet(const Rows& r, int64_t T, int64_t D) {
  if (T == 1 || r.heads == 1 || r.t - (r.heads - 1) * r.h >= D || r.h - (T - 1) * r.t >= D) return false;
  for (int64_t k = 1; k < r.heads; ++k) {
    const int64_t below = k * r.h / r.t, off = k * r.h - below * r.t;
    if ((below >= 1 && below < T && off < D) || (below + 1 < T && r.t - off < D)) return true;
  }
  return false;
}

// Whether a row of a meets a row of b, elements of `size` bytes.  Exact where the tensors have one token stride
// (views of one buffer do) and up to 2^20 pairs of heads; else spans that reach into one another count.
bool rows_meet(const Rows& a, const Rows& b, int64_t T, int64_t D, int64_t size) {
  const int64_t an = span_of(a, T, D), bn = span_of(b, T, D);
  if (a.at + uintptr_t(an * size) <= b.at || b.at + uintptr_t(bn * size) <= a.at) return false;
  if (T > 1 && a.t != b.t) return true;
  const int64_t step = T > 1 ? a.t : 0, from = (int64_t(b.at) - int64_t(a.at)) / size;
  // the heads of a token side by side in each, and b's in the gap between a's
  const int64_t aw = (a.heads - 1) * a.h + D, bw = (b.heads - 1) * b.h + D;
  if (step > 0) {
    const int64_t gap = (from % step + step) % step;
    if (gap >= aw && gap + bw <= step) return false;
  }
  if (a.heads * b.heads > 1 << 20) return true;
  for (int64_t i = 0; i < a.heads; ++i)
    for (int64_t j = 0; j < b.heads; ++j) {
      const int64_t off = from + j * b.h - i * a.h;           // tokens apart by k: off + k step
      if (off > -D && off < D) return true;
      if (step == 0) continue;
      const int64_t far = off < 0 ? -off : off, below = far / step, rest = far - below * step;
      if ((below < T && rest < D) || (below + 1 < T && step - rest < D)) return true;
    }
  return false;
}

// A tensor [T][heads][D] that is turned, as the entry points get it.
struct TurnedPart {
  const void* in;
  int64_t in_t, in_h;
  void* out;
  int64_t out_t, out_h, heads;
};

bool apart(const void* a, int64_t an, const void* b, int64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x + uintptr_t(an) <= y || y + uintptr_t(bn) <= x;
}

// A tensor as bytes in memory.
struct Extent {
  const void* at;
  int64_t bytes;
};

// Whether the tensors that are not turned (NULL: none) lie apart from what is written, from each output's first element to
// its last.
bool apart_from_outputs(const TurnedPart (&part)[2], int32_t dtype, int64_t T, int64_t D,
                        std::initializer_list<Extent> others) {
  for (const auto& p : part) {
    if (p.heads == 0) continue;
    const int64_t span = span_of(Rows{0, p.out_t, p.out_h, p.heads}, T, D) * int64_t(elem_size(dtype));
    for (const Extent& o : others)
      if (o.at != nullptr && !apart(p.out, span, o.at, o.bytes)) return false;
  }
  return true;
}

// What the entry points for rotary positions refuse; *nothing: there is nothing to do.
int check_turned(const TurnedPart (&part)[2], int32_t dtype, int64_t T, int64_t D, int64_t R, const int64_t* pos,
                 const float* inv_freq, bool* nothing) {
  const size_t size = elem_size(dtype);
  if (size == 0) return CONVROT_ERR_DTYPE;
  if (T < 0 || T > kIntMax || part[0].heads < 0 || part[1].heads < 0 || D < 1 || R < 2 || R % 2 != 0 || R > D) return CONVROT_ERR_SHAPE;
  if (D > 1024 || part[0].heads > 65535 || part[1].heads > 65535 - part[0].heads || !launch_fits(T, 256)) return CONVROT_ERR_UNSUPPORTED;
  for (const auto& p : part) {
    if (p.heads == 0 || T == 0) continue;
    if (!stride_ok(p.in_t) || !stride_ok(p.in_h) || !stride_ok(p.out_t) || !stride_ok(p.out_h))
      return CONVROT_ERR_SHAPE;
    // rows of the output must not meet
    const Rows out{reinterpret_cast<uintptr_t>(p.out), p.out_t, p.out_h, p.heads};
    if ((p.heads > 1 && p.out_h < D) || (T > 1 && p.out_t < D) || span_of(out, T, D) < 0 || rows_meet(out, T, D))
      return CONVROT_ERR_SHAPE;
    if (p.in == p.out && ((T > 1 && p.in_t != p.out_t) || (p.heads > 1 && p.in_h != p.out_h)))
      return CONVROT_ERR_SHAPE;
    if (span_of(Rows{0, p.in_t, p.in_h, p.heads}, T, D) < 0) return CONVROT_ERR_SHAPE;
  }
  *nothing = T == 0 || part[0].heads + part[1].heads == 0;
  if (*nothing) return CONVROT_OK;
  for (const auto& p : part) {
    if (p.heads == 0) continue;
    if (p.in == nullptr || p.out == nullptr) return CONVROT_ERR_NULL;
    if (!aligned(p.in, size) || !aligned(p.out, size)) return CONVROT_ERR_ALIGN;
  }
  // an output is its own input, or meets no tensor of the call
  for (int i = 0; i < 2; ++i) {
    const auto &p = part[i], &other = part[1 - i];
    if (p.heads == 0) continue;
    const Rows out{reinterpret_cast<uintptr_t>(p.out), p.out_t, p.out_h, p.heads};
    const Rows in{reinterpret_cast<uintptr_t>(p.in), p.in_t, p.in_h, p.heads};
    if (p.in != p.out && rows_meet(out, in, T, D, int64_t(size))) return CONVROT_ERR_SHAPE;
    if (other.heads == 0) continue;
    if (rows_meet(out, Rows{reinterpret_cast<uintptr_t>(other.in), other.in_t, other.in_h, other.heads}, T, D,
                  int64_t(size)) ||
        rows_meet(out, Rows{reinterpret_cast<uintptr_t>(other.out), other.out_t, other.out_h, other.heads}, T, D,
                  int64_t(size)))
      return CONVROT_ERR_SHAPE;
  }
  if (pos == nullptr || inv_freq == nullptr) return CONVROT_ERR_NULL;
  if (!aligned(pos, 8) || !aligned(inv_freq, 4)) return CONVROT_ERR_ALIGN;
  return CONVROT_OK;
}

}  // namespace
