// C ABI of the decoding operators: host-side argument validation and launches.
// Semantics: include/convrot.h.
#include "convrot.h"
#include "convrot_internal.h"

#include <math.h>

namespace {

constexpr int64_t kIntMax = 0x7FFFFFFF;
// A launch takes fewer than 2^32 threads along x; what would need more is refused here, before it
// becomes an error that the runtime keeps for a later call to find.
constexpr int64_t kMaxThreads = 0xFFFFFFFF;
constexpr int64_t kMaxStride = int64_t(1) << 46;   // elements; keeps every offset within 63 bits

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

int check_w4a16(int64_t M, int64_t N, int64_t K, int64_t g, int64_t sg, int64_t* kp) {
  const int st = check_window(g, 1024);
  if (st != CONVROT_OK) return st;
  *kp = convrot_w4a16_padded_k(K, g, sg);
  if (*kp < 0) return int(*kp);
  if (M < 0 || N < 0 || M > kIntMax || N > kIntMax) return CONVROT_ERR_SHAPE;
  if (*kp > CONVROT_MAX_KP || M > 65535 * int64_t(64)) return CONVROT_ERR_UNSUPPORTED;
  // workgroups of at least 16 weight rows and 512 threads; preparing x takes a wave for 1024 columns
  if (!launch_fits((N + 15) / 16, 512) || !launch_fits((M * ((*kp + 1023) / 1024) + 3) / 4, 256))
    return CONVROT_ERR_UNSUPPORTED;
  return CONVROT_OK;
}

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

}  // namespace

extern "C" {

int64_t convrot_w4a16_padded_k(int64_t K, int64_t g, int64_t sg) {
  const int st = check_window(g, 1024);
  if (st != CONVROT_OK) return st;
  if (sg != 32 && sg != 64 && sg != 128) return CONVROT_ERR_UNSUPPORTED;
  const int64_t unit = g > sg ? g : sg;
  if (K < 1 || K > INT64_MAX - unit) return CONVROT_ERR_SHAPE;
  return (K + unit - 1) / unit * unit;
}

int convrot_quant_weight_g4(const void* w, int32_t w_dtype, int64_t N, int64_t K, int64_t g, int64_t sg,
                            uint8_t* wq, void* ws, void* stream) {
  int64_t kp = 0;
  const int st = check_w4a16(0, N, K, g, sg, &kp);
  if (st != CONVROT_OK) return st;
  if (!launch_fits((N * ((kp + 1023) / 1024) + 3) / 4, 256)) return CONVROT_ERR_UNSUPPORTED;
  if (elem_size(w_dtype) == 0) return CONVROT_ERR_DTYPE;
  if (N == 0) return CONVROT_OK;
  if (w == nullptr || wq == nullptr || ws == nullptr) return CONVROT_ERR_NULL;
  if (!aligned(w, elem_size(w_dtype)) || !aligned(wq, 16) || !aligned(ws, 2)) return CONVROT_ERR_ALIGN;
  return status_of(convrot::launch_quant_weight_g4(w, w_dtype, N, K, int(g), int(sg), kp, wq,
                                                   static_cast<uint16_t*>(ws),
                                                   static_cast<hipStream_t>(stream)));
}

size_t convrot_w4a16_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t g, int64_t sg) {
  int64_t kp = 0;
  if (check_w4a16(M, N, K, g, sg, &kp) != CONVROT_OK || M == 0 || N == 0) return 0;
  const convrot::W4A16Plan p = convrot::plan_w4a16(M, kp, int(g));
  return p.operand_bytes + p.factor_bytes;
}

int convrot_w4a16_linear(const void* x, int32_t x_dtype, int64_t M, int64_t K, int64_t ldx, int64_t g, int64_t sg,
                         const uint8_t* wq, const void* ws, int64_t N, const void* bias, void* y,
                         void* workspace, size_t ws_bytes, void* stream) {
  int64_t kp = 0;
  const int st = check_w4a16(M, N, K, g, sg, &kp);
  if (st != CONVROT_OK) return st;
  if (elem_size(x_dtype) == 0) return CONVROT_ERR_DTYPE;
  if (ldx < K || !stride_ok(ldx)) return CONVROT_ERR_SHAPE;
  if (M == 0 || N == 0) return CONVROT_OK;
  if (x == nullptr || wq == nullptr || ws == nullptr || y == nullptr) return CONVROT_ERR_NULL;
  if (!aligned(x, elem_size(x_dtype)) || !aligned(wq, 16) || !aligned(ws, 2) || !aligned(y, 2) ||
      !aligned(bias, 2) || !aligned(workspace, 256))
    return CONVROT_ERR_ALIGN;
  const size_t need = convrot_w4a16_workspace_bytes(M, N, K, g, sg);
  if (need > 0 && workspace == nullptr) return CONVROT_ERR_NULL;
  if (ws_bytes < need) return CONVROT_ERR_WORKSPACE;
  return status_of(convrot::launch_w4a16_linear(x, x_dtype, M, K, ldx, int(g), int(sg), kp, wq,
                                                static_cast<const uint16_t*>(ws), N,
                                                static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(y),
                                                workspace, static_cast<hipStream_t>(stream)));
}

int convrot_rotary_frequencies(int64_t R, double base, int32_t scaling, double factor, double original,
                               double low, double high, float* out) {
  if (R < 2 || R > 1024 || R % 2 != 0) return CONVROT_ERR_SHAPE;
  if (scaling < CONVROT_ROPE_PLAIN || scaling > CONVROT_ROPE_BANDS || !(base > 0.0) || !isfinite(base))
    return CONVROT_ERR_UNSUPPORTED;
  if (scaling != CONVROT_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return CONVROT_ERR_UNSUPPORTED;
  if (scaling == CONVROT_ROPE_NTK && R == 2) return CONVROT_ERR_UNSUPPORTED;
  if (scaling == CONVROT_ROPE_BANDS &&
      (!(original > 0.0) || !(low >= 0.0) || !(high > low) || !isfinite(original) || !isfinite(high)))
    return CONVROT_ERR_UNSUPPORTED;
  if (out == nullptr) return CONVROT_ERR_NULL;
  if (scaling == CONVROT_ROPE_NTK) base *= pow(factor, double(R) / double(R - 2));
  for (int64_t i = 0; i < R / 2; ++i) {
    double f = pow(base, -2.0 * double(i) / double(R));
    if (scaling == CONVROT_ROPE_LINEAR) f /= factor;
    if (scaling == CONVROT_ROPE_BANDS) {
      const double turns = original * f / 6.283185307179586;
      const double w = fmin(fmax((turns - low) / (high - low), 0.0), 1.0);
      f *= w + (1.0 - w) / factor;
    }
    out[i] = float(f);
  }
  return CONVROT_OK;
}

int convrot_rotary(const void* q, int64_t q_t, int64_t q_h, void* q_out, int64_t qo_t, int64_t qo_h, int64_t Hq,
                   const void* k, int64_t k_t, int64_t k_h, void* k_out, int64_t ko_t, int64_t ko_h, int64_t Hk,
                   int32_t dtype, int64_t T, int64_t D, int64_t R, const int64_t* pos, const float* inv_freq,
                   int32_t interleaved, float factor, int32_t inverse, void* stream) {
  const size_t size = elem_size(dtype);
  if (size == 0) return CONVROT_ERR_DTYPE;
  if (T < 0 || T > kIntMax || Hq < 0 || Hk < 0 || D < 1 || R < 2 || R % 2 != 0 || R > D) return CONVROT_ERR_SHAPE;
  if (D > 1024 || Hq > 65535 || Hk > 65535 - Hq || !launch_fits(T, 256)) return CONVROT_ERR_UNSUPPORTED;
  const struct {
    const void* in;
    int64_t in_t, in_h;
    void* out;
    int64_t out_t, out_h, heads;
  } part[2] = {{q, q_t, q_h, q_out, qo_t, qo_h, Hq}, {k, k_t, k_h, k_out, ko_t, ko_h, Hk}};
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
  if (T == 0 || Hq + Hk == 0) return CONVROT_OK;
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
  convrot::RotaryArgs a{{q, q_out, q_t, q_h, qo_t, qo_h, int(Hq)}, {k, k_out, k_t, k_h, ko_t, ko_h, int(Hk)},
                        pos, inv_freq, factor, int(D), int(R), interleaved != 0, inverse != 0};
  return status_of(convrot::launch_rotary(a, dtype, T, static_cast<hipStream_t>(stream)));
}

int convrot_kv8_append(const void* k, int64_t k_t, int64_t k_h, const void* v, int64_t v_t, int64_t v_h,
                       int32_t dtype, int64_t T, const int32_t* cu, const int32_t* lens, const int32_t* table,
                       int64_t table_ld, int64_t B, int64_t max_pages, int8_t* kc, float* ks, int8_t* vc,
                       float* vs, int64_t num_pages, int64_t page, int64_t H, int64_t D, int64_t g,
                       int64_t max_new, void* stream) {
  int st = check_cache(num_pages, page, H, D, g, B, T, max_pages, table_ld);
  if (st != CONVROT_OK) return st;
  if (elem_size(dtype) == 0) return CONVROT_ERR_DTYPE;
  if (!stride_ok(k_t) || !stride_ok(k_h) || !stride_ok(v_t) || !stride_ok(v_h) || max_new < 0)
    return CONVROT_ERR_SHAPE;
  if (T == 0 || B == 0) return CONVROT_OK;
  if (k == nullptr || v == nullptr) return CONVROT_ERR_NULL;
  st = check_batch_pointers(cu, lens, table, max_pages, kc, ks, vc, vs);
  if (st != CONVROT_OK) return st;
  if (!aligned(k, elem_size(dtype)) || !aligned(v, elem_size(dtype))) return CONVROT_ERR_ALIGN;
  const convrot::Kv8Batch batch{cu, lens, table, B, T, table_ld, max_pages};
  const convrot::Kv8Cache cache{kc, ks, vc, vs, num_pages, int(page), int(H), int(D)};
  return status_of(convrot::launch_kv8_append(k, v, dtype, k_t, k_h, v_t, v_h, batch, cache, int(g),
                                              max_new < T ? max_new : T, static_cast<hipStream_t>(stream)));
}

int convrot_kv8_read(const int32_t* cu, const int32_t* lens, const int32_t* table, int64_t table_ld, int64_t B,
                     int64_t max_pages, const int8_t* kc, const float* ks, const int8_t* vc, const float* vs,
                     int64_t num_pages, int64_t page, int64_t H, int64_t D, int64_t g, int64_t max_new, int64_t T,
                     void* k, void* v, void* stream) {
  int st = check_cache(num_pages, page, H, D, g, B, T, max_pages, table_ld);
  if (st != CONVROT_OK) return st;
  if (max_new < 0) return CONVROT_ERR_SHAPE;
  if (T == 0 || B == 0) return CONVROT_OK;
  if (k == nullptr || v == nullptr) return CONVROT_ERR_NULL;
  st = check_batch_pointers(cu, lens, table, max_pages, kc, ks, vc, vs);
  if (st != CONVROT_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16)) return CONVROT_ERR_ALIGN;
  const convrot::Kv8Batch batch{cu, lens, table, B, T, table_ld, max_pages};
  const convrot::Kv8Cache cache{const_cast<int8_t*>(kc), const_cast<float*>(ks), const_cast<int8_t*>(vc),
                                const_cast<float*>(vs), num_pages, int(page), int(H), int(D)};
  return status_of(convrot::launch_kv8_read(batch, cache, int(g), max_new < T ? max_new : T,
                                            static_cast<uint16_t*>(k), static_cast<uint16_t*>(v),
                                            static_cast<hipStream_t>(stream)));
}

size_t convrot_kv8_attention_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t D,
                                             int64_t max_new, int64_t max_len) {
  if (!attention_shape_ok(T, B, Hq, H, D, max_new, max_len) || !attention_plannable(T, B, Hq, H) || T == 0 ||
      B == 0 || D > 256 || D % 16 != 0)
    return 0;
  return convrot::plan_kv8_attention(B, T, Hq, H, D, max_new, max_len).bytes;
}

int convrot_kv8_attention(const void* q, int64_t q_t, int64_t q_h, int32_t dtype, int64_t T, int64_t Hq,
                          const int32_t* cu, const int32_t* lens, const int32_t* table, int64_t table_ld,
                          int64_t B, int64_t max_pages, const int8_t* kc, const float* ks, const int8_t* vc,
                          const float* vs, int64_t num_pages, int64_t page, int64_t H, int64_t D, int64_t g,
                          float scale, int64_t max_new, int64_t max_len, void* out, void* workspace,
                          size_t ws_bytes, void* stream) {
  int st = check_cache(num_pages, page, H, D, g, B, T, max_pages, table_ld);
  if (st != CONVROT_OK) return st;
  if (elem_size(dtype) == 0) return CONVROT_ERR_DTYPE;
  if (!attention_shape_ok(T, B, Hq, H, D, max_new, max_len) || !stride_ok(q_t) || !stride_ok(q_h))
    return CONVROT_ERR_SHAPE;
  if (T == 0 || B == 0) return CONVROT_OK;
  if (!attention_plannable(T, B, Hq, H)) return CONVROT_ERR_UNSUPPORTED;
  const convrot::Kv8Plan plan = convrot::plan_kv8_attention(B, T, Hq, H, D, max_new, max_len);
  // workgroups of 256 threads for few rows, 512 for many; joining the splits takes one to a row at most
  if (plan.row_blocks > kMaxThreads / (plan.row_tiles <= 4 ? 256 : 512) / plan.splits / H / B ||
      (plan.splits > 1 && !launch_fits(T * Hq, 256)))
    return CONVROT_ERR_UNSUPPORTED;
  if (q == nullptr || out == nullptr || (plan.bytes > 0 && workspace == nullptr)) return CONVROT_ERR_NULL;
  st = check_batch_pointers(cu, lens, table, max_pages, kc, ks, vc, vs);
  if (st != CONVROT_OK) return st;
  if (!aligned(q, elem_size(dtype)) || !aligned(out, 16) || !aligned(workspace, 256)) return CONVROT_ERR_ALIGN;
  if (ws_bytes < plan.bytes) return CONVROT_ERR_WORKSPACE;
  const convrot::Kv8Batch batch{cu, lens, table, B, T, table_ld, max_pages};
  const convrot::Kv8Cache cache{const_cast<int8_t*>(kc), const_cast<float*>(ks), const_cast<int8_t*>(vc),
                                const_cast<float*>(vs), num_pages, int(page), int(H), int(D)};
  return status_of(convrot::launch_kv8_attention(q, dtype, q_t, q_h, Hq, batch, cache, int(g), scale, plan,
                                                 static_cast<uint16_t*>(out), workspace,
                                                 static_cast<hipStream_t>(stream)));
}

}  // extern "C"
