// C ABI of the decoding operators: host-side argument validation and launches.
// Semantics: include/convrot.h.
#include "api_checks.h"

#include <math.h>

namespace {

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
  const TurnedPart part[2] = {{q, q_t, q_h, q_out, qo_t, qo_h, Hq}, {k, k_t, k_h, k_out, ko_t, ko_h, Hk}};
  bool nothing = false;
  const int st = check_turned(part, dtype, T, D, R, pos, inv_freq, &nothing);
  if (st != CONVROT_OK || nothing) return st;
  if (!apart_from_outputs(part, dtype, T, D, {{pos, 8 * T}, {inv_freq, 2 * R}})) return CONVROT_ERR_SHAPE;
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
  return attention_workspace(convrot::plan_kv8_attention, T, B, Hq, H, D, max_new, max_len);
}

int convrot_kv8_attention(const void* q, int64_t q_t, int64_t q_h, int32_t dtype, int64_t T, int64_t Hq,
                          const int32_t* cu, const int32_t* lens, const int32_t* table, int64_t table_ld,
                          int64_t B, int64_t max_pages, const int8_t* kc, const float* ks, const int8_t* vc,
                          const float* vs, int64_t num_pages, int64_t page, int64_t H, int64_t D, int64_t g,
                          float scale, int64_t max_new, int64_t max_len, void* out, void* workspace,
                          size_t ws_bytes, void* stream) {
  convrot::Kv8Plan plan;
  bool nothing = false;
  const int st = check_attention(q, q_t, q_h, dtype, T, Hq, cu, lens, table, table_ld, B, max_pages, kc, ks, vc, vs,
                                 num_pages, page, H, D, g, max_new, max_len, out, workspace, ws_bytes,
                                 convrot::plan_kv8_attention, &plan, &nothing);
  if (st != CONVROT_OK || nothing) return st;
  const convrot::Kv8Batch batch{cu, lens, table, B, T, table_ld, max_pages};
  const convrot::Kv8Cache cache{const_cast<int8_t*>(kc), const_cast<float*>(ks), const_cast<int8_t*>(vc),
                                const_cast<float*>(vs), num_pages, int(page), int(H), int(D)};
  return status_of(convrot::launch_kv8_attention(q, dtype, q_t, q_h, Hq, batch, cache, int(g), scale, plan,
                                                 static_cast<uint16_t*>(out), workspace,
                                                 static_cast<hipStream_t>(stream)));
}

}  // extern "C"
