// C ABI of the operators for normed heads, drafted tokens, moved pages and adapters: host-side argument
// validation and launches.  Semantics: include/convrot.h.
#include "api_checks.h"

namespace {

constexpr int64_t kMaxWords = 1024, kMaxAdapters = 1 << 24, kMaxPageBytes = 1 << 29;
constexpr float kLeastEps = 7.888609052210118e-31f;     // 2^-100

int check_lora(int64_t M, int64_t K, int64_t r, int64_t L) {
  if (M < 0 || M > kIntMax || K < 1 || K > kIntMax || r < 1 || L < 1 || L > kIntMax - 1) return CONVROT_ERR_SHAPE;
  return M <= 65535 * int64_t(64) && r <= 256 && L <= kMaxAdapters ? CONVROT_OK : CONVROT_ERR_UNSUPPORTED;
}

// Bytes from a matrix' first element to behind its last; strides are within kMaxStride.
int64_t bytes_of(int64_t rows, int64_t cols, int64_t ld, int64_t size) { return ((rows - 1) * ld + cols) * size; }

}  // namespace

extern "C" {

int convrot_norm_rotary(const void* q, int64_t q_t, int64_t q_h, void* q_out, int64_t qo_t, int64_t qo_h, int64_t Hq,
                        const void* k, int64_t k_t, int64_t k_h, void* k_out, int64_t ko_t, int64_t ko_h, int64_t Hk,
                        int32_t dtype, int64_t T, int64_t D, int64_t R, const int64_t* pos, const float* inv_freq,
                        const void* q_weight, const void* k_weight, int32_t w_dtype, float eps, int32_t interleaved,
                        float factor, void* stream) {
  if (elem_size(w_dtype) == 0) return CONVROT_ERR_DTYPE;
  if (!(eps >= kLeastEps && eps <= 1.0f)) return CONVROT_ERR_UNSUPPORTED;
  const TurnedPart part[2] = {{q, q_t, q_h, q_out, qo_t, qo_h, Hq}, {k, k_t, k_h, k_out, ko_t, ko_h, Hk}};
  bool nothing = false;
  const int st = check_turned(part, dtype, T, D, R, pos, inv_freq, &nothing);
  if (st != CONVROT_OK || nothing) return st;
  if (!aligned(q_weight, elem_size(w_dtype)) || !aligned(k_weight, elem_size(w_dtype))) return CONVROT_ERR_ALIGN;
  const int64_t bytes = D * int64_t(elem_size(w_dtype));
  if (!apart_from_outputs(part, dtype, T, D, {{pos, 8 * T}, {inv_freq, 2 * R}, {q_weight, bytes}, {k_weight, bytes}}))
    return CONVROT_ERR_SHAPE;
  const convrot::NormRotaryArgs a{{{q, q_out, q_t, q_h, qo_t, qo_h, int(Hq)}, {k, k_out, k_t, k_h, ko_t, ko_h, int(Hk)},
                                   pos, inv_freq, factor, int(D), int(R), interleaved != 0, 0},
                                  q_weight, k_weight, w_dtype, eps};
  return status_of(convrot::launch_norm_rotary(a, dtype, T, static_cast<hipStream_t>(stream)));
}

int convrot_tree_masks(const int32_t* parents, const int32_t* cu, const int32_t* lens, int64_t B, int64_t T,
                       int64_t max_new, int64_t words, uint64_t* mask, int64_t* pos, void* stream) {
  if (B < 0 || B > kIntMax || T < 0 || T > kIntMax || max_new < 0 || words < 1) return CONVROT_ERR_SHAPE;
  if (words > kMaxWords || !launch_fits(B, 256)) return CONVROT_ERR_UNSUPPORTED;
  if (T == 0 || B == 0) return CONVROT_OK;
  if (parents == nullptr || cu == nullptr || lens == nullptr || mask == nullptr || pos == nullptr) return CONVROT_ERR_NULL;
  if (!aligned(parents, 4) || !aligned(cu, 4) || !aligned(lens, 4) || !aligned(mask, 8) || !aligned(pos, 8))
    return CONVROT_ERR_ALIGN;
  for (const auto& [out, bytes] : {Extent{mask, 8 * T * words}, {pos, 8 * T}})
    if (!apart(out, bytes, parents, 4 * T) || !apart(out, bytes, cu, 4 * (B + 1)) || !apart(out, bytes, lens, 4 * B))
      return CONVROT_ERR_SHAPE;
  if (!apart(mask, 8 * T * words, pos, 8 * T)) return CONVROT_ERR_SHAPE;
  const convrot::Kv8Batch batch{cu, lens, nullptr, B, T, 0, 0};
  return status_of(convrot::launch_tree_masks(parents, batch, words, max_new < T ? max_new : T, mask, pos,
                                              static_cast<hipStream_t>(stream)));
}

size_t convrot_kv8_tree_attention_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t D,
                                                  int64_t max_new, int64_t max_len) {
  return attention_workspace(convrot::plan_kv8_tree, T, B, Hq, H, D, max_new, max_len);
}

int convrot_kv8_tree_attention(const void* q, int64_t q_t, int64_t q_h, int32_t dtype, int64_t T, int64_t Hq,
                               const uint64_t* mask, int64_t words, const int32_t* cu, const int32_t* lens,
                               const int32_t* table, int64_t table_ld, int64_t B, int64_t max_pages, const int8_t* kc,
                               const float* ks, const int8_t* vc, const float* vs, int64_t num_pages, int64_t page,
                               int64_t H, int64_t D, int64_t g, float scale, int64_t max_new, int64_t max_len,
                               void* out, void* workspace, size_t ws_bytes, void* stream) {
  if (words < 1) return CONVROT_ERR_SHAPE;
  if (words > kMaxWords) return CONVROT_ERR_UNSUPPORTED;
  convrot::Kv8Plan plan;
  bool nothing = false;
  const int st = check_attention(q, q_t, q_h, dtype, T, Hq, cu, lens, table, table_ld, B, max_pages, kc, ks, vc, vs,
                                 num_pages, page, H, D, g, max_new, max_len, out, workspace, ws_bytes,
                                 convrot::plan_kv8_tree, &plan, &nothing);
  if (st != CONVROT_OK || nothing) return st;
  if (mask == nullptr) return CONVROT_ERR_NULL;
  if (!aligned(mask, 8)) return CONVROT_ERR_ALIGN;
  const convrot::Kv8Batch batch{cu, lens, table, B, T, table_ld, max_pages};
  const convrot::Kv8Cache cache{const_cast<int8_t*>(kc), const_cast<float*>(ks), const_cast<int8_t*>(vc),
                                const_cast<float*>(vs), num_pages, int(page), int(H), int(D)};
  return status_of(convrot::launch_kv8_tree_attention(q, dtype, q_t, q_h, Hq, mask, words, batch, cache, int(g), scale,
                                                      plan, static_cast<uint16_t*>(out), workspace,
                                                      static_cast<hipStream_t>(stream)));
}

size_t convrot_kv8_keep_workspace_bytes(int64_t T, int64_t B, int64_t H, int64_t D) {
  if (check_cache(1, 16, H, D, 0, B, T, 0, 0) != CONVROT_OK || T == 0 || B == 0) return 0;
  return convrot::kv8_keep_bytes(T, B, H, D);
}

int convrot_kv8_keep(const int32_t* kept, int64_t T, const int32_t* cu, const int32_t* lens, const int32_t* table,
                     int64_t table_ld, int64_t B, int64_t max_pages, int8_t* kc, float* ks, int8_t* vc, float* vs,
                     int64_t num_pages, int64_t page, int64_t H, int64_t D, int64_t max_new, int32_t* lens_out,
                     void* workspace, size_t ws_bytes, void* stream) {
  int st = check_cache(num_pages, page, H, D, 0, B, T, max_pages, table_ld);
  if (st != CONVROT_OK) return st;
  if (max_new < 0) return CONVROT_ERR_SHAPE;
  if (T == 0 || B == 0) return CONVROT_OK;
  if (kept == nullptr || workspace == nullptr) return CONVROT_ERR_NULL;
  st = check_batch_pointers(cu, lens, table, max_pages, kc, ks, vc, vs);
  if (st != CONVROT_OK) return st;
  if (!aligned(kept, 4) || !aligned(lens_out, 4) || !aligned(workspace, 256)) return CONVROT_ERR_ALIGN;
  if (lens_out != nullptr && (!apart(lens_out, 4 * B, lens, 4 * B) || !apart(lens_out, 4 * B, cu, 4 * (B + 1)) ||
                              !apart(lens_out, 4 * B, kept, 4 * T) ||
                              (max_pages > 0 && !apart(lens_out, 4 * B, table, bytes_of(B, max_pages, table_ld, 4)))))
    return CONVROT_ERR_SHAPE;
  const int64_t need = int64_t(convrot::kv8_keep_bytes(T, B, H, D)), codes = num_pages * H * page * D, scales = 4 * num_pages * H;
  if (ws_bytes < size_t(need)) return CONVROT_ERR_WORKSPACE;
  if (lens_out != nullptr && (!apart(lens_out, 4 * B, kc, codes) || !apart(lens_out, 4 * B, ks, scales) ||
                              !apart(lens_out, 4 * B, vc, codes) || !apart(lens_out, 4 * B, vs, scales) ||
                              !apart(lens_out, 4 * B, workspace, need)))
    return CONVROT_ERR_SHAPE;
  const convrot::Kv8Batch batch{cu, lens, table, B, T, table_ld, max_pages};
  const convrot::Kv8Cache cache{kc, ks, vc, vs, num_pages, int(page), int(H), int(D)};
  return status_of(convrot::launch_kv8_keep(kept, batch, cache, max_new < T ? max_new : T, lens_out, workspace,
                                            static_cast<hipStream_t>(stream)));
}

int convrot_kv8_copy(const int32_t* src, const int32_t* dst, int64_t n, int8_t* kc, float* ks, int8_t* vc, float* vs,
                     int64_t num_pages, int64_t page, int64_t H, int64_t D, void* stream) {
  const int st = check_cache(num_pages, page, H, D, 0, 0, 0, 0, 0);
  if (st != CONVROT_OK) return st;
  if (n < 0 || n > kIntMax) return CONVROT_ERR_SHAPE;
  const convrot::Kv8Cache cache{kc, ks, vc, vs, num_pages, int(page), int(H), int(D)};
  if (!launch_fits(n, 256) || H * page * D > kMaxPageBytes) return CONVROT_ERR_UNSUPPORTED;
  if (n == 0) return CONVROT_OK;
  if (src == nullptr || dst == nullptr || kc == nullptr || ks == nullptr || vc == nullptr || vs == nullptr)
    return CONVROT_ERR_NULL;
  if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(kc, 16) || !aligned(vc, 16) || !aligned(ks, 4) || !aligned(vs, 4))
    return CONVROT_ERR_ALIGN;
  return status_of(convrot::launch_kv8_copy(src, dst, n, cache, static_cast<hipStream_t>(stream)));
}

size_t convrot_lora_workspace_bytes(int64_t M, int64_t K, int64_t r, int64_t L) {
  if (check_lora(M, K, r, L) != CONVROT_OK || M == 0) return 0;
  return convrot::lora_workspace_bytes(M, K, r, L);
}

int convrot_lora(const void* x, int32_t x_dtype, int64_t M, int64_t K, int64_t ldx, const int32_t* ids, const void* a,
                 const void* b, const float* scale, int64_t r, int64_t L, const void* y, int64_t ldy, int64_t N, void* out,
                 int64_t ldo, void* workspace, size_t ws_bytes, void* stream) {
  const int st = check_lora(M, K, r, L);
  if (st != CONVROT_OK) return st;
  const int64_t size = int64_t(elem_size(x_dtype));
  if (size == 0) return CONVROT_ERR_DTYPE;
  if (N < 0 || N > kIntMax || ldx < K || ldy < N || ldo < N || !stride_ok(ldx) ||
      !stride_ok(ldy) || !stride_ok(ldo))
    return CONVROT_ERR_SHAPE;
  // the offsets of all adapters, and of all rows, stay within 63 bits
  if (ldx > kMaxBytes / 8 / (M + 1) || ldy > kMaxBytes / 8 / (M + 1) || ldo > kMaxBytes / 8 / (M + 1) ||
      K > kMaxBytes / 2 / r / L || N > kMaxBytes / 2 / r / L)
    return CONVROT_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return CONVROT_OK;
  if (x == nullptr || ids == nullptr || a == nullptr || b == nullptr || scale == nullptr || y == nullptr ||
      out == nullptr || workspace == nullptr)
    return CONVROT_ERR_NULL;
  if (!aligned(x, size_t(size)) || !aligned(ids, 4) || !aligned(a, 2) || !aligned(b, 2) || !aligned(scale, 4) ||
      !aligned(y, 2) || !aligned(out, 2) || !aligned(workspace, 256))
    return CONVROT_ERR_ALIGN;
  if (out == y ? M > 1 && ldy != ldo : !apart(out, bytes_of(M, N, ldo, 2), y, bytes_of(M, N, ldy, 2)))
    return CONVROT_ERR_SHAPE;
  if (!apart(out, bytes_of(M, N, ldo, 2), x, bytes_of(M, K, ldx, size))) return CONVROT_ERR_SHAPE;
  const int64_t need = int64_t(convrot_lora_workspace_bytes(M, K, r, L));
  if (ws_bytes < size_t(need)) return CONVROT_ERR_WORKSPACE;
  for (const auto& [other, bytes] : {Extent{ids, 4 * M}, {a, 2 * L * r * K}, {b, 2 * L * N * r}, {scale, 4 * L}, {workspace, need}})
    if (!apart(out, bytes_of(M, N, ldo, 2), other, bytes)) return CONVROT_ERR_SHAPE;
  convrot::LoraArgs args{};
  args.x = x;
  args.ldx = ldx;
  args.M = M;
  args.K = K;
  args.ids = ids;
  args.a = static_cast<const uint16_t*>(a);
  args.b = static_cast<const uint16_t*>(b);
  args.scale = scale;
  args.r = r;
  args.L = L;
  args.N = N;
  args.y = static_cast<const uint16_t*>(y);
  args.ldy = ldy;
  args.out = static_cast<uint16_t*>(out);
  args.ldo = ldo;
  return status_of(convrot::launch_lora(args, x_dtype, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
