// The paged 8-bit key/value cache as its kernels see it, and the attention over it (kv8.hip,
// kv8_tree.hip): the work of one workgroup, for rows that see the tokens up to their own and for rows that
// see a mask's.
#pragma once

#include "decode_device.h"

#include <algorithm>
#include <type_traits>

namespace convrot {
namespace {

// The least scale that is stored; pages whose values are all below 127 times this hold zeros.
// Attention divides by scales in fp32: 2^80 times the weights of all tokens, 2^15 each, stays finite.
constexpr float kLeastScale = 8.271806125530277e-25f;   // 2^-80
constexpr float kLeastLog = -80.0f;

struct Sequence {
  int64_t row0, n, len;   // first row, new rows, tokens in all (the rows' included)
};

// A sequence as the device arrays state it; counts that do not fit the T rows give none.
__device__ __forceinline__ Sequence sequence_of(const Kv8Batch& b, int64_t i) {
  const int64_t from = b.cu[i], to = b.cu[i + 1];
  Sequence s{from, to - from, b.lens[i]};
  if (from < 0 || to < from || to > b.T) s.n = 0;
  return s;
}

// Page number of a sequence's page, -1 where the table has none that exists.
__device__ __forceinline__ int64_t page_of(const Kv8Batch& b, const Kv8Cache& c, int64_t i, int64_t col) {
  if (col < 0 || col >= b.max_pages) return -1;
  const int64_t id = b.table[i * b.table_ld + col];
  return id >= 0 && id < c.num_pages ? id : -1;
}


// Four kept codes under a grown scale: rne(code * ratio).
__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float ratio) {
  uint32_t r = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    r |= uint32_t(int(rintf(float(int8_t(w >> (8 * e))) * ratio)) & 255) << (8 * e);
  return r;
}

// ------------------------------------------------------------------------------- attention
constexpr float kNothing = -1e30f;   // reference of a row before its first token
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kShift = 7.0f;       // weights are kept times 2^kShift ...
constexpr float kSlack = 8.0f;       // ... and may pass their reference by 2^kSlack: 2^15 fits fp16

// Eight int8 codes to fp16, exactly: 0x6400 + (code + 128) is the fp16 1024 + code + 128.
__device__ __forceinline__ half8 decode_i8(uint32_t a, uint32_t b) {
  const half2_t off = {(_Float16)1152.0f, (_Float16)1152.0f};
  a ^= 0x80808080u;
  b ^= 0x80808080u;
  const half2_t p = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, a, 0x04010400u)) - off;
  const half2_t q = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u)) - off;
  const half2_t r = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u)) - off;
  const half2_t s = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u)) - off;
  return half8{p[0], p[1], q[0], q[1], r[0], r[1], s[0], s[1]};
}

__device__ __forceinline__ half8 pack_half8(const float4_t& a, const float4_t& b) {
  typedef float float2_v __attribute__((ext_vector_type(2)));
  const half2_t p = __builtin_convertvector((float2_v{a[0], a[1]}), half2_t);
  const half2_t q = __builtin_convertvector((float2_v{a[2], a[3]}), half2_t);
  const half2_t r = __builtin_convertvector((float2_v{b[0], b[1]}), half2_t);
  const half2_t s = __builtin_convertvector((float2_v{b[2], b[3]}), half2_t);
  return half8{p[0], p[1], q[0], q[1], r[0], r[1], s[0], s[1]};
}

// Over the four lane rows (lanes 16 apart): swapping a register with itself gives a lane its own value
// and that of the lane 16, or 32, away, without LDS.
__device__ __forceinline__ float max_over_lane_rows(float v) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float sum_over_lane_rows(float v) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

struct AttentionArgs {
  const void* q;
  int64_t q_t, q_h;
  bool q_wide;
  int Hq, digits, splits;
  float scale;
  int64_t row_blocks, rows;       // rows: T * Hq, of the partial results
  uint16_t* out;
  float* partial;                 // [splits][rows][D] (but for TreeTokens::whole), or NULL: one split, straight to out
  float2* stats;                  // [splits][rows]: reference and sum
};

// [splits][rows], behind the statistics: where partial has a piece's row, for TreeTokens::whole.
__host__ __device__ __forceinline__ uint32_t* places_of(const AttentionArgs& a) {
  return reinterpret_cast<uint32_t*>(a.stats + a.splits * a.rows);
}

// What a workgroup works on: a block of the rows of one sequence and cached head, and a share of
// the sequence's tokens in blocks of 64.
struct Work {
  Sequence seq;
  int64_t b, h, len, before, rows, rb, split;
};

__device__ __forceinline__ Work work_of(const AttentionArgs& a, const Kv8Batch& batch, const Kv8Cache& cache) {
  // the cached head varies fastest: with 8 of them each of the chip's 8 L2s sees one head; the
  // rows that see most come first
  Work w;
  uint32_t id = blockIdx.x;
  const uint32_t heads = uint32_t(cache.H), splits = uint32_t(a.splits), row_blocks = uint32_t(a.row_blocks);
  w.h = id % heads;
  id /= heads;
  w.split = id % splits;
  id /= splits;
  w.rb = row_blocks - 1 - id % row_blocks;
  w.b = id / row_blocks;
  w.seq = sequence_of(batch, w.b);
  w.rows = w.seq.n * (a.Hq / cache.H);
  w.len = max(min(w.seq.len, batch.max_pages * cache.page), int64_t(0));
  w.before = w.seq.len - w.seq.n;
  return w;
}

// A sequence's pages as a lane sees them.  A look-up is a plain load that nothing waits for or
// branches on (its column is that of a token below the limit, so it is in the table); what it gave is
// checked when it is used, a block or two later.
struct Pages {
  const int32_t* row;           // of the table
  const int8_t *k, *v;          // of the cached head, in page 0
  const float *ks, *vs;
  uint32_t num_pages, stride, heads, limit, mask;
  int log;

  __device__ __forceinline__ int32_t find(uint32_t base, uint32_t off) const {
    return row[min(min(base, limit) + off, limit - 1) >> log];
  }
  __device__ __forceinline__ bool there(int32_t id, uint32_t base, uint32_t off) const {
    return uint32_t(id) < num_pages && base < limit && off < limit - base;
  }
  __device__ __forceinline__ uint32_t safe(int32_t id) const { return uint32_t(id) < num_pages ? uint32_t(id) : 0u; }
  __device__ __forceinline__ const int8_t* keys(int32_t id) const { return k + uint64_t(safe(id)) * stride; }
  __device__ __forceinline__ const int8_t* values(int32_t id) const { return v + uint64_t(safe(id)) * stride; }
};

__device__ __forceinline__ Pages pages_of(const Kv8Batch& batch, const Kv8Cache& cache, const Work& w, int64_t limit) {
  const int64_t head = w.h * cache.page * cache.D;
  return Pages{batch.table + w.b * batch.table_ld, cache.kc + head, cache.vc + head, cache.ks + w.h, cache.vs + w.h,
               uint32_t(cache.num_pages), uint32_t(cache.H) * uint32_t(cache.page * cache.D), uint32_t(cache.H),
               uint32_t(limit), uint32_t(cache.page - 1), 31 - __clz(cache.page)};
}

// Sixteen values of query rows of a (sequence, cached head), `step` rows apart from row r on; a row of 16 lanes holds a
// row.  Rows behind the last are the last one: their answers go nowhere.  T Hq is below 2^31.
template <typename TIn, int ROWS>
__device__ __forceinline__ void load_queries(const AttentionArgs& a, const Kv8Cache& cache, const Work& w, int64_t r,
                                             int step, int n, float (&v)[ROWS][16]) {
  const uint32_t G = uint32_t(a.Hq / cache.H);
  const TIn* p[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const uint32_t at = uint32_t(min(r + i * step, w.rows - 1)), t = at / G;
    p[i] = static_cast<const TIn*>(a.q) + ((w.seq.row0 + t) * a.q_t + (w.h * G + at - t * G) * a.q_h + (n * 16 < cache.D ? n * 16 : 0));
  }
  if (a.q_wide) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) load16<TIn>(p[i], 16, true, v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) load16<TIn>(p[i], 16, false, v[i]);
  }
}

// These, rotated and scaled into fp16's range, to 16 places of LDS; `factor` takes the row's score scale, in powers
// of two.  A negative scale's sign goes to the query, so that score scales are never negative.  A row that
// holds an Inf or a NaN becomes NaN as a whole: unrotated, an Inf that meets codes of one sign would make scores of
// -Inf, which is how tokens that are not seen are marked.
template <int DT>
__device__ __forceinline__ void place_query(const AttentionArgs& a, int D, int n, float (&v)[16], _Float16* row,
                                            float* factor) {
  float up, back;
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = n * 16 < D ? v[e] : 0.0f;
  const uint32_t bits = row_max(abs_max16(v));
  half_range(bits, a.digits, &up, &back);
  up = bits >= 0x7F800000u ? back : a.scale < 0.0f ? -up : up;        // back is NaN there
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] *= up;
  rotate16(v, a.digits);
  if (n * 16 < DT) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      half8 o;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = (_Float16)v[8 * k + e];
      *reinterpret_cast<half8*>(&row[n * 16 + 8 * k]) = o;
    }
  }
  if (n == 0) *factor = back * fabsf(a.scale) * kLog2e;
}

// The page scales of the 16 tokens whose scores a lane holds.
struct PageScale {
  float ks, vs;
  bool there;
};

// A token's place from the share's first one, -1 for all before it.  Lengths are int32, so the places of a
// share's tokens are too, to the end of its last block of 64; what is compared with them stays at 2^31 - 1.
__device__ __forceinline__ int from_here(int64_t token, int64_t first) {
  return int(max(min(token - first, int64_t(0x7FFFFFFF)), int64_t(-1)));
}

__device__ __forceinline__ PageScale scale_of(const Pages& p, int32_t id, uint32_t base, uint32_t off) {
  const uint64_t at = uint64_t(p.safe(id)) * p.heads;
  return PageScale{p.ks[at], p.vs[at], p.there(id, base, off)};
}

// Which tokens a row sees.  EarlierTokens: those up to its own.  TreeTokens: those before the sequence's rows,
// and of the rows' own tokens those whose bits are set in the row's words of the mask.
struct EarlierTokens {};
struct TreeTokens {
  const uint64_t* mask;         // [T][words]
  int64_t words;
  // many rows: what one workgroup has seen all of goes straight to out; partial has two slots of rows for every
  // workgroup, for the group that it begins within and the one that it begins but does not end, and places_of says
  // where it has a row of a piece
  bool whole;
};

// A lane's row.  hide: scores of the lane's 16 tokens from `token` on become -infinity where they are not seen
// (`none`: all of them) or at `limit` or beyond; token and limit count from the share's first token.
template <typename Seen>
struct RowSees;

template <>
struct RowSees<EarlierTokens> {
  int last;                     // token that the row sees

  __device__ __forceinline__ void set(const EarlierTokens&, const Work& w, int64_t r, int G, int64_t first) {
    last = r < w.rows ? from_here(w.before + uint32_t(r) / uint32_t(G), first) : -1;
  }
  template <int RT>
  __device__ __forceinline__ void hide(float4_t (&s)[4][RT], int rt, bool none, int token, int limit) const {
    const int seen = none ? -1 : min(last, limit - 1) - token;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * t + i > seen) s[t][rt][i] = -INFINITY;
  }
};

template <>
struct RowSees<TreeTokens> {
  int row;                      // of the mask, -1: none
  const uint64_t* mask;
  int64_t words, first;         // first: the share's first token, from the sequence's first row on

  __device__ __forceinline__ void set(const TreeTokens& tree, const Work& w, int64_t r, int G, int64_t from) {
    row = r < w.rows ? int(w.seq.row0 + uint32_t(r) / uint32_t(G)) : -1;
    mask = tree.mask;
    words = tree.words;
    first = from - w.before;
  }
  // Of the tokens j ... j + 15 of the sequence's rows (below 0: before them), which are seen.  The words are loaded here and
  // waited for here: a load that may still be on its way where the paths meet again would make every block wait for
  // all loads (many_rows' blocks 3.7 us instead of 1.9).
  __device__ __forceinline__ uint32_t bits_at(int64_t j) const {
    if (j <= -16) return 0xFFFFu;
    const uint64_t* const line = mask + row * words;
    const int64_t at = max(j, int64_t(0)), word = at >> 6;
    uint64_t low = word < words ? line[word] : 0, high = word + 1 < words ? line[word + 1] : 0;
    __builtin_amdgcn_s_waitcnt(0x0F70);                // vmcnt(0), nothing else
    if (j < 0) return uint32_t(low << -j) | ((1u << -j) - 1);
    const int shift = int(j & 63);
    return uint32_t(low >> shift) | (shift > 48 ? uint32_t(high << (64 - shift)) : 0u);
  }
  template <int RT>
  __device__ __forceinline__ void hide(float4_t (&s)[4][RT], int rt, bool none, int token, int limit) const {
    uint32_t bits = none || row < 0 ? 0u : bits_at(first + token);
    const int left = limit - token;
    if (left < 16) bits &= left > 0 ? (1u << left) - 1 : 0u;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((bits >> (4 * t + i) & 1) == 0) s[t][rt][i] = -INFINITY;
  }
};

// The tokens that any of the rows r ... end - 1 of a sequence sees, and the last one that all rows from r on see,
// up to which there is nothing to hide.
template <typename Seen>
__device__ __forceinline__ int64_t tokens_seen(const Work& w, int64_t end, int G) {
  if constexpr (std::is_same_v<Seen, TreeTokens>) return w.len;
  else return min(w.len, w.before + (end - 1) / G + 1);
}
template <typename Seen>
__device__ __forceinline__ int64_t seen_by_all(const Work& w, int64_t r, int G) {
  if constexpr (std::is_same_v<Seen, TreeTokens>) return w.before - 1;
  else return w.before + r / G;
}

// A block of 64 scores a row (16 of them in each lane) becomes weights, with a running reference m, sum l
// and output o of each row.  With s_j = scale q.k_j in powers of two, vs_j the page's value scale and
// R the reference, at most kSlack below max(s_j + log2 vs_j):
//   w_j = 2^(s_j + log2 vs_j - R + kShift),   o = sum w_j vcode_j,   l = sum w_j / vs_j,
// so o / l is the answer, the page scale of the values costs nothing in the second product, and w_j
// rounded to fp16 (2^-11 relative; below 2^-21 of the reference an absolute 2^-32 of it) uses that
// type's range.  The reference moves only when a score passes it by 2^kSlack, so that o is rarely
// scaled again.
// Pages of zeros (vs_j = 0) add to l only.  To the reference they count as pages of the least scale: any
// larger one would push the weights of pages that have values out of fp16's range, and with none l could
// overflow.  Their weights are 2^(s_j - R + kShift), at most 2^95 in fp32, and are dropped before the product.
struct BlockScale {
  float ks, lv, over_vs;      // lv: for the reference; pages of zeros have 0 in the weights
  // bit 0: the lane's 16 tokens have no page; 1: their values' scale is 0; 2 and 3: so it is for some lane
  int bits;
};

__device__ __forceinline__ BlockScale settle(const PageScale& page) {
  const bool zero = page.vs == 0.0f;
  const float lv = zero ? kLeastLog : __builtin_amdgcn_logf(page.vs);
  return BlockScale{page.ks, lv, zero ? 1.0f : __builtin_amdgcn_exp2f(-lv),
                    (page.there ? 0 : 1) | (zero ? 2 : 0) | (__any(!page.there) ? 4 : 0) | (__any(zero) ? 8 : 0)};
}

// A sum l under a reference that is higher by -d >= 0: l 2^d in two steps, since l may be as large as 2^d is
// small (a share that saw pages of zeros only, next to one of large values) and 2^d alone would be 0.
__device__ __forceinline__ float lowered(float l, float d) {
  const float half = __builtin_amdgcn_exp2f(0.5f * d);
  return l * half * half;
}

// First half: scores of tokens that are not there or not seen to -infinity (`ragged`: there are some;
// token, the lane's first, and limit count from the share's first), and the references.
template <int RT, int TILES, typename Seen>
__device__ __forceinline__ void refer(float4_t (&s)[4][RT], const BlockScale& bs, bool ragged, int token, int limit,
                                      const float (&row_scale)[RT], const RowSees<Seen> (&sees)[RT], float (&m)[RT],
                                      float (&l)[RT], float4_t (&o)[TILES][RT], float (&mul)[RT]) {
  if (ragged) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) sees[rt].hide(s, rt, bs.bits & 1, token, limit);
  }
  float high[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    mul[rt] = row_scale[rt] * bs.ks;
    float top[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) top[t] = fmaxf(fmaxf(s[t][rt][0], s[t][rt][1]), fmaxf(s[t][rt][2], s[t][rt][3]));
    top[0] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    high[rt] = fmaxf(kNothing, top[0] * mul[rt] + bs.lv);
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) high[rt] = max_over_lane_rows(high[rt]);
  bool grown = false;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) grown = grown || high[rt] > m[rt] + kSlack;
  if (__any(grown)) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float now = fmaxf(m[rt], high[rt]);
      const float down = __builtin_amdgcn_exp2f(m[rt] - now);
      l[rt] = lowered(l[rt], m[rt] - now);
      m[rt] = now;
#pragma unroll
      for (int dt = 0; dt < TILES; ++dt) o[dt][rt] *= down;
    }
  }
}

// Second half: the weights, in the layout of the second product's operand.
template <bool RAGGED, int RT>
__device__ __forceinline__ void weigh(const float4_t (&s)[4][RT], const BlockScale& bs, const float (&mul)[RT],
                                      const float (&m)[RT], float (&l)[RT], half8 (&w0)[RT], half8 (&w1)[RT]) {
  float4_t w[4][RT];
  float add[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) add[rt] = (bs.bits & 2 ? 0.0f : bs.lv) - m[rt] + kShift;
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[t][rt][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][rt][i], mul[rt], add[rt]));
        if (RAGGED && s[t][rt][i] == -INFINITY) w[t][rt][i] = 0.0f;     // also where mul or add is NaN
      }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    float4_t part;
#pragma unroll
    for (int i = 0; i < 4; ++i) part[i] = (w[0][rt][i] + w[1][rt][i]) + (w[2][rt][i] + w[3][rt][i]);
    const float sum = (part[0] + part[1]) + (part[2] + part[3]);
    l[rt] += sum == 0.0f ? 0.0f : sum * bs.over_vs;
    w0[rt] = pack_half8(w[0][rt], w[1][rt]);
    w1[rt] = pack_half8(w[2][rt], w[3][rt]);
  }
}

// Values of a page whose scale is 0 count as zeros, whatever their codes.
template <int RT>
__device__ __forceinline__ void drop_zero_values(const BlockScale& bs, half8 (&w0)[RT], half8 (&w1)[RT]) {
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
    if (bs.bits & 2) w0[rt] = w1[rt] = half8{};
}

__device__ __forceinline__ uint2_t pack_bf16x4(const float4_t& v, float mul) {
  uint2_t w;
  w[0] = uint32_t(f32_to_bf16(v[0] * mul)) | (uint32_t(f32_to_bf16(v[1] * mul)) << 16);
  w[1] = uint32_t(f32_to_bf16(v[2] * mul)) | (uint32_t(f32_to_bf16(v[3] * mul)) << 16);
  return w;
}

// Four values of a row's answer, or of its share of the sums.
__device__ __forceinline__ void put(const AttentionArgs& a, float* partial, int D, int64_t place, int64_t row, int d,
                                    const float4_t& v, float over_l) {
  if (partial != nullptr) *reinterpret_cast<float4_t*>(partial + place * D + d) = v;
  else *reinterpret_cast<uint2_t*>(a.out + row * D + d) = pack_bf16x4(v, over_l);
}

// Both products run on v_mfma_f32_16x16x32_f16 with the codes exact in fp16.  Scores are computed
// transposed, tokens x rows: a lane then holds one row's scores of 16 tokens that follow one
// another (lane row c: tokens 16 c ... of a block of 64), which is the layout the second product's
// operand needs, so the weights never leave the registers; the row statistics need two lane
// exchanges a block.  Rows are (query, head of the group) pairs of one cached head.

// Few rows: a workgroup takes 16 * TILES rows of a cached head, each of its four waves 16 of them and
// every (4 / TILES)th block of tokens, straight from memory into its registers (waves with the same
// tokens find them in the L1 cache); the waves of a tile add up through LDS at the end.  The cache's
// bytes are the bound: a block's keys are asked for as soon as the last block's are used, its values as
// soon as those are.  40 ragged sequences of up to 12000 tokens, 64 / 8 heads of 128: 126 us (4.5 TB/s; a
// plain read of as much reaches 6), where waves that end early are what is left; one sequence of 200000
// tokens, 32 / 8 heads: 87 us (4.7 TB/s), join included; one of 300 tokens: 7.3 us.  Less to read is further
// from that rate: 40 sequences with one cached head 25 us (2.9 TB/s), 20000 tokens of 8 heads of 256 27 us
// (3.0 TB/s, one workgroup of four waves a compute unit), 5 to 6 us of each for the join.
template <int DT>
constexpr size_t few_rows_lds_bytes() {
  return size_t(4) * 16 * (DT + 4) * 4;
}

template <typename TIn, int DT, int TILES, typename Seen>
__global__ __launch_bounds__(256, DT <= 128 ? 2 : 1) void few_rows_kernel(AttentionArgs a, Kv8Batch batch, Kv8Cache cache,
                                                                          Seen seen) {
  constexpr int RT = 1, kPhases = 4 / TILES, kStep = 64 * kPhases;
  constexpr int kRows = TILES * 16, kQStride = DT + 8, kPieces = DT / 64, kTilesD = DT / 16;
  constexpr int kOStride = DT + 4;
  extern __shared__ __align__(16) uint8_t lds[];     // few_rows_lds_bytes: the queries, later the sums
  __shared__ float factor[kRows];
  __shared__ float wave_m[4][16], wave_l[4][16];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, c = lane >> 4;
  const int tile = wave % TILES, phase = wave / TILES;
  const Work w = work_of(a, batch, cache);
  const int G = a.Hq / cache.H;
  _Float16* const q_lds = reinterpret_cast<_Float16*>(lds);

  for (int64_t rb = w.rb; rb * kRows < w.rows; rb += a.row_blocks) {
    const int64_t r0 = rb * kRows;
    // tokens that any of these rows sees, in blocks of 64; this split's share of them
    const int64_t limit = tokens_seen<Seen>(w, min(r0 + kRows, w.rows), G);
    const int64_t blocks = limit > 0 ? (limit + 63) / 64 : 0;
    const int64_t per = (blocks + a.splits - 1) / a.splits, from = w.split * per;
    const int count = int(max(min(per, blocks - from), int64_t(0)));
    // from here on tokens count from the share's first
    const int rel_limit = from_here(limit, from * 64);
    const int all_see = from_here(seen_by_all<Seen>(w, r0, G), from * 64);   // every row sees the tokens up to it

    // tokens of a block that concern the lane: the 16 whose keys it loads (16 (n / 4) ...), and the 16
    // whose values and scores it holds (16 c ...)
    const Pages pages = pages_of(batch, cache, w, limit);
    const uint32_t off_k = 16 * (n >> 2), off_v = 16 * c, base0 = uint32_t(from) * 64 + phase * 64;
    int32_t idk = -1, idv = -1, idk1 = -1, idv1 = -1;            // of the first block and the next
    if (phase < count) {
      idk = pages.find(base0, off_k);
      idv = pages.find(base0, off_v);
      idk1 = pages.find(base0 + kStep, off_k);
      idv1 = pages.find(base0 + kStep, off_v);
    }
    float raw[TILES][16];
    load_queries<TIn>(a, cache, w, r0 + wave * 4 + c, 16, n, raw);

    uint4_t kw[4][kPieces], vw[kTilesD];
    const auto load_keys = [&](uint32_t base, int32_t id) {
      const int8_t* const kp = pages.keys(id) + (((base + off_k) & pages.mask) + (n & 3)) * cache.D;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const int d = 64 * p + 16 * c;
          kw[t][p] = *reinterpret_cast<const uint4_t*>(kp + 4 * t * cache.D + (d < cache.D ? d : 0));
        }
    };
    const auto load_values = [&](uint32_t base, int32_t id) {
      const int8_t* const vp = pages.values(id) + ((base + off_v) & pages.mask);
#pragma unroll
      for (int dt = 0; dt < kTilesD; ++dt) {
        const int d = 16 * dt + n;
        vw[dt] = *reinterpret_cast<const uint4_t*>(vp + (d < cache.D ? d : 0) * cache.page);
      }
    };
    // the keys are on their way while the queries go to LDS, the values only then: with both, 20000 tokens of 8 heads
    // of 256 take 22.1 us instead of 20.7, 3000 of 128 11.3 instead of 10.6
    PageScale page{};
    if (phase < count) {
      load_keys(base0, idk);
      page = scale_of(pages, idv, base0, off_v);
    }
    lds_barrier();                  // no wave reads the sums of the rows before any more
#pragma unroll
    for (int it = 0; it < TILES; ++it) {
      const int i = wave * 4 + c + 16 * it;
      place_query<DT>(a, cache.D, n, raw[it], q_lds + i * kQStride, factor + i);
    }
    if (phase < count) load_values(base0, idv);
    idk = idk1;
    idv = idv1;
    lds_barrier();                  // the queries are there; the codes may still be on their way

    half8 q[RT][kPieces][2];
    float row_scale[RT], m[RT], l[RT];
    RowSees<Seen> sees[RT];
    float4_t o[kTilesD][RT] = {};
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          q[rt][p][k] = *reinterpret_cast<const half8*>(&q_lds[(tile * 16 + n) * kQStride + 64 * p + 16 * c + 8 * k]);
      const int64_t r = r0 + tile * 16 + n;
      row_scale[rt] = factor[tile * 16 + n];
      sees[rt].set(seen, w, r, G, from * 64);
      m[rt] = kNothing;
      l[rt] = 0.0f;
    }
    // one block; `more`: another follows, whose codes are asked for meanwhile.  Every value that a load
    // brings for it is asked for after its last use here, and the last block has a copy of the code
    // of its own, so that nothing has to be moved, or waited for, while it is on its way.
    const auto step = [&](auto tag, int blk) {
      constexpr bool more = decltype(tag)::value;
      const int base = blk * 64;
      float4_t s[4][RT];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          s[t][rt] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const half8 key = decode_i8(kw[t][p][2 * k], kw[t][p][2 * k + 1]);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
              s[t][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key, q[rt][p][k], s[t][rt], 0, 0, 0);
          }
      const uint32_t ahead = uint32_t(from + blk + kPhases) * 64;
      if constexpr (more) {
        load_keys(ahead, idk);
        idk = pages.find(ahead + kStep, off_k);
      }
      __builtin_amdgcn_sched_barrier(0);
      const BlockScale bs = settle(page);
      const int some = __builtin_amdgcn_readfirstlane(bs.bits);
      const bool ragged = base + 63 > all_see || base + 63 >= rel_limit || (some & 4);
      half8 w0[RT], w1[RT];
      float mul[RT];
      refer(s, bs, ragged, base + 16 * c, rel_limit, row_scale, sees, m, l, o, mul);
      if (ragged) weigh<true>(s, bs, mul, m, l, w0, w1);
      else weigh<false>(s, bs, mul, m, l, w0, w1);
      if (some & 8) drop_zero_values(bs, w0, w1);
      if constexpr (more) page = scale_of(pages, idv, ahead, off_v);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int dt = 0; dt < kTilesD; ++dt) {
          const half8 v = decode_i8(vw[dt][2 * k], vw[dt][2 * k + 1]);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            o[dt][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, k == 0 ? w0[rt] : w1[rt], o[dt][rt], 0, 0, 0);
        }
      if constexpr (more) {
        load_values(ahead, idv);
        idv = pages.find(ahead + kStep, off_v);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    int blk = phase;
    for (; blk + kPhases < count; blk += kPhases) step(std::true_type{}, blk);
    if (blk < count) step(std::false_type{}, blk);

#pragma unroll
    for (int rt = 0; rt < RT; ++rt) l[rt] = sum_over_lane_rows(l[rt]);
    // the sums of a tile's waves, added in their order
    if (c == 0) {
      wave_m[wave][n] = m[0];
      wave_l[wave][n] = l[0];
    }
    __syncthreads();                // also: no wave reads the queries any more
    float* const sums = reinterpret_cast<float*>(lds);
    const auto top_of = [&](int t, int i) {
      float top = wave_m[t][i];
#pragma unroll
      for (int k = 1; k < kPhases; ++k) top = fmaxf(top, wave_m[t + k * TILES][i]);
      return top;
    };
    const float down = __builtin_amdgcn_exp2f(m[0] - top_of(tile, n));
#pragma unroll
    for (int dt = 0; dt < kTilesD; ++dt)
      *reinterpret_cast<float4_t*>(&sums[(wave * 16 + n) * kOStride + 16 * dt + 4 * c]) = o[dt][0] * down;
    __syncthreads();
    // a row of 16 lanes to a row
    for (int k = threadIdx.x >> 4; k < kRows; k += 16) {
      const int64_t r = r0 + k;
      const int t = k >> 4, i = k & 15;
      if (r >= w.rows) continue;
      const float top = top_of(t, i);
      float sum = 0.0f;
#pragma unroll
      for (int p = 0; p < kPhases; ++p)
        sum += lowered(wave_l[t + p * TILES][i], wave_m[t + p * TILES][i] - top);
      const int64_t row = (w.seq.row0 + uint32_t(r) / uint32_t(G)) * a.Hq + w.h * G + uint32_t(r) % uint32_t(G);
      if (a.partial != nullptr && n == 0) a.stats[w.split * a.rows + row] = make_float2(top, sum);
      const float over_l = sum == 0.0f ? 0.0f : 1.0f / sum;
      for (int d = n * 4; d < cache.D; d += 64) {
        float4_t v = *reinterpret_cast<const float4_t*>(&sums[(t * 16 + i) * kOStride + d]);
#pragma unroll
        for (int p = 1; p < kPhases; ++p)
          v += *reinterpret_cast<const float4_t*>(&sums[((t + p * TILES) * 16 + i) * kOStride + d]);
        put(a, a.partial, cache.D, w.split * a.rows + row, row, d, v, over_l);
      }
    }
  }
}

constexpr int kAhead = 6;      // operand reads from LDS that are ahead of their use

// Many rows: a workgroup of eight waves takes 8 * 16 * RT rows.  Every block of 64 tokens is decoded
// once, an eighth by each wave, into the operand layout in LDS (blocks of 1 KB that a wave reads as
// they are), where all eight waves use it.
//
// A block is two phases of a wave, one of vector arithmetic (its weights) and one of matrix
// instructions (its values' product, then the next block's scores) with the decoding of coming blocks
// between them.  The two waves of a SIMD, w and w + 4, are kept one phase apart by a barrier after
// each, so that the matrix cores work for one while the other has its weights computed; the matrix phase
// has the higher priority.  3x900 rows over 6000 tokens, 32 / 8 heads of 128: 244 us; 262 with one priority,
// 278 with the groups in step, 315 with waves 2 i and 2 i + 1 apart, which share no SIMD.  Heads of 256
// (16 / 4; one tile of rows a wave) 254, 265, 265 and 379.  With phases counted over both groups, waves 0-3 do the weights of block i in phase 2 i and its products in 2 i + 1, waves
// 4-7 one later: keys of block j are read in phases 2 j - 1 and 2 j, values in 2 j + 1 and 2 j + 2.  In its
// product phase of block i a wave writes its part of the keys of block i + 2 and of the values of block
// i + 1: two buffers each are enough, and four places for the page scales (read in phases 2 j - 1 to
// 2 j + 1, written in 2 j - 3 and 2 j - 2).
template <int DT, int RT>
constexpr size_t many_rows_lds_bytes() {               // two blocks of keys and values and the scales, or the queries
  const size_t blocks = size_t(DT / 8) * 2048 * 2 + 4 * 64, queries = size_t(8) * RT * 16 * (DT + 8) * 2;
  return blocks > queries ? blocks : queries;
}

template <typename TIn, int DT, int RT, typename Seen>
__device__ __forceinline__ void many_rows(const AttentionArgs& a, const Kv8Batch& batch, const Kv8Cache& cache,
                                          const Seen& seen, const Work& w, int64_t rb, int64_t limit, int64_t from,
                                          int count) {
  constexpr int kWaveRows = RT * 16, kRows = 8 * kWaveRows;
  constexpr int kPieces = DT / 64, kTilesD = DT / 16, kQStride = DT + 8;
  constexpr int kHalf = 4 * kPieces * 2048;            // the keys, or the values, of a block
  constexpr int kMine = (4 * kPieces + 7) / 8;         // 2 KB jobs of a wave in each half
  extern __shared__ __align__(16) uint8_t lds[];       // many_rows_lds_bytes
  uint8_t* const key_lds = lds;
  uint8_t* const value_lds = lds + 2 * kHalf;
  float* const scale_lds = reinterpret_cast<float*>(lds + 4 * kHalf);
  static_assert(4 * kPieces == kTilesD, "as many key tiles as value tiles");
  __shared__ float factor[kRows];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, c = lane >> 4;
  const int G = a.Hq / cache.H;
  const int64_t r0 = rb * kRows + wave * kWaveRows;
  half8 q[RT][kPieces][2];
  float row_scale[RT], m[RT], l[RT];
  RowSees<Seen> sees[RT];
  // a wave's queries, four rows of each of its lane rows asked for at once
  float raw_q[4][16];
  load_queries<TIn>(a, cache, w, r0 + c, 4, n, raw_q);
  const bool active = r0 < w.rows;                               // the wave has rows
  // from here on tokens count from the share's first
  const int rel_limit = from_here(limit, from * 64);
  const int all_see = from_here(seen_by_all<Seen>(w, r0, G), from * 64);   // every row of the wave sees the tokens up to it
  const Pages pages = pages_of(batch, cache, w, limit);
  const uint32_t off_k = 16 * (n >> 2), off_v = 16 * c, base0 = uint32_t(from) * 64;
  uint4_t raw_k[kMine], raw_v[kMine];
  PageScale raw_page{};
  const bool works = kTilesD >= 8 || wave < kTilesD;      // with D <= 64 half the waves have no part
  const auto load_keys = [&](uint32_t base, int32_t id) {
    const int8_t* const kp = pages.keys(id) + (((base + off_k) & pages.mask) + (n & 3)) * cache.D;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int job = i * 8 + wave, d = 64 * (job / 4) + 16 * c;
      if (works) raw_k[i] = *reinterpret_cast<const uint4_t*>(kp + 4 * (job % 4) * cache.D + (d < cache.D ? d : 0));
    }
  };
  const auto load_values = [&](uint32_t base, int32_t id) {
    const int8_t* const vp = pages.values(id) + ((base + off_v) & pages.mask);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int d = 16 * (i * 8 + wave) + n;
      if (works) raw_v[i] = *reinterpret_cast<const uint4_t*>(vp + (d < cache.D ? d : 0) * cache.page);
    }
  };
  // the first block's codes, and the pages of the next two, are on their way while the queries go through LDS in
  // the buffers' place
  int32_t k0 = 0, v0 = 0, k1 = 0, v1 = 0, k2 = 0, v2 = 0;
  if (count > 0) {
    k0 = pages.find(base0, off_k), v0 = pages.find(base0, off_v);
    k1 = pages.find(base0 + 64, off_k), v1 = pages.find(base0 + 64, off_v);
    k2 = pages.find(base0 + 128, off_k), v2 = pages.find(base0 + 128, off_v);
    load_keys(base0, k0);
    load_values(base0, v0);
    raw_page = scale_of(pages, v0, base0, off_v);
  }
  lds_barrier();                                       // no wave reads what a piece of work before this one left
  _Float16* const q_lds = reinterpret_cast<_Float16*>(lds) + wave * kWaveRows * kQStride;
#pragma nounroll
  for (int part = 0; part < kWaveRows / 4; part += 4) {
    if (part > 0) load_queries<TIn>(a, cache, w, r0 + c + 4 * part, 4, n, raw_q);
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int i = c + 4 * (part + it);
      place_query<DT>(a, cache.D, n, raw_q[it], q_lds + i * kQStride, factor + wave * kWaveRows + i);
    }
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int p = 0; p < kPieces; ++p)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        q[rt][p][k] = *reinterpret_cast<const half8*>(&q_lds[(rt * 16 + n) * kQStride + 64 * p + 16 * c + 8 * k]);
  lds_barrier();
  float4_t o[kTilesD][RT] = {};
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int64_t r = r0 + rt * 16 + n;
    row_scale[rt] = factor[wave * kWaveRows + rt * 16 + n];
    sees[rt].set(seen, w, r, G, from * 64);
    m[rt] = kNothing;
    l[rt] = 0.0f;
  }
  // half h of job i of a wave's part, decoded and written
  const auto write = [&](uint8_t* at, const uint4_t& raw, int i, int h) {
    if (works) reinterpret_cast<half8*>(at + (i * 8 + wave) * 2048)[64 * h + lane] = decode_i8(raw[2 * h], raw[2 * h + 1]);
  };
  const auto write_all = [&](uint8_t* at, const uint4_t (&raw)[kMine]) {
#pragma unroll
    for (int i = 0; i < 2 * kMine; ++i) write(at, raw[i / 2], i / 2, i % 2);
  };
  const auto write_scale = [&](int i) {                   // by every lane that knows it, all alike
    const BlockScale bs = settle(raw_page);
    reinterpret_cast<float4_t*>(scale_lds)[(i & 3) * 4 + c] = float4_t{bs.ks, bs.lv, bs.over_vs, __int_as_float(bs.bits)};
  };
  float4_t s[4][RT];
  // operand blocks of the scores: piece j / 8, half j / 4 % 2, token tile j % 4; of the values' product:
  // half j / kTilesD of the tokens, channel tile j % kTilesD
  constexpr int kReads = 2 * kTilesD;
  const auto key_block = [&](const uint8_t* at, int j) {
    return reinterpret_cast<const half8*>(at + (j / 8 * 4 + j % 4) * 2048)[j / 4 % 2 * 64 + lane];
  };
  const auto value_block = [&](const uint8_t* at, int j) {
    return reinterpret_cast<const half8*>(at + j % kTilesD * 2048)[j / kTilesD * 64 + lane];
  };
  const auto score_step = [&](const half8& key, int j) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      s[j % 4][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
          key, q[rt][j / 8][j / 4 % 2], j < 4 ? float4_t{0.0f, 0.0f, 0.0f, 0.0f} : s[j % 4][rt], 0, 0, 0);
  };

  if (count > 0) {
    // blocks 0 and 1 of the keys and 0 of the values, then what the first phases write
    write_all(key_lds, raw_k);
    write_all(value_lds, raw_v);
    write_scale(0);
    load_keys(base0 + 64, k1);
    raw_page = scale_of(pages, v1, base0 + 64, off_v);
    write_all(key_lds + kHalf, raw_k);
    write_scale(1);
    load_keys(base0 + 128, k2);
    raw_page = scale_of(pages, v2, base0 + 128, off_v);
    load_values(base0 + 64, v1);
    // pages that the product phase of block i needs: for the keys and the scales of block i + 3, for the
    // values of i + 2.  Past the share's end blocks are loaded from its last token's page and never
    // used.
    int32_t idk = pages.find(base0 + 192, off_k), ids = pages.find(base0 + 192, off_v), idv = v2;
    lds_barrier();
#pragma unroll
    for (int j = 0; j < kReads; ++j) score_step(key_block(key_lds, j), j);
    if (wave >= 4) lds_barrier();
    BlockScale bs{};
    const auto read_scale = [&](int i) {
      const float4_t v = reinterpret_cast<const float4_t*>(scale_lds)[(i & 3) * 4 + c];
      bs = BlockScale{v[0], v[1], v[2], __float_as_int(v[3])};
    };
    // what a wave does beside the products of block i, in pieces
    constexpr int kPieceCount = 4 * kMine + 6;
    const auto piece = [&](int i, int p) {
      const uint32_t ahead = uint32_t(from + i) * 64;
      if (p < 2 * kMine) write(value_lds + ((i + 1) & 1) * kHalf, raw_v[p / 2], p / 2, p % 2);
      else if (p < 4 * kMine) write(key_lds + (i & 1) * kHalf, raw_k[p / 2 - kMine], p / 2 - kMine, p % 2);
      else if (p == 4 * kMine) write_scale(i + 2);
      else if (p == 4 * kMine + 1) load_values(ahead + 128, idv);
      else if (p == 4 * kMine + 2) load_keys(ahead + 192, idk);
      else if (p == 4 * kMine + 3) raw_page = scale_of(pages, ids, ahead + 192, off_v);
      else if (p == 4 * kMine + 4) idv = pages.find(ahead + 192, off_v), idk = pages.find(ahead + 256, off_k);
      else ids = pages.find(ahead + 256, off_v), read_scale(i + 1);
    };
    read_scale(0);
    if (active) {
      for (int i = 0; i < count; ++i) {
        const int some = __builtin_amdgcn_readfirstlane(bs.bits);
        const bool ragged = i * 64 + 63 > all_see || i * 64 + 63 >= rel_limit || (some & 4);
        float mul[RT];
        half8 w0[RT], w1[RT];
        refer(s, bs, ragged, i * 64 + 16 * c, rel_limit, row_scale, sees, m, l, o, mul);
        if (ragged) weigh<true>(s, bs, mul, m, l, w0, w1);
        else weigh<false>(s, bs, mul, m, l, w0, w1);
        if (some & 8) drop_zero_values(bs, w0, w1);
        lds_barrier();
        __builtin_amdgcn_s_setprio(1);
        // both products as one run of matrix instructions, each operand block read kAhead blocks before
        // its use, and the other work in pieces between them; the compiler keeps this order.  A loop for
        // each product: as one of 64 rounds (heads above 128) the compiler does not write it out, and
        // every array that it indexes moves to scratch memory (3x900 rows over 6000 tokens, 16 / 4
        // heads of 256: 69 ms so, 254 us in two loops)
        const uint8_t* const values = value_lds + (i & 1) * kHalf;
        const uint8_t* const keys = key_lds + ((i + 1) & 1) * kHalf;
        half8 ring[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) ring[j] = value_block(values, j);
        const auto beside = [&](int j) {
#pragma unroll
          for (int p = 0; p < kPieceCount; ++p)
            if (p * 2 * kReads / kPieceCount == j) piece(i, p);
          __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int j = 0; j < kReads; ++j) {
          const half8 operand = ring[j % kAhead];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            o[j % kTilesD][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(operand, j < kTilesD ? w0[rt] : w1[rt],
                                                                       o[j % kTilesD][rt], 0, 0, 0);
          ring[j % kAhead] = j + kAhead < kReads ? value_block(values, j + kAhead) : key_block(keys, j + kAhead - kReads);
          beside(j);
        }
#pragma unroll
        for (int j = kReads; j < 2 * kReads; ++j) {
          const half8 operand = ring[j % kAhead];
          score_step(operand, j - kReads);
          if (j + kAhead < 2 * kReads) ring[j % kAhead] = key_block(keys, j + kAhead - kReads);
          beside(j);
        }
        __builtin_amdgcn_s_setprio(0);
        lds_barrier();
      }
    } else {                                               // a loop of its own: see few_rows_kernel's step
      for (int i = 0; i < count; ++i) {
        lds_barrier();
#pragma unroll
        for (int p = 0; p < kPieceCount; ++p) piece(i, p);
        lds_barrier();
      }
    }
    if (wave < 4) lds_barrier();
  }

#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    l[rt] = sum_over_lane_rows(l[rt]);
    const int64_t r = r0 + rt * 16 + n;
    if (r >= w.rows) continue;
    const int64_t row = (w.seq.row0 + uint32_t(r) / uint32_t(G)) * a.Hq + w.h * G + uint32_t(r) % uint32_t(G);
    const int64_t at = max(w.split, int64_t(0)) * a.rows + row;
    int64_t place = at;
    if constexpr (std::is_same_v<Seen, TreeTokens>)
      if (seen.whole) place = (2 * int64_t(blockIdx.x) + (from == 0)) * kRows + (r - rb * kRows);
    if (a.partial != nullptr && c == 0) {
      a.stats[at] = make_float2(m[rt], w.split < 0 ? -1.0f : l[rt]);
      if constexpr (std::is_same_v<Seen, TreeTokens>)
        if (seen.whole) places_of(a)[at] = uint32_t(place);
    }
    const float over_l = l[rt] == 0.0f ? 0.0f : 1.0f / l[rt];
#pragma unroll
    for (int dt = 0; dt < kTilesD; ++dt) {
      const int d = 16 * dt + 4 * c;
      if (d < cache.D) put(a, w.split < 0 ? nullptr : a.partial, cache.D, place, row, d, o[dt][rt], over_l);
    }
  }
}

template <typename TIn, int DT, int RT>
__global__ __launch_bounds__(512) void many_rows_kernel(AttentionArgs a, Kv8Batch batch, Kv8Cache cache, EarlierTokens seen) {
  constexpr int kRows = 8 * RT * 16;
  const Work w = work_of(a, batch, cache);
  for (int64_t rb = w.rb; rb * kRows < w.rows; rb += a.row_blocks) {
    // tokens that any of these rows sees, in blocks of 64; this split's share of them
    const int64_t limit = tokens_seen<EarlierTokens>(w, min(rb * kRows + kRows, w.rows), a.Hq / cache.H);
    const int64_t blocks = limit > 0 ? (limit + 63) / 64 : 0;
    const int64_t per = (blocks + a.splits - 1) / a.splits, from = w.split * per;
    many_rows<TIn, DT, RT>(a, batch, cache, seen, w, rb, limit, from, int(max(min(per, blocks - from), int64_t(0))));
  }
}

// Joins the splits of a row, WAVES waves to a row, each of which takes every WAVES-th split; always in the
// same order.  64 splits of 32 rows of 128: 6.5 us with four waves to a row, 68 with one.
template <int WAVES>
__global__ __launch_bounds__(256) void join_splits_kernel(Kv8Batch batch, int Hq, int D, int splits, int64_t rows,
                                                          const float* __restrict__ partial,
                                                          const float2* __restrict__ stats,
                                                          uint16_t* __restrict__ out) {
  constexpr int kPerBlock = 4 / WAVES;
  __shared__ __align__(16) float4_t part[WAVES == 1 ? 1 : 4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = int64_t(blockIdx.x) * kPerBlock + wave / WAVES;
  if (row >= rows) return;
  const int64_t t = row / Hq;
  bool there = false;
  for (int64_t i = lane; i < batch.B; i += 64) {
    const Sequence seq = sequence_of(batch, i);
    there = there || (t >= seq.row0 && t < seq.row0 + seq.n);
  }
  if (!__any(there)) return;                                  // a row of no sequence: left as it is
  float top = kNothing;
  for (int s = lane; s < splits; s += 64) top = fmaxf(top, stats[s * rows + row].x);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
  float sum = 0.0f;
  for (int s = lane; s < splits; s += 64) {
    const float2 st = stats[s * rows + row];
    sum += lowered(st.y, st.x - top);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
  const float over_l = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int first = WAVES == 1 ? 0 : wave;
  float4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
  const int d = lane * 4;                                     // D <= 256: a wave holds a row
  if (d < D) {
#pragma unroll 4
    for (int s = first; s < splits; s += WAVES) {
      const float2 st = stats[s * rows + row];
      if (st.y == 0.0f) continue;                             // nothing seen there, nothing written
      const float f = __builtin_amdgcn_exp2f(st.x - top);
      const float4_t p = *reinterpret_cast<const float4_t*>(partial + (s * rows + row) * D + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(p[i], f, v[i]);
    }
  }
  if constexpr (WAVES > 1) {
    part[wave][lane] = v;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int k = 1; k < WAVES; ++k) v += part[k][lane];
  }
  if (d < D) *reinterpret_cast<uint2_t*>(out + row * D + d) = pack_bf16x4(v, over_l);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

bool wide_rows(const void* p, int64_t t, int64_t h, int dtype) {
  const int per = dtype == 0 ? 4 : 8;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && t % per == 0 && h % per == 0;
}

template <typename Kernel, typename Seen>
hipError_t run_kernel(Kernel* kernel, int64_t groups, int threads, size_t lds, const AttentionArgs& a,
                      const Kv8Batch& b, const Kv8Cache& c, const Seen& seen, hipStream_t stream) {
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
    if (e != hipSuccess) return e;
  }
  return launch_kernel(kernel, dim3(unsigned(groups)), dim3(threads), lds, stream, a, b, c, seen);
}

// Many rows of trees, and the join of their pieces (kv8_tree.hip).
template <typename TIn, int DT>
hipError_t run_tree(const AttentionArgs& a, const Kv8Batch& b, const Kv8Cache& c, const TreeTokens& tree,
                    const Kv8Plan& p, hipStream_t stream);
hipError_t join_pieces(const AttentionArgs& a, const Kv8Batch& b, const Kv8Cache& c, const TreeTokens& tree,
                       const Kv8Plan& p, hipStream_t stream);

template <typename TIn, int DT, typename Seen>
hipError_t run_attention(const AttentionArgs& a, const Kv8Batch& b, const Kv8Cache& c, const Seen& seen,
                         const Kv8Plan& p, hipStream_t stream) {
  const int64_t groups = b.B * c.H * p.row_blocks * p.splits;
  constexpr size_t kFew = few_rows_lds_bytes<DT>();
  if (p.row_tiles == 1) return run_kernel(few_rows_kernel<TIn, DT, 1, Seen>, groups, 256, kFew, a, b, c, seen, stream);
  if (p.row_tiles == 2) return run_kernel(few_rows_kernel<TIn, DT, 2, Seen>, groups, 256, kFew, a, b, c, seen, stream);
  if (p.row_tiles == 4) return run_kernel(few_rows_kernel<TIn, DT, 4, Seen>, groups, 256, kFew, a, b, c, seen, stream);
  if constexpr (std::is_same_v<Seen, TreeTokens>) return run_tree<TIn, DT>(a, b, c, seen, p, stream);
  else {
    constexpr int RT = DT == 256 ? 1 : 2;
    return run_kernel(many_rows_kernel<TIn, DT, RT>, groups, 512, many_rows_lds_bytes<DT, RT>(), a, b, c, seen, stream);
  }
}

template <typename TIn, typename Seen>
hipError_t run_attention(const AttentionArgs& a, const Kv8Batch& b, const Kv8Cache& c, const Seen& seen,
                         const Kv8Plan& p, hipStream_t stream) {
  if (c.D <= 64) return run_attention<TIn, 64>(a, b, c, seen, p, stream);
  if (c.D <= 128) return run_attention<TIn, 128>(a, b, c, seen, p, stream);
  return run_attention<TIn, 256>(a, b, c, seen, p, stream);
}

// The attention of a call: the kernel of its plan, and the join of its splits.
template <typename Seen>
hipError_t attend(const void* q, int dtype, int64_t q_t, int64_t q_h, int64_t Hq, const Kv8Batch& b,
                  const Kv8Cache& c, const Seen& seen, int g, float scale, const Kv8Plan& p, uint16_t* out,
                  void* workspace, hipStream_t stream) {
  AttentionArgs a{};
  a.q = q;
  a.q_t = q_t;
  a.q_h = q_h;
  a.q_wide = wide_rows(q, q_t, q_h, dtype);
  a.Hq = int(Hq);
  a.digits = digits_of(g);
  a.splits = p.splits;
  a.scale = scale;
  a.row_blocks = p.row_blocks;
  a.rows = b.T * Hq;
  a.out = out;
  if (p.splits > 1) {
    a.partial = static_cast<float*>(workspace);
    a.stats = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + round256(size_t(p.sums) * c.D * 4));
  }
  const hipError_t e = dtype == 0 ? run_attention<float>(a, b, c, seen, p, stream)
                                  : run_attention<uint16_t>(a, b, c, seen, p, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  if constexpr (std::is_same_v<Seen, TreeTokens>)
    if (p.row_tiles > 4) return join_pieces(a, b, c, seen, p, stream);
  // a wave to a row; four where there are many splits
  if (p.splits <= 8)
    return launch_kernel(join_splits_kernel<1>, dim3(unsigned(ceil_div(a.rows, 4))), dim3(256), 0, stream, b,
                         int(Hq), c.D, p.splits, a.rows, a.partial, a.stats, out);
  return launch_kernel(join_splits_kernel<4>, dim3(unsigned(a.rows)), dim3(256), 0, stream, b, int(Hq), c.D,
                       p.splits, a.rows, a.partial, a.stats, out);
}

}  // namespace
}  // namespace convrot
