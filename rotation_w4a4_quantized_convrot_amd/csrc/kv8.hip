// The paged 8-bit key/value cache: append (convrot_kv8_append), read back (convrot_kv8_read) and
// attention (convrot_kv8_attention).
//
// A page holds `page` tokens of one sequence; for each page and head there are int8 codes and one
// fp32 scale for the keys and one for the values.  Keys [page][head][slot][D] are rotated in
// windows of g before they are quantized (their few large channels spread over the window) and
// queries are rotated alike: H_g / sqrt(g) is orthogonal, so the scores stay.  Values stand
// transposed, [page][head][D][slot]: 16 tokens of a channel are 16 bytes, what one lane feeds
// into the matrix instructions of P V.
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

__device__ __forceinline__ uint32_t pack_codes(const float* v, float scale) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    int q = 0;
    if (scale > 0.0f) q = int(fminf(fmaxf(rintf(__fdiv_rn(v[e], scale)), -127.0f), 127.0f));
    w |= uint32_t(q & 255) << (8 * e);
  }
  return w;
}

// Four kept codes under a grown scale: rne(code * ratio).
__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float ratio) {
  uint32_t r = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    r |= uint32_t(int(rintf(float(int8_t(w >> (8 * e))) * ratio)) & 255) << (8 * e);
  return r;
}

constexpr int kThreads = 256;

struct KvRows {
  const void *k, *v;
  int64_t k_t, k_h, v_t, v_h;
  bool k_wide, v_wide;
};

// One workgroup per (sequence, page the new tokens reach, head, keys or values): it alone
// touches that page's codes and scale, so the page's largest value, the new scale, the kept
// codes and the new ones take one launch and no atomics.  ITER * 16 tokens to a page, a row of 16
// lanes to a token.
//
// Six ragged prompts of up to 2500 rows, 8 heads of 128 (bf16, pages of 64; 60 MB): 38.4 us, 1.6 TB/s;
// what is beyond the copy's 12 us is the values' way through LDS byte by byte and a page's three steps
// (load, maximum, codes) that nothing overlaps in a workgroup.  48 x 1 rows: 7.2 us, the launch and three
// trips to memory one after another (the sequence, its page, the page's codes).
template <typename TIn, int ITER>
__global__ __launch_bounds__(kThreads) void append_kernel(KvRows rows, Kv8Batch batch, Kv8Cache cache, int digits) {
  constexpr int kPage = 16 * ITER, kStride = kPage + 16;
  extern __shared__ __align__(16) uint8_t tile[];          // values only: [D][kStride]
  __shared__ uint32_t wave_max[kThreads / 64];
  const bool values = blockIdx.x & 1;
  const int64_t h = (blockIdx.x >> 1) % cache.H, b = (blockIdx.x >> 1) / cache.H;
  const Sequence seq = sequence_of(batch, b);
  if (seq.n == 0 || seq.len < seq.n) return;
  const int64_t before = seq.len - seq.n;
  const int row = threadIdx.x >> 4, d = (threadIdx.x & 15) * 16;
  const TIn* src = values ? static_cast<const TIn*>(rows.v) + h * rows.v_h : static_cast<const TIn*>(rows.k) + h * rows.k_h;
  const int64_t src_t = values ? rows.v_t : rows.k_t;
  const bool wide = values ? rows.v_wide : rows.k_wide;

  for (int64_t col = before / kPage + blockIdx.y; col <= (seq.len - 1) / kPage; col += gridDim.y) {
    const int64_t id = page_of(batch, cache, b, col);
    if (id < 0) continue;
    const int lo = int(max(before - col * kPage, int64_t(0)));
    const int hi = int(min(seq.len - col * kPage, int64_t(kPage)));
    float v[ITER][16];
    uint32_t bits = 0;
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const int slot = it * 16 + row;
      const bool here = slot >= lo && slot < hi && d < cache.D;
      const int64_t t = seq.row0 + col * kPage + slot - before;
      load16<TIn>(here ? src + t * src_t + d : src, here ? 16 : 0, wide, v[it]);
      if (!values) rotate16(v[it], digits);
      bits = max(bits, abs_max16(v[it]));
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) bits = max(bits, uint32_t(__shfl_xor(int(bits), o)));
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = bits;
    float* const scale_at = (values ? cache.vs : cache.ks) + id * cache.H + h;
    const float old = lo > 0 ? *scale_at : 0.0f;
    __syncthreads();
    bits = max(max(wave_max[0], wave_max[1]), max(wave_max[2], wave_max[3]));
    float scale = __fdiv_rn(__uint_as_float(bits), 127.0f);
    if (scale < kLeastScale) scale = 0.0f;
    const bool finite = bits < 0x7F800000u && old == old;
    scale = finite ? fmaxf(scale, old) : __uint_as_float(0x7FC00000u);
    const bool again = lo > 0 && finite && scale != old;      // the kept codes change
    const float ratio = again ? __fdiv_rn(old, scale) : 1.0f;
    if (threadIdx.x == 0) *scale_at = scale;

    if (!values) {
      int8_t* const page = cache.kc + (id * cache.H + h) * kPage * cache.D;
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int slot = it * 16 + row;
        if (d >= cache.D || slot >= hi) continue;
        uint4_t* const at = reinterpret_cast<uint4_t*>(page + slot * cache.D + d);
        uint4_t w;
        if (slot >= lo) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = pack_codes(&v[it][4 * j], scale);
          *at = w;
        } else if (again) {
          w = *at;
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = rescale_codes(w[j], ratio);
          *at = w;
        }
      }
    } else {
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int slot = it * 16 + row;
        if (d >= cache.D || slot < lo || slot >= hi) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = pack_codes(&v[it][4 * j], scale);
#pragma unroll
          for (int e = 0; e < 4; ++e) tile[(d + 4 * j + e) * kStride + slot] = uint8_t(w >> (8 * e));
        }
      }
      __syncthreads();
      int8_t* const page = cache.vc + (id * cache.H + h) * kPage * cache.D;
      for (int i = threadIdx.x; i < cache.D * ITER; i += kThreads) {
        const int channel = i / ITER, s = (i % ITER) * 16;        // 16 slots of a channel
        if (s >= hi || (s + 16 <= lo && !again)) continue;
        uint4_t* const at = reinterpret_cast<uint4_t*>(page + channel * kPage + s);
        uint4_t w = *reinterpret_cast<const uint4_t*>(&tile[channel * kStride + s]);
        if (s < lo || s + 16 > hi) {
          const uint4_t was = *at;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t kept = again ? rescale_codes(was[j], ratio) : was[j];
            uint32_t r = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int slot = s + 4 * j + e;
              const uint32_t from = slot < lo ? kept : slot < hi ? w[j] : was[j];
              r |= from & (0xFFu << (8 * e));
            }
            w[j] = r;
          }
        }
        *at = w;
      }
    }
    __syncthreads();   // wave_max and the tile are written again
  }
}

// The last n tokens of each sequence as bf16 rows, keys turned back (the rotation is its own
// inverse).  The same workgroups as append; values go through LDS to stand by token again.  The six
// prompts above: 29.9 us, 2.0 TB/s.
template <int ITER>
__global__ __launch_bounds__(kThreads) void read_kernel(Kv8Batch batch, Kv8Cache cache, int digits,
                                                        uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  constexpr int kPage = 16 * ITER, kStride = kPage + 16;
  extern __shared__ __align__(16) uint8_t tile[];
  const bool values = blockIdx.x & 1;
  const int64_t h = (blockIdx.x >> 1) % cache.H, b = (blockIdx.x >> 1) / cache.H;
  const Sequence seq = sequence_of(batch, b);
  if (seq.n == 0 || seq.len < seq.n) return;
  const int64_t before = seq.len - seq.n;
  const int row = threadIdx.x >> 4, d = (threadIdx.x & 15) * 16;
  uint16_t* const out = values ? v : k;

  for (int64_t col = before / kPage + blockIdx.y; col <= (seq.len - 1) / kPage; col += gridDim.y) {
    const int64_t id = page_of(batch, cache, b, col);
    const int lo = int(max(before - col * kPage, int64_t(0)));
    const int hi = int(min(seq.len - col * kPage, int64_t(kPage)));
    const float scale = id < 0 ? 0.0f : (values ? cache.vs : cache.ks)[id * cache.H + h];
    const int8_t* const page = (values ? cache.vc : cache.kc) + max(id, int64_t(0)) * cache.H * kPage * cache.D +
                               h * kPage * cache.D;
    if (values && id >= 0) {
      for (int i = threadIdx.x; i < cache.D * ITER; i += kThreads) {
        const int channel = i / ITER, s = (i % ITER) * 16;
        if (s >= hi || s + 16 <= lo) continue;
        *reinterpret_cast<uint4_t*>(&tile[channel * kStride + s]) =
            *reinterpret_cast<const uint4_t*>(page + channel * kPage + s);
      }
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const int slot = it * 16 + row;
      const bool here = slot >= lo && slot < hi && d < cache.D;
      float x[16];
      if (!here || id < 0) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = 0.0f;
      } else if (values) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = float(int8_t(tile[(d + e) * kStride + slot])) * scale;
      } else {
        const uint4_t w = *reinterpret_cast<const uint4_t*>(page + slot * cache.D + d);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = float(int8_t(w[e >> 2] >> (8 * (e & 3)))) * scale;
      }
      if (!values) rotate16(x, digits);
      if (here) {
        const int64_t t = seq.row0 + col * kPage + slot - before;
        uint4_t* const at = reinterpret_cast<uint4_t*>(out + (t * cache.H + h) * cache.D + d);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint4_t w;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = uint32_t(f32_to_bf16(x[8 * i + 2 * j])) | (uint32_t(f32_to_bf16(x[8 * i + 2 * j + 1])) << 16);
          at[i] = w;
        }
      }
    }
    __syncthreads();
  }
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
  float* partial;                 // [splits][rows][D], or NULL: one split, straight to out
  float2* stats;                  // [splits][rows]: reference and sum
};

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
  int64_t id = blockIdx.x;
  w.h = id % cache.H;
  id /= cache.H;
  w.split = id % a.splits;
  id /= a.splits;
  w.rb = a.row_blocks - 1 - id % a.row_blocks;
  w.b = id / a.row_blocks;
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

// Sixteen values of query row r of a (sequence, cached head), rotated and scaled into fp16's range, to
// 16 places of LDS; `factor` takes the row's score scale, in powers of two.  A row of 16 lanes
// holds the row.  A negative scale's sign goes to the query, so that score scales are never
// negative.  A row that holds an Inf or a NaN becomes NaN as a whole: unrotated, an Inf that meets codes of
// one sign would make scores of -Inf, which is how tokens that are not seen are marked.
template <typename TIn, int DT>
__device__ __forceinline__ void stage_query(const AttentionArgs& a, const Kv8Cache& cache, const Work& w, int64_t r,
                                            int n, _Float16* row, float* factor) {
  const int G = a.Hq / cache.H;
  const bool there = r < w.rows && n * 16 < cache.D;
  const int64_t t = w.seq.row0 + (there ? r / G : 0), hq = w.h * G + (there ? r % G : 0);
  const TIn* p = static_cast<const TIn*>(a.q) + (there ? t * a.q_t + hq * a.q_h + n * 16 : 0);
  float v[16];
  load16<TIn>(p, there ? 16 : 0, a.q_wide, v);
  float up, back;
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
// token, the lane's first, limit and sees, a row's last token, count from the share's first), and the
// references.
template <int RT, int TILES>
__device__ __forceinline__ void refer(float4_t (&s)[4][RT], const BlockScale& bs, bool ragged, int token, int limit,
                                      const float (&row_scale)[RT], const int (&sees)[RT], float (&m)[RT],
                                      float (&l)[RT], float4_t (&o)[TILES][RT], float (&mul)[RT]) {
  if (ragged) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int seen = bs.bits & 1 ? -1 : min(sees[rt], limit - 1) - token;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * t + i > seen) s[t][rt][i] = -INFINITY;
    }
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
__device__ __forceinline__ void put(const AttentionArgs& a, int D, int64_t split, int64_t row, int d,
                                    const float4_t& v, float over_l) {
  if (a.partial != nullptr) *reinterpret_cast<float4_t*>(a.partial + (split * a.rows + row) * D + d) = v;
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
// soon as those are.  40 ragged sequences of up to 12000 tokens, 64 / 8 heads of 128: 130 us (4.4 TB/s; a
// plain read of as much reaches 6), where waves that end early are what is left; one sequence of 200000
// tokens, 32 / 8 heads: 92 us (4.5 TB/s), join included; one of 300 tokens: 7.4 us.  Less to read is further
// from that rate: 40 sequences with one cached head 27 us (2.7 TB/s), 20000 tokens of 8 heads of 256 27 us
// (3.0 TB/s, one workgroup of four waves a compute unit), 5 to 6 us of each for the join.
template <int DT>
constexpr size_t few_rows_lds_bytes() {
  return size_t(4) * 16 * (DT + 4) * 4;
}

template <typename TIn, int DT, int TILES>
__global__ __launch_bounds__(256, DT <= 128 ? 2 : 1) void few_rows_kernel(AttentionArgs a, Kv8Batch batch, Kv8Cache cache) {
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
    const int64_t limit = min(w.len, w.before + (min(r0 + kRows, w.rows) - 1) / G + 1);
    const int64_t blocks = limit > 0 ? (limit + 63) / 64 : 0;
    const int64_t per = (blocks + a.splits - 1) / a.splits, from = w.split * per;
    const int count = int(max(min(per, blocks - from), int64_t(0)));
    // from here on tokens count from the share's first
    const int rel_limit = from_here(limit, from * 64);
    const int all_see = from_here(w.before + r0 / G, from * 64);   // every row sees the tokens up to it

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
    __syncthreads();
    for (int i = wave * 4 + c; i < kRows; i += 16)
      stage_query<TIn, DT>(a, cache, w, r0 + i, n, q_lds + i * kQStride, factor + i);

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
    PageScale page{};
    if (phase < count) {
      load_keys(base0, idk);
      page = scale_of(pages, idv, base0, off_v);
      load_values(base0, idv);
    }
    idk = idk1;
    idv = idv1;
    lds_barrier();                  // the queries are there; the codes may still be on their way

    half8 q[RT][kPieces][2];
    float row_scale[RT], m[RT], l[RT];
    int sees[RT];                   // last token that the lane's row may see
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
      sees[rt] = r < w.rows ? from_here(w.before + r / G, from * 64) : -1;
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
      const int64_t row = (w.seq.row0 + r / G) * a.Hq + w.h * G + r % G;
      if (a.partial != nullptr && n == 0) a.stats[w.split * a.rows + row] = make_float2(top, sum);
      const float over_l = sum == 0.0f ? 0.0f : 1.0f / sum;
      for (int d = n * 4; d < cache.D; d += 64) {
        float4_t v = *reinterpret_cast<const float4_t*>(&sums[(t * 16 + i) * kOStride + d]);
#pragma unroll
        for (int p = 1; p < kPhases; ++p)
          v += *reinterpret_cast<const float4_t*>(&sums[((t + p * TILES) * 16 + i) * kOStride + d]);
        put(a, cache.D, w.split, row, d, v, over_l);
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
// has the higher priority.  3x900 rows over 6000 tokens, 32 / 8 heads of 128: 240 us; 262 with one priority,
// 278 with the groups in step, 315 with waves 2 i and 2 i + 1 apart, which share no SIMD.  Heads of 256
// (16 / 4; one tile of rows a wave) 264, 265, 265 and 379.  With phases counted over both groups, waves 0-3 do the weights of block i in phase 2 i and its products in 2 i + 1, waves
// 4-7 one later: keys of block j are read in phases 2 j - 1 and 2 j, values in 2 j + 1 and 2 j + 2.  In its
// product phase of block i a wave writes its part of the keys of block i + 2 and of the values of block
// i + 1: two buffers each are enough, and four places for the page scales (read in phases 2 j - 1 to
// 2 j + 1, written in 2 j - 3 and 2 j - 2).
template <int DT>
constexpr size_t many_rows_lds_bytes() {
  return size_t(DT / 8) * 2048 * 2 + 4 * 64;
}

template <typename TIn, int DT, int RT>
__global__ __launch_bounds__(512) void many_rows_kernel(AttentionArgs a, Kv8Batch batch, Kv8Cache cache) {
  constexpr int kWaveRows = RT * 16, kRows = 8 * kWaveRows;
  constexpr int kPieces = DT / 64, kTilesD = DT / 16, kQStride = DT + 8;
  constexpr int kHalf = 4 * kPieces * 2048;            // the keys, or the values, of a block
  constexpr int kMine = (4 * kPieces + 7) / 8;         // 2 KB jobs of a wave in each half
  extern __shared__ __align__(16) uint8_t lds[];       // many_rows_lds_bytes
  uint8_t* const key_lds = lds;
  uint8_t* const value_lds = lds + 2 * kHalf;
  float* const scale_lds = reinterpret_cast<float*>(lds + 4 * kHalf);
  static_assert(4 * kPieces == kTilesD, "as many key tiles as value tiles");
  static_assert(kWaveRows * kQStride * 2 * 4 <= 4 * kHalf, "the queries of half the waves fit the buffers");
  __shared__ float factor[kRows];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, c = lane >> 4;
  const Work w = work_of(a, batch, cache);
  const int G = a.Hq / cache.H;

  for (int64_t rb = w.rb; rb * kRows < w.rows; rb += a.row_blocks) {
    const int64_t r0 = rb * kRows + wave * kWaveRows;
    half8 q[RT][kPieces][2];
    float row_scale[RT], m[RT], l[RT];
    int sees[RT];
    float4_t o[kTilesD][RT] = {};
    // the queries go through LDS in the buffers' place, four waves at a time
    for (int turn = 0; turn < 2; ++turn) {
      __syncthreads();
      if ((wave >> 2) == turn) {
        _Float16* const q_lds = reinterpret_cast<_Float16*>(lds) + (wave & 3) * kWaveRows * kQStride;
        for (int i = c; i < kWaveRows; i += 4)
          stage_query<TIn, DT>(a, cache, w, r0 + i, n, q_lds + i * kQStride, factor + wave * kWaveRows + i);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int p = 0; p < kPieces; ++p)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              q[rt][p][k] = *reinterpret_cast<const half8*>(&q_lds[(rt * 16 + n) * kQStride + 64 * p + 16 * c + 8 * k]);
      }
    }
    __syncthreads();
    const bool active = r0 < w.rows;                               // the wave has rows
    // tokens that any row of the workgroup sees, in blocks of 64; this split's share of them
    const int64_t limit = min(w.len, w.before + (min(rb * kRows + kRows, w.rows) - 1) / G + 1);
    const int64_t blocks = limit > 0 ? (limit + 63) / 64 : 0;
    const int64_t per = (blocks + a.splits - 1) / a.splits;
    const int64_t from = w.split * per;
    const int count = int(max(min(per, blocks - from), int64_t(0)));
    // from here on tokens count from the share's first
    const int rel_limit = from_here(limit, from * 64);
    const int all_see = from_here(w.before + r0 / G, from * 64);   // every row of the wave sees the tokens up to it
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int64_t r = r0 + rt * 16 + n;
      row_scale[rt] = factor[wave * kWaveRows + rt * 16 + n];
      sees[rt] = r < w.rows ? from_here(w.before + r / G, from * 64) : -1;
      m[rt] = kNothing;
      l[rt] = 0.0f;
    }

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
      const int32_t k0 = pages.find(base0, off_k), v0 = pages.find(base0, off_v);
      const int32_t k1 = pages.find(base0 + 64, off_k), v1 = pages.find(base0 + 64, off_v);
      const int32_t k2 = pages.find(base0 + 128, off_k), v2 = pages.find(base0 + 128, off_v);
      load_keys(base0, k0);
      load_values(base0, v0);
      raw_page = scale_of(pages, v0, base0, off_v);
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
          // heads of 256: 69 ms so, 264 us in two loops)
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
      const int64_t row = (w.seq.row0 + r / G) * a.Hq + w.h * G + r % G;
      if (a.partial != nullptr && c == 0) a.stats[w.split * a.rows + row] = make_float2(m[rt], l[rt]);
      const float over_l = l[rt] == 0.0f ? 0.0f : 1.0f / l[rt];
#pragma unroll
      for (int dt = 0; dt < kTilesD; ++dt) {
        const int d = 16 * dt + 4 * c;
        if (d < cache.D) put(a, cache.D, w.split, row, d, o[dt][rt], over_l);
      }
    }
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

template <typename TIn>
hipError_t run_append(const KvRows& rows, const Kv8Batch& b, const Kv8Cache& c, int g, dim3 grid,
                      hipStream_t stream) {
  auto kernel = c.page == 16 ? append_kernel<TIn, 1> : c.page == 32 ? append_kernel<TIn, 2>
                : c.page == 64 ? append_kernel<TIn, 4> : append_kernel<TIn, 8>;
  return launch_kernel(kernel, grid, dim3(kThreads), size_t(c.D) * (c.page + 16), stream, rows, b, c,
                       digits_of(g));
}

// Pages that max_new tokens can reach, at most 65535 (the kernels loop over what is left).
unsigned page_slots(int64_t max_new, int page) {
  return unsigned(std::min<int64_t>(ceil_div(std::max<int64_t>(max_new, 1) - 1, page) + 1, 65535));
}

template <typename Kernel>
hipError_t run_kernel(Kernel* kernel, int64_t groups, int threads, size_t lds, const AttentionArgs& a,
                      const Kv8Batch& b, const Kv8Cache& c, hipStream_t stream) {
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
    if (e != hipSuccess) return e;
  }
  return launch_kernel(kernel, dim3(unsigned(groups)), dim3(threads), lds, stream, a, b, c);
}

template <typename TIn, int DT>
hipError_t run_attention(const AttentionArgs& a, const Kv8Batch& b, const Kv8Cache& c, const Kv8Plan& p,
                         hipStream_t stream) {
  constexpr int RT = DT == 256 ? 1 : 2;
  const int64_t groups = b.B * c.H * p.row_blocks * p.splits;
  constexpr size_t kFew = few_rows_lds_bytes<DT>();
  if (p.row_tiles == 1) return run_kernel(few_rows_kernel<TIn, DT, 1>, groups, 256, kFew, a, b, c, stream);
  if (p.row_tiles == 2) return run_kernel(few_rows_kernel<TIn, DT, 2>, groups, 256, kFew, a, b, c, stream);
  if (p.row_tiles == 4) return run_kernel(few_rows_kernel<TIn, DT, 4>, groups, 256, kFew, a, b, c, stream);
  return run_kernel(many_rows_kernel<TIn, DT, RT>, groups, 512, many_rows_lds_bytes<DT>(), a, b, c, stream);
}

template <typename TIn>
hipError_t run_attention(const AttentionArgs& a, const Kv8Batch& b, const Kv8Cache& c, const Kv8Plan& p,
                         hipStream_t stream) {
  if (c.D <= 64) return run_attention<TIn, 64>(a, b, c, p, stream);
  if (c.D <= 128) return run_attention<TIn, 128>(a, b, c, p, stream);
  return run_attention<TIn, 256>(a, b, c, p, stream);
}

bool wide_rows(const void* p, int64_t t, int64_t h, int dtype) {
  const int per = dtype == 0 ? 4 : 8;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && t % per == 0 && h % per == 0;
}

}  // namespace

hipError_t launch_kv8_append(const void* k, const void* v, int dtype, int64_t k_t, int64_t k_h, int64_t v_t,
                             int64_t v_h, const Kv8Batch& b, const Kv8Cache& c, int g, int64_t max_new,
                             hipStream_t stream) {
  const KvRows rows{k, v, k_t, k_h, v_t, v_h, wide_rows(k, k_t, k_h, dtype), wide_rows(v, v_t, v_h, dtype)};
  const dim3 grid(unsigned(2 * b.B * c.H), page_slots(max_new, c.page));
  return dtype == 0 ? run_append<float>(rows, b, c, g, grid, stream)
                    : run_append<uint16_t>(rows, b, c, g, grid, stream);
}

hipError_t launch_kv8_read(const Kv8Batch& b, const Kv8Cache& c, int g, int64_t max_new, uint16_t* k,
                           uint16_t* v, hipStream_t stream) {
  const dim3 grid(unsigned(2 * b.B * c.H), page_slots(max_new, c.page));
  auto kernel = c.page == 16 ? read_kernel<1> : c.page == 32 ? read_kernel<2>
                : c.page == 64 ? read_kernel<4> : read_kernel<8>;
  return launch_kernel(kernel, grid, dim3(kThreads), size_t(c.D) * (c.page + 16), stream, b, c, digits_of(g), k,
                       v);
}

Kv8Plan plan_kv8_attention(int64_t B, int64_t T, int64_t Hq, int64_t H, int64_t D, int64_t max_new,
                           int64_t max_len) {
  Kv8Plan p{};
  const int64_t rows = std::max<int64_t>(std::min(max_new, T), 1) * (Hq / H);
  const bool many = rows > 64;
  p.row_tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : !many ? 4 : D > 128 ? 8 : 16;
  p.row_blocks = ceil_div(rows, 16 * p.row_tiles);
  const int64_t groups = B * H * p.row_blocks;
  const int64_t blocks = std::max<int64_t>(1, ceil_div(max_len, 64));
  // Tokens are split where the groups alone do not fill the chip: into about the workgroups that it
  // holds at once (two a compute unit, one for heads of more than 128 or for many rows), since each
  // one costs some 5 us to start and to end, and joining costs another 4: 200000 tokens of 8 heads
  // take 86 us with 512 workgroups and 112 with 1536.  No split has fewer than 8 blocks of 64 tokens
  // (300 tokens of 16 heads: 7.4 us in one, 10.4 in two).
  const int64_t hold = many || D > 128 ? 256 : 512;
  const int64_t wish = many ? hold / groups : ceil_div(hold, groups);
  p.splits = int(std::min<int64_t>(std::max<int64_t>(1, wish), std::min<int64_t>(std::max<int64_t>(1, blocks / 8), 256)));
  if (p.splits > 1)
    p.bytes = round256(size_t(p.splits) * T * Hq * D * 4) + round256(size_t(p.splits) * T * Hq * 8);
  return p;
}

hipError_t launch_kv8_attention(const void* q, int dtype, int64_t q_t, int64_t q_h, int64_t Hq,
                                const Kv8Batch& b, const Kv8Cache& c, int g, float scale, const Kv8Plan& p,
                                uint16_t* out, void* workspace, hipStream_t stream) {
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
    a.stats = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) +
                                        round256(size_t(p.splits) * a.rows * c.D * 4));
  }
  const hipError_t e = dtype == 0 ? run_attention<float>(a, b, c, p, stream)
                                  : run_attention<uint16_t>(a, b, c, p, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  // a wave to a row; four where there are many splits
  if (p.splits <= 8)
    return launch_kernel(join_splits_kernel<1>, dim3(unsigned(ceil_div(a.rows, 4))), dim3(256), 0, stream, b,
                         int(Hq), c.D, p.splits, a.rows, a.partial, a.stats, out);
  return launch_kernel(join_splits_kernel<4>, dim3(unsigned(a.rows)), dim3(256), 0, stream, b, int(Hq), c.D,
                       p.splits, a.rows, a.partial, a.stats, out);
}

}  // namespace convrot
