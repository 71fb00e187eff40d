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

namespace convrot {
namespace {

// The least scale that is stored; pages whose values are all below 127 times this hold zeros.
// Attention divides by scales in fp32: 2^80 times a sum of 2^21 tokens' weights stays finite.
constexpr float kLeastScale = 8.271806125530277e-25f;   // 2^-80

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
// inverse).  The same workgroups as append; values go through LDS to stand by token again.
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
constexpr float kNothing = -1e30f;   // running maximum before the first token
constexpr float kLog2e = 1.4426950408889634f;

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

__device__ __forceinline__ float max_over_lane_rows(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum_over_lane_rows(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
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
  float2* stats;                  // [splits][rows]: running maximum and sum
};

// One pass over the tokens with a running maximum.  With s_j = scale q.k_j in powers of two and
// page scale vs_j, the kept sums are relative to M = max(s_j + log2 vs_j):
//   w_j = 2^(s_j + log2 vs_j - M + 14),   O = sum w_j vcode_j,   l = sum w_j / vs_j,
// so that O / l is the answer, the page scale of the values costs nothing in P V, and w_j rounded to
// fp16 uses that type's range from 2^14 down (a weight 2^-28 of the largest is still normal).
//
// Both products run on v_mfma_f32_16x16x32_f16 with the codes exact in fp16.  Scores are computed
// transposed, tokens x rows: a lane then holds one row's 16 tokens of the 16 that follow one
// another (lane row c: tokens 16 c ... of a block of 64), which is the layout the second product's
// operand needs, so the weights never leave the registers; the row statistics need two lane
// exchanges a block.  Rows are (query, head of the group) pairs of one cached head.
//
// SHARE (few rows): the four waves of a workgroup take every fourth block of tokens of the same
// RT * 16 rows and add up through LDS at the end.  Else each wave has RT * 16 rows of its own.
template <typename TIn, int DT, int RT, bool SHARE>
__global__ __launch_bounds__(256) void attention_kernel(AttentionArgs a, Kv8Batch batch, Kv8Cache cache) {
  constexpr int kRows = RT * 16, kQStride = DT + 8, kPieces = DT / 64, kTilesD = DT / 16;
  constexpr int kOStride = DT + 4;
  constexpr int kQBytes = (SHARE ? 1 : 4) * kRows * kQStride * 2;
  constexpr int kOBytes = SHARE ? kRows * kOStride * 4 : 0;
  __shared__ __align__(16) uint8_t lds[kQBytes > kOBytes ? kQBytes : kOBytes];
  __shared__ float row_factor[(SHARE ? 1 : 4) * kRows];
  __shared__ float wave_m[SHARE ? 4 : 1][kRows], wave_l[SHARE ? 4 : 1][kRows];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, c = lane >> 4;
  // the cached head varies fastest: with 8 of them each of the chip's 8 L2s sees one head
  int64_t id = blockIdx.x;
  const int64_t h = id % cache.H;
  id /= cache.H;
  const int split = int(id % a.splits);
  id /= a.splits;
  const int64_t rb_first = a.row_blocks - 1 - id % a.row_blocks, b = id / a.row_blocks;
  const Sequence seq = sequence_of(batch, b);
  const int G = a.Hq / cache.H;
  const int64_t rows = seq.n * G;
  const int64_t len = max(min(seq.len, batch.max_pages * cache.page), int64_t(0));
  const int64_t before = seq.len - seq.n;
  const int page_log = 31 - __clz(cache.page);
  const int64_t page_bytes = int64_t(cache.page) * cache.D;

  _Float16* const q_lds = reinterpret_cast<_Float16*>(lds) + (SHARE ? 0 : wave * kRows * kQStride);
  float* const factor = row_factor + (SHARE ? 0 : wave * kRows);

  for (int64_t rb = rb_first; rb * (SHARE ? kRows : 4 * kRows) < rows; rb += a.row_blocks) {
    const int64_t r0 = SHARE ? rb * kRows : (rb * 4 + wave) * kRows;
    if constexpr (SHARE) __syncthreads();
    // the queries: rotated, scaled into fp16's range, to LDS
    for (int i = (SHARE ? wave * 4 : 0) + c; i < kRows; i += SHARE ? 16 : 4) {
      const int64_t r = r0 + i;
      const bool there = r < rows && n * 16 < cache.D;
      const int64_t t = seq.row0 + (there ? r / G : 0), hq = h * G + (there ? r % G : 0);
      const TIn* p = static_cast<const TIn*>(a.q) + (there ? t * a.q_t + hq * a.q_h + n * 16 : 0);
      float v[16];
      load16<TIn>(p, there ? 16 : 0, a.q_wide, v);
      float up, back;
      half_range(row_max(abs_max16(v)), a.digits, &up, &back);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= up;
      rotate16(v, a.digits);
      if (n * 16 < DT) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          half8 o;
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = (_Float16)v[8 * k + e];
          *reinterpret_cast<half8*>(&q_lds[i * kQStride + n * 16 + 8 * k]) = o;
        }
      }
      if (n == 0) factor[i] = back * a.scale * kLog2e;
    }
    if constexpr (SHARE) __syncthreads();
    else __builtin_amdgcn_wave_barrier();

    half8 q[RT == 1 ? kPieces : 1][2];
    if constexpr (RT == 1) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          q[p][k] = *reinterpret_cast<const half8*>(&q_lds[n * kQStride + 64 * p + 16 * c + 8 * k]);
    }
    float row_scale[RT], m[RT], l[RT];
    int64_t sees[RT];               // last token that the lane's row may see
    float4_t o[kTilesD][RT] = {};
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int64_t r = r0 + rt * 16 + n;
      row_scale[rt] = factor[rt * 16 + n];
      sees[rt] = r < rows ? before + r / G : int64_t(-1);
      m[rt] = kNothing;
      l[rt] = 0.0f;
    }
    // tokens that any of these rows sees, in blocks of 64; this split's share of them
    const int64_t r_last = min(r0 + kRows, rows) - 1;
    const int64_t limit = r0 < rows ? min(len, before + r_last / G + 1) : int64_t(0);
    const int64_t all_see = r0 < rows ? before + r0 / G : int64_t(-1);   // every row sees tokens up to it
    const int64_t blocks = limit > 0 ? (limit + 63) / 64 : 0;
    const int64_t per = (blocks + a.splits - 1) / a.splits;
    const int64_t from = split * per, to = min(from + per, blocks);

    for (int64_t blk = from + (SHARE ? wave : 0); blk < to; blk += SHARE ? 4 : 1) {
      const int64_t base = blk * 64;
      // pages: of the 16 tokens whose keys the lane loads (16 (n / 4) ...), and of those whose
      // values and scores it holds (16 c ...)
      const int64_t tk = base + 16 * (n >> 2), tv = base + 16 * c;
      const int64_t idk = tk < limit ? page_of(batch, cache, b, tk >> page_log) : -1;
      const int64_t idv = tv < limit ? page_of(batch, cache, b, tv >> page_log) : -1;
      const int64_t hk = max(idk, int64_t(0)) * cache.H + h, hv = max(idv, int64_t(0)) * cache.H + h;
      const int8_t* const kp = cache.kc + hk * page_bytes + ((tk & (cache.page - 1)) + (n & 3)) * cache.D;
      const int8_t* const vp = cache.vc + hv * page_bytes + (tv & (cache.page - 1));
      uint4_t kw[4][kPieces], vw[kTilesD];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const int d = 64 * p + 16 * c;
          kw[t][p] = *reinterpret_cast<const uint4_t*>(kp + 4 * t * cache.D + (d < cache.D ? d : 0));
        }
      const float ks = cache.ks[hv], vs = cache.vs[hv];     // of the scores the lane holds
#pragma unroll
      for (int dt = 0; dt < kTilesD; ++dt) {
        const int d = 16 * dt + n;
        vw[dt] = *reinterpret_cast<const uint4_t*>(vp + (d < cache.D ? d : 0) * cache.page);
      }

      float4_t s[4][RT];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) s[t][rt] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        half8 qf[RT][2];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if constexpr (RT == 1) qf[rt][k] = q[p][k];
            else qf[rt][k] = *reinterpret_cast<const half8*>(&q_lds[(rt * 16 + n) * kQStride + 64 * p + 16 * c + 8 * k]);
          }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const half8 k0 = decode_i8(kw[t][p][0], kw[t][p][1]), k1 = decode_i8(kw[t][p][2], kw[t][p][3]);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            s[t][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[rt][0], s[t][rt], 0, 0, 0);
            s[t][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qf[rt][1], s[t][rt], 0, 0, 0);
          }
        }
      }

      const float lv = vs == 0.0f ? 0.0f : __builtin_amdgcn_logf(vs);
      const float over_vs = __builtin_amdgcn_exp2f(-lv);
      const bool ragged = base + 63 > all_see || base + 64 > limit || __any(idv < 0);
      const bool no_values = __any(vs == 0.0f);
      half8 w0[RT], w1[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float mul = row_scale[rt] * ks;
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x = s[t][rt][i] * mul;
            if (ragged && (tv + 4 * t + i > sees[rt] || tv + 4 * t + i >= limit || idv < 0)) x = -INFINITY;
            s[t][rt][i] = x;
            top = fmaxf(top, x);
          }
        const float m_new = fmaxf(m[rt], max_over_lane_rows(top + lv));
        if (__any(m_new > m[rt])) {
          const float down = __builtin_amdgcn_exp2f(m[rt] - m_new);
          l[rt] *= down;
#pragma unroll
          for (int dt = 0; dt < kTilesD; ++dt) o[dt][rt] *= down;
          m[rt] = m_new;
        }
        const float add = lv - m[rt] + 14.0f;
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float w = __builtin_amdgcn_exp2f(s[t][rt][i] + add);
            if (ragged && s[t][rt][i] == -INFINITY) w = 0.0f;      // also where `add` is NaN
            s[t][rt][i] = w;
            sum += w;
          }
        l[rt] += sum == 0.0f ? 0.0f : sum * over_vs;
        w0[rt] = pack_half8(s[0][rt], s[1][rt]);
        w1[rt] = pack_half8(s[2][rt], s[3][rt]);
        if (no_values && vs == 0.0f) w0[rt] = w1[rt] = half8{};
      }
#pragma unroll
      for (int dt = 0; dt < kTilesD; ++dt) {
        const half8 v0 = decode_i8(vw[dt][0], vw[dt][1]), v1 = decode_i8(vw[dt][2], vw[dt][3]);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          o[dt][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w0[rt], o[dt][rt], 0, 0, 0);
          o[dt][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w1[rt], o[dt][rt], 0, 0, 0);
        }
      }
    }

#pragma unroll
    for (int rt = 0; rt < RT; ++rt) l[rt] = sum_over_lane_rows(l[rt]);

    if constexpr (SHARE) {
      // the four waves' sums, added in wave order
      if (c == 0) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          wave_m[wave][rt * 16 + n] = m[rt];
          wave_l[wave][rt * 16 + n] = l[rt];
        }
      }
      __syncthreads();
      float* const sums = reinterpret_cast<float*>(lds);
      for (int w = 0; w < 4; ++w) {
        if (wave == w) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const int r = rt * 16 + n;
            const float top = fmaxf(fmaxf(wave_m[0][r], wave_m[1][r]), fmaxf(wave_m[2][r], wave_m[3][r]));
            const float down = __builtin_amdgcn_exp2f(m[rt] - top);
#pragma unroll
            for (int dt = 0; dt < kTilesD; ++dt) {
              float4_t* const at = reinterpret_cast<float4_t*>(&sums[r * kOStride + 16 * dt + 4 * c]);
              float4_t v = w == 0 ? float4_t{0.0f, 0.0f, 0.0f, 0.0f} : *at;
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(o[dt][rt][i], down, v[i]);
              *at = v;
            }
          }
        }
        __syncthreads();
      }
      // a row of 16 lanes to a row: 16 values a lane
      for (int i = threadIdx.x >> 4; i < kRows; i += 16) {
        const int64_t r = r0 + i;
        const float top = fmaxf(fmaxf(wave_m[0][i], wave_m[1][i]), fmaxf(wave_m[2][i], wave_m[3][i]));
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) sum += wave_l[w][i] * __builtin_amdgcn_exp2f(wave_m[w][i] - top);
        if (r >= rows) continue;
        const int64_t row = (seq.row0 + r / G) * a.Hq + h * G + r % G;
        if (a.partial != nullptr && n == 0) a.stats[split * a.rows + row] = make_float2(top, sum);
        for (int d = n * 4; d < cache.D; d += 64) {
          float4_t v = *reinterpret_cast<const float4_t*>(&sums[i * kOStride + d]);
          if (a.partial != nullptr) {
            *reinterpret_cast<float4_t*>(a.partial + (split * a.rows + row) * cache.D + d) = v;
          } else {
            const float div = sum == 0.0f ? 0.0f : 1.0f / sum;
            uint2_t w;
            w[0] = uint32_t(f32_to_bf16(v[0] * div)) | (uint32_t(f32_to_bf16(v[1] * div)) << 16);
            w[1] = uint32_t(f32_to_bf16(v[2] * div)) | (uint32_t(f32_to_bf16(v[3] * div)) << 16);
            *reinterpret_cast<uint2_t*>(a.out + row * cache.D + d) = w;
          }
        }
      }
    } else {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int64_t r = r0 + rt * 16 + n;
        if (r >= rows) continue;
        const int64_t row = (seq.row0 + r / G) * a.Hq + h * G + r % G;
        if (a.partial != nullptr && c == 0) a.stats[split * a.rows + row] = make_float2(m[rt], l[rt]);
        const float div = l[rt] == 0.0f ? 0.0f : 1.0f / l[rt];
#pragma unroll
        for (int dt = 0; dt < kTilesD; ++dt) {
          const int d = 16 * dt + 4 * c;
          if (d >= cache.D) continue;
          const float4_t v = o[dt][rt];
          if (a.partial != nullptr) {
            *reinterpret_cast<float4_t*>(a.partial + (split * a.rows + row) * cache.D + d) = v;
          } else {
            uint2_t w;
            w[0] = uint32_t(f32_to_bf16(v[0] * div)) | (uint32_t(f32_to_bf16(v[1] * div)) << 16);
            w[1] = uint32_t(f32_to_bf16(v[2] * div)) | (uint32_t(f32_to_bf16(v[3] * div)) << 16);
            *reinterpret_cast<uint2_t*>(a.out + row * cache.D + d) = w;
          }
        }
      }
      __builtin_amdgcn_wave_barrier();   // the wave's queries are read before the next ones come
    }
  }
}

// Joins the splits of a row in their order: a wave to a row.
__global__ __launch_bounds__(256) void join_splits_kernel(Kv8Batch batch, int Hq, int D, int splits, int64_t rows,
                                                          const float* __restrict__ partial,
                                                          const float2* __restrict__ stats,
                                                          uint16_t* __restrict__ out) {
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int64_t t = row / Hq;
  if (t < batch.cu[0] || t >= batch.cu[batch.B]) return;      // a row of no sequence: left as it is
  float top = kNothing, sum = 0.0f;
  for (int s = 0; s < splits; ++s) top = fmaxf(top, stats[s * rows + row].x);
  for (int s = 0; s < splits; ++s) {
    const float2 st = stats[s * rows + row];
    sum += st.y * __builtin_amdgcn_exp2f(st.x - top);
  }
  const float div = sum == 0.0f ? 0.0f : 1.0f / sum;
  for (int d = (threadIdx.x & 63) * 4; d < D; d += 256) {
    float4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < splits; ++s) {
      const float2 st = stats[s * rows + row];
      if (st.y == 0.0f) continue;
      const float f = __builtin_amdgcn_exp2f(st.x - top);
      const float4_t p = *reinterpret_cast<const float4_t*>(partial + (s * rows + row) * D + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(p[i], f, v[i]);
    }
    uint2_t w;
    w[0] = uint32_t(f32_to_bf16(v[0] * div)) | (uint32_t(f32_to_bf16(v[1] * div)) << 16);
    w[1] = uint32_t(f32_to_bf16(v[2] * div)) | (uint32_t(f32_to_bf16(v[3] * div)) << 16);
    *reinterpret_cast<uint2_t*>(out + row * D + d) = w;
  }
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

template <typename TIn, int DT, int RT, bool SHARE>
hipError_t run_attention(const AttentionArgs& a, const Kv8Batch& b, const Kv8Cache& c, const Kv8Plan& p,
                         hipStream_t stream) {
  const int64_t groups = b.B * c.H * p.row_blocks * p.splits;
  return launch_kernel(attention_kernel<TIn, DT, RT, SHARE>, dim3(unsigned(groups)), dim3(256), 0, stream, a,
                       b, c);
}

template <typename TIn, int DT>
hipError_t run_attention(const AttentionArgs& a, const Kv8Batch& b, const Kv8Cache& c, const Kv8Plan& p,
                         hipStream_t stream) {
  constexpr int kMost = DT == 256 ? 2 : 4;
  if (!p.share) return run_attention<TIn, DT, kMost, false>(a, b, c, p, stream);
  if (p.row_tiles == 1) return run_attention<TIn, DT, 1, true>(a, b, c, p, stream);
  if (p.row_tiles == 2) return run_attention<TIn, DT, 2, true>(a, b, c, p, stream);
  return run_attention<TIn, DT, kMost, true>(a, b, c, p, stream);
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
  const int most = D > 128 ? 2 : 4;
  p.row_tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : most;
  p.share = rows <= 64 * most;      // up to four workgroups' rows: tokens over the waves
  p.row_blocks = ceil_div(rows, (p.share ? 16 : 64) * p.row_tiles);
  // about three workgroups a compute unit, each with at least four blocks of 64 tokens
  const int64_t groups = B * H * p.row_blocks;
  const int64_t most_splits = std::max<int64_t>(1, max_len / (p.share ? 256 : 512));
  p.splits = int(std::min<int64_t>(std::max<int64_t>(1, 768 / groups), std::min<int64_t>(most_splits, 256)));
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
  return launch_kernel(join_splits_kernel, dim3(unsigned(ceil_div(a.rows, 4))), dim3(256), 0, stream, b, int(Hq),
                       c.D, p.splits, a.rows, a.partial, a.stats, out);
}

}  // namespace convrot
