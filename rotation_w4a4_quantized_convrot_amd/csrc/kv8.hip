// The paged 8-bit key/value cache: append (convrot_kv8_append), read back (convrot_kv8_read) and
// attention (convrot_kv8_attention).
//
// A page holds `page` tokens of one sequence; for each page and head there are int8 codes and one
// fp32 scale for the keys and one for the values.  Keys [page][head][slot][D] are rotated in
// windows of g before they are quantized (their few large channels spread over the window) and
// queries are rotated alike: H_g / sqrt(g) is orthogonal, so the scores stay.  Values stand
// transposed, [page][head][D][slot]: 16 tokens of a channel are 16 bytes, what one lane feeds
// into the matrix instructions of P V.
#include "kv8_device.h"

namespace convrot {
namespace {

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
// inverse).  The same workgroups as append; values go through LDS to stand by token again, a thread taking 4 slots
// of 16 channels, 4 bytes at a time; blocks of 16 channels are 16 bytes further apart than their codes, so that the
// lanes of a wave read from banks of their own.  The six prompts above: 17 us (30 with a
// thread's 16 bytes from LDS one by one, for one token at a time, and without the conversion to bf16 by instruction),
// 2500 pages of 64 tokens of 8 heads of 128 (983 MB, written for the most part) 228 us; 48 x 1 rows from pages of 64 4.5 us,
// 5.5 where they are not treated apart.
template <int ITER>
__global__ __launch_bounds__(kThreads) void read_kernel(Kv8Batch batch, Kv8Cache cache, int digits,
                                                        uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  constexpr int kPage = 16 * ITER;
  extern __shared__ __align__(16) uint8_t tile[];
  const bool values = blockIdx.x & 1;
  const int64_t h = (blockIdx.x >> 1) % cache.H, b = (blockIdx.x >> 1) / cache.H;
  const Sequence seq = sequence_of(batch, b);
  if (seq.n == 0 || seq.len < seq.n) return;
  const int64_t before = seq.len - seq.n;
  const int row = threadIdx.x >> 4, d = (threadIdx.x & 15) * 16;
  uint16_t* const out = values ? v : k;
  const auto put = [&](const float (&x)[16], int64_t t) {
    typedef float float8 __attribute__((ext_vector_type(8)));
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    bf16x8* const at = reinterpret_cast<bf16x8*>(out + (t * cache.H + h) * cache.D + d);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float8 w;
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = x[8 * i + e];
      at[i] = __builtin_convertvector(w, bf16x8);      // to nearest even, two at once
    }
  };

  for (int64_t col = before / kPage + blockIdx.y; col <= (seq.len - 1) / kPage; col += gridDim.y) {
    const int64_t id = page_of(batch, cache, b, col);
    const int lo = int(max(before - col * kPage, int64_t(0)));
    const int hi = int(min(seq.len - col * kPage, int64_t(kPage)));
    const int64_t t0 = seq.row0 + col * kPage - before;        // the row of the page's first slot
    const float scale = id < 0 ? 0.0f : (values ? cache.vs : cache.ks)[id * cache.H + h];
    const int8_t* const page = (values ? cache.vc : cache.kc) + max(id, int64_t(0)) * cache.H * kPage * cache.D +
                               h * kPage * cache.D;
    const bool few = hi - lo <= 16;                              // a thread takes 16 channels of one token
    if (!values && few) {
      const int slot = lo + row;
      const bool here = slot < hi && d < cache.D;
      uint4_t w = {0, 0, 0, 0};
      if (here && id >= 0) w = *reinterpret_cast<const uint4_t*>(page + slot * cache.D + d);
      float x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = id < 0 ? 0.0f : float(int8_t(w[e >> 2] >> (8 * (e & 3)))) * scale;
      rotate16(x, digits);
      if (here) put(x, t0 + slot);
      continue;
    }
    if (!values) {
      uint4_t w[ITER];
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int slot = it * 16 + row;
        w[it] = uint4_t{0, 0, 0, 0};
        if (slot >= lo && slot < hi && d < cache.D && id >= 0)
          w[it] = *reinterpret_cast<const uint4_t*>(page + slot * cache.D + d);
      }
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int slot = it * 16 + row;
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = id < 0 ? 0.0f : float(int8_t(w[it][e >> 2] >> (8 * (e & 3)))) * scale;
        rotate16(x, digits);
        if (slot >= lo && slot < hi && d < cache.D) put(x, t0 + slot);
      }
      continue;
    }
    if (id >= 0) {
      for (int i = threadIdx.x; i < cache.D * ITER; i += kThreads) {
        const int channel = i / ITER, s = (i % ITER) * 16;
        if (s >= hi || s + 16 <= lo) continue;
        *reinterpret_cast<uint4_t*>(&tile[channel * kPage + (channel >> 4) * 16 + s]) =
            *reinterpret_cast<const uint4_t*>(page + channel * kPage + s);
      }
    }
    __syncthreads();
    if (few) {
      const int s = lo + row;
      if (s < hi && d < cache.D) {
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = id < 0 ? 0.0f : float(int8_t(tile[(d + e) * kPage + d + s])) * scale;
        put(x, t0 + s);
      }
      __syncthreads();
      continue;
    }
    for (int s = row * 4; s < kPage; s += 64) {
      if (d >= cache.D || s >= hi || s + 4 <= lo) continue;
      uint32_t w[16];                                          // 4 slots of each channel
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e] = *reinterpret_cast<const uint32_t*>(&tile[(d + e) * kPage + d + s]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = id < 0 ? 0.0f : float(int8_t(w[e] >> (8 * i))) * scale;
        if (s + i >= lo && s + i < hi) put(x, t0 + s + i);
      }
    }
    __syncthreads();
  }
}

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
  p.sums = p.splits * T * Hq;
  if (p.splits > 1) p.bytes = round256(size_t(p.sums) * D * 4) + round256(size_t(p.sums) * 8);
  // joining the splits takes up to a workgroup a row
  p.threads = std::max(groups * p.splits * (many ? 512 : 256), p.splits > 1 ? T * Hq * 256 : 0);
  return p;
}

hipError_t launch_kv8_attention(const void* q, int dtype, int64_t q_t, int64_t q_h, int64_t Hq,
                                const Kv8Batch& b, const Kv8Cache& c, int g, float scale, const Kv8Plan& p,
                                uint16_t* out, void* workspace, hipStream_t stream) {
  return attend(q, dtype, q_t, q_h, Hq, b, c, EarlierTokens{}, g, scale, p, out, workspace, stream);
}

}  // namespace convrot
