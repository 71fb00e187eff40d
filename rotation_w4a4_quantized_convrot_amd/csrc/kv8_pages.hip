// The pages of the 8-bit cache moved about: drafted tokens that stay (convrot_kv8_keep) and whole pages
// (convrot_kv8_copy).
#include "kv8_device.h"

namespace convrot {
namespace {

constexpr int kThreads = 256;

// The length of a sequence's list, as far as this thread's entries tell: it ends at its first entry that does not name a
// later token than the one before it.
__device__ __forceinline__ bool list_ends(const int32_t at, const int32_t last, int64_t k, int64_t n) {
  return at <= (k > 0 ? max(last, -1) : -1) || at >= n;
}

__device__ __forceinline__ int list_length(const int32_t* __restrict__ list, int64_t n) {
  constexpr int kBatch = 4;
  int low = int(n);
  for (int64_t base = threadIdx.x; base < n; base += kBatch * kThreads) {
    int32_t at[kBatch], last[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t k = min(base + i * kThreads, n - 1);
      at[i] = list[k];
      last[i] = list[max(k - 1, int64_t(0))];
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t k = base + i * kThreads;
      if (k < n && list_ends(at[i], last[i], k, n)) low = min(low, int(k));
    }
  }
  return low;
}

// The smallest of a workgroup's values; everyone has to come here.
__device__ __forceinline__ int block_min(int v) {
  __shared__ int lowest[kThreads / 64];
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = min(v, __shfl_xor(v, o));
  if ((threadIdx.x & 63) == 0) lowest[threadIdx.x >> 6] = v;
  __syncthreads();
  return min(min(lowest[0], lowest[1]), min(lowest[2], lowest[3]));
}

// Few kept tokens move in one launch: a workgroup takes a (sequence, head, keys or values) and goes through the pages that
// receive tokens, first to last.  Tokens move towards the front only, so no page is read after it was written: a
// page's codes are gathered into registers, then, behind a barrier, written.  The scales and roundings are those of
// place_kernel.  Loads that wait for one another bound it: 48 sequences of 24 rows, 8 heads of 128, 10.4 us.
template <int ITER>
__global__ __launch_bounds__(kThreads) void keep_kernel(const int32_t* __restrict__ kept, Kv8Batch batch, Kv8Cache cache,
                                                        int32_t* __restrict__ lens_out) {
  constexpr int kPage = 16 * ITER;
  __shared__ int64_t from[kPage];           // where a slot's first code stands, -1: it has no page
  __shared__ float ratio[kPage];            // 1: the codes as they are
  __shared__ uint32_t shared_scale;
  const bool values = blockIdx.x & 1;
  const int64_t h = (blockIdx.x >> 1) % cache.H, b = (blockIdx.x >> 1) / cache.H;
  const Sequence seq = sequence_of(batch, b);
  const bool tells = !values && h == 0 && threadIdx.x == 0 && lens_out != nullptr;
  if (seq.n == 0 || seq.len < seq.n) {
    if (tells) lens_out[b] = int32_t(seq.len);
    return;
  }
  const int64_t before = seq.len - seq.n;
  const int32_t* const list = kept + seq.row0;
  const int64_t count = block_min(list_length(list, seq.n));
  if (tells) lens_out[b] = int32_t(before + count);
  if (count == 0) return;
  const int row = threadIdx.x >> 4, d = (threadIdx.x & 15) * 16, slot = threadIdx.x;
  float* const scales = values ? cache.vs : cache.ks;
  int8_t* const codes = values ? cache.vc : cache.kc;
  const int step = values ? 1 : cache.D;

  for (int64_t col = before / kPage; col <= (before + count - 1) / kPage; ++col) {
    const int64_t id = page_of(batch, cache, b, col);
    if (id < 0) continue;
    const int lo = int(max(before - col * kPage, int64_t(0)));
    const int hi = int(min(before + count - col * kPage, int64_t(kPage)));
    if (threadIdx.x == 0) shared_scale = 0;
    __syncthreads();
    int64_t src = id;
    int src_slot = slot;
    float scale = -1.0f;
    if (slot < hi) {
      if (slot >= lo) {
        const int64_t token = before + list[col * kPage + slot - before];
        src = page_of(batch, cache, b, token / kPage);
        src_slot = int(token % kPage);
      }
      if (src >= 0) {
        scale = scales[src * cache.H + h];
        atomicMax(&shared_scale, __float_as_uint(scale));      // scales are not negative; a NaN is above all
      }
    }
    __syncthreads();
    const float top = __uint_as_float(shared_scale);
    bool change = false;
    if (slot < kPage) {
      const bool again = !(scale < 0.0f) && scale != top && top == top;
      from[slot] = src < 0 ? -1 : (src * cache.H + h) * kPage * cache.D + src_slot * step;
      ratio[slot] = again ? __fdiv_rn(scale, top) : 1.0f;
      change = again || src != id || src_slot != slot;
    }
    if (!__syncthreads_or(change)) continue;
    uint4_t w[ITER];                        // D <= 256: at most ITER pieces of 16 codes a thread
    int8_t* const page = codes + (id * cache.H + h) * kPage * cache.D;
    if (!values) {
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int s = it * 16 + row;
        w[it] = uint4_t{0, 0, 0, 0};
        if (d < cache.D && s < hi && from[s] >= 0) w[it] = *reinterpret_cast<const uint4_t*>(codes + from[s] + d);
      }
      __syncthreads();
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int s = it * 16 + row;
        if (d >= cache.D || s >= hi) continue;
        if (ratio[s] != 1.0f) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[it][j] = rescale_codes(w[it][j], ratio[s]);
        }
        *reinterpret_cast<uint4_t*>(page + s * cache.D + d) = w[it];
      }
    } else {
      const int s0 = threadIdx.x % ITER * 16;
      int64_t at[16];
      float by[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) at[e] = from[s0 + e], by[e] = ratio[s0 + e];
#pragma unroll
      for (int n = 0; n < ITER; ++n) {
        const int channel = threadIdx.x / ITER + n * (kThreads / ITER);
        w[n] = uint4_t{0, 0, 0, 0};
        if (channel >= cache.D || s0 >= hi) continue;
        uint8_t code[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) code[e] = uint8_t(codes[max(at[e], int64_t(0)) + channel * kPage]);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float c = at[e] < 0 ? 0.0f : float(int8_t(code[e]));
          w[n][e >> 2] |= uint32_t(int(rintf(c * by[e])) & 255) << (8 * (e & 3));
        }
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < ITER; ++n) {
        const int channel = threadIdx.x / ITER + n * (kThreads / ITER);
        if (channel < cache.D && s0 < hi) *reinterpret_cast<uint4_t*>(page + channel * kPage + s0) = w[n];
      }
    }
    if (threadIdx.x == 0) scales[id * cache.H + h] = top;
    __syncthreads();                        // the slots' sources are written again
  }
}

// More of them move in two launches, so that every page of every sequence can be read and written by a workgroup of
// its own: the first one takes the tokens that stay, and their pages' scales, to the workspace, the second one puts
// them into their pages.
struct Staged {
  int32_t* count;     // [B]: tokens that stay
  float* scale[2];    // keys, values: [T][H], below 0: a token without a page
  int8_t* keys;       // [T][H][D]
  int8_t* values;     // [H][D][stride]: as in a page, 16 tokens of a channel in a row
  int64_t stride;
};

// A workgroup takes a page's share of the kept tokens of a (sequence, head, keys or values).  48 sequences of 24 rows, 8
// heads of 128: 8.2 us, then 6.4 to place them; 6 of up to 3000 rows of which half stay: 31 and 16 us, 140 in one launch.
template <int ITER>
__global__ __launch_bounds__(kThreads) void stage_kernel(const int32_t* __restrict__ kept, Kv8Batch batch, Kv8Cache cache,
                                                         Staged staged, int32_t* __restrict__ lens_out) {
  constexpr int kPage = 16 * ITER;
  __shared__ int64_t from[kPage];           // where a token's first code stands, -1: it has no page
  const bool values = blockIdx.x & 1;
  const int64_t h = (blockIdx.x >> 1) % cache.H, b = (blockIdx.x >> 1) / cache.H;
  const Sequence seq = sequence_of(batch, b);
  const bool tells = !values && h == 0 && threadIdx.x == 0 && blockIdx.y == 0;
  if (seq.n == 0 || seq.len < seq.n) {
    if (tells) {
      staged.count[b] = 0;
      if (lens_out != nullptr) lens_out[b] = int32_t(seq.len);
    }
    return;
  }
  const int64_t before = seq.len - seq.n;
  const int32_t* const list = kept + seq.row0;
  // workgroups whose own first entry ends the list are behind its end
  const int64_t first = int64_t(blockIdx.y) * kPage;
  if (first > 0 && (first >= seq.n || list_ends(list[first], list[first - 1], first, seq.n))) return;
  const int64_t count = block_min(list_length(list, seq.n));
  if (tells) {
    staged.count[b] = int32_t(count);
    if (lens_out != nullptr) lens_out[b] = int32_t(before + count);
  }
  const int8_t* const codes = values ? cache.vc : cache.kc;
  const float* const scales = values ? cache.vs : cache.ks;
  const int row = threadIdx.x >> 4, d = (threadIdx.x & 15) * 16, piece = threadIdx.x % ITER * 16;
  for (int64_t k0 = first; k0 < count; k0 += int64_t(gridDim.y) * kPage) {
    const int here = int(min(count - k0, int64_t(kPage)));
    const int64_t row0 = seq.row0 + k0;
    if (threadIdx.x < kPage) {
      from[threadIdx.x] = -1;
      if (threadIdx.x < here) {
        const int64_t token = before + list[k0 + threadIdx.x], id = page_of(batch, cache, b, token / kPage);
        if (id >= 0)
          from[threadIdx.x] = (id * cache.H + h) * kPage * cache.D + token % kPage * (values ? 1 : cache.D);
        staged.scale[values][(row0 + threadIdx.x) * cache.H + h] = id >= 0 ? scales[id * cache.H + h] : -1.0f;
      }
    }
    __syncthreads();
    if (!values) {
      uint4_t w[ITER];
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int64_t at = from[it * 16 + row];
        w[it] = uint4_t{0, 0, 0, 0};
        if (at >= 0 && d < cache.D) w[it] = *reinterpret_cast<const uint4_t*>(codes + at + d);
      }
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int s = it * 16 + row;
        if (s < here && d < cache.D)
          *reinterpret_cast<uint4_t*>(staged.keys + ((row0 + s) * cache.H + h) * cache.D + d) = w[it];
      }
    } else if (piece < here) {
      int64_t at[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) at[e] = from[piece + e];
      bool none[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) none[e] = at[e] < 0, at[e] = max(at[e], int64_t(0));
      for (int channel = threadIdx.x / ITER; channel < cache.D; channel += kThreads / ITER) {
        uint8_t code[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) code[e] = uint8_t(codes[at[e] + channel * kPage]);
#pragma unroll
        for (int e = 0; e < 16; ++e) code[e] = none[e] ? uint8_t(0) : code[e];
        int8_t* const to = staged.values + (h * cache.D + channel) * staged.stride + row0 + piece;
        if (piece + 16 <= here) {
          __builtin_memcpy(to, code, 16);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (piece + e < here) to[e] = int8_t(code[e]);
        }
      }
    }
    __syncthreads();                        // the sources are written again
  }
}

// A workgroup takes a page that receives tokens.  Its new scale is the largest of the pages' that they come from, and
// of its own if tokens stand before them; codes under another scale become rne(code * fp32(their scale / it)).
template <int ITER>
__global__ __launch_bounds__(kThreads) void place_kernel(Kv8Batch batch, Kv8Cache cache, Staged staged) {
  constexpr int kPage = 16 * ITER;
  __shared__ float ratio[kPage];            // of each slot, 1: the code as it is
  __shared__ uint32_t shared_scale;
  const bool values = blockIdx.x & 1;
  const int64_t h = (blockIdx.x >> 1) % cache.H, b = (blockIdx.x >> 1) / cache.H;
  const Sequence seq = sequence_of(batch, b);
  const int64_t count = staged.count[b];
  if (count == 0) return;
  const int64_t before = seq.len - seq.n;
  const int row = threadIdx.x >> 4, d = (threadIdx.x & 15) * 16, slot = threadIdx.x, piece = threadIdx.x % ITER * 16;
  for (int64_t col = before / kPage + blockIdx.y; col <= (before + count - 1) / kPage; col += gridDim.y) {
    const int64_t id = page_of(batch, cache, b, col);
    if (id < 0) continue;
    const int lo = int(max(before - col * kPage, int64_t(0)));
    const int hi = int(min(before + count - col * kPage, int64_t(kPage)));
    const int64_t row0 = seq.row0 + col * kPage - before;      // the workspace's row for slot 0
    float* const own = (values ? cache.vs : cache.ks) + id * cache.H + h;
    if (threadIdx.x == 0) shared_scale = 0;
    __syncthreads();
    float scale = -1.0f;
    if (slot < lo) scale = *own;
    else if (slot < hi) scale = staged.scale[values][(row0 + slot) * cache.H + h];
    // scales are not negative; a NaN is above all
    if (!(scale < 0.0f)) atomicMax(&shared_scale, __float_as_uint(scale));
    __syncthreads();
    const float top = __uint_as_float(shared_scale);
    if (slot < kPage) ratio[slot] = !(scale < 0.0f) && scale != top && top == top ? __fdiv_rn(scale, top) : 1.0f;
    __syncthreads();
    if (threadIdx.x == 0) *own = top;
    if (!values) {
      int8_t* const page = cache.kc + (id * cache.H + h) * kPage * cache.D;
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const int s = it * 16 + row;
        if (d >= cache.D || s >= hi || (s < lo && ratio[s] == 1.0f)) continue;
        uint4_t* const to = reinterpret_cast<uint4_t*>(page + s * cache.D + d);
        uint4_t w = s < lo ? *to : *reinterpret_cast<const uint4_t*>(staged.keys + ((row0 + s) * cache.H + h) * cache.D + d);
        if (ratio[s] != 1.0f) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = rescale_codes(w[j], ratio[s]);
        }
        *to = w;
      }
    } else if (piece < hi) {
      int8_t* const page = cache.vc + (id * cache.H + h) * kPage * cache.D;
      float by[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) by[e] = ratio[piece + e];
      for (int channel = threadIdx.x / ITER; channel < cache.D; channel += kThreads / ITER) {
        uint4_t* const to = reinterpret_cast<uint4_t*>(page + channel * kPage + piece);
        const int8_t* const in = staged.values + (h * cache.D + channel) * staged.stride + row0 + piece;
        uint32_t w[4];
        if (piece >= lo && piece + 16 <= hi) {
          __builtin_memcpy(w, in, 16);
        } else {
          const uint4_t was = *to;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const bool comes = piece + e >= lo && piece + e < hi;
            const uint32_t code = comes ? uint8_t(in[e]) : was[e >> 2] >> (8 * (e & 3)) & 255;
            w[e >> 2] = (e & 3) == 0 ? code : w[e >> 2] | code << (8 * (e & 3));
          }
        }
        uint4_t o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t r = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            r |= uint32_t(int(rintf(float(int8_t(w[j] >> (8 * e))) * by[4 * j + e])) & 255) << (8 * e);
          o[j] = r;
        }
        *to = o;
      }
    }
    __syncthreads();                        // the ratios are written again
  }
}

constexpr int kCopyBytes = kThreads * 16 * 4;     // of a workgroup

// A page's keys, and its values, of all heads are one run of bytes each.  Reading and writing them bounds it: 2500 pages
// of 64 tokens, 8 heads of 128 (655 MB): 127 to 137 us, 5.0 TB/s, as a large copy; 13 small pages 3.5 us, the launch.
__global__ __launch_bounds__(kThreads) void copy_kernel(const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
                                                        Kv8Cache cache) {
  const bool values = blockIdx.z;
  const int64_t from = src[blockIdx.x], to = dst[blockIdx.x];
  if (from < 0 || from >= cache.num_pages || to < 0 || to >= cache.num_pages || from == to) return;
  const int64_t bytes = int64_t(cache.H) * cache.page * cache.D;
  int8_t* const codes = values ? cache.vc : cache.kc;
  const int64_t part = int64_t(blockIdx.y) * kCopyBytes;
  const uint4_t* const in = reinterpret_cast<const uint4_t*>(codes + from * bytes + part);
  uint4_t* const out = reinterpret_cast<uint4_t*>(codes + to * bytes + part);
  const int64_t left = (bytes - part) / 16;
  uint4_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (threadIdx.x + i * kThreads < left) w[i] = in[threadIdx.x + i * kThreads];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (threadIdx.x + i * kThreads < left) out[threadIdx.x + i * kThreads] = w[i];
  if (blockIdx.y == 0) {
    float* const scales = values ? cache.vs : cache.ks;
    for (int h = threadIdx.x; h < cache.H; h += kThreads) scales[to * cache.H + h] = scales[from * cache.H + h];
  }
}

}  // namespace

namespace {

// The parts of the workspace, in their order; at: its start, or NULL for the size alone.
size_t stage(int64_t T, int64_t B, int64_t H, int64_t D, uint8_t* at, Staged* s) {
  size_t bytes = 0;
  const auto part = [&](size_t size) {
    uint8_t* const p = at + bytes;
    bytes += round256(size);
    return p;
  };
  s->stride = (T + 15) / 16 * 16;
  s->count = reinterpret_cast<int32_t*>(part(size_t(B) * 4));
  for (auto& scale : s->scale) scale = reinterpret_cast<float*>(part(size_t(T) * H * 4));
  s->keys = reinterpret_cast<int8_t*>(part(size_t(T) * H * D));
  s->values = reinterpret_cast<int8_t*>(part(size_t(s->stride) * H * D));
  return bytes;
}

}  // namespace

size_t kv8_keep_bytes(int64_t T, int64_t B, int64_t H, int64_t D) {
  Staged s;
  return stage(T, B, H, D, nullptr, &s);
}

// Rows of a sequence up to which one launch does it (page 64, 8 heads of 128; one launch, the two): 4 sequences of 64 rows
// 11.7 us, 6.7 + 7.8; of 128 rows 17.3, 7.3 + 7.9; of 256 rows 18.4, 7.0 + 7.8; 48 sequences of 64 rows 17.3, 14.1 +
// 10.1; of 256 rows 29.3, 25.0 + 16.3.  A launch costs the host about 2.5 us.
constexpr int kFewKept = 128;

hipError_t launch_kv8_keep(const int32_t* kept, const Kv8Batch& b, const Kv8Cache& c, int64_t max_new, int32_t* lens_out,
                           void* workspace, hipStream_t stream) {
  if (max_new <= kFewKept) {
    auto kernel = c.page == 16 ? keep_kernel<1> : c.page == 32 ? keep_kernel<2>
                  : c.page == 64 ? keep_kernel<4> : keep_kernel<8>;
    return launch_kernel(kernel, dim3(unsigned(2 * b.B * c.H)), dim3(kThreads), 0, stream, kept, b, c, lens_out);
  }
  Staged s;
  stage(b.T, b.B, c.H, c.D, static_cast<uint8_t*>(workspace), &s);
  const int64_t pages = std::min<int64_t>(ceil_div(std::max<int64_t>(max_new, 1), c.page), 65534);
  auto take = c.page == 16 ? stage_kernel<1> : c.page == 32 ? stage_kernel<2> : c.page == 64 ? stage_kernel<4> : stage_kernel<8>;
  auto put = c.page == 16 ? place_kernel<1> : c.page == 32 ? place_kernel<2> : c.page == 64 ? place_kernel<4> : place_kernel<8>;
  const hipError_t e = launch_kernel(take, dim3(unsigned(2 * b.B * c.H), unsigned(pages)), dim3(kThreads), 0, stream, kept,
                                     b, c, s, lens_out);
  if (e != hipSuccess) return e;
  return launch_kernel(put, dim3(unsigned(2 * b.B * c.H), unsigned(pages + 1)), dim3(kThreads), 0, stream, b, c, s);
}

hipError_t launch_kv8_copy(const int32_t* src, const int32_t* dst, int64_t n, const Kv8Cache& c, hipStream_t stream) {
  const int64_t parts = ceil_div(int64_t(c.H) * c.page * c.D, kCopyBytes);      // 2^15 for the largest page
  return launch_kernel(copy_kernel, dim3(unsigned(n), unsigned(parts), 2), dim3(kThreads), 0, stream, src, dst, c);
}

}  // namespace convrot
