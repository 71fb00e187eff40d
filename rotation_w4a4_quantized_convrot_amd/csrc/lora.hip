// Low-rank adapters of many requests beside a shared projection (convrot_lora): for each row m with
// adapter l = ids[m],
//   out[m][n] = bf16( y[m][n] + scale[l] sum_j h[m][j] B[l][n][j] ),   h[m][j] = sum_k x[m][k] A[l][j][k].
//
// h first, in fp32, split over K into partial sums that the second launch adds up in their order.  Both
// products run on v_mfma_f32_16x16x32_bf16; A and B are bf16 already, fp32 operands (x where it is fp32, and h)
// enter as two bf16 pieces, the value cut off and its rest: 2^-16 relative, below 2^-133 an absolute 2^-134.  A
// row's sums do not depend on what the rows beside it hold, nor on its place in a tile; how they are split goes by M.
//
// Few rows: a workgroup to each row of a tile of 16, of which the first with its adapter goes on, for all rows
// of the tile that have it; operands go straight into registers.  Many rows: the rows are sorted by adapter
// first, and tiles of 64 rows with one adapter go through LDS.
#include "decode_device.h"

#include <algorithm>

namespace convrot {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t ushort8 __attribute__((ext_vector_type(8)));
typedef int16_t short8 __attribute__((ext_vector_type(8)));
typedef float float8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4;

// What lanes of a wave wrote to LDS is there for its other lanes.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A value cut off to bf16, and the rest in fp32; Inf and NaN have no rest.
__device__ __forceinline__ uint16_t cut(float v) {
  const uint32_t u = __float_as_uint(v);
  return uint16_t((u & 0x7FFFFFFFu) > 0x7F800000u ? 0x7FC0u : u >> 16);
}
__device__ __forceinline__ float rest(float v) {
  const uint32_t u = __float_as_uint(v);
  return (u & 0x7F800000u) == 0x7F800000u ? 0.0f : v - __uint_as_float(u & 0xFFFF0000u);
}

// What a second piece is multiplied with: the values, but the largest finite ones in the place of Inf and NaN.  The first
// piece makes the Inf or NaN of such a weight; a second piece of 0 would make a NaN of an Inf.  Its sign is the first one's, so
// that its product agrees with the Inf even where it overflows.
__device__ __forceinline__ bf16x8 finite(const bf16x8& v) {
  const ushort8 below = __builtin_elementwise_min(__builtin_bit_cast(ushort8, v), ushort8(0xFF7F));       // negative ones
  return __builtin_bit_cast(bf16x8, __builtin_elementwise_min(__builtin_bit_cast(short8, below), short8(0x7F7F)));
}

// Eight neighbouring elements as they stand in memory.  Rows need no alignment beyond their elements'.
template <typename T>
struct Raw {
  uint4_t w[sizeof(T) / 2];

  __device__ __forceinline__ void from(const T* p) { __builtin_memcpy(w, p, sizeof(w)); }
  // `left` of them are there, the others 0
  __device__ __forceinline__ void from(const T* p, int64_t left) {
    if (left >= 8) return from(p);
    T v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? p[e] : T(0);
    __builtin_memcpy(w, v, sizeof(w));
  }
};

// bf16( y + scale s ), eight at once.
__device__ __forceinline__ void add_scaled(uint16_t (&y)[8], const float (&s)[8], float scale) {
  float8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(scale, s[e], bf16_to_f32(y[e]));
  const bf16x8 o = __builtin_convertvector(v, bf16x8);
  __builtin_memcpy(y, &o, sizeof(o));
}

// Eight operand values: as they are, or in two pieces.
struct Operand {
  bf16x8 high, low;

  __device__ __forceinline__ explicit Operand(const Raw<uint16_t>& raw) : high(__builtin_bit_cast(bf16x8, raw.w[0])), low{} {}
  __device__ __forceinline__ explicit Operand(const float (&v)[8]) {
    ushort8 h;
    float8 l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[e] = cut(v[e]);
      l[e] = rest(v[e]);
    }
    high = __builtin_bit_cast(bf16x8, h);
    low = __builtin_convertvector(l, bf16x8);
  }
  __device__ __forceinline__ static Operand two(const Raw<float>& raw) {
    float v[8];
    __builtin_memcpy(v, raw.w, sizeof(v));
    return Operand(v);
  }
};
__device__ __forceinline__ Operand operand(const Raw<uint16_t>& raw) { return Operand(raw); }
__device__ __forceinline__ Operand operand(const Raw<float>& raw) { return Operand::two(raw); }

// The adapter of a row, -1: none.
__device__ __forceinline__ int adapter_of(const LoraArgs& a, int64_t m) {
  if (m >= a.M) return -2;                     // no row
  const int id = a.ids[m];
  return id >= 0 && id < a.L ? id : -1;
}

// The rows of a tile (lanes 0-15 hold their adapters) that have the adapter of row `lead`, if that is the first
// one with it; else none.
__device__ __forceinline__ uint32_t led_by(int id, int lead, int* adapter) {
  *adapter = __builtin_amdgcn_readlane(id, lead);
  const uint32_t rows = uint32_t(__ballot(id == *adapter)) & 0xFFFFu;
  return *adapter >= -1 && __builtin_ctz(rows) == lead ? rows : 0;
}

// h of rows of a tile of 16: ranks 16 RT z ... of split y.  The waves share the split's part of K and add up
// through LDS.  50 rows of 8192, r = 32, an adapter each (26 MB): 8.5 us; one row of 4096 2.0 to 3.0 us.
template <typename TIn, int RT>
__global__ __launch_bounds__(kWaves * 64) void few_shrink_kernel(LoraArgs a) {
  __shared__ float red[kWaves][16 * RT * 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, c = lane >> 4;
  const int64_t m0 = int64_t(blockIdx.x / 16) * 16;
  int adapter;
  const uint32_t rows = led_by(adapter_of(a, m0 + n), blockIdx.x % 16, &adapter);
  if (rows == 0 || adapter < 0) return;
  // this wave's part of K in steps of 64
  const int64_t steps = (a.K + 63) / 64, parts = int64_t(a.splits) * kWaves, part = int64_t(blockIdx.y) * kWaves + wave;
  const int64_t from = steps * part / parts, to = steps * (part + 1) / parts, whole = min(to, a.K / 64);
  const int r0 = blockIdx.z * RT * 16;
  // rows of other adapters repeat one of this one's; their sums are not used, nor those of ranks past the last
  const int64_t m = m0 + (rows >> n & 1 ? n : __builtin_ctz(rows));
  const TIn* const x = static_cast<const TIn*>(a.x) + m * a.ldx;
  const uint16_t* w[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
    w[rt] = a.a + (int64_t(adapter) * a.r + min(int64_t(r0 + rt * 16 + n), a.r - 1)) * a.K;
  float4_t sum[RT] = {};
  // a step's 64 columns, in any order: a lane holds 16 that follow one another
  struct Step {
    Raw<TIn> x[2];
    Raw<uint16_t> w[RT][2];
  };
  const auto load = [&](Step& s, int64_t step) {
    const int64_t k = step * 64 + 16 * c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s.x[i].from(x + k + 8 * i);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s.w[rt][i].from(w[rt] + k + 8 * i);
    }
  };
  const auto multiply = [&](const Step& s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Operand xs = operand(s.x[i]);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const Operand ws(s.w[rt][i]);
        sum[rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xs.high, ws.high, sum[rt], 0, 0, 0);
        if (sizeof(TIn) == 4) sum[rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xs.low, finite(ws.high), sum[rt], 0, 0, 0);
      }
    }
  };
  // the next step is on its way while one is multiplied
  if (from < whole) {
    Step one, two;
    load(one, from);
    int64_t step = from;
    for (; step + 1 < whole; step += 2) {
      load(two, step + 1);
      multiply(one);
      load(one, min(step + 2, whole - 1));
      multiply(two);
    }
    if (step < whole) multiply(one);
  }
  if (to > whole) {                                  // K's end within a step
    Step s;
    const int64_t k = whole * 64 + 16 * c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t at = min(k + 8 * i, a.K), there = a.K - at;
      s.x[i].from(x + at, there);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s.w[rt][i].from(w[rt] + at, there);
    }
    multiply(s);
  }
  float* const h = a.h + int64_t(blockIdx.y) * a.M * a.ranks;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][(4 * c + i) * (RT * 16) + rt * 16 + n] = sum[rt][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * RT * 16; i += kWaves * 64) {
    const int row = i / (RT * 16), j = r0 + i % (RT * 16);
    float s = 0.0f;
#pragma unroll
    for (int p = 0; p < kWaves; ++p) s += red[p][i];
    if ((rows >> row & 1) && j < a.ranks) h[(m0 + row) * a.ranks + j] = j < a.r ? s : 0.0f;
  }
}

// Rows of out, 64 columns a step.  The products are taken transposed (columns of out x rows), with
// the columns of a step dealt so that a lane ends up with 16 that follow one another of one row: column
// 16 c + 4 t + i stands in tile t, row 4 c + i.  KS * 32 ranks.  To 8192 columns for the 50 rows above: 10 to 12 us, the
// trips to memory for the adapter, then B and h, and four steps a wave; one step a wave 15, eight 13.
template <int KS>
__global__ __launch_bounds__(kWaves * 64) void few_expand_kernel(LoraArgs a, int col_steps) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, c = lane >> 4;
  const int64_t m0 = int64_t(blockIdx.y / 16) * 16;
  int adapter;
  const uint32_t rows = led_by(adapter_of(a, m0 + n), blockIdx.y % 16, &adapter);
  if (rows == 0 || (adapter < 0 && a.out == a.y)) return;
  const int64_t first = (int64_t(blockIdx.x) * kWaves + wave) * col_steps * 64;
  const bool mine = rows >> n & 1;
  const int64_t m = m0 + (mine ? n : __builtin_ctz(rows));
  const float scale = adapter >= 0 ? a.scale[adapter] : 0.0f;
  // what a step reads: rows of B, and 16 columns of y
  struct Step {
    Raw<uint16_t> b[4][KS], y[2];
  };
  const auto load = [&](Step& s, int64_t n0) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int64_t col = min(n0 + 16 * (n >> 2) + 4 * t + (n & 3), a.N - 1);
      const uint16_t* const b = a.b + (max(adapter, 0) * a.N + col) * a.r;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int64_t j = min(int64_t(32 * ks + 8 * c), a.r);
        s.b[t][ks].from(b + j, a.r - j);
      }
    }
    const int64_t col = min(n0 + 16 * c, a.N);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t at = min(col + 8 * i, a.N);
      s.y[i].from(a.y + m * a.ldy + at, a.N - at);
    }
  };
  const int64_t last = min(first + int64_t(col_steps) * 64, a.N);
  if (first >= last) return;
  Step one;
  load(one, first);
  // h of the rows: the splits' sums in their order
  float v[KS][8] = {};
  if (adapter >= 0) {
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
      const float* const row = a.h + (s * a.M + m) * a.ranks;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int j = 32 * ks + 8 * c;
        if (j >= a.ranks) continue;
        float part[8];
        __builtin_memcpy(part, __builtin_assume_aligned(row + j, 16), sizeof(part));
#pragma unroll
        for (int e = 0; e < 8; ++e) v[ks][e] += part[e];
      }
    }
  }
  const auto finish = [&](const Step& s, int64_t n0) {
    float4_t sum[4] = {};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Operand h(v[ks]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const Operand bs(s.b[t][ks]);
        sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bs.high, h.high, sum[t], 0, 0, 0);
        sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(finite(bs.high), h.low, sum[t], 0, 0, 0);
      }
    }
    const int64_t col = n0 + 16 * c, there = a.N - col;
    if (!mine || there <= 0) return;
    uint16_t* const out = a.out + m * a.ldo + col;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint16_t o[8];
      __builtin_memcpy(o, s.y[i].w, sizeof(o));
      if (adapter >= 0) {
        float eight[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) eight[e] = sum[2 * i + (e >> 2)][e & 3];
        add_scaled(o, eight, scale);
      }
      if (there >= 8 * i + 8) {
        __builtin_memcpy(out + 8 * i, o, sizeof(o));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (8 * i + e < there) out[8 * i + e] = o[e];
      }
    }
  };
  if constexpr (KS <= 2) {                             // the next step is on its way while one is finished
    Step two;
    for (int64_t n0 = first; n0 < last; n0 += 128) {
      if (n0 + 64 < last) load(two, n0 + 64);
      finish(one, n0);
      if (n0 + 64 >= last) break;
      if (n0 + 128 < last) load(one, n0 + 128);
      finish(two, n0 + 64);
    }
  } else {                                             // registers hold one
    for (int64_t n0 = first; n0 < last; n0 += 64) {
      if (n0 > first) load(one, n0);
      finish(one, n0);
    }
  }
}

// ------------------------------------------------------------------------------- many rows
constexpr int kTileRows = 64, kSortThreads = 1024;
constexpr int kSortGroups = 4096;      // adapters and the group without one whose counts fit the sort's LDS

// Sorts the rows by adapter, those without one last (left out where out is y), and cuts each adapter's rows into tiles
// of up to 64.  One workgroup; rows are placed by atomics, in no fixed order within an adapter, on which no result
// depends.  5000 rows of 6 adapters: 6.6 us, 100 rows 4.0; the launch and three trips to memory.
__global__ __launch_bounds__(kSortThreads) void sort_kernel(LoraArgs a) {
  __shared__ int lds[3 * kSortGroups];
  __shared__ int sums[2][kSortThreads / 64];
  const int groups = int(a.L) + 1, used = a.out == a.y ? groups - 1 : groups;
  int* const count = groups <= kSortGroups ? lds : a.scratch;
  int* const next = count + groups;            // where a group's next row goes
  int* const tile = next + groups;             // its first tile
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // the rows' groups, kBatch of a thread's rows at once
  constexpr int kBatch = 8;
  const auto every_row = [&](const auto& with) {
    for (int64_t base = threadIdx.x; base < a.M; base += kBatch * kSortThreads) {
      int id[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) id[i] = a.ids[min(base + i * kSortThreads, a.M - 1)];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (base + i * kSortThreads < a.M) with(base + i * kSortThreads, id[i] >= 0 && id[i] < a.L ? id[i] : groups - 1);
    }
  };
  // adds 1 to at[group] for every lane; a wave whose lanes have one group adds once
  const auto take = [&](int* at, int group) {
    const uint64_t here = __ballot(1);
    const int first = __builtin_amdgcn_readfirstlane(group);
    if (__ballot(group == first) != here) return atomicAdd(&at[group], 1);
    const int rank = __builtin_amdgcn_mbcnt_hi(uint32_t(here >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(here), 0));
    int base = 0;
    if (rank == 0) base = atomicAdd(&at[group], __builtin_popcountll(here));
    return __builtin_amdgcn_readfirstlane(base) + rank;
  };
  for (int g = threadIdx.x; g < groups; g += kSortThreads) count[g] = 0;
  __syncthreads();
  every_row([&](int64_t, int group) { take(count, group); });
  __syncthreads();
  // running sums of the rows and tiles; a thread takes neighbouring groups
  const int per = (used + kSortThreads - 1) / kSortThreads, from = min(int(threadIdx.x) * per, used), to = min(from + per, used);
  int rows = 0, tiles = 0;
  for (int g = from; g < to; ++g) {
    rows += count[g];
    tiles += (count[g] + kTileRows - 1) / kTileRows;
  }
  int rows_to = rows, tiles_to = tiles;        // up to this thread's
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int r = __shfl_up(rows_to, o), t = __shfl_up(tiles_to, o);
    if (lane >= o) {
      rows_to += r;
      tiles_to += t;
    }
  }
  if (lane == 63) {
    sums[0][wave] = rows_to;
    sums[1][wave] = tiles_to;
  }
  __syncthreads();
  int all = 0;
  for (int w = 0; w < kSortThreads / 64; ++w) {
    if (w < wave) {
      rows_to += sums[0][w];
      tiles_to += sums[1][w];
    }
    all += sums[1][w];
  }
  rows_to -= rows;
  tiles_to -= tiles;
  for (int g = from; g < to; ++g) {
    next[g] = rows_to;
    tile[g] = tiles_to;
    rows_to += count[g];
    tiles_to += (count[g] + kTileRows - 1) / kTileRows;
  }
  __syncthreads();
  for (int64_t t = threadIdx.x; t < a.max_tiles; t += kSortThreads) {
    LoraTile of{-1, 0, 0};
    if (t < all) {                             // the last group whose first tile is not behind t and that has rows
      int lo = 0, hi = used;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (tile[mid] <= t) lo = mid;
        else hi = mid;
      }
      const int done = (int(t) - tile[lo]) * kTileRows;
      of = LoraTile{lo < a.L ? lo : -1, next[lo] + done, min(count[lo] - done, kTileRows)};
    }
    a.tiles[t] = of;
  }
  __syncthreads();
  every_row([&](int64_t m, int group) {
    if (group < used) a.rows[take(next, group)] = int32_t(m);
  });
}

// h of a tile of 64 rows, by their place in the sorted order: ranks 16 RT z ... of split y.  Steps of 64 columns of x and A
// go through LDS, the next one on its way meanwhile; each wave takes 16 rows.  The columns are split until there are
// some 320 workgroups: 5000 x 4096, r = 64: 17 us (41 MB of x at 2.4 TB/s); with 768 15, but what follows then reads
// more partial sums and takes 6 us more; 24 with 160.  Operands straight from memory into registers, as for few rows:
// 48 us, since a load of 64 lanes touches 16 rows and the L1 cache takes the pieces one by one.  379 fp32 rows of 10058:
// 17 us (23 without the conversion to bf16 by instruction).
template <typename TIn, int RT>
__global__ __launch_bounds__(kWaves * 64) void many_shrink_kernel(LoraArgs a) {
  constexpr int kStride = 64 + 8, kRanks = RT * 16;
  constexpr int kPieces = sizeof(TIn) == 4 ? 2 : 1;                       // bf16 pieces of a value of x
  constexpr int kXs = kTileRows * 8 / (kWaves * 64), kAs = (kRanks * 8 + kWaves * 64 - 1) / (kWaves * 64);   // loads of a thread
  __shared__ __align__(16) uint16_t x_lds[2][kPieces][kTileRows * kStride];
  __shared__ __align__(16) uint16_t a_lds[2][kRanks * kStride];
  const LoraTile tile = a.tiles[blockIdx.x];
  if (tile.rows == 0 || tile.adapter < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, c = lane >> 4;
  const int64_t steps = (a.K + 63) / 64, from = steps * blockIdx.y / a.splits, to = steps * (blockIdx.y + 1) / a.splits;
  const int r0 = blockIdx.z * kRanks;
  // a thread's pieces of 8 columns: 8 of them a row; rows past the tile's last are its first one, ranks past r the last
  const int piece = threadIdx.x & 7, row = threadIdx.x >> 3;
  const TIn* x[kXs];
  const uint16_t* w[kAs];
#pragma unroll
  for (int i = 0; i < kXs; ++i) {
    const int r = row + i * (kWaves * 8);
    x[i] = static_cast<const TIn*>(a.x) + int64_t(a.rows[tile.first + (r < tile.rows ? r : 0)]) * a.ldx;
  }
#pragma unroll
  for (int i = 0; i < kAs; ++i)
    w[i] = a.a + (int64_t(tile.adapter) * a.r + min(int64_t(r0 + row + i * (kWaves * 8)), a.r - 1)) * a.K;
  Raw<TIn> xs[kXs];
  Raw<uint16_t> ws[kAs];
  const auto load = [&](int64_t step) {
    const int64_t k = min(step * 64 + piece * 8, a.K), there = a.K - k;
#pragma unroll
    for (int i = 0; i < kXs; ++i) xs[i].from(x[i] + k, there);
#pragma unroll
    for (int i = 0; i < kAs; ++i) ws[i].from(w[i] + k, there);
  };
  const auto put = [&](int buffer) {
#pragma unroll
    for (int i = 0; i < kXs; ++i) {
      const Operand o = operand(xs[i]);
      const int at = (row + i * (kWaves * 8)) * kStride + piece * 8;
      *reinterpret_cast<bf16x8*>(&x_lds[buffer][0][at]) = o.high;
      if (kPieces == 2) *reinterpret_cast<bf16x8*>(&x_lds[buffer][kPieces - 1][at]) = o.low;
    }
#pragma unroll
    for (int i = 0; i < kAs; ++i)
      if (row + i * (kWaves * 8) < kRanks)
        *reinterpret_cast<uint4_t*>(&a_lds[buffer][(row + i * (kWaves * 8)) * kStride + piece * 8]) = ws[i].w[0];
  };
  float4_t sum[RT] = {};
  if (from < to) load(from);
  for (int64_t step = from; step < to; ++step) {
    const int buffer = int(step - from) & 1;
    put(buffer);
    lds_barrier();                                     // a wave writes a buffer again two barriers later
    if (step + 1 < to) load(step + 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = 32 * i + 8 * c;
      bf16x8 v[kPieces];
#pragma unroll
      for (int p = 0; p < kPieces; ++p) v[p] = *reinterpret_cast<const bf16x8*>(&x_lds[buffer][p][(wave * 16 + n) * kStride + at]);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const bf16x8 u = *reinterpret_cast<const bf16x8*>(&a_lds[buffer][(rt * 16 + n) * kStride + at]);
#pragma unroll
        for (int p = 0; p < kPieces; ++p) sum[rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[p], p == 0 ? u : finite(u), sum[rt], 0, 0, 0);
      }
    }
  }
  float* const h = a.h + (int64_t(blockIdx.y) * a.M + tile.first) * a.ranks;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = wave * 16 + 4 * c + i, j = r0 + rt * 16 + n;
      if (r < tile.rows && j < a.ranks) h[r * a.ranks + j] = j < a.r ? sum[rt][i] : 0.0f;
    }
}

// Rows of out of a tile, 128 columns a step; KS * 32 ranks.  h of the tile is summed over the splits into LDS once and from
// there into each wave's registers (16 rows), rows of B go through LDS, the sums too, so that y and out are
// accessed in runs of 128 bytes; B of the next step, and y as soon as its registers are free, are on their way
// meanwhile.  5000 rows to 6144 columns, r = 64: 35 us (123 MB, 3.5 TB/s), to 6111 columns, whose rows start
// anywhere, 49; 62 and 77 with y asked for at the start of its step, 96 and 112 with lanes that access 16 columns of a
// row each.
template <int KS>
constexpr size_t many_expand_lds_bytes() {
  const size_t h = size_t(2) * kTileRows * (32 * KS + 8) * 2, b = size_t(128) * (32 * KS + 8) * 2 + kWaves * 16 * 68 * 4;
  return h > b ? h : b;
}

template <int KS>
__global__ __launch_bounds__(kWaves * 64) void many_expand_kernel(LoraArgs a, int col_steps) {
  constexpr int kStride = 32 * KS + 8, kCols = 128, kLoads = kCols * 4 * KS / (kWaves * 64);
  extern __shared__ __align__(16) uint16_t lds[];      // many_expand_lds_bytes
  uint16_t* const b_lds = lds;
  const LoraTile tile = a.tiles[blockIdx.x];
  if (tile.rows == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, c = lane >> 4;
  float* const sum_lds = reinterpret_cast<float*>(lds + kCols * kStride) + wave * 16 * 68;
  const int64_t first = int64_t(blockIdx.y) * col_steps * kCols, last = min(first + int64_t(col_steps) * kCols, a.N);
  // a lane's rows where y and out are accessed: 8 lanes to a row, 8 rows at a time
  const int piece = lane & 7;
  int64_t m[2];
  bool mine[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int r = wave * 16 + p * 8 + (lane >> 3);
    mine[p] = r < tile.rows;
    m[p] = a.rows[tile.first + (mine[p] ? r : 0)];
  }
  const auto finish = [&](const Raw<uint16_t>& y, const float* sums, float scale, int p, int64_t col) {
    if (!mine[p] || col >= a.N) return;
    uint16_t o[8];
    __builtin_memcpy(o, y.w, sizeof(o));
    if (sums != nullptr) {
      float s[8];
      __builtin_memcpy(s, __builtin_assume_aligned(sums, 16), sizeof(s));
      add_scaled(o, s, scale);
    }
    uint16_t* const out = a.out + m[p] * a.ldo + col;
    if (a.N - col >= 8) {
      __builtin_memcpy(out, o, sizeof(o));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e < a.N) out[e] = o[e];
    }
  };
  const auto load_y = [&](Raw<uint16_t>& y, int p, int64_t col) {
    const int64_t at = min(col, a.N);
    y.from(a.y + m[p] * a.ldy + at, a.N - at);
  };
  if (tile.adapter < 0) {                              // y as it is
    for (int64_t n0 = first; n0 < last; n0 += 64)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        Raw<uint16_t> y;
        load_y(y, p, n0 + 8 * piece);
        finish(y, nullptr, 0.0f, p, n0 + 8 * piece);
      }
    return;
  }
  const float scale = a.scale[tile.adapter];
  // rows of B: 4 KS pieces of 8 ranks each
  Raw<uint16_t> bs[kLoads];
  const auto load_b = [&](int64_t n0) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = threadIdx.x + i * (kWaves * 64);
      const int64_t col = min(n0 + at / (4 * KS), a.N - 1), j = min(int64_t(at % (4 * KS) * 8), a.r);
      bs[i].from(a.b + (int64_t(tile.adapter) * a.N + col) * a.r + j, a.r - j);
    }
  };
  load_b(first);
  // h: the splits' sums in their order, cut into two pieces
  for (int i = threadIdx.x; i < kTileRows * 4 * KS; i += kWaves * 64) {
    const int r = i / (4 * KS), j = i % (4 * KS) * 8;
    float v[8] = {};
    if (r < tile.rows && j < a.ranks) {
      const float* const h = a.h + (int64_t(tile.first) + r) * a.ranks + j;
#pragma unroll 4
      for (int s = 0; s < a.splits; ++s) {
        float part[8];
        __builtin_memcpy(part, __builtin_assume_aligned(h + s * a.M * a.ranks, 16), sizeof(part));
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += part[e];
      }
    }
    const Operand o(v);
    *reinterpret_cast<bf16x8*>(&lds[r * kStride + j]) = o.high;
    *reinterpret_cast<bf16x8*>(&lds[(kTileRows + r) * kStride + j]) = o.low;
  }
  __syncthreads();
  bf16x8 high[KS], low[KS];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    high[ks] = *reinterpret_cast<const bf16x8*>(&lds[(wave * 16 + n) * kStride + 32 * ks + 8 * c]);
    low[ks] = *reinterpret_cast<const bf16x8*>(&lds[(kTileRows + wave * 16 + n) * kStride + 32 * ks + 8 * c]);
  }
  __syncthreads();                                     // B takes h's place
  Raw<uint16_t> y[2][2];                               // of the next step as soon as this one's is used
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int p = 0; p < 2; ++p) load_y(y[half][p], p, first + 64 * half + 8 * piece);
  for (int64_t n0 = first; n0 < last; n0 += kCols) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = threadIdx.x + i * (kWaves * 64);
      *reinterpret_cast<uint4_t*>(&b_lds[at / (4 * KS) * kStride + at % (4 * KS) * 8]) = bs[i].w[0];
    }
    lds_barrier();
    if (n0 + kCols < last) load_b(n0 + kCols);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        float4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const bf16x8 b = *reinterpret_cast<const bf16x8*>(&b_lds[(64 * half + 16 * t + n) * kStride + 32 * ks + 8 * c]);
          sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, high[ks], sum, 0, 0, 0);
          sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(finite(b), low[ks], sum, 0, 0, 0);
        }
        *reinterpret_cast<float4_t*>(&sum_lds[n * 68 + 16 * t + 4 * c]) = sum;     // columns x rows: 4 columns of row n
      }
      wave_fence();
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int64_t col = n0 + 64 * half + 8 * piece;
        finish(y[half][p], &sum_lds[(p * 8 + (lane >> 3)) * 68 + 8 * piece], scale, p, col);
        if (n0 + kCols < last) load_y(y[half][p], p, col + kCols);
      }
      wave_fence();
    }
    lds_barrier();                                     // B is written again
  }
}

// Both ways, whole calls of 8192 -> 8192, r = 32: 100 rows of one adapter 26 us as few, 18 as many rows, of 64 adapters 26
// and 39; 256 rows 34 and 19, 42 and 40; 64 rows of one or 64 adapters 18 and 21 as few.  How many adapters the rows use is
// known to the device only; the rule takes them for few.
constexpr int64_t kFewRows = 64;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

template <typename TIn>
hipError_t run_shrink(const LoraArgs& a, bool few, hipStream_t stream) {
  const int rt = a.r <= 16 ? 1 : a.r <= 32 ? 2 : 4;
  const dim3 grid(unsigned(few ? ceil_div(a.M, 16) * 16 : a.max_tiles), unsigned(a.splits), unsigned(ceil_div(a.r, 16 * rt)));
  auto kernel = few ? (rt == 1 ? few_shrink_kernel<TIn, 1> : rt == 2 ? few_shrink_kernel<TIn, 2> : few_shrink_kernel<TIn, 4>)
                    : (rt == 1 ? many_shrink_kernel<TIn, 1> : rt == 2 ? many_shrink_kernel<TIn, 2> : many_shrink_kernel<TIn, 4>);
  return launch_kernel(kernel, grid, dim3(kWaves * 64), 0, stream, a);
}

hipError_t run_few_expand(const LoraArgs& a, hipStream_t stream) {
  const int steps = int(std::min<int64_t>(4, std::max<int64_t>(1, a.M * ceil_div(a.N, 64) / 1024)));
  const dim3 grid(unsigned(ceil_div(a.N, steps * 64 * kWaves)), unsigned(ceil_div(a.M, 16) * 16));
  auto kernel = a.r <= 32 ? few_expand_kernel<1> : a.r <= 64 ? few_expand_kernel<2>
                : a.r <= 128 ? few_expand_kernel<4> : few_expand_kernel<8>;
  return launch_kernel(kernel, grid, dim3(kWaves * 64), 0, stream, a, steps);
}

template <int KS>
hipError_t run_many_expand(const LoraArgs& a, hipStream_t stream) {
  constexpr size_t lds = many_expand_lds_bytes<KS>();
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(many_expand_kernel<KS>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
    if (e != hipSuccess) return e;
  }
  const int64_t tiles = ceil_div(a.M, kTileRows), steps = ceil_div(a.N, 128);
  const int64_t each = std::max<int64_t>(ceil_div(steps, 65535), std::min<int64_t>(8, std::max<int64_t>(1, tiles * steps / 512)));
  return launch_kernel(many_expand_kernel<KS>, dim3(unsigned(a.max_tiles), unsigned(ceil_div(steps, each))), dim3(kWaves * 64),
                       lds, stream, a, int(each));
}

// The parts of the workspace, in their order.
struct LoraSpace {
  size_t h, rows, tiles, scratch, bytes;
  int64_t ranks, max_tiles;
  int splits;
};

LoraSpace space_of(int64_t M, int64_t K, int64_t r, int64_t L) {
  LoraSpace s{};
  const bool few = M <= kFewRows;
  s.ranks = ceil_div(r, 16) * 16;
  // workgroups for every compute unit twice or more, in parts of at least 512 (256) columns
  const int64_t groups = few ? M : ceil_div(M, kTileRows);
  s.splits = int(std::max<int64_t>(1, std::min<int64_t>({ceil_div(few ? 512 : 320, groups), K / (few ? 512 : 256), 16})));
  s.max_tiles = few ? 0 : ceil_div(M, kTileRows) + std::min(L + 1, M);      // every adapter may have one that is not full
  s.rows = round256(size_t(s.splits) * M * s.ranks * 4);
  s.tiles = s.rows + (few ? 0 : round256(size_t(M) * 4));
  s.scratch = s.tiles + round256(size_t(s.max_tiles) * sizeof(LoraTile));
  s.bytes = s.scratch + (few || L + 1 <= kSortGroups ? 0 : round256(size_t(L + 1) * 12));
  return s;
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t r, int64_t L) { return space_of(M, K, r, L).bytes; }

hipError_t launch_lora(LoraArgs a, int x_dtype, void* workspace, hipStream_t stream) {
  const LoraSpace s = space_of(a.M, a.K, a.r, a.L);
  uint8_t* const base = static_cast<uint8_t*>(workspace);
  a.h = reinterpret_cast<float*>(base);
  a.rows = reinterpret_cast<int32_t*>(base + s.rows);
  a.tiles = reinterpret_cast<LoraTile*>(base + s.tiles);
  a.scratch = reinterpret_cast<int*>(base + s.scratch);
  a.ranks = s.ranks;
  a.max_tiles = s.max_tiles;
  a.splits = s.splits;
  const bool few = a.M <= kFewRows;
  hipError_t e = few ? hipSuccess : launch_kernel(sort_kernel, dim3(1), dim3(kSortThreads), 0, stream, a);
  if (e == hipSuccess) e = x_dtype == 0 ? run_shrink<float>(a, few, stream) : run_shrink<uint16_t>(a, few, stream);
  if (e != hipSuccess) return e;
  if (few) return run_few_expand(a, stream);
  return a.r <= 32 ? run_many_expand<1>(a, stream) : a.r <= 64 ? run_many_expand<2>(a, stream)
         : a.r <= 128 ? run_many_expand<4>(a, stream) : run_many_expand<8>(a, stream);
}

}  // namespace convrot
