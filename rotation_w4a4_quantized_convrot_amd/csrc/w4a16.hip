// The linear layer for few activation rows: 4-bit weights with one bf16 scale per group of sg
// values of a row, activations kept at 16 bits or more (convrot_w4a16_linear), and its offline
// weight path (convrot_quant_weight_g4).
//
//   y[m][n] = bf16( sum_j s[n][j] sum_{k in group j} q[n][k] xr[m][k]  +  bias[n] )
//
// xr = x rotated in windows of g by H_g / sqrt(g) (g = 0: x itself).
//
// The weights are the traffic: N K'/2 bytes of codes, each read once for every 64 rows.  The products run on
// v_mfma_f32_16x16x32_f16 with the codes exact in fp16 and the activations rounded to fp16
// after an exact power-of-two scaling per unit of 256 values (decode_device.h, half_range): a
// rounding of 2^-11 relative to each value, eight times finer than bf16's, where the output is
// rounded to bf16 (2^-8) anyway; all sums are fp32.
#include "decode_device.h"

#include <type_traits>

namespace convrot {
namespace {

constexpr int kUnit = 256;     // k values that share an activation factor; one 128-byte line of codes

// Sum order of the eight values of a dword in a matrix operand: nibbles i and i + 4 of a dword
// come out of one mask, so the activations are stored in this order.
__device__ __forceinline__ constexpr int order_of(int e) { return (e & 1) * 4 + e / 2; }

__device__ __forceinline__ half2_t as_half2(uint32_t u) { return __builtin_bit_cast(half2_t, u); }

// Eight two's complement codes to fp16, exactly.  1024 + (code + 8) is the fp16 with the biased
// nibble in its low mantissa bits; one nibble higher it is 1024 + 16 (code + 8).  Nine or ten
// VALU instructions for eight codes.
__device__ __forceinline__ half8 decode8(uint32_t q) {
  const half2_t off_lo = {(_Float16)1032.0f, (_Float16)1032.0f};
  const half2_t off_hi = {(_Float16)-72.0f, (_Float16)-72.0f};
  const half2_t sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
  const uint32_t r = q >> 8;
  const half2_t a = as_half2((q & 0x000F000Fu) ^ 0x64086408u) - off_lo;
  const half2_t b = __builtin_elementwise_fma(as_half2((q & 0x00F000F0u) ^ 0x64806480u), sixteenth, off_hi);
  const half2_t c = as_half2((r & 0x000F000Fu) ^ 0x64086408u) - off_lo;
  const half2_t d = __builtin_elementwise_fma(as_half2((r & 0x00F000F0u) ^ 0x64806480u), sixteenth, off_hi);
  return half8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Sixteen bytes of a lane (32 codes of one row: four dwords) against the three lanes 16, 32 and
// 48 further on: afterwards dword j of lane row c is what dword c of lane row j was, so that one
// matrix instruction covers 32 neighbouring codes and none spans two scale groups.
__device__ __forceinline__ void transpose4(uint4_t& w) {
  const auto p = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto q = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto a = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
  w = uint4_t{a[0], a[1], b[0], b[1]};
}

// Where 8 activations (row m, columns k .. k + 7, k a multiple of 8) stand in the operand
// layout: 1 KB blocks that a wave loads as they are, 16 bytes a lane.  Folded (M <= 8): rows
// 0-7 of the operand hold the first half of a unit, rows 8-15 the second.
template <bool FOLD>
__device__ __forceinline__ int64_t operand_at(int64_t m, int64_t k, int64_t units) {
  const int64_t u = k / kUnit;
  const int h = int(k / 128) & 1, j = int(k / 32) & 3, c = int(k / 8) & 3;
  if (FOLD) return ((u * 4 + j) * 64 + c * 16 + h * 8 + m) * 8;
  return ((((m / 16) * units + u) * 8 + h * 4 + j) * 64 + c * 16 + (m & 15)) * 8;
}

// Pads, rotates, scales and rounds the activations into the operand layout.  A wave takes 1024
// columns of a row, 16 to a lane.  5 x 4100: 3.7 us, 32 x 12288: 5.8 us; the launch and one trip to
// memory are most of it.
template <typename TIn, bool FOLD>
__global__ __launch_bounds__(256) void prepare_kernel(const TIn* __restrict__ x, int64_t M, int64_t K,
                                                      int64_t ldx, bool wide, int digits, int64_t units,
                                                      int64_t rows_padded, _Float16* __restrict__ op,
                                                      float* __restrict__ factor) {
  const int lane = threadIdx.x & 63;
  const int64_t spans = (units + 3) / 4;
  const int64_t job = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (job >= M * spans) return;
  const int64_t m = job / spans, k = (job - m * spans) * 1024 + lane * 16;
  float v[16];
  load16<TIn>(x + m * ldx + k, K - k, wide, v);
  float up, back;
  half_range(unit_max(abs_max16(v), digits), digits, &up, &back);
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] *= up;
  rotate16(v, digits);
  if (k >= units * kUnit) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    half8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (_Float16)v[8 * i + order_of(e)];
    *reinterpret_cast<half8*>(op + operand_at<FOLD>(m, k + 8 * i, units)) = o;
  }
  if ((lane & 15) == 0) factor[(k / kUnit) * rows_padded + m] = back;
}

struct Weights {
  const uint8_t* codes;    // [N][row_bytes]
  const uint16_t* scales;  // [N][groups], bf16
  int64_t N, row_bytes, groups;
};

// The codes of one load: 16 bytes at `byte` of a row; past the row's end (its activations are
// zero there) its first ones.
__device__ __forceinline__ uint4_t load_codes(const Weights& w, int64_t row, int64_t byte) {
  byte = byte < w.row_bytes ? byte : 0;
  return *reinterpret_cast<const uint4_t*>(w.codes + row * w.row_bytes + byte);
}

template <int GC>
__device__ __forceinline__ float load_scale(const Weights& w, int64_t row, int64_t chunk) {
  const int64_t j = min(chunk / GC, w.groups - 1);
  return bf16_to_f32(w.scales[row * w.groups + j]);
}

// acc[m-tile] += the products of one load (32 codes a lane, columns 128 * half ... of a unit)
// with the activation operand; GC matrix instructions share a scale.
template <int MB, int GC>
__device__ __forceinline__ void multiply(uint4_t codes, const float (&scale)[4 / GC],
                                         const half8 (&x)[MB][4], float4_t (&acc)[MB]) {
  transpose4(codes);
  half8 w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = decode8(codes[j]);
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
    for (int i = 0; i < 4 / GC; ++i) {
      float4_t part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = i * GC; j < (i + 1) * GC; ++j)
        part = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[mb][j], w[j], part, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[mb][r] = __builtin_fmaf(scale[i], part[r], acc[mb][r]);
    }
  }
}

constexpr int kWaves = 8;

// The end of a tile, behind a barrier: the waves' sums over their parts of K are added in wave order, then
// bias and rounding.
template <int ROWS, int COLS, int PARTS>
__device__ __forceinline__ void finish(const float (*red)[ROWS * COLS], int64_t m0, int64_t n0, int64_t M,
                                       int64_t N, const uint16_t* __restrict__ bias,
                                       uint16_t* __restrict__ y) {
  for (int i = threadIdx.x; i < ROWS * COLS; i += kWaves * 64) {
    const int64_t m = m0 + i / COLS, n = n0 + i % COLS;
    if (m >= M || n >= N) continue;
    float s = 0.0f;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) s += red[p][i];
    if (bias != nullptr) s += bf16_to_f32(bias[n]);
    y[m * N + n] = f32_to_bf16(s);
  }
}

// Scale groups as the kernels see them: GC loads' 32-code chunks share a scale; WHOLE: rows are whole
// loads of 128 codes (K' is a multiple of 128), so a load's scales are neighbours in one row.
template <int GC_, bool WHOLE_>
struct Groups {
  static constexpr int GC = GC_;
  static constexpr bool WHOLE = WHOLE_ || GC_ == 4;
};

// Eight or sixteen weight rows as a lane sees them: the first row's address is the wave's, the lane's row
// from there an offset of 32 bits (16 rows of at most 32 KB).  Rows past the last are the last one.
struct Rows {
  const uint8_t* codes;
  const uint16_t* scales;
  uint32_t row_codes, row_scales;     // offsets of the lane's row, in bytes and in scales

  __device__ __forceinline__ void set(const Weights& w, int64_t first, int lane_row) {
    const int64_t row = min(first, w.N - 1);
    codes = w.codes + row * w.row_bytes;
    scales = w.scales + row * w.groups;
    const uint32_t r = uint32_t(min(int64_t(lane_row), w.N - 1 - row));
    row_codes = r * uint32_t(w.row_bytes);
    row_scales = r * uint32_t(w.groups);
  }
};

// One load of a row: 16 bytes of codes (32 of them) at chunk + c, and the 4 / GC scales of the chunks
// chunk ... chunk + 3.  Past the row's end (the activations are zero there) its first ones.  Nothing is
// computed from what is loaded before it is used, and it stays where it was loaded to, so that
// nothing waits for loads that are on their way.
template <typename G>
struct Load {
  uint4_t codes;
  uint16_t scale[G::WHOLE && G::GC != 4 ? 1 : 4 / G::GC];      // raw bf16, or as loaded together:
  uint32_t pair[G::WHOLE && G::GC < 4 ? 2 / G::GC : 1];

  __device__ __forceinline__ void from(const Weights& w, const Rows& rows, int chunk, int c) {
    const uint32_t byte = uint32_t(chunk + c) * 16;
    codes = *reinterpret_cast<const uint4_t*>(rows.codes + (rows.row_codes + (byte < uint32_t(w.row_bytes) ? byte : 0u)));
    uint32_t j = uint32_t(chunk) / G::GC;
    if constexpr (G::WHOLE) {
      j = rows.row_scales + (j < uint32_t(w.groups) ? j : 0u);
      if constexpr (G::GC == 4) scale[0] = rows.scales[j];
      else __builtin_memcpy(pair, rows.scales + j, 8 / G::GC);
    } else {            // the row may end between them
#pragma unroll
      for (int i = 0; i < 4 / G::GC; ++i) scale[i] = rows.scales[rows.row_scales + min(j + i, uint32_t(w.groups - 1))];
    }
  }

  __device__ __forceinline__ void scales(float (&out)[4 / G::GC]) const {
#pragma unroll
    for (int i = 0; i < 4 / G::GC; ++i) {
      if constexpr (G::WHOLE && G::GC < 4)
        out[i] = __uint_as_float(i % 2 ? pair[i / 2] & 0xFFFF0000u : pair[i / 2] << 16);
      else
        out[i] = bf16_to_f32(scale[i]);
    }
  }
};

// The product for prepared activations.  A workgroup takes NT tiles of weight rows and 16 * MB
// (FOLD: 8) activation rows; its eight waves take parts of K, so that each weight line is read by
// one wave and the activation operand goes straight into registers.  FOLD, for M <= 8: a load
// covers 8 rows times a whole 128-byte line, columns 0-7 of the matrix instruction being the
// rows' first halves and columns 8-15 their second, against activation rows 0-7 and 8-15; the
// two quadrants where they meet are the result.
//
// 5 x 4100 to 4111 (fp32, groups of 32): 8.3 us, a load's way to memory for each of a wave's two units.
// 8192 to 28672: 16 rows 51.5 us, 32 rows 66, 64 rows 97, 512 rows 547 (activations included): nothing is asked
// for ahead of its use, every workgroup reads the whole operand (1 MB for 64 rows) from its L2, and
// from 65 rows on the weights are read and decoded again for every 64.
template <int MB, bool FOLD, int NT, int GC>
__global__ __launch_bounds__(kWaves * 64) void product_kernel(
    Weights w, const _Float16* __restrict__ op, const float* __restrict__ factor, int64_t rows_padded,
    int64_t M, int64_t units, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y) {
  constexpr int kHalves = FOLD ? 1 : 2;
  constexpr int kTile = FOLD ? 8 : 16, kRows = FOLD ? 8 : 16 * MB;
  __shared__ float red[FOLD ? 2 * kWaves : kWaves][kRows * kTile * NT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, c = lane >> 4;
  const int64_t n0 = int64_t(blockIdx.x) * (kTile * NT), m0 = int64_t(blockIdx.y) * kRows;
  const int64_t first = wave * units / kWaves, last = (wave + 1) * units / kWaves;

  float4_t acc[NT][MB] = {};
  int64_t row[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) row[t] = min(n0 + kTile * t + (FOLD ? n & 7 : n), w.N - 1);

  for (int64_t u = first; u < last; ++u) {
    uint4_t codes[NT][kHalves];
    float scale[NT][kHalves][4 / GC];
    half8 x[kHalves][MB][4];
    float4_t f[MB];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const int half = FOLD ? n >> 3 : h;
        codes[t][h] = load_codes(w, row[t], u * 128 + half * 64 + c * 16);
#pragma unroll
        for (int i = 0; i < 4 / GC; ++i)
          scale[t][h][i] = load_scale<GC>(w, row[t], u * 8 + half * 4 + i * GC);
      }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const int64_t tile = int64_t(blockIdx.y) * MB + mb;
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t block = FOLD ? u * 4 + j : (tile * units + u) * 8 + h * 4 + j;
          x[h][mb][j] = *reinterpret_cast<const half8*>(op + (block * 64 + lane) * 8);
        }
      f[mb] = *reinterpret_cast<const float4_t*>(factor + u * rows_padded +
                                                 (FOLD ? (4 * c) & 7 : m0 + 16 * mb + 4 * c));
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float4_t sum[MB] = {};
#pragma unroll
      for (int h = 0; h < kHalves; ++h) multiply<MB, GC>(codes[t][h], scale[t][h], x[h], sum);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t][mb][r] = __builtin_fmaf(f[mb][r], sum[mb][r], acc[t][mb][r]);
    }
  }

#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (FOLD) {
          if ((n >> 3) == (c >> 1))
            red[2 * wave + (n >> 3)][((4 * c + r) & 7) * (kTile * NT) + kTile * t + (n & 7)] = acc[t][mb][r];
        } else {
          red[wave][(16 * mb + 4 * c + r) * (kTile * NT) + kTile * t + n] = acc[t][mb][r];
        }
      }
  __syncthreads();
  finish<kRows, kTile * NT, FOLD ? 2 * kWaves : kWaves>(red, m0, n0, M, w.N, bias, y);
}

// The product for prepared activations where tiles of 32 weight rows are too few for the chip: one tile of
// 16, the waves' parts of K in steps of one load (128 columns), and what the next step needs asked for as
// soon as this one has used the same registers.  With the activations' launch, here and in product_kernel's
// tiles of 32, which leave half the compute units idle: 32 x 12288 to 4096 22.6 and 32.3 us, 16, 32 and 64 rows
// of 4096 to 4096 8.8 and 11.6, 10.4 and 14.6, 14.2 and 16.5.  Where there are enough of those the operand,
// read once a tile, decides instead: 16, 32 and 64 rows of 8192 to 28672 take 60.6, 82 and 126 us so, 55, 69
// and 100 in tiles of 32.
template <int MB, typename G>
__global__ __launch_bounds__(kWaves * 64, 2) void narrow_kernel(Weights w, const _Float16* __restrict__ op,
                                                                const float* __restrict__ factor,
                                                                int64_t rows_padded, int64_t M, int64_t units,
                                                                const uint16_t* __restrict__ bias,
                                                                uint16_t* __restrict__ y) {
  constexpr int kRows = 16 * MB;
  __shared__ float red[kWaves][kRows * 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, c = lane >> 4;
  const int64_t n0 = int64_t(blockIdx.x) * 16, m0 = int64_t(blockIdx.y) * kRows;
  const int steps = int(units) * 2, first = wave * steps / kWaves, last = (wave + 1) * steps / kWaves;

  float4_t acc[MB] = {};
  Rows rows;
  rows.set(w, n0, n);
  Load<G> weights;
  half8 x[MB][4];
  float4_t f[MB];
  const auto load_x = [&](int step) {
    const int64_t u = step / 2;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const int64_t tile = int64_t(blockIdx.y) * MB + mb;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t block = (tile * units + u) * 8 + (step & 1) * 4 + j;
        x[mb][j] = *reinterpret_cast<const half8*>(op + (block * 64 + lane) * 8);
      }
      f[mb] = *reinterpret_cast<const float4_t*>(factor + u * rows_padded + m0 + 16 * mb + 4 * c);
    }
  };
  const auto advance = [&](auto more, int step) {
    float scale[4 / G::GC];
    weights.scales(scale);
    float4_t sum[MB] = {};
    multiply<MB, G::GC>(weights.codes, scale, x, sum);
    if constexpr (decltype(more)::value) weights.from(w, rows, (step + 1) * 4, c);
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[mb][r] = __builtin_fmaf(f[mb][r], sum[mb][r], acc[mb][r]);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (decltype(more)::value) load_x(step + 1);
  };
  if (first < last) {
    weights.from(w, rows, first * 4, c);
    load_x(first);
    for (int step = first; step + 1 < last; ++step) advance(std::true_type{}, step);
    advance(std::false_type{}, last - 1);
  }

#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][(16 * mb + 4 * c + r) * 16 + n] = acc[mb][r];
  __syncthreads();
  finish<kRows, 16, kWaves>(red, m0, n0, M, w.N, bias, y);
}

// One launch for one or two rows of up to 64 units.  A wave takes U units of K of every tile that its
// workgroup goes through (8 NT weight rows, folded as above): it rotates its columns of the activations once,
// into LDS of its own (no barrier), with its first weights already on their way, and asks for a load of the
// next tile as soon as it has used the same one of this tile.  A row of 16 lanes rotates one unit of one
// activation row, four of them at a time (a window of 1024: the four units of one row).
//
// The weights' bytes bound it.  1 x 8192 to 28672 (121 MB): 28.5 us, 4.2 TB/s, where a plain read of as
// much reaches 5.5; 35.7 us with x rotated again for every tile (long_vector_kernel).  One workgroup a
// compute unit with 256 registers a lane: in an earlier form 35.9 us so and 40.7 with two workgroups of 128
// registers, which do not hold the loads.  1 x 4096 to 4096: 6.3 us; 1 x 1024 to 1024: 5.0 us, of which the
// launch is most.  Groups of 32 have four scales a load, and from K' = 4097 on their registers spill: 1 x 8192 to
// 28672 takes 38.5 us, 1 x 16384 to 4096 27.8 (groups of 128: 13.3).
template <int U>
__host__ __device__ constexpr size_t vector_lds_bytes(int M) {
  return size_t(kWaves) * M * U * (2 * 136 * 2 + 4);      // a unit's halves 16 bytes apart in the banks
}

template <typename TIn, int U, int NT, typename G>
__global__ __launch_bounds__(kWaves * 64, U >= 2 ? 2 : 4) void vector_kernel(
    Weights w, const TIn* __restrict__ x, int M, int64_t K, int64_t ldx, bool wide, int digits, int units,
    int tiles, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y) {
  constexpr int kStride = 2 * 136, kRows = 2, kSize = kRows * 8 * NT;
  extern __shared__ __align__(16) _Float16 lds[];         // vector_lds_bytes
  __shared__ float red[2][2 * kWaves][kSize];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, c = lane >> 4, half = n >> 3;
  // parts of K: whole units, whole windows of 1024 where there are such
  const int quads = (units + 3) / 4;
  const int first = digits >= 5 ? wave * quads / kWaves * 4 : wave * units / kWaves;
  const int last = digits >= 5 ? min((wave + 1) * quads / kWaves * 4, units) : (wave + 1) * units / kWaves;
  _Float16* const operand = lds + wave * M * U * kStride;
  float* const factor = reinterpret_cast<float*>(lds + kWaves * M * U * kStride) + wave * M * U;

  Load<G> weights[U][NT];
  Rows rows[NT];
  const auto rows_of = [&](int tile) {
#pragma unroll
    for (int t = 0; t < NT; ++t) rows[t].set(w, int64_t(tile) * (8 * NT) + 8 * t, n & 7);
  };
  // a unit that the wave does not have reads the row's first codes, against activations of zero
  const auto chunk_of = [&](int u) { return first + u < last ? (first + u) * 8 + half * 4 : 1 << 20; };
  rows_of(blockIdx.x);
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int t = 0; t < NT; ++t)
      weights[u][t].from(w, rows[t], chunk_of(u), c);

  // job j: unit j % kSpan of row j / kSpan; with windows of 1024 four jobs are one window
  constexpr int kSpan = U;
  for (int j0 = 0; j0 < M * kSpan; j0 += 4) {
    const int j = j0 + c, u = j % kSpan;
    const int m = min(j / kSpan, M - 1);
    const bool there = j < M * kSpan && first + u < last;
    const int64_t k = int64_t(first + u) * kUnit + n * 16;
    float v[16];
    load16<TIn>(x + m * ldx + (there ? k : 0), there ? K - k : 0, wide, v);
    const uint32_t bits = unit_max(abs_max16(v), digits);
    float up, back;
    half_range(bits, digits, &up, &back);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] *= up;
    rotate16(v, digits);
    if (j >= M * kSpan) continue;
    _Float16* const at = operand + (m * U + u) * kStride + (n >> 3) * 136 + (n & 7) * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      half8 o;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = (_Float16)v[8 * i + order_of(e)];
      *reinterpret_cast<half8*>(at + 8 * i) = o;
    }
    if (n == 0) factor[m * U + u] = back;
  }
  __builtin_amdgcn_wave_barrier();

  const int m = min(n & 7, M - 1);
  int buffer = 0;
  const auto advance = [&](auto more, int tile) {
    float4_t acc[NT] = {};
    if constexpr (decltype(more)::value) rows_of(tile + gridDim.x);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      half8 a[1][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a[0][j] = *reinterpret_cast<const half8*>(&operand[(m * U + u) * kStride + half * 136 + 32 * j + 8 * c]);
      float f[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) f[r] = factor[min((4 * c + r) & 7, M - 1) * U + u];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float scale[4 / G::GC];
        weights[u][t].scales(scale);
        float4_t sum[1] = {};
        multiply<1, G::GC>(weights[u][t].codes, scale, a, sum);
        if constexpr (decltype(more)::value)
          weights[u][t].from(w, rows[t], chunk_of(u), c);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t][r] = __builtin_fmaf(f[r], sum[0][r], acc[t][r]);
        __builtin_amdgcn_sched_barrier(0);      // one load's values at a time in registers
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int mr = (4 * c + r) & 7;
        if (half == (c >> 1) && mr < M) red[buffer][2 * wave + half][mr * (8 * NT) + 8 * t + (n & 7)] = acc[t][r];
      }
    lds_barrier();      // the next tile's weights stay on their way
    finish<kRows, 8 * NT, 2 * kWaves>(red[buffer], 0, int64_t(tile) * (8 * NT), M, w.N, bias, y);
    buffer ^= 1;        // the other one was read before this barrier
  };
  int tile = blockIdx.x;
  for (; tile + int(gridDim.x) < tiles; tile += gridDim.x) advance(std::true_type{}, tile);
  advance(std::false_type{}, tile);
}

// One launch for one or two rows that are longer: as above, but a wave goes through its part of K four
// units at a time, for one tile, so that x is rotated again for every tile.  1 x 28672 to 8192 (121 MB): 35 us,
// 3.4 TB/s.
template <typename TIn, int NT, int GC>
__global__ __launch_bounds__(kWaves * 64) void long_vector_kernel(
    Weights w, const TIn* __restrict__ x, int M, int64_t K, int64_t ldx, bool wide, int digits, int64_t units,
    const uint16_t* __restrict__ bias, uint16_t* __restrict__ y) {
  constexpr int kRows = 2, kPass = 4, kStride = 2 * 136;   // a unit's halves 16 bytes apart in the banks
  __shared__ float red[2 * kWaves][kRows * 8 * NT];
  __shared__ __align__(16) _Float16 operand[kWaves][kRows][kPass][kStride];
  __shared__ float factor[kWaves][kRows][kPass];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, c = lane >> 4, half = n >> 3;
  const int64_t n0 = int64_t(blockIdx.x) * (8 * NT);
  // parts of whole passes of four units, which a window of 1024 fills exactly
  const int64_t passes = (units + kPass - 1) / kPass;

  float4_t acc[NT] = {};
  int64_t row[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) row[t] = min(n0 + 8 * t + (n & 7), w.N - 1);

  for (int64_t p = wave; p < passes; p += kWaves) {
    uint4_t codes[kPass][NT];
    float scale[kPass][NT][4 / GC];
#pragma unroll
    for (int i = 0; i < kPass; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int64_t u = p * kPass + i;
        codes[i][t] = load_codes(w, row[t], u * 128 + half * 64 + c * 16);
#pragma unroll
        for (int s = 0; s < 4 / GC; ++s) scale[i][t][s] = load_scale<GC>(w, row[t], u * 8 + half * 4 + s * GC);
      }
    for (int m = 0; m < M; ++m) {
      const int64_t k = p * (kPass * kUnit) + lane * 16;
      float v[16];
      load16<TIn>(x + m * ldx + k, K - k, wide, v);
      float up, back;
      half_range(unit_max(abs_max16(v), digits), digits, &up, &back);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= up;
      rotate16(v, digits);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        half8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (_Float16)v[8 * i + order_of(e)];
        const int at = (lane & 15) * 16 + 8 * i;                     // column of the unit
        *reinterpret_cast<half8*>(&operand[wave][m][c][(at >> 7) * 136 + (at & 127)]) = o;
      }
      if (n == 0) factor[wave][m][c] = back;
    }
    __builtin_amdgcn_wave_barrier();
    const int m = min(n & 7, M - 1);
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      half8 a[1][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a[0][j] = *reinterpret_cast<const half8*>(&operand[wave][m][i][half * 136 + 32 * j + 8 * c]);
      float f[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) f[r] = factor[wave][min((4 * c + r) & 7, M - 1)][i];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float4_t sum[1] = {};
        multiply<1, GC>(codes[i][t], scale[i][t], a, sum);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t][r] = __builtin_fmaf(f[r], sum[0][r], acc[t][r]);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = (4 * c + r) & 7;
      if (half == (c >> 1) && m < kRows) red[2 * wave + half][m * (8 * NT) + 8 * t + (n & 7)] = acc[t][r];
    }
  __syncthreads();
  finish<kRows, 8 * NT, 2 * kWaves>(red, 0, n0, M, w.N, bias, y);
}

// Weights, offline: rotate, one scale bf16(max / 7) per group, codes clamp(rne(value / scale)).  The
// scale is rounded before the codes are taken, so that they are right for the scale that is kept.  28672 x 8192
// in bf16: 208 us, 2.8 TB/s, once for a model.
template <typename TIn>
__global__ __launch_bounds__(256) void quant_weight_kernel(const TIn* __restrict__ w, int64_t N, int64_t K,
                                                           bool wide, int digits, int64_t Kp, int sg,
                                                           uint8_t* __restrict__ codes,
                                                           uint16_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int64_t spans = (Kp + 1023) / 1024;
  const int64_t job = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (job >= N * spans) return;
  const int64_t n = job / spans, k = (job - n * spans) * 1024 + lane * 16;
  float v[16];
  load16<TIn>(w + n * K + k, K - k, wide, v);
  rotate16(v, digits);
  uint32_t bits = abs_max16(v);
  for (int o = 1; o < sg / 16; o <<= 1) bits = max(bits, uint32_t(__shfl_xor(int(bits), o)));
  const bool finite = bits < 0x7F800000u;
  const uint16_t s16 = finite ? f32_to_bf16(__fdiv_rn(__uint_as_float(bits), 7.0f)) : uint16_t(0x7FC0);
  const float s = bf16_to_f32(s16);
  uint32_t packed[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    int q = 0;
    if (s > 0.0f) q = int(fminf(fmaxf(rintf(__fdiv_rn(v[e], s)), -8.0f), 7.0f));
    packed[e >> 3] |= uint32_t(q & 15) << (4 * (e & 7));
  }
  if (k >= Kp) return;
  *reinterpret_cast<uint2_t*>(codes + n * (Kp / 2) + k / 2) = uint2_t{packed[0], packed[1]};
  if (lane % (sg / 16) == 0) scales[n * (Kp / sg) + k / sg] = s16;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Calls `run` with the Groups that a scale group of sg values and rows of row_bytes make.
template <typename Run>
hipError_t with_groups(const Weights& w, int sg, Run run) {
  const bool whole = w.row_bytes % 64 == 0;
  if (sg == 128) return run(Groups<4, true>{});
  if (sg == 64) return whole ? run(Groups<2, true>{}) : run(Groups<2, false>{});
  return whole ? run(Groups<1, true>{}) : run(Groups<1, false>{});
}

template <int MB>
hipError_t run_narrow(const Weights& w, int sg, const _Float16* op, const float* factor, const W4A16Plan& p,
                      int64_t M, const uint16_t* bias, uint16_t* y, hipStream_t stream) {
  const dim3 grid(unsigned(ceil_div(w.N, 16)), unsigned(ceil_div(M, 16 * MB)));
  return with_groups(w, sg, [&](auto groups) {
    return launch_kernel(narrow_kernel<MB, decltype(groups)>, grid, dim3(kWaves * 64), 0, stream, w, op, factor,
                         p.rows_padded, M, p.units, bias, y);
  });
}

template <int MB, bool FOLD, int NT>
hipError_t run_product(const Weights& w, int sg, const _Float16* op, const float* factor,
                       const W4A16Plan& p, int64_t M, const uint16_t* bias, uint16_t* y,
                       hipStream_t stream) {
  const int tile = (FOLD ? 8 : 16) * NT, rows = FOLD ? 8 : 16 * MB;
  const dim3 grid(unsigned(ceil_div(w.N, tile)), unsigned(ceil_div(M, rows)));
  auto kernel = sg == 32 ? product_kernel<MB, FOLD, NT, 1>
                : sg == 64 ? product_kernel<MB, FOLD, NT, 2> : product_kernel<MB, FOLD, NT, 4>;
  return launch_kernel(kernel, grid, dim3(kWaves * 64), 0, stream, w, op, factor, p.rows_padded, M, p.units,
                       bias, y);
}

template <typename TIn, int U, int NT>
hipError_t run_vector(const Weights& w, int sg, const TIn* x, int64_t M, int64_t K, int64_t ldx, bool wide,
                      int g, const W4A16Plan& p, const uint16_t* bias, uint16_t* y, hipStream_t stream) {
  const size_t lds = vector_lds_bytes<U>(int(M));
  // what the chip holds at once: one unit a wave leaves registers for two workgroups a compute unit
  const int64_t tiles = ceil_div(w.N, 8 * NT), hold = U >= 2 ? 256 : 512;
  return with_groups(w, sg, [&](auto groups) {
    const auto kernel = vector_kernel<TIn, U, NT, decltype(groups)>;
    if (lds > 65536) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
      if (e != hipSuccess) return e;
    }
    return launch_kernel(kernel, dim3(unsigned(tiles < hold ? tiles : hold)), dim3(kWaves * 64), lds, stream, w, x,
                         int(M), K, ldx, wide, digits_of(g), int(p.units), int(tiles), bias, y);
  });
}

template <typename TIn, int NT>
hipError_t run_long_vector(const Weights& w, int sg, const TIn* x, int64_t M, int64_t K, int64_t ldx, bool wide,
                           int g, const W4A16Plan& p, const uint16_t* bias, uint16_t* y, hipStream_t stream) {
  auto kernel = sg == 32 ? long_vector_kernel<TIn, NT, 1>
                : sg == 64 ? long_vector_kernel<TIn, NT, 2> : long_vector_kernel<TIn, NT, 4>;
  return launch_kernel(kernel, dim3(unsigned(ceil_div(w.N, 8 * NT))), dim3(kWaves * 64), 0, stream, w, x,
                       int(M), K, ldx, wide, digits_of(g), p.units, bias, y);
}

template <typename TIn>
hipError_t run_linear(const TIn* x, int64_t M, int64_t K, int64_t ldx, int g, int sg, const Weights& w,
                      const uint16_t* bias, uint16_t* y, const W4A16Plan& p, uint8_t* workspace,
                      hipStream_t stream) {
  const bool wide = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (ldx * sizeof(TIn)) % 16 == 0;
  if (p.vector_units == 1) return run_vector<TIn, 1, 2>(w, sg, x, M, K, ldx, wide, g, p, bias, y, stream);
  if (p.vector_units == 2) return run_vector<TIn, 2, 2>(w, sg, x, M, K, ldx, wide, g, p, bias, y, stream);
  if (p.vector_units == 4) return run_vector<TIn, 4, 2>(w, sg, x, M, K, ldx, wide, g, p, bias, y, stream);
  if (p.vector_units == 8) return run_vector<TIn, 8, 1>(w, sg, x, M, K, ldx, wide, g, p, bias, y, stream);
  if (p.rows_padded == 0) return run_long_vector<TIn, 2>(w, sg, x, M, K, ldx, wide, g, p, bias, y, stream);
  _Float16* op = reinterpret_cast<_Float16*>(workspace);
  float* factor = reinterpret_cast<float*>(workspace + p.operand_bytes);
  const bool fold = M <= 8;
  const int64_t jobs = M * ceil_div(p.units, 4);
  const hipError_t e = launch_kernel(fold ? prepare_kernel<TIn, true> : prepare_kernel<TIn, false>,
                               dim3(unsigned(ceil_div(jobs, 4))), dim3(256), 0, stream, x, M, K, ldx, wide,
                               digits_of(g), p.units, p.rows_padded, op, factor);
  if (e != hipSuccess) return e;
  if (fold) return run_product<1, true, 2>(w, sg, op, factor, p, M, bias, y, stream);
  // tiles of 32 weight rows once they make a workgroup for each of the 256 compute units
  if (ceil_div(w.N, 32) * ceil_div(M, 64) < 256) {
    if (M <= 16) return run_narrow<1>(w, sg, op, factor, p, M, bias, y, stream);
    if (M <= 32) return run_narrow<2>(w, sg, op, factor, p, M, bias, y, stream);
    return run_narrow<4>(w, sg, op, factor, p, M, bias, y, stream);
  }
  if (M <= 16) return run_product<1, false, 2>(w, sg, op, factor, p, M, bias, y, stream);
  if (M <= 32) return run_product<2, false, 2>(w, sg, op, factor, p, M, bias, y, stream);
  return run_product<4, false, 2>(w, sg, op, factor, p, M, bias, y, stream);
}

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

W4A16Plan plan_w4a16(int64_t M, int64_t Kp, int g) {
  W4A16Plan p{};
  p.units = ceil_div(Kp, kUnit);
  // One or two rows: a single launch, no workspace.  From three on the activations are prepared once, in a
  // launch of their own: 5 x 4100 to 4111 takes 12.4 us so, and 18.5 in the single launch, where every
  // workgroup rotates all five rows.
  if (M <= 2) {
    const int64_t most = g == 1024 ? ceil_div(p.units / 4, kWaves) * 4 : ceil_div(p.units, kWaves);
    p.vector_units = most <= 1 ? 1 : most <= 2 ? 2 : most <= 4 ? 4 : most <= 8 ? 8 : 0;
    return p;
  }
  p.rows_padded = M <= 8 ? 8 : M <= 16 ? 16 : M <= 32 ? 32 : ceil_div(M, 64) * 64;
  p.operand_bytes = round256(size_t(p.rows_padded) * p.units * kUnit * 2);
  p.factor_bytes = round256(size_t(p.rows_padded) * p.units * 4);
  return p;
}

hipError_t launch_w4a16_linear(const void* x, int x_dtype, int64_t M, int64_t K, int64_t ldx, int g, int sg,
                               int64_t Kp, const uint8_t* wq, const uint16_t* ws, int64_t N,
                               const uint16_t* bias, uint16_t* y, void* workspace, hipStream_t stream) {
  const W4A16Plan p = plan_w4a16(M, Kp, g);
  const Weights w{wq, ws, N, Kp / 2, Kp / sg};
  uint8_t* work = static_cast<uint8_t*>(workspace);
  if (x_dtype == 0)
    return run_linear(static_cast<const float*>(x), M, K, ldx, g, sg, w, bias, y, p, work, stream);
  return run_linear(static_cast<const uint16_t*>(x), M, K, ldx, g, sg, w, bias, y, p, work, stream);
}

hipError_t launch_quant_weight_g4(const void* w, int w_dtype, int64_t N, int64_t K, int g, int sg, int64_t Kp,
                                  uint8_t* wq, uint16_t* ws, hipStream_t stream) {
  const int64_t jobs = N * ceil_div(Kp, 1024);
  const dim3 grid(unsigned(ceil_div(jobs, 4)));
  const uintptr_t a = reinterpret_cast<uintptr_t>(w);
  if (w_dtype == 0)
    return launch_kernel(quant_weight_kernel<float>, grid, dim3(256), 0, stream, static_cast<const float*>(w),
                         N, K, a % 16 == 0 && K % 4 == 0, digits_of(g), Kp, sg, wq, ws);
  return launch_kernel(quant_weight_kernel<uint16_t>, grid, dim3(256), 0, stream,
                       static_cast<const uint16_t*>(w), N, K, a % 16 == 0 && K % 8 == 0, digits_of(g), Kp, sg,
                       wq, ws);
}

}  // namespace convrot
