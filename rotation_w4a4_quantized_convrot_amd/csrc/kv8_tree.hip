// Trees of drafted tokens behind the sequences of the 8-bit cache: who descends from whom
// (convrot_tree_masks) and the attention of their rows (convrot_kv8_tree_attention), which sees the tokens
// before them and those that a mask names.
#include "kv8_device.h"

namespace convrot {
namespace {

constexpr int kThreads = 256;
constexpr int kStaged = 4096;     // parents that a workgroup keeps in LDS
constexpr int kParts = 256;       // a workgroup of eight waves for every compute unit

// A thread takes a row and walks up to the context: parents come before their children, so the bits of a word of
// its mask are set one after another, from the row's own word down, and each word is written once.  Loads that wait for one
// another bound it, and the longest line of descent: one tree of 12 tokens 2.3 us, two of 300 5.3.
__global__ __launch_bounds__(kThreads) void tree_masks_kernel(const int32_t* __restrict__ parents, Kv8Batch batch,
                                                              int64_t words, uint64_t* __restrict__ mask,
                                                              int64_t* __restrict__ pos) {
  __shared__ int32_t staged[kStaged];
  const int64_t b = blockIdx.x;
  const Sequence seq = sequence_of(batch, b);
  const int64_t first = int64_t(blockIdx.y) * kThreads, step = int64_t(gridDim.y) * kThreads;
  if (first >= seq.n) return;
  const int32_t* const up = parents + seq.row0;
  const int near = int(min(seq.n, int64_t(kStaged)));
  for (int i = threadIdx.x; i < near; i += kThreads) staged[i] = up[i];
  __syncthreads();
  for (int64_t i = first + threadIdx.x; i < seq.n; i += step) {
    uint64_t* const line = mask + (seq.row0 + i) * words;
    int64_t word = i >> 6, depth = 0, j = i;
    for (int64_t w = words - 1; w > word; --w) line[w] = 0;
    uint64_t bits = 0;
    while (true) {
      for (; word > j >> 6; --word) {
        if (word < words) line[word] = bits;
        bits = 0;
      }
      bits |= uint64_t(1) << (j & 63);
      const int64_t parent = j < kStaged ? staged[j] : up[j];
      if (parent < 0 || parent >= j) break;                   // follows the context itself
      j = parent;
      ++depth;
    }
    for (; word >= 0; --word) {
      if (word < words) line[word] = bits;
      bits = 0;
    }
    pos[seq.row0 + i] = seq.len - seq.n + depth;
  }
}

// Many rows: as many workgroups as the chip holds share all the work there is.  A group is a block of rows of a
// sequence and cached head, with the sequence's tokens in blocks of 64; groups are cut into up to a.splits pieces.
// Few groups: pieces of up to `share` blocks, a workgroup to each.  Many: the groups stand in a row, each kStart units for
// what it costs to begin with it and one for each block, and a workgroup takes the next `share` units; where
// that ends within a group the next one goes on there, unless it would leave fewer than kLeast blocks on one side.
// A group that is not cut may be written as it is, with a mark for the join (writes_whole); else every piece leaves its sums in the
// workspace, and the last one of a group says so for the pieces that it does not have.  Where groups that are not cut are
// written, a workgroup has two slots for the sums of the others: 512 slots of 256 rows, 67 MB for heads of 128, whatever
// the number of rows (with sums for every row and piece, 100 trees of 64 with 32 heads of 128 took 420 MB).  The lengths
// are the device's, so each workgroup finds its part by going over the batch.
//
// Trees of 300 and 159 tokens over 20000 and 8545, 64 / 8 heads of 128: 340 us (720 TFLOP/s;
// with splits of the longest context, as for rows that see the tokens up to their own, about 630); 16 trees of up to 26 over up
// to 8000 tokens, 32 / 8 heads: 78 us, 12 of them to begin and 1.4 a block, which the eight waves' reading of its
// codes from LDS (0.85) bounds.
constexpr int kStart = 8, kLeast = 4, kShare = 8;

// A value that all lanes hold, as one of the wave.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return int64_t(uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(v)))) |
                 uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(v >> 32)))) << 32);
}

// The groups of a sequence and the blocks of tokens of each; none count as one.
struct Groups {
  int64_t count, blocks;
};
__device__ __forceinline__ Groups groups_of(const Kv8Batch& batch, const Kv8Cache& cache, int64_t b, int G, int rows_each) {
  const Sequence seq = sequence_of(batch, b);
  return Groups{(seq.n * G + rows_each - 1) / rows_each * cache.H,
                (max(min(seq.len, batch.max_pages * cache.page), int64_t(1)) + 63) / 64};
}

__device__ __forceinline__ int64_t wave_sum(int64_t v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ int64_t wave_top(int64_t v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = max(v, int64_t(__shfl_xor(v, o)));
  return v;
}

template <typename TIn, int DT, int RT>
__global__ __launch_bounds__(512) void many_rows_tree_kernel(AttentionArgs a, Kv8Batch batch, Kv8Cache cache, TreeTokens tree) {
  constexpr int kRows = 8 * RT * 16;
  __shared__ int64_t sums[3][8];
  __shared__ int64_t found[2];            // the sequence that the part starts in, and the units before it
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int G = a.Hq / cache.H;
  int64_t blocks = 0, groups = 0, longest = 0;
  for (int64_t b = threadIdx.x; b < batch.B; b += 512) {
    const Groups g = groups_of(batch, cache, b, G, kRows);
    blocks += g.count * g.blocks;
    groups += g.count;
    if (g.count > 0) longest = max(longest, g.blocks);
  }
  blocks = wave_sum(blocks);
  groups = wave_sum(groups);
  longest = wave_top(longest);
  if (lane == 0) {
    sums[0][wave] = blocks;
    sums[1][wave] = groups;
    sums[2][wave] = longest;
  }
  __syncthreads();
  blocks = groups = longest = 0;
  for (int i = 0; i < 8; ++i) {
    blocks += sums[0][i];
    groups += sums[1][i];
    longest = max(longest, sums[2][i]);
  }
  blocks = uniform(blocks), groups = uniform(groups), longest = uniform(longest);
  const int64_t parts = gridDim.x;
  if (groups == 0) return;
  // units for each workgroup if they stand in a row, within the pieces that the workspace has room for
  int64_t share = uniform(max(max((blocks + groups * kStart + parts - 1) / parts, min(longest + kStart, int64_t(2 * kStart))),
                              (longest + kStart + a.splits - 2) / (a.splits - 1)));
  // blocks for each if it takes one piece; these are no more than `parts` then
  const int64_t each = groups < parts ? uniform(max(max((blocks + parts - groups - 1) / (parts - groups), int64_t(kShare)),
                                                    (longest + a.splits - 1) / a.splits)) : longest + share;
  const bool single = each <= share;
  if (single) share = each;
  const auto units_of = [&](const Groups& g) { return single ? (g.blocks + share - 1) / share : g.blocks + kStart; };
  const int64_t from = blockIdx.x * (single ? 1 : share), to = from + (single ? 1 : share);
  int64_t before = 0;                     // of the sequences gone over
  for (int64_t base = 0; base < batch.B; base += 512) {
    __syncthreads();
    int64_t own = 0;
    if (base + threadIdx.x < batch.B) {
      const Groups g = groups_of(batch, cache, base + threadIdx.x, G, kRows);
      own = g.count * units_of(g);
    }
    int64_t upto = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 63) sums[0][wave] = upto;
    __syncthreads();
    for (int i = 0; i < wave; ++i) upto += sums[0][i];
    upto += before;
    if (from >= upto - own && from < upto) {
      found[0] = base + threadIdx.x;
      found[1] = upto - own;
    }
    for (int i = 0; i < 8; ++i) before += sums[0][i];
    if (from < before) break;
  }
  __syncthreads();
  if (from >= uniform(before)) return;    // no work left
  int64_t b = uniform(found[0]), start = uniform(found[1]);
  while (start < to && b < batch.B) {
    const Groups g = groups_of(batch, cache, b, G, kRows);
    const int64_t units = uniform(units_of(g)), count = uniform(g.count);
    // the sequence's groups that the part reaches
    for (int64_t i = from > start ? uniform((from - start) / units) : 0; i < count && start + i * units < to; ++i) {
      const int64_t first = start + i * units;
      Work w;
      int64_t block, end;
      if (single) {                       // equal pieces
        w.split = from - first;
        block = uniform(w.split * g.blocks / units);
        end = uniform((w.split + 1) * g.blocks / units);
      } else {
        // where the part's ends cut the group, in units from its start: at its ends if they leave too little
        const auto cut = [&](int64_t at) {
          return at >= units ? units : at < kStart + kLeast ? int64_t(0) : at > units - kLeast ? units : at;
        };
        const int64_t lo = cut(from - first), hi = cut(to - first);
        if (lo >= hi) continue;
        // pieces before this one: parts whose start cuts the group, up to this one's
        w.split = lo == 0 ? 0 : blockIdx.x - uniform((first + kStart + kLeast - 1) / share);
        block = max(lo - kStart, int64_t(0)), end = hi - kStart;
      }
      const bool whole = tree.whole && block == 0 && end == g.blocks;
      if (whole) w.split = -1;
      w.seq = sequence_of(batch, b);
      w.b = b;
      w.rb = uniform(i / cache.H);
      w.h = i - w.rb * cache.H;
      w.rows = w.seq.n * G;
      w.len = max(min(w.seq.len, batch.max_pages * cache.page), int64_t(0));
      w.before = w.seq.len - w.seq.n;
      many_rows<TIn, DT, RT>(a, batch, cache, tree, w, w.rb, w.len, block, w.len > 0 ? int(end - block) : 0);
      if (end == g.blocks && !whole)
        for (int64_t k = threadIdx.x; k < kRows * (a.splits - 1 - w.split); k += 512) {
          const int64_t r = w.rb * kRows + k % kRows;
          if (r >= w.rows) continue;
          const int64_t row = (w.seq.row0 + uint32_t(r) / uint32_t(G)) * a.Hq + w.h * G + uint32_t(r) % uint32_t(G);
          a.stats[(w.split + 1 + k / kRows) * a.rows + row] = make_float2(kNothing, 0.0f);
        }
    }
    start += count * units;
    ++b;
  }
}

int join_lanes(int D) { return D <= 64 ? 16 : D <= 128 ? 32 : 64; }

// Whether groups that are not cut are written as they are.  The join then looks for their marks, which costs it a trip to
// memory and some 1 us; many more rows than the chip holds at once are worth it: 204800 rows of 128, none cut, 51
// us joined, 11 so; 52800 15.5 and 11; 29376, all cut, 13.3 and 14.8.
bool writes_whole(int64_t rows, int D) { return rows * join_lanes(D) > int64_t(4096) * 256; }

// Joins the pieces of a row, LANES lanes to a row of up to 4 LANES values, always in the same order; most rows have few
// of the splits.  As join_splits_kernel, which reads them one after another (24 us for the trees of 300 above, 13 so).
template <int LANES, bool WHOLE>
__global__ __launch_bounds__(256) void join_pieces_kernel(Kv8Batch batch, int Hq, int D, int splits, int64_t rows,
                                                          const float* __restrict__ partial,
                                                          const float2* __restrict__ stats,
                                                          const uint32_t* __restrict__ places, uint16_t* __restrict__ out) {
  constexpr int kBatch = 8;
  const int lane = threadIdx.x & 63, n = lane & (LANES - 1);
  const int64_t row = (int64_t(blockIdx.x) * 256 + threadIdx.x) / LANES;
  const bool real = row < rows;
  const int64_t at = real ? row : 0, t = uint32_t(at) / uint32_t(Hq);
  if (WHOLE && __all(stats[at].y < 0.0f)) return;         // these rows are there
  bool there = false;
  for (int64_t i = n; i < batch.B; i += LANES) {
    const Sequence seq = sequence_of(batch, i);
    there = there || (t >= seq.row0 && t < seq.row0 + seq.n);
  }
  constexpr uint64_t kMask = LANES == 64 ? ~uint64_t(0) : (uint64_t(1) << (LANES & 63)) - 1;
  const bool some = (__ballot(there) >> (lane & ~(LANES - 1)) & kMask) != 0;
  float2 st[kBatch];
  uint32_t place[WHOLE ? kBatch : 1];     // of the piece's row in partial
  const auto load = [&](int from) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t piece = int64_t(min(from + i, splits - 1)) * rows + at;
      st[i] = stats[piece];
      if constexpr (WHOLE) place[i] = places[piece];
    }
  };
  float top = kNothing;
  bool open = true;
  for (int from = 0; from < splits; from += kBatch) {
    load(from);
    if (WHOLE && from == 0) open = !(st[0].y < 0.0f);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top = fmaxf(top, st[i].x);
  }
  float sum = 0.0f;
  float4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int from = 0; from < splits; from += kBatch) {
    if (splits > kBatch) load(from);
    float4_t p[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      p[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
      // nothing seen there, nothing written; and places of rows of no sequence are not to be followed
      if ((!WHOLE || some) && open && from + i < splits && st[i].y != 0.0f && n * 4 < D) {
        int64_t from_row = (from + i) * rows + at;
        if constexpr (WHOLE) from_row = place[i];
        p[i] = *reinterpret_cast<const float4_t*>(partial + from_row * D + n * 4);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (from + i >= splits || st[i].y == 0.0f) continue;
      const float f = __builtin_amdgcn_exp2f(st[i].x - top);
      sum += lowered(st[i].y, st[i].x - top);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(p[i][e], f, v[e]);
    }
  }
  const float over_l = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (real && some && open && n * 4 < D) *reinterpret_cast<uint2_t*>(out + row * D + n * 4) = pack_bf16x4(v, over_l);
}

template <typename TIn, int DT>
hipError_t run_tree(const AttentionArgs& a, const Kv8Batch& b, const Kv8Cache& c, const TreeTokens& tree,
                    const Kv8Plan& p, hipStream_t stream) {
  if (p.row_tiles == 8)
    return run_kernel(many_rows_tree_kernel<TIn, DT, 1>, kParts, 512, many_rows_lds_bytes<DT, 1>(), a, b, c, tree, stream);
  if constexpr (DT < 256)
    return run_kernel(many_rows_tree_kernel<TIn, DT, 2>, kParts, 512, many_rows_lds_bytes<DT, 2>(), a, b, c, tree, stream);
  else return hipErrorInvalidValue;                    // no plan has such tiles
}

hipError_t join_pieces(const AttentionArgs& a, const Kv8Batch& b, const Kv8Cache& c, const TreeTokens& tree,
                       const Kv8Plan& p, hipStream_t stream) {
  const int lanes = join_lanes(c.D);
  const bool whole = tree.whole;
  auto kernel = lanes == 16 ? (whole ? join_pieces_kernel<16, true> : join_pieces_kernel<16, false>)
                : lanes == 32 ? (whole ? join_pieces_kernel<32, true> : join_pieces_kernel<32, false>)
                              : (whole ? join_pieces_kernel<64, true> : join_pieces_kernel<64, false>);
  return launch_kernel(kernel, dim3(unsigned(ceil_div(a.rows, 256 / lanes))), dim3(256), 0, stream, b, a.Hq, c.D, p.splits,
                       a.rows, a.partial, a.stats, places_of(a), a.out);
}

}  // namespace

hipError_t launch_tree_masks(const int32_t* parents, const Kv8Batch& b, int64_t words, int64_t max_new,
                             uint64_t* mask, int64_t* pos, hipStream_t stream) {
  const int64_t slots = std::min<int64_t>(ceil_div(std::max<int64_t>(max_new, 1), kThreads), 65535);
  return launch_kernel(tree_masks_kernel, dim3(unsigned(b.B), unsigned(slots)), dim3(kThreads), 0, stream, parents, b,
                       words, mask, pos);
}

Kv8Plan plan_kv8_tree(int64_t B, int64_t T, int64_t Hq, int64_t H, int64_t D, int64_t max_new, int64_t max_len) {
  Kv8Plan p = plan_kv8_attention(B, T, Hq, H, D, max_new, max_len);
  if (p.row_tiles <= 4) return p;
  const int64_t rows = std::max<int64_t>(std::min(max_new, T), 1) * (Hq / H);
  const int64_t blocks = ceil_div(std::max<int64_t>(max_len, 1), 64);
  if (D <= 128) {
    // tiles of 256 rows or of 128: a workgroup's start, and its blocks (in tenths of us, measured), for sequences of
    // the mean number of rows.  16 trees of up to 40 tokens, 32 / 8 heads, 25 in the mean: 96 us in tiles of 128, 106 of 256;
    // two of up to 300, 64 / 8 heads: 422 and 345
    const int64_t mean = std::max<int64_t>(std::min(max_new, ceil_div(T, B)), 1) * (Hq / H);
    const auto cost = [&](int64_t each, int64_t start, int64_t block) {
      return start + block * std::max<int64_t>(std::min<int64_t>(kShare, blocks), ceil_div(B * H * ceil_div(mean, each) * blocks, kParts));
    };
    if (cost(128, 120, 14) < cost(256, 160, 19)) p.row_tiles = 8;
  }
  p.row_blocks = ceil_div(rows, 16 * p.row_tiles);
  // pieces: twice what equal sequences have of equal parts for every workgroup, for ragged ones
  const int64_t groups = B * H * p.row_blocks;
  p.splits = int(2 + 2 * std::min<int64_t>(ceil_div(kParts, groups), ceil_div(blocks, kShare)));
  const size_t all = size_t(p.splits) * T * Hq;
  const bool whole = writes_whole(T * Hq, int(D));
  p.sums = whole ? 2 * kParts * 16 * p.row_tiles : int64_t(all);
  p.bytes = round256(size_t(p.sums) * D * 4) + round256(all * (whole ? 12 : 8));
  const int lanes = join_lanes(int(D));
  p.threads = std::max<int64_t>(kParts * 512, ceil_div(T * Hq, 256 / lanes) * 256);
  return p;
}

hipError_t launch_kv8_tree_attention(const void* q, int dtype, int64_t q_t, int64_t q_h, int64_t Hq,
                                     const uint64_t* mask, int64_t words, const Kv8Batch& b, const Kv8Cache& c, int g,
                                     float scale, const Kv8Plan& p, uint16_t* out, void* workspace,
                                     hipStream_t stream) {
  return attend(q, dtype, q_t, q_h, Hq, b, c, TreeTokens{mask, words, writes_whole(b.T * Hq, c.D)}, g, scale, p, out, workspace, stream);
}

}  // namespace convrot
