// Rotary positions of queries and keys (convrot_rotary): for each pair (a, b) of a head's first R
// elements, with angle = pos * inv_freq[i],
//   (a, b) -> f (a cos - b sin, b cos + a sin),
// pairs (2i, 2i + 1) or (i, i + R/2); elements from R on are copied.  The inverse turns by
// -angle, which is also the transpose: the gradient's way back.
//
// Angles of far positions do not fit fp32 (position 10^6 times a frequency near 1 has an error of
// 0.06 rad there), so each angle is taken in fp64 in turns and only its fraction goes to fp32.
// A workgroup takes a token: its R/2 cosines and sines go to LDS once, for all of its heads.
//
// Every element is read and written once, which bounds it: 16384 tokens of 40 heads of 128 in bf16
// (336 MB) take 82.8 us, 4.05 TB/s (a large copy: 4.95); 8 tokens 4.2 us, the launch.
#include "decode_device.h"

#include <algorithm>

namespace convrot {
namespace {

constexpr int kThreads = 256;

template <typename T> __device__ __forceinline__ T to_elem(float f);
template <> __device__ __forceinline__ float to_elem<float>(float f) { return f; }
template <> __device__ __forceinline__ uint16_t to_elem<uint16_t>(float f) { return f32_to_bf16(f); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T e[V];
};

// An item is V pairs, V neighbouring elements of each half, or V / 2 pairs that are neighbours
// themselves (INTERLEAVED); V = 1: one pair.
template <typename T, int V, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, int heads_per_block) {
  extern __shared__ float2 turn[];                       // f cos, f sin of each pair
  const int64_t t = blockIdx.x;
  const double pos = double(a.pos[t]);
  for (int i = threadIdx.x; i < a.R / 2; i += kThreads) {
    // pos * inv_freq / 2 pi with the product and the turns in two fp64 pieces each: good to about 2^-50 of
    // a turn for positions below 2^53, which fp64 holds (from 2^29 on, 53 - 24 bits, the product has a
    // second piece)
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591104e-18;   // 1 / (2 pi)
    const double f = double(a.inv_freq[i]);
    const double p = pos * f, p_lo = __builtin_fma(pos, f, -p);
    const double hi = p * kHi;
    const double lo = __builtin_fma(p, kHi, -hi) + __builtin_fma(p, kLo, p_lo * kHi);
    const double frac = (hi - __builtin_rint(hi)) + lo;
    float s, c;
    sincospif(float(2.0 * frac), &s, &c);
    turn[i] = make_float2(a.factor * c, a.factor * (a.inverse ? -s : s));
  }
  __syncthreads();

  const int first = blockIdx.y * heads_per_block;
  const int last = min(first + heads_per_block, a.q.heads + a.k.heads);
  const int turned = INTERLEAVED && V > 1 ? a.R / V : a.R / (2 * V);   // items that hold pairs
  const int items = turned + (a.D - a.R) / V;                 // and those that are copied
  for (int i = threadIdx.x; i < (last - first) * items; i += kThreads) {
    const int head = first + i / items, item = i - (i / items) * items;
    const bool is_q = head < a.q.heads;
    const RotaryPart& part = is_q ? a.q : a.k;
    const int64_t h = is_q ? head : head - a.q.heads;
    const T* in = static_cast<const T*>(part.in) + t * part.in_t + h * part.in_h;
    T* out = static_cast<T*>(part.out) + t * part.out_t + h * part.out_h;
    if (item >= turned) {
      const int at = a.R + (item - turned) * V;
      *reinterpret_cast<Pack<T, V>*>(out + at) = *reinterpret_cast<const Pack<T, V>*>(in + at);
    } else if constexpr (V == 1) {
      const int ix = INTERLEAVED ? 2 * item : item, iy = INTERLEAVED ? ix + 1 : item + a.R / 2;
      const float2 cs = turn[item];
      const float x = load_one<T>(in + ix), y = load_one<T>(in + iy);
      out[ix] = to_elem<T>(__builtin_fmaf(x, cs.x, -(y * cs.y)));
      out[iy] = to_elem<T>(__builtin_fmaf(y, cs.x, x * cs.y));
    } else if constexpr (INTERLEAVED) {
      Pack<T, V> v = *reinterpret_cast<const Pack<T, V>*>(in + item * V);
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const float2 cs = turn[(item * V + e) / 2];
        const float x = load_one<T>(&v.e[e]), y = load_one<T>(&v.e[e + 1]);
        v.e[e] = to_elem<T>(__builtin_fmaf(x, cs.x, -(y * cs.y)));
        v.e[e + 1] = to_elem<T>(__builtin_fmaf(y, cs.x, x * cs.y));
      }
      *reinterpret_cast<Pack<T, V>*>(out + item * V) = v;
    } else {
      const int half = a.R / 2, at = item * V;
      Pack<T, V> u = *reinterpret_cast<const Pack<T, V>*>(in + at);
      Pack<T, V> v = *reinterpret_cast<const Pack<T, V>*>(in + half + at);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float2 cs = turn[at + e];
        const float x = load_one<T>(&u.e[e]), y = load_one<T>(&v.e[e]);
        u.e[e] = to_elem<T>(__builtin_fmaf(x, cs.x, -(y * cs.y)));
        v.e[e] = to_elem<T>(__builtin_fmaf(y, cs.x, x * cs.y));
      }
      *reinterpret_cast<Pack<T, V>*>(out + at) = u;
      *reinterpret_cast<Pack<T, V>*>(out + half + at) = v;
    }
  }
}

template <typename T, int V>
hipError_t run(const RotaryArgs& a, int64_t T_, hipStream_t stream) {
  // a token's heads over several workgroups while there are few tokens
  const int heads = a.q.heads + a.k.heads;
  int blocks = int(std::min<int64_t>(heads, std::max<int64_t>(1, 1024 / T_)));
  const int per = (heads + blocks - 1) / blocks;
  blocks = (heads + per - 1) / per;
  const size_t lds = size_t(a.R / 2) * sizeof(float2);
  return launch_kernel(a.interleaved ? rotary_kernel<T, V, true> : rotary_kernel<T, V, false>,
                       dim3(unsigned(T_), unsigned(blocks)), dim3(kThreads), lds, stream, a, per);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, int dtype, int64_t T, hipStream_t stream) {
  // 16-byte accesses where every piece of every head starts on 16 bytes: the head and token
  // strides, R, and R/2 too when the halves are apart.  Else pair by pair.
  const int V = dtype == 0 ? 4 : 8;
  bool wide = a.R % V == 0 && a.D % V == 0 && (a.interleaved || (a.R / 2) % V == 0);
  for (const RotaryPart* p : {&a.q, &a.k}) {
    if (p->heads == 0) continue;
    wide = wide && reinterpret_cast<uintptr_t>(p->in) % 16 == 0 && reinterpret_cast<uintptr_t>(p->out) % 16 == 0 &&
           p->in_t % V == 0 && p->in_h % V == 0 && p->out_t % V == 0 && p->out_h % V == 0;
  }
  if (wide) return dtype == 0 ? run<float, 4>(a, T, stream) : run<uint16_t, 8>(a, T, stream);
  return dtype == 0 ? run<float, 1>(a, T, stream) : run<uint16_t, 1>(a, T, stream);
}

}  // namespace convrot
