// Rotary positions: the angle of a pair, and the kernel that rotates queries (or gradients).
//
// A pair (a, b) of a token at position p with frequency f (radians a position) and gain g becomes
//   a' = g (a cos pf - b sin pf),  b' = g (a sin pf + b cos pf);
// the transpose (the gradient's map) has the angle negated.  Pair i of n/2 is columns (i, i + n/2) of
// the rotated part in the half layout and (2i, 2i + 1) in the interleaved one.
//
// The angle is taken in turns, in fp64: fp32 would lose it (at position 10^6 an fp32 angle of frequency
// 1 is off by 0.03 rad).  p f / 2 pi takes three roundings (1 / 2 pi and two products), 3 2^-53 of it: below
// 1.2 10^-7 turns at the largest int32 position and frequency 1, in proportion to the frequency.  Its distance to
// the nearest whole turn is rounded to fp32 (2^-24 of it) for sincospif.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

namespace lkv {

__device__ __forceinline__ float2 rope_cos_sin(int pos, double freq, float gain) {
  const double turns = static_cast<double>(pos) * freq * 0.15915494309189533577;  // 1 / (2 pi)
  float s, c;
  sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
  return make_float2(gain * c, gain * s);
}

struct RopeParams {
  const void* x;
  void* out;
  long long x_ts, x_hs, o_ts, o_hs;  // token and head strides, elements
  const int* pos;
  const double* freqs;
  long long n_tok;
  int heads, d, first, rot;
  int inverse, copy;  // copy: the columns outside the rotated part go to `out` too
  float gain;
  int tok_block;   // tokens of a block
  int head_block;  // heads of a block (all of them where tok_block > 1)
};

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 512;
constexpr int kRopeTable = 2048;  // (cos, sin) entries of a block: 16 KB

template <typename T>
__device__ __forceinline__ float rope_up(T v);
template <>
__device__ __forceinline__ float rope_up<float>(float v) { return v; }
template <>
__device__ __forceinline__ float rope_up<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T rope_down(float v);
template <>
__device__ __forceinline__ float rope_down<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rope_down<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int V>
struct alignas(sizeof(T) * V) RopeVec {
  T v[V];
};

// Threads x run along a head's items, threads y along the block's (token, head) rows.  An item is V columns of the half
// layout's lower half with their partners, 2 columns or V of the interleaved layout, or V copied columns.  Every element
// is read and written once, by one thread, so x and out may be the same array.  With many heads the kernel is bound by memory,
// and what it takes is warps: one row a thread at a time with eight blocks an SM reads and writes 8192 x 128 x 192 bf16,
// interleaved, in 156 us (5.1 TB/s), four rows at a time with the four blocks that their registers leave in 214 us.  Eight
// blocks leave 32 registers, of which the half layout in bf16 spills a few: 175 us (4.6 TB/s).  A block's (cos, sin) table
// costs one fp64 angle a pair and is shared by its heads; its first loads are issued before the table is built.  With one
// head there is nothing to share and the angles bound it: 65536 x 1 x 64 bf16 takes 13 us interleaved and 14 us in halves,
// 1.2-1.3 TB/s.
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 table[kRopeTable];
  constexpr int kIV = kInterleaved && V == 1 ? 2 : V;  // columns of an interleaved item
  using Vec = RopeVec<T, V>;
  const int half = p.rot / 2;
  const int rot_items = kInterleaved ? p.rot / kIV : half / V;
  const int left = p.first / V;  // copied items before the rotated part
  const int items = rot_items + (p.copy ? (p.d - p.rot) / V : 0);
  const int ty = threadIdx.y, by = blockDim.y, tid = ty * blockDim.x + threadIdx.x;
  const int h0 = blockIdx.y * p.head_block;
  const long long tok0 = static_cast<long long>(blockIdx.x) * p.tok_block;
  const int nh = min(p.head_block, p.heads - h0);
  const int nt = static_cast<int>(min(static_cast<long long>(p.tok_block), p.n_tok - tok0));
  const int rows = nt * nh;
  const T* x = static_cast<const T*>(p.x) + tok0 * p.x_ts + h0 * p.x_hs;
  T* out = static_cast<T*>(p.out) + tok0 * p.o_ts + h0 * p.o_hs;
  bool fresh = true;  // the table is still to be built
  for (int it0 = 0; it0 < items; it0 += blockDim.x) {
    const int it = it0 + threadIdx.x;
    const bool live = it < items;
    // columns of this item: c0 (and c1, its partners in the half layout)
    int c0, c1 = 0, pair0 = -1;
    if (it < rot_items) {
      c0 = p.first + it * (kInterleaved ? kIV : V);
      c1 = kInterleaved && V == 1 ? c0 + 1 : c0 + half;
      pair0 = kInterleaved ? it * kIV / 2 : it * V;
    } else {
      const int k = it - rot_items;
      c0 = k < left ? k * V : p.rot + k * V;
    }
    const bool two = pair0 >= 0 && (!kInterleaved || V == 1);
    for (int r = ty; r - ty < rows; r += by) {
      const bool mine = live && r < rows;
      const int t = nt == 1 ? 0 : r / nh;
      Vec a, b;
      if (mine) {
        const T* row = x + t * p.x_ts + (r - t * nh) * p.x_hs;
        a = *reinterpret_cast<const Vec*>(row + c0);
        if (two) b = *reinterpret_cast<const Vec*>(row + c1);
      }
      if (fresh) {  // the first pass of every thread
        for (int e = tid; e < nt * half; e += blockDim.x * by) {
          const int k = nt == 1 ? 0 : e / half;
          float2 cs = rope_cos_sin(p.pos[tok0 + k], p.freqs[e - k * half], p.gain);
          if (p.inverse) cs.y = -cs.y;
          table[e] = cs;
        }
        __syncthreads();
        fresh = false;
      }
      if (!mine) continue;
      T* row = out + t * p.o_ts + (r - t * nh) * p.o_hs;
      if (pair0 >= 0) {
        const float2* cs = table + t * half + pair0;
        if (two) {
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const float fa = rope_up(a.v[k]), fb = rope_up(b.v[k]);
            a.v[k] = rope_down<T>(fa * cs[k].x - fb * cs[k].y);
            b.v[k] = rope_down<T>(fa * cs[k].y + fb * cs[k].x);
          }
          *reinterpret_cast<Vec*>(row + c1) = b;
        } else {
#pragma unroll
          for (int k = 0; k + 1 < V; k += 2) {
            const float fa = rope_up(a.v[k]), fb = rope_up(a.v[k + 1]);
            a.v[k] = rope_down<T>(fa * cs[k / 2].x - fb * cs[k / 2].y);
            a.v[k + 1] = rope_down<T>(fa * cs[k / 2].y + fb * cs[k / 2].x);
          }
        }
      }
      *reinterpret_cast<Vec*>(row + c0) = a;
    }
  }
}

}  // namespace lkv
