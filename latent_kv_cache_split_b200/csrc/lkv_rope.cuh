// Rotary positions: the angle of a pair, and the kernel that rotates queries (or gradients).
//
// A pair (a, b) of a token at position p with frequency f (radians a position) and gain g becomes
//   a' = g (a cos pf - b sin pf),  b' = g (a sin pf + b cos pf);
// the transpose (the gradient's map) has the angle negated.  Pair i of n/2 is columns (i, i + n/2) of
// the rotated part in the half layout and (2i, 2i + 1) in the interleaved one.
//
// The angle is taken in turns, in fp64: fp32 would lose it (at position 10^6 an fp32 angle of frequency
// 1 is off by 0.03 rad).  p f / 2 pi is off by at most 3 ulp, under 10^-7 turns at the largest int32
// position; its distance to the nearest whole turn is rounded to fp32 (2^-24 of it) for sincospif.
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
  int bx, by;      // threads: bx along a head's items, by along (token, head) rows
  int tok_block;   // tokens of a block
  int head_block;  // heads of a block (tok_block is 1 where this is less than all)
};

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;  // (token, head) rows of a thread, all loaded before any is used
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

// One item is V columns of the half layout's lower half with their partners, 2 columns or V of the
// interleaved layout, or V copied columns.  Every element is read and written once, by one thread, so
// x and out may be the same array.  The kernel is bound by memory: a block's (cos, sin) table costs one
// fp64 angle a pair and is shared by its heads, and its loads are issued before the table is built.
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  __shared__ float2 table[kRopeTable];
  constexpr int kIV = kInterleaved && V == 1 ? 2 : V;  // columns of an interleaved item
  using Vec = RopeVec<T, V>;
  const int half = p.rot / 2;
  const int rot_items = kInterleaved ? p.rot / kIV : half / V;
  const int left = p.first / V;  // copied items before the rotated part
  const int items = rot_items + (p.copy ? (p.d - p.rot) / V : 0);
  const int tid = threadIdx.x;
  const int tx = tid % p.bx, ty = tid / p.bx;
  const int head_chunks = (p.heads + p.head_block - 1) / p.head_block;
  const long long tok0 = static_cast<long long>(blockIdx.x / head_chunks) * p.tok_block;
  const int h0 = (blockIdx.x % head_chunks) * p.head_block;
  const int nh = min(p.head_block, p.heads - h0);
  const int nt = static_cast<int>(min(static_cast<long long>(p.tok_block), p.n_tok - tok0));
  const int rows = nt * nh;
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);
  bool first_pass = true;
  for (int it0 = 0; it0 < items; it0 += p.bx) {
    const int it = it0 + tx;
    const bool live = it < items && ty < p.by;
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
    for (int r0 = 0; r0 < rows; r0 += p.by * kRopeUnroll) {
      Vec a[kRopeUnroll], b[kRopeUnroll];
      int tok[kRopeUnroll], head[kRopeUnroll];
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        const int r = r0 + u * p.by + ty;
        tok[u] = -1;
        if (live && r < rows) {
          tok[u] = r / nh;
          head[u] = h0 + r - tok[u] * nh;
          const T* row = x + (tok0 + tok[u]) * p.x_ts + head[u] * p.x_hs;
          a[u] = *reinterpret_cast<const Vec*>(row + c0);
          if (two) b[u] = *reinterpret_cast<const Vec*>(row + c1);
        }
      }
      if (first_pass) {
        for (int e = tid; e < nt * half; e += kRopeThreads) {
          const int t = e / half;
          float2 cs = rope_cos_sin(p.pos[tok0 + t], p.freqs[e - t * half], p.gain);
          if (p.inverse) cs.y = -cs.y;
          table[e] = cs;
        }
        __syncthreads();
        first_pass = false;
      }
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        if (tok[u] < 0) continue;
        T* row = out + (tok0 + tok[u]) * p.o_ts + head[u] * p.o_hs;
        if (pair0 >= 0) {
          const float2* cs = table + tok[u] * half + pair0;
          if (two) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
              const float fa = rope_up(a[u].v[k]), fb = rope_up(b[u].v[k]);
              a[u].v[k] = rope_down<T>(fa * cs[k].x - fb * cs[k].y);
              b[u].v[k] = rope_down<T>(fa * cs[k].y + fb * cs[k].x);
            }
            *reinterpret_cast<Vec*>(row + c1) = b[u];
          } else {
#pragma unroll
            for (int k = 0; k + 1 < V; k += 2) {
              const float fa = rope_up(a[u].v[k]), fb = rope_up(a[u].v[k + 1]);
              a[u].v[k] = rope_down<T>(fa * cs[k / 2].x - fb * cs[k / 2].y);
              a[u].v[k + 1] = rope_down<T>(fa * cs[k / 2].y + fb * cs[k / 2].x);
            }
          }
        }
        *reinterpret_cast<Vec*>(row + c0) = a[u];
      }
    }
  }
}

}  // namespace lkv
