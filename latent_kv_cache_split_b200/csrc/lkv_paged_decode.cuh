// Decode attention over paged 4-bit cache rows (lkv_int4.cuh): the tied forms, where the state of a
// group is its key (with the shared RoPE key) and its value.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include "lkv_int4.cuh"
#include "lkv_ptx.cuh"

namespace lkv {

struct PagedDecodeParams {
  Paged pages;
  const __nv_bfloat16* q;       // [B, s_q, h_q, d]
  const __nv_bfloat16* q_rope;  // [B, s_q, h_q, d_rope]
  int B, s_q, h_q, G, hpg, d, d_rope;
  float scale;
  __nv_bfloat16* out;  // [B, s_q, h_q, d]
  float* lse;          // [B, s_q, h_q]
  int* err;
};

constexpr int kPagedThreads = 128;
constexpr int kPagedChunk = 128;
constexpr int kPagedMaxD = 512;

__device__ __forceinline__ float int4_at(const uint8_t* row, int r, int c) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(row + (c / 8) * 4);
  const int e = c % 8;
  const int u = (w >> (4 * (e / 2) + 16 * (e & 1))) & 15;
  return static_cast<float>(u - 8) * __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row + r / 2)[c / kInt4Block]);
}

// One CTA per (request, query token, head), keys in chunks with a running maximum and sum.
__global__ void __launch_bounds__(kPagedThreads) paged_decode_kernel(const PagedDecodeParams p) {
  __shared__ float qs[kPagedMaxD + 256];
  __shared__ float ps[kPagedChunk];
  __shared__ long long at[kPagedChunk];
  __shared__ float red[kPagedThreads / 32];
  const int h = blockIdx.x % p.h_q, i = (blockIdx.x / p.h_q) % p.s_q, b = blockIdx.x / (p.h_q * p.s_q);
  const int j = h / p.hpg, tid = threadIdx.x, r = p.G * p.d;
  const int nvis = max(0, __ldg(p.pages.seq_lens + b)) - p.s_q + i + 1;
  const size_t qrow = (static_cast<size_t>(b) * p.s_q + i) * p.h_q + h;
  for (int c = tid; c < p.d; c += kPagedThreads) qs[c] = __bfloat162float(p.q[qrow * p.d + c]);
  for (int c = tid; c < p.d_rope; c += kPagedThreads) qs[p.d + c] = __bfloat162float(p.q_rope[qrow * p.d_rope + c]);
  float acc[kPagedMaxD / kPagedThreads] = {};
  float m = -INFINITY, l = 0.f;
  for (int t0 = 0; t0 < nvis; t0 += kPagedChunk) {
    const int n = min(kPagedChunk, nvis - t0);
    __syncthreads();
    float s = -INFINITY;
    if (tid < n) {
      at[tid] = paged_row(p.pages, b, t0 + tid);
      if (at[tid] < 0) record_error(p.err, LKV_SITE_BAD_ROW);
      s = 0.f;
      if (at[tid] >= 0) {
        const uint8_t* row = p.pages.pool + at[tid];
        for (int c = 0; c < p.d; ++c) s = fmaf(qs[c], int4_at(row, r, j * p.d + c), s);
        const __nv_bfloat16* kr = reinterpret_cast<const __nv_bfloat16*>(row + int4_rope_at(r));
        for (int c = 0; c < p.d_rope; ++c) s = fmaf(qs[p.d + c], __bfloat162float(kr[c]), s);
      }
      s *= p.scale;
    }
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float alpha = m == -INFINITY ? 0.f : expf(m - mn);
    const float e = tid < n ? expf(s - mn) : 0.f;
    ps[tid] = e;
    float sum = e;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    l = l * alpha + ((red[0] + red[1]) + (red[2] + red[3]));
    m = mn;
#pragma unroll
    for (int a = 0; a < kPagedMaxD / kPagedThreads; ++a) {
      const int c = tid + a * kPagedThreads;
      if (c >= p.d) continue;
      float o = 0.f;
      for (int t = 0; t < n; ++t)
        if (at[t] >= 0) o = fmaf(ps[t], int4_at(p.pages.pool + at[t], r, j * p.d + c), o);
      acc[a] = acc[a] * alpha + o;
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int a = 0; a < kPagedMaxD / kPagedThreads; ++a) {
    const int c = tid + a * kPagedThreads;
    if (c < p.d) p.out[qrow * p.d + c] = __float2bfloat16_rn(acc[a] * inv);
  }
  if (tid == 0) p.lse[qrow] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace lkv
