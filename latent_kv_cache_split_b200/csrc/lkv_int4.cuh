// 4-bit cache rows in a paged pool: the row format, the page lookup and the append.
//
// A row of r latent columns and d_rope RoPE columns (one token) is
//   [0, r / 2)              4-bit codes, u = code + 8 with code in [-7, 7]; eight columns share a 32-bit
//                           word, column 2i of the eight in bits 4i .. 4i + 3, column 2i + 1 in bits
//                           16 + 4i .. 19 + 4i, so that (word >> 4i) & 0x000f000f is a pair of columns
//   [r / 2, + 2 (r / 32))   bf16 scales, one for every 32 columns, the field padded to 16 bytes
//   then                    d_rope bf16 values: the rotated RoPE key
// and every field starts on a 16-byte boundary.  A scale is the smallest number of 4 significant bits
// that reaches amax / 7, so code * scale has at most 7 significant bits and is exact in bf16: a decode
// computes on bf16 operands that are the very values the row stands for.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include "lkv_ptx.cuh"
#include "lkv_rope.cuh"
#include "../../include/lkv.h"

namespace lkv {

constexpr int kInt4Block = 32;       // columns that share a scale
constexpr int kInt4MaxLatent = 1024;

__host__ __device__ __forceinline__ int int4_scale_bytes(int r) { return (r / 16 + 15) / 16 * 16; }
__host__ __device__ __forceinline__ int int4_rope_at(int r) { return r / 2 + int4_scale_bytes(r); }

// Pages of a pool and the table that places a request's tokens in them.
struct Paged {
  uint8_t* pool;
  long long page_stride, row_stride;  // bytes
  long long n_pages;
  int page_size, page_shift;  // page_shift: log2 of page_size, or -1 where it is no power of two
  const int* table;  // [batch, max_pages], row stride table_stride
  long long table_stride;
  int max_pages;
  const int* seq_lens;  // [batch]
};

// Byte offset of token t of request b in the pool, or -1 where the table has no page for it.
__device__ __forceinline__ long long paged_row(const Paged& g, int b, int t) {
  const int k = t / g.page_size;
  if (k >= g.max_pages) return -1;
  const int page = __ldg(g.table + b * g.table_stride + k);
  if (page < 0 || page >= g.n_pages) return -1;
  return page * g.page_stride + static_cast<long long>(t - k * g.page_size) * g.row_stride;
}

// Eight codes times their scale: bf16 pairs of columns (2i, 2i + 1).  mask and magic are 0x000f000f and 0x43004300
// in registers, so that one lop3 takes both.
__device__ __forceinline__ uint4 int4_expand(uint32_t w, uint32_t mask, uint32_t magic, __nv_bfloat162 s, __nv_bfloat162 off) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(u) : "r"(w >> (4 * i)), "r"(mask), "r"(magic));
    __nv_bfloat162 v = __hfma2(*reinterpret_cast<__nv_bfloat162*>(&u), s, off);
    o[i] = *reinterpret_cast<uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

struct AppendParams {
  Paged pages;
  const __nv_bfloat16* rows;  // [n_new, r + d_rope]
  long long row_stride;       // elements
  long long n_new;
  const int* cu_new;  // [batch + 1], or NULL: n_new / batch rows a request
  int batch, per;     // per: rows a request without cu_new
  int r, d_rope;
  const double* freqs;  // [d_rope / 2], or NULL: the keys are stored as they come
  int interleaved;
  float gain;
  __nv_bfloat16* held;  // [n_new, r + d_rope] the values the cache then holds, or NULL
  long long held_stride;
  int* err;
};

// The larger value, NaN where either is (fmaxf passes over NaN).
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

constexpr int kAppendThreads = 256;

// Request of new row w: the last b with cu[b] <= w, its rows [begin, end) and its token count.  One step looks at 32
// places of the range at once, and the last one brings the request's own numbers with it, so that a batch of up to 32
// costs one load's latency.
__device__ __forceinline__ int request_of(const int* cu, const int* seq_lens, int batch, long long w, int lane, int& begin, int& end,
                                          int& len) {
  int lo = 0, hi = batch;  // cu[lo] <= w < cu[hi]
  while (true) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const int c = at < hi ? __ldg(cu + at) : 0, l = step == 1 && at < hi ? __ldg(seq_lens + at) : 0;
    const int next = step == 1 && at < hi ? __ldg(cu + at + 1) : 0;
    const unsigned below = __ballot_sync(0xffffffffu, at < hi && c <= w);
    const int k = below ? 31 - __clz(below) : 0;
    if (step == 1) {
      begin = __shfl_sync(0xffffffffu, c, k);
      end = __shfl_sync(0xffffffffu, next, k);
      len = __shfl_sync(0xffffffffu, l, k);
      return lo + k;
    }
    lo += k * step;
    hi = min(hi, lo + step);
  }
}

// One warp a row: lane l takes columns 8 (l + 32 k) .. + 7, so 4 lanes share a scale and every load and
// store of the warp is contiguous.  Bound by instruction issue, some 600 a row: 78k rows of 576 take 36.4 us
// where their bytes (the row in, the cache's row and the held values out) would take 22.5.
//
// The code is x / s rounded to the nearest integer, ties to even, without a division: x is 8 significant
// bits and s = n 2^k with n in 8 .. 15, so x / s is a tie or at least 1/1920 away from one.  fma(x, 1 / s,
// 1536) rounds x / s (off by under 2^-20) to a multiple of 2^-13, which puts ties back on the tie and
// moves nothing else across one; adding 12582920 - 1536 then rounds to an integer, and leaves code + 8 in
// the low bits of the sum's pattern.  A block with a NaN or an infinity gets a NaN for its scale, whatever
// its codes (78k rows of 576: 36.0 us with a maximum that passes over NaN, 36.4 with one that keeps it).
__global__ void __launch_bounds__(kAppendThreads) append_int4_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const long long w = (static_cast<long long>(blockIdx.x) * kAppendThreads + threadIdx.x) >> 5;
  if (w >= p.n_new) return;
  const __nv_bfloat16* src = p.rows + w * p.row_stride;
  const int chunks = p.r / 8;
  constexpr int kK = kInt4MaxLatent / 256;
  uint4 v[kK];
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int c = lane + 32 * k;
    v[k] = c < chunks ? reinterpret_cast<const uint4*>(src)[c] : make_uint4(0u, 0u, 0u, 0u);
  }
  // the first pair of the RoPE key, ahead of the chain of loads that finds the row's place
  const int half = p.d_rope / 2;
  auto pair_at = [&](int i, int& c0, int& c1) {
    c0 = p.interleaved ? 2 * i : i;
    c1 = p.interleaved ? 2 * i + 1 : i + half;
  };
  __nv_bfloat16 ka = __float2bfloat16_rn(0.f), kb = ka;
  double freq = 0.;
  if (lane < half) {
    int c0, c1;
    pair_at(lane, c0, c1);
    ka = src[p.r + c0];
    kb = src[p.r + c1];
    if (p.freqs) freq = __ldg(p.freqs + lane);
  }
  int b, pos;
  if (p.cu_new) {
    int begin, end, len;
    b = request_of(p.cu_new, p.pages.seq_lens, p.batch, w, lane, begin, end, len);
    if (w < begin || w >= end) return;  // behind the last request's rows
    pos = max(len, 0) - (end - static_cast<int>(w));
  } else {
    b = static_cast<int>(w / p.per);
    pos = max(__ldg(p.pages.seq_lens + b), 0) - p.per + static_cast<int>(w - static_cast<long long>(b) * p.per);
  }
  if (pos < 0) return;  // an idle slot: no such token
  const long long at = paged_row(p.pages, b, pos);
  if (at < 0) {
    if (lane == 0) record_error(p.err, LKV_SITE_BAD_ROW);
    return;
  }
  uint8_t* dst = p.pages.pool + at;
  __nv_bfloat16* held = p.held ? p.held + w * p.held_stride : nullptr;
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int c = lane + 32 * k;
    if (32 * k >= chunks) break;  // the same for the whole warp
    const uint32_t word[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    float x[8];
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(word[e] << 16);
      x[2 * e + 1] = __uint_as_float(word[e] & 0xffff0000u);
      amax = max_or_nan(amax, max_or_nan(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
    }
    amax = max_or_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max_or_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // amax = m 2^(e - 134) with m in 128 .. 255; the least n with 7 n 2 >= m, or else with 7 n 4 >= m
    const uint32_t bits = __float_as_uint(amax);
    const int m = static_cast<int>((bits >> 16) & 0x7fu) | 0x80, e = static_cast<int>(bits >> 23);
    const bool low = m <= 210;
    const int n = low ? (m + 13) / 14 : (m + 27) / 28;
    // 0 below 2^-100, NaN where amax is infinite or none
    const float s = static_cast<uint32_t>(e - 27) < 228u ? static_cast<float>(n) * __uint_as_float(static_cast<uint32_t>(e - (low ? 6 : 5)) << 23)
                                                         : amax * 0.f;
    const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
    uint32_t code = 0u - (0x4b400000u + (0x4b400000u << 4) + (0x4b400000u << 8));  // the sums' patterns above their low bits
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f0 = fmaf(x[2 * i], inv, 1536.f) + (12582920.f - 1536.f);
      const float f1 = fmaf(x[2 * i + 1], inv, 1536.f) + (12582920.f - 1536.f);
      code += (__float_as_uint(f0) << (4 * i)) + (__float_as_uint(f1) << (4 * i + 16));
    }
    if (c < chunks) {
      reinterpret_cast<uint32_t*>(dst)[c] = code;
      if ((lane & 3) == 0) reinterpret_cast<__nv_bfloat16*>(dst + p.r / 2)[c / 4] = __float2bfloat16_rn(s);
      if (held) {
        const __nv_bfloat162 s2 = __float2bfloat162_rn(s);
        reinterpret_cast<uint4*>(held)[c] = int4_expand(code, 0x000f000fu, 0x43004300u, s2, __hmul2(s2, __float2bfloat162_rn(-136.f)));
      }
    }
  }
  // the padding of the scales' field
  for (int c = p.r / kInt4Block + lane; c < int4_scale_bytes(p.r) / 2; c += 32)
    reinterpret_cast<uint16_t*>(dst + p.r / 2)[c] = 0;
  __nv_bfloat16* kd = reinterpret_cast<__nv_bfloat16*>(dst + int4_rope_at(p.r));
  for (int i = lane; i < half; i += 32) {
    int c0, c1;
    pair_at(i, c0, c1);
    __nv_bfloat16 a = ka, bb = kb;
    if (i >= 32) {
      a = src[p.r + c0];
      bb = src[p.r + c1];
      if (p.freqs) freq = __ldg(p.freqs + i);
    }
    if (p.freqs) {
      const float2 cs = rope_cos_sin(pos, freq, p.gain);
      const float fa = __bfloat162float(a), fb = __bfloat162float(bb);
      a = __float2bfloat16_rn(fa * cs.x - fb * cs.y);
      bb = __float2bfloat16_rn(fa * cs.y + fb * cs.x);
    }
    kd[c0] = a;
    kd[c1] = bb;
    if (held) {
      held[p.r + c0] = a;
      held[p.r + c1] = bb;
    }
  }
}

}  // namespace lkv
