// Decode attention over paged 4-bit cache rows for units of at most 16 query rows (d = 128 or 256), on
// warp-level matrix instructions.
//
// A unit of 16 rows gives a tcgen05 MMA of the keys-in-M form (lkv_paged_decode.cuh) N = 16 columns for the
// 128 x 16 operand that it reads, and each tile passes through eight barriers between four roles.  Here a
// warp keeps everything of 16 keys in registers: it expands the codes straight into the B operand of QK,
// transposes those registers into the B operand of PV, and keeps its own running sums, references and
// output; warps meet only at a segment's end.  mma.sync runs at a third of the tcgen05 rate (555 TFLOP/s
// measured), which 16 rows do not reach.
//
//   S[row, key] = Q[row, :] . K[key, :]    m16n8k16, A = Q, B = K: thread 4g + t has of key g (of 8) the 32
//                                          columns 32 t .. + 31 (one scale) of every 128, in the order of the
//                                          codes; the k index runs through them as it falls, Q alike
//   O[row, c]  += P[row, key] V[key, c]    A = P from the accumulators of S, B = V: movmatrix turns register
//                                          i of K (8 keys x columns 32 t + 2i, + 1) into (8 columns x 8 keys)
//
// Warp w of eight takes keys 16 w .. + 15 of every 128-key tile.  Its rows come by cp.async into a ring of its
// own, kWarpStages deep, a row without a token as zeros.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include "lkv_int4.cuh"
#include "lkv_paged_decode.cuh"
#include "lkv_ptx.cuh"

namespace lkv {

constexpr int kWarpThreads = 256;
constexpr int kWarpRows = 16;
constexpr int kWarpStages = 4;

template <int D>
struct WarpCfg {
  static constexpr int kH = D / 128;
  static constexpr int kCodeBytes = 16 * (D / 2), kScaleBytes = 16 * (D / 16), kRopeBytes = 16 * 128;
  static constexpr int kStage = kCodeBytes + kScaleBytes + kRopeBytes;  // 16 keys
  static constexpr int kRing = kWarpStages * kStage;                    // of a warp
  // The warps' outputs on their way to their sum: 64 columns of every 128 at a time, as float2, rows padded against
  // bank conflicts.
  static constexpr int kSumRow = 32 * kH + 4;
  static constexpr int kSumBytes = 8 * kWarpRows * kSumRow * 8;
  static constexpr bool kQRegs = D == 128;  // Q stays in registers (D = 256: the output takes them, Q is read from smem)
  static constexpr int kQRow = (D + 64) * 2 + 16;
  static constexpr size_t kSmem = 8 * static_cast<size_t>(kRing) + kSumBytes + (kQRegs ? 0 : kWarpRows * kQRow);
  static_assert(kStage % 16 == 0 && kSmem <= 232448 - 8192, "shared memory budget");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const uint8_t* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const uint8_t* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds2(uint32_t a) {
  uint32_t v;
  asm volatile("{\n\t.reg .u16 h;\n\tld.shared.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct __align__(16) WarpSmem {
  float m[8][kWarpRows], l[8][kWarpRows];
  PagedCursor walk[8], ahead[8];
  PagedSegment seg[8], ahead_seg[8];
};

template <int D>
__global__ void __launch_bounds__(kWarpThreads, 1) paged_warp_kernel(const __grid_constant__ PagedDecodeParams p) {
  using Cfg = WarpCfg<D>;
  constexpr int H = Cfg::kH, TN = kPagedTile;
  extern __shared__ __align__(1024) uint8_t warp_smem_raw[];
  __shared__ WarpSmem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int range = blockIdx.x;
  const int r = p.G * D;
  const uint32_t ring = smem_u32(warp_smem_raw) + warp * Cfg::kRing;
  float2* sums = reinterpret_cast<float2*>(warp_smem_raw + 8 * Cfg::kRing);
  uint8_t* qsm = warp_smem_raw + 8 * Cfg::kRing + Cfg::kSumBytes;  // the unit's Q, where it is not in registers

  if (tid < 2) p.seg_info[2 * range + tid] = -1;
  {
    const PagedCursor c = paged_locate(p, range, lane);
    if (lane == 0) {
      sm.walk[warp] = c;
      sm.ahead[warp] = c;
    }
  }
  griddep_launch_dependents();  // the combine may start launching
  // idle requests: no tile is walked for them
  for (int b = range; b < p.B; b += p.P) {
    if (__ldg(p.pages.seq_lens + b) > 0) continue;
    const size_t rows = static_cast<size_t>(p.s_q) * p.h_q;
    uint4* o = reinterpret_cast<uint4*>(p.out + b * rows * D);
    for (size_t e = tid; e < rows * D / 8; e += kWarpThreads) o[e] = make_uint4(0u, 0u, 0u, 0u);
    for (size_t e = tid; e < rows; e += kWarpThreads) p.lse[b * rows + e] = -INFINITY;
  }

  // -------------------------------------------------------------------- the copies, kWarpStages - 1 steps ahead
  int a_tile = 0, a_hi = 0, a_group = 0, a_key = 0;
  bool a_live = false;         // this lane's key (lanes 0 .. 15) is one of the request's
  int a_page = -1, a_slot = 0;
  bool a_more = true;
  // move to the next tile and ask for the page of this lane's key; used by the next copy
  auto ask = [&] {
    if (a_tile >= a_hi) {
      a_more = paged_next(p, kWarpRows, sm.ahead[warp], sm.ahead_seg[warp], lane);
      if (!a_more) {
        a_live = false;
        return;
      }
      a_tile = sm.ahead_seg[warp].tile_lo;
      a_hi = sm.ahead_seg[warp].tile_hi;
      a_group = sm.ahead_seg[warp].group;
    }
    a_key = a_tile * TN + 16 * warp + (lane & 15);
    ++a_tile;
    a_live = a_key < sm.ahead_seg[warp].L;
    a_page = -1;
    if (a_live) {
      const int k = p.pages.page_shift >= 0 ? a_key >> p.pages.page_shift : a_key / p.pages.page_size;
      a_slot = a_key - k * p.pages.page_size;
      if (k < p.pages.max_pages) a_page = __ldg(p.pages.table + sm.ahead_seg[warp].b * p.pages.table_stride + k);
    }
  };
  // lane 4g + t copies of keys g and g + 8 the 16-byte pieces t (+ 4): 64 contiguous bytes of eight rows at a time
  auto copy = [&](int stage) {
    if (a_more) {
      long long off = -1;
      if (a_live) {
        if (a_page >= 0 && a_page < p.pages.n_pages)
          off = a_page * p.pages.page_stride + a_slot * p.pages.row_stride;
        else if (lane < 16)
          record_error(p.err, LKV_SITE_BAD_ROW);
      }
      const uint32_t base = ring + stage * Cfg::kStage;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const long long at = __shfl_sync(0xffffffffu, off, g + 8 * k);
        const uint8_t* row = p.pages.pool + (at < 0 ? 0 : at);
        const int n16 = at < 0 ? 0 : 16;
        const int key = g + 8 * k;
        const uint8_t* cp = row + a_group * (D / 2);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const int c = t + 4 * h;
          cp_async16(base + key * (D / 2) + ((D == 256 ? c ^ (4 * (key & 1)) : c) << 4), cp + 16 * c, n16);
        }
        const uint8_t* kp = row + int4_rope_at(r);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = t + 4 * h;
          cp_async16(base + Cfg::kCodeBytes + Cfg::kScaleBytes + key * 128 + ((c ^ (key & 1)) << 4), kp + 16 * c, n16);
        }
      }
      if (lane < 16) {
        const uint8_t* sp = p.pages.pool + (off < 0 ? 0 : off) + r / 2 + a_group * (D / 16);
        const uint32_t dst = base + Cfg::kCodeBytes + lane * (D / 16);
        if (D == 128)
          cp_async8(dst, sp, off < 0 ? 0 : 8);
        else
          cp_async16(dst, sp, off < 0 ? 0 : 16);
      }
    }
    cp_async_commit();
    if (a_more) ask();
  };
  ask();
#pragma unroll 1
  for (int s = 0; s < kWarpStages - 1; ++s) copy(s);

  // -------------------------------------------------------------------- Q
  // k step s of a 128-column block: columns 32 t + 4 s .. + 3 of rows g and g + 8; of the RoPE part 16 t + 4 s .. + 3
  uint32_t qa[Cfg::kQRegs ? 12 : 1][4];
  auto q_row = [&](const PagedSegment& s, int row) -> long long {
    const int gr = s.row0 + row;
    if (gr >= p.R) return -1;
    const int i = gr >= p.hpg;
    return (static_cast<long long>(s.b) * p.s_q + i) * p.h_q + s.group * p.hpg + (gr - i * p.hpg);
  };
  auto load_q = [&](const PagedSegment& s) {
    if constexpr (Cfg::kQRegs) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const long long row = q_row(s, g + 8 * k);
#pragma unroll
        for (int v = 0; v < 6; ++v) {
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if (row >= 0)
            x = v < 4 ? __ldg(reinterpret_cast<const uint4*>(p.q + row * D + 32 * t) + v)
                      : __ldg(reinterpret_cast<const uint4*>(p.q_rope + row * 64 + 16 * t) + (v - 4));
          qa[2 * v][k] = x.x;
          qa[2 * v][2 + k] = x.y;
          qa[2 * v + 1][k] = x.z;
          qa[2 * v + 1][2 + k] = x.w;
        }
      }
    } else {
      for (int idx = tid; idx < kWarpRows * (D + 64) / 8; idx += kWarpThreads) {
        const int row = idx / ((D + 64) / 8), c = idx % ((D + 64) / 8);
        const long long at = q_row(s, row);
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (at >= 0)
          x = c < D / 8 ? __ldg(reinterpret_cast<const uint4*>(p.q + at * D) + c)
                        : __ldg(reinterpret_cast<const uint4*>(p.q_rope + at * 64) + (c - D / 8));
        *reinterpret_cast<uint4*>(qsm + row * Cfg::kQRow + 16 * c) = x;
      }
    }
  };

  uint32_t mask = 0x000f000fu, magic = 0x43004300u;
  asm volatile("" : "+r"(mask), "+r"(magic));
  int step = 0;
  bool have = paged_next(p, kWarpRows, sm.walk[warp], sm.seg[warp], lane);
  if (have) load_q(sm.seg[warp]);
  while (have) {
    const PagedSegment sg = sm.seg[warp];
    if (!Cfg::kQRegs) __syncthreads();  // the unit's Q is in shared memory
    const uint32_t qbase = smem_u32(qsm);
    float o[16 * H][4];
#pragma unroll
    for (int i = 0; i < 16 * H; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float ref0 = 0.f, ref1 = 0.f, l0 = 0.f, l1 = 0.f;  // of rows g and g + 8, this thread's keys
    const int lim0 = sg.L - p.s_q;                      // query i sees keys 0 .. lim0 + i
    const int late0 = sg.row0 + g >= p.hpg, late1 = sg.row0 + g + 8 >= p.hpg;  // which query the rows are of
    for (int tile = sg.tile_lo; tile < sg.tile_hi; ++tile, ++step) {
      cp_async_wait<kWarpStages - 2>();
      __syncwarp();  // the step's rows have landed, and every lane is done with the stage that is copied into next
      copy((step + kWarpStages - 1) % kWarpStages);
      const int key0 = tile * TN + 16 * warp;
      if (key0 >= sg.L) continue;
      const uint32_t base = ring + (step % kWarpStages) * Cfg::kStage;
      // ---- expand and QK
      float s[2][4] = {};
      uint32_t kv[H][2][16];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        const int key = 8 * nb + g;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const int c = t + 4 * h;
          const uint4 v = lds16(base + key * (D / 2) + ((D == 256 ? c ^ (4 * (key & 1)) : c) << 4));
          const uint32_t s2 = lds2(base + Cfg::kCodeBytes + key * (D / 16) + 2 * c) * 0x10001u;
          const __nv_bfloat162 sc = *reinterpret_cast<const __nv_bfloat162*>(&s2);
          const __nv_bfloat162 off = __hmul2(sc, __float2bfloat162_rn(-136.f));
          const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4 x = int4_expand(word[e], mask, magic, sc, off);
            kv[h][nb][4 * e] = x.x, kv[h][nb][4 * e + 1] = x.y, kv[h][nb][4 * e + 2] = x.z, kv[h][nb][4 * e + 3] = x.w;
          }
        }
      }
      uint32_t kr[2][8];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        const int key = 8 * nb + g;
        const uint32_t kb = base + Cfg::kCodeBytes + Cfg::kScaleBytes + key * 128;
        const uint4 x = lds16(kb + (((2 * t) ^ (key & 1)) << 4)), y = lds16(kb + (((2 * t + 1) ^ (key & 1)) << 4));
        kr[nb][0] = x.x, kr[nb][1] = x.y, kr[nb][2] = x.z, kr[nb][3] = x.w;
        kr[nb][4] = y.x, kr[nb][5] = y.y, kr[nb][6] = y.z, kr[nb][7] = y.w;
      }
#pragma unroll
      for (int v = 0; v < 4 * H + 2; ++v) {  // two k steps each
        uint32_t a[2][4];
        if constexpr (Cfg::kQRegs) {
#pragma unroll
          for (int k = 0; k < 4; ++k) a[0][k] = qa[2 * v][k], a[1][k] = qa[2 * v + 1][k];
        } else {
          const int col = v < 4 * H ? 128 * (v >> 2) + 32 * t + 8 * (v & 3) : D + 16 * t + 8 * (v - 4 * H);
          const uint4 x = lds16(qbase + g * Cfg::kQRow + 2 * col), y = lds16(qbase + (g + 8) * Cfg::kQRow + 2 * col);
          a[0][0] = x.x, a[0][2] = x.y, a[1][0] = x.z, a[1][2] = x.w;
          a[0][1] = y.x, a[0][3] = y.y, a[1][1] = y.z, a[1][3] = y.w;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int nb = 0; nb < 2; ++nb) {
            const uint32_t b0 = v < 4 * H ? kv[v >> 2 < H ? v >> 2 : 0][nb][4 * (v & 3) + 2 * u] : kr[nb][4 * (v - 4 * H) + 2 * u];
            const uint32_t b1 = v < 4 * H ? kv[v >> 2 < H ? v >> 2 : 0][nb][4 * (v & 3) + 2 * u + 1] : kr[nb][4 * (v - 4 * H) + 2 * u + 1];
            mma16816(s[nb], a[u][0], a[u][1], a[u][2], a[u][3], b0, b1);
          }
        }
      }
      // ---- softmax against the rows' references
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        s[nb][0] = fmaf(s[nb][0], p.sl2, -ref0);
        s[nb][1] = fmaf(s[nb][1], p.sl2, -ref0);
        s[nb][2] = fmaf(s[nb][2], p.sl2, -ref1);
        s[nb][3] = fmaf(s[nb][3], p.sl2, -ref1);
      }
      if (key0 + 15 > lim0) {
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int ahead = key0 + 8 * nb + 2 * t + e - lim0;
            if (ahead > late0) s[nb][e] = -INFINITY;
            if (ahead > late1) s[nb][2 + e] = -INFINITY;
          }
        }
      }
      const bool first = tile == sg.tile_lo;
      const float top0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      const float top1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
      if (first || __any_sync(0xffffffffu, fmaxf(top0, top1) > kPagedRaise)) {
        float m0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 1)), m1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 1));
        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, 2));
        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, 2));
        // a row that sees no key of the first tile sees none of the later ones: its reference stays 0
        const float up0 = first ? (m0 == -INFINITY ? 0.f : m0) : fmaxf(m0, 0.f);
        const float up1 = first ? (m1 == -INFINITY ? 0.f : m1) : fmaxf(m1, 0.f);
        ref0 += up0;
        ref1 += up1;
        if (!first) {
          const float f0 = ex2_approx(-up0), f1 = ex2_approx(-up1);
          l0 *= f0;
          l1 *= f1;
#pragma unroll
          for (int i = 0; i < 16 * H; ++i) o[i][0] *= f0, o[i][1] *= f0, o[i][2] *= f1, o[i][3] *= f1;
        }
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) s[nb][0] -= up0, s[nb][1] -= up0, s[nb][2] -= up1, s[nb][3] -= up1;
      }
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nb][e] = ex2_approx(s[nb][e]);
      }
      l0 += (s[0][0] + s[0][1]) + (s[1][0] + s[1][1]);
      l1 += (s[0][2] + s[0][3]) + (s[1][2] + s[1][3]);
      // the weights are rounded to bf16 as the A operand of PV; l sums them unrounded
      const uint32_t pa0 = pack_bf16x2(s[0][0], s[0][1]), pa1 = pack_bf16x2(s[0][2], s[0][3]);
      const uint32_t pa2 = pack_bf16x2(s[1][0], s[1][1]), pa3 = pack_bf16x2(s[1][2], s[1][3]);
      // ---- PV
#pragma unroll
      for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int i = 0; i < 16; ++i) mma16816(o[16 * h + i], pa0, pa1, pa2, pa3, movmatrix(kv[h][0][i]), movmatrix(kv[h][1][i]));
      }
    }
    // ------------------------------------------------------------------ the segment's end: sum the warps
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (t == 0) {
      sm.m[warp][g] = ref0, sm.m[warp][g + 8] = ref1;
      sm.l[warp][g] = l0, sm.l[warp][g + 8] = l1;
    }
    have = paged_next(p, kWarpRows, sm.walk[warp], sm.seg[warp], lane);
    if (Cfg::kQRegs && have) load_q(sm.seg[warp]);
    __syncthreads();
    if (!Cfg::kQRegs && have) load_q(sm.seg[warp]);  // no warp reads the last unit's any more
    // this thread's row of the sum, and the warps' factors for it
    const int row = tid >> 4, part = tid & 15;
    float m = -INFINITY, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w)
      if (sm.l[w][row] != 0.f) m = fmaxf(m, sm.m[w][row]);
    float f[8];
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float lw = sm.l[w][row];
      f[w] = lw == 0.f ? 0.f : ex2_approx(sm.m[w][row] - m);  // a NaN sum stays one in both results
      lsum += f[w] * lw;
    }
    const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
    const int gr = sg.row0 + row, qi = gr >= p.hpg;
    const bool live = gr < p.R;
    const size_t orow = (static_cast<size_t>(sg.b) * p.s_q + qi) * p.h_q + sg.group * p.hpg + (gr - qi * p.hpg);
    const size_t prow = static_cast<size_t>(2 * range + (sg.slot < 0 ? 0 : sg.slot)) * kWarpRows + row;
    if (live && part == 0) {
      const float lse = lsum == 0.f ? -INFINITY : (m + log2f(lsum)) * 0.69314718055994531f;
      if (sg.slot < 0)
        p.lse[orow] = lse;
      else
        p.part_lse[prow] = lse;
    }
    if (tid == 0 && sg.slot >= 0) p.seg_info[2 * range + sg.slot] = 4 * sg.unit + sg.first + 2 * sg.last;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {  // registers 8 pass .. + 7 of every 128 columns
      if (pass) __syncthreads();
#pragma unroll
      for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float2* dst = sums + (warp * kWarpRows + g) * Cfg::kSumRow + 32 * h + 4 * i + t;
          dst[0] = make_float2(o[16 * h + 8 * pass + i][0], o[16 * h + 8 * pass + i][1]);
          dst[8 * Cfg::kSumRow] = make_float2(o[16 * h + 8 * pass + i][2], o[16 * h + 8 * pass + i][3]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 2 * H; ++e) {
        const int slot = part + 16 * e;  // 4 i + t of block slot / 32
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float2 v = sums[(w * kWarpRows + row) * Cfg::kSumRow + slot];
          a.x = fmaf(f[w], v.x, a.x);
          a.y = fmaf(f[w], v.y, a.y);
        }
        const int col = 128 * (slot >> 5) + 32 * (slot & 3) + 2 * (8 * pass + ((slot & 31) >> 2));
        if (live) {
          if (sg.slot < 0)
            *reinterpret_cast<uint32_t*>(p.out + orow * D + col) = pack_bf16x2(a.x * inv, a.y * inv);
          else
            *reinterpret_cast<float2*>(p.part_o + prow * D + col) = make_float2(a.x * inv, a.y * inv);
        }
      }
    }
  }
  cp_async_wait<0>();
}

}  // namespace lkv
