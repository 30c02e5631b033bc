// Decode attention over paged 4-bit cache rows (lkv_int4.cuh): the tied forms, where the state of a
// group (D columns of the latent) is its key, with the shared RoPE key, and its value.
//
// A unit is a block of at most N query rows (heads of one group times new tokens) of one request.  The
// products are taken with the keys in the MMA's M dimension, since a unit has few rows:
//   S^T[key, row] = K[key, :] . Q[row, :]          M = 128 keys, N rows, K = D + 64 columns
//   O^T[c, row]  += V^T[c, key] . P^T[key, row]    M = 128 value columns (D / 128 blocks), N rows, K = 128 keys
// A 128-key tile costs (D + 64) / 16 + D / 16 MMAs.  With K in tensor memory one takes 16 cycles at N = 32 and 32 at N = 64,
// with both operands in shared memory, as PV's are, 40 and 48 (it reads 4 KB of A): some 570 cycles a tile of the 1900 that
// one takes at D = 128, N = 32.
//
// 4-bit codes are no operand of these MMAs, so converter warps turn each tile into bf16, exactly: (word >> 4i) & 0x000f000f |
// 0x43004300 is a pair of bf16 128 + u, and one fma by the scale s with -136 s (17 x 4 bits: exact) leaves (u - 8) s.  A key
// behind the request's end or without a page gets scales of 0, so that nothing of it reaches PV; the scores behind the end are
// masked, and the RoPE key of a token without a page is zeros.
//
// Softmax in the exp2 domain against a reference per row instead of the running maximum: 16 above the
// first tile's maximum, raised only when some score passes it by 8, so by 24 the maximum it was set to
// (log2 units; a weight's relative precision does not depend on it).  Weights of a row's largest score
// so far lie between 2^-16 and 2^8: a sum of 2^20 of them times values below 2^100, as the cache may
// hold, stays below fp32's 2^128, and the least values, 2^-103, keep their place above 2^-126.  A tile
// then needs no reduction over its keys, only a vote of the softmax warps on whether any score passed.
//
// Warps: 0 QK issuer and TMEM owner, 1 PV issuer, 2 and 3 the copies of codes, scales and RoPE keys (idle where the
// converters load for themselves), 4 to 19 softmax and epilogue (warp w: TMEM lane quadrant w % 4; a thread owns one key of
// the tile, or one value column of O^T), 20 to 27 converters.
//
// What bounds it is neither bytes nor FLOPs but the length of a tile's way through these warps against the tiles that shared
// memory holds: from the copy to PV's end a tile takes about 8000 cycles (of them 1500 for the copy, 1000 for the conversion, 2400
// for the softmax), with three to six tiles on the way.  64 requests of 8192 tokens: 8 groups of 128 with 32 rows 252 us (1.50
// TB/s, 340 TFLOP/s), MLA's 512 columns with 128 rows at half the length 182 us (400 TFLOP/s: a single stage, so conversion and
// products alternate); 8 of 131072 with 2 groups of 256, 64 rows, 229 us (1.91 TB/s, 674 TFLOP/s).
#pragma once
#include <cstdint>
#include <type_traits>
#include <utility>
#include <cuda_bf16.h>
#include "lkv_int4.cuh"
#include "lkv_paged_ptx.cuh"

namespace lkv {

constexpr int kPagedConv = 8;                          // converter warps
constexpr int kPagedSoft = 16;                         // softmax warps
constexpr int kPagedThreads = 32 * (4 + kPagedSoft + kPagedConv);  // issuers, softmax, converters
constexpr int kPagedTile = 128;
constexpr float kPagedShift = 16.f;  // log2 units from a tile's maximum to the reference that it sets
constexpr float kPagedRaise = 8.f;   // log2 units a score may pass its row's reference by

struct PagedDecodeParams {
  Paged pages;
  const __nv_bfloat16* q;       // [B, s_q, h_q, D]
  const __nv_bfloat16* q_rope;  // [B, s_q, h_q, 64]
  int B, s_q, h_q, G, hpg;
  int R;         // rows of a group: s_q * hpg
  int RB;        // row blocks of a group
  int U;         // units of a request: G * RB
  int P;         // ranges (CTAs)
  int unit_cost; // tiles that a unit's start and end count for
  int lockstep;  // the U units of a request run on neighbouring CTAs at the same pace
  float sl2;     // scale * log2(e)
  __nv_bfloat16* out;  // [B, s_q, h_q, D]
  float* lse;          // [B, s_q, h_q]
  int* seg_info;       // [2P] 4 * unit + (1: holds the unit's first tile) + (2: its last); -1: no partial
  float* part_lse;     // [2P][N]
  float* part_o;       // [2P][N][D]
  int* err;
  unsigned long long wait_limit_ns;
  int box_rows;  // rows of a copy: the largest power of two in the page size, 128 at most
};

// The pool as three-dimensional tensors of bytes {row, page_size, n_pages} for the copies of a group's codes, of 16 bytes
// of scales and of the RoPE key (128-byte swizzle), box_rows rows each.
struct PagedMaps {
  CUtensorMap codes, scales, keys;
};

// ------------------------------------------------------------------------------------------
// Work partition.  The tiles of all units, and before a unit's first one the cost of the unit itself (its queries' load and its
// result's store, as unit_cost tiles), are laid end to end (request-major) and cut into P equal ranges; in lockstep the
// requests' are cut into P / U blocks, and range p walks block p / U for unit p % U, so that the units of a request read its RoPE
// keys and scales from L2.  A range is walked as segments, the runs of its tiles that belong to one unit; a segment that is
// not a whole unit leaves a partial (slot 0 the range's first segment, 1 its last).
// ------------------------------------------------------------------------------------------
struct PagedSegment {
  int b, unit, group, row0;  // unit = b * U + u; row0: the unit's first row in its group
  int L, tile_lo, tile_hi;
  int first, last;           // holds the unit's first / last tile
  int slot;                  // partial slot; -1 where the segment is the whole unit
};

__device__ __forceinline__ int paged_tiles_of(int L) { return L / kPagedTile + (L % kPagedTile != 0); }

struct PagedCursor {
  long long t_begin, t_end, t0;  // t0: where unit (b, u) begins
  int b, u, produced;

  __device__ __forceinline__ bool next(const PagedDecodeParams& p, int rows, PagedSegment& s) {
    while (b < p.B && t0 < t_end) {
      const int L = max(0, __ldg(p.pages.seq_lens + b));
      const int nt = paged_tiles_of(L);
      const long long at = t0 + p.unit_cost;  // of the unit's first tile
      const long long lo = t_begin > at ? t_begin - at : 0;
      const long long hi = t_end - at < nt ? t_end - at : nt;
      const int cb = b, cu = u;
      t0 += nt > 0 ? p.unit_cost + nt : 0;
      if (p.lockstep || ++u == p.U) {
        if (!p.lockstep) u = 0;
        ++b;
      }
      if (hi <= lo) continue;
      s.b = cb;
      s.unit = cb * p.U + cu;
      s.group = cu / p.RB;
      s.row0 = (cu - s.group * p.RB) * rows;
      s.L = L;
      s.tile_lo = static_cast<int>(lo);
      s.tile_hi = static_cast<int>(hi);
      s.first = lo == 0;
      s.last = hi == nt;
      s.slot = s.first && s.last ? -1 : (produced == 0 ? 0 : 1);
      ++produced;
      return true;
    }
    return false;
  }
};

// What a unit of request b counts for.
__device__ __forceinline__ long long paged_cost(const PagedDecodeParams& p, int b) {
  const int nt = b < p.B ? paged_tiles_of(max(0, __ldg(p.pages.seq_lens + b))) : 0;
  return nt > 0 ? p.unit_cost + nt : 0;
}

// Start of range `range`; called by one full warp.
__device__ __forceinline__ PagedCursor paged_locate(const PagedDecodeParams& p, int range, int lane) {
  const int mult = p.lockstep ? 1 : p.U;
  long long total = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) total += paged_cost(p, b0 + lane);
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  total *= mult;
  const int n = p.lockstep ? p.P / p.U : p.P, k = p.lockstep ? range / p.U : range;
  PagedCursor c;
  c.t_begin = total * k / n;
  c.t_end = total * (k + 1) / n;
  c.produced = 0;
  c.u = p.lockstep ? range % p.U : 0;
  c.b = p.B;
  c.t0 = total;
  long long acc = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const long long t = paged_cost(p, b0 + lane) * mult;
    long long incl = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, acc + incl > c.t_begin);
    if (hit) {
      const int l0 = __ffs(hit) - 1;
      c.b = b0 + l0;
      c.t0 = acc + __shfl_sync(0xffffffffu, incl - t, l0);
      const long long per = __shfl_sync(0xffffffffu, t, l0) / mult;
      if (!p.lockstep) {
        c.u = static_cast<int>((c.t_begin - c.t0) / per);
        c.t0 += c.u * per;
      }
      break;
    }
    acc += __shfl_sync(0xffffffffu, incl, 31);
  }
  return c;
}

// ------------------------------------------------------------------------------------------
// kTma: codes, scales and RoPE keys come by TMA into a ring of raw tiles; else the converters load them themselves.
template <int D, int N, bool kTma>
struct PagedCfg {
  static_assert(!kTma || D <= 256, "no shared memory for raw tiles");
  static constexpr int kBox = kPagedTile * 128;  // 128 keys x 64 bf16, 128-byte swizzle
  static constexpr int kVBoxes = D / 64;
  static constexpr int kVStage = kVBoxes * kBox;  // the state in shared memory: the value operand
  // QK takes the state from TMEM where that has the columns (an MMA with both operands in shared memory reads 4 KB of
  // A there, 32 cycles of its bandwidth; from TMEM it runs at the tensor core's rate, 16 cycles at N = 32; GTA 385 -> 378 us,
  // not measured apart at d = 256), else from the value operand's tile.
  static constexpr bool kTS = D <= 256;
  // QK reads the RoPE key from the raw tile (the copy leaves it as an MMA wants it) where the ring is deep enough to hold
  // the tile that long, else the converters put it into TMEM.
  static constexpr bool kKeyRaw = kTma && D == 128;
  static constexpr bool kWide = kTma && D == 256;  // codes in rows of 128 bytes, which the copy swizzles
  // Converters: two groups that take turns at the tiles with 32 keys a warp, or one with 16 keys a warp of every tile.  A warp's
  // tile is a chain of waits, reads, stores and fences whose length hardly depends on the keys (GTA 273 -> 252 us).
  static constexpr int kTurns = kTma && D == 128 ? 2 : 1;
  static constexpr int kCW = kPagedConv / kTurns;  // warps of a group
  static constexpr int kKCols = (kTS ? D / 2 : 0) + (kKeyRaw ? 0 : 32);  // TMEM columns of a stage: the key operand
  static constexpr int kStages = D == 128 ? 3 : D == 256 ? 2 : 1;
  // Where a tile is converted in one pass, stages are handed on in blocks of 128 columns: QK starts on the first columns while the
  // rest is converted, and the next tile's conversion while PV runs over the last columns (MLA 224 -> 218 us).  In two passes
  // the barriers cost more than that gives (each some 200 cycles of a converter's way; GLA-2 232 us with blocks, 229 us without).
  static constexpr int kBlocks = kTma ? 1 : D / 128;
  // K and V of a tile in two passes over its codes: K's TMEM is free once QK is done, long before PV leaves V's shared memory, so
  // that the next tile's QK and softmax do not wait for it (GTA 268 -> 252 us, GLA-2 250 -> 229 us).
  static constexpr bool kSplit = kTma;
  static constexpr int kRaws = !kTma ? 1 : D == 256 ? (N == 16 ? 2 : 1) : N == 64 ? 2 : 3;  // raw tiles
  static constexpr int kCodeBytes = kPagedTile * (D / 2), kScaleBytes = kPagedTile * 16;
  static constexpr int kRawBytes = kTma ? kBox + kCodeBytes + kScaleBytes : 0;  // RoPE keys, codes, scales
  // Softmax: sets of four warps, one for each TMEM lane quadrant, with kRW rows each; at N <= 32 two groups of two sets
  // take turns at the tiles, each with accumulators, references and sums of its own, joined at the segment's end (a
  // group is bound by the latency of its chain of instructions, not by their number).
  static constexpr int kGroups = N == 64 ? 1 : 2;
  static constexpr int kGW = kPagedSoft / kGroups;  // warps of a group
  static constexpr int kRW = 4 * N / kGW;           // rows of a softmax warp
  static constexpr int kSBufs = D == 256 && N == 64 ? 1 : 2;  // S^T buffers
  static constexpr int kPs = N == 64 && (D == 512 || (D == 256 && kTma)) ? 1 : 2;  // P buffers
  static constexpr int kQBox = N * 128;
  static constexpr int kQBytes = (kVBoxes + 1) * kQBox;
  static constexpr int kPBytes = kPagedTile * N * 2;
  static constexpr int kMB = D / 128;            // M blocks of PV
  static constexpr uint32_t kO0 = kSBufs * N, kK0 = (kO0 + kGroups * kMB * N + 31) / 32 * 32;  // TMEM: S^T buffers, O^T, key stages
  static constexpr int kTmemNeed = kK0 + kStages * kKCols;
  static constexpr int kTmemCols = kTmemNeed <= 128 ? 128 : kTmemNeed <= 256 ? 256 : 512;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kVStage + static_cast<size_t>(kRaws) * kRawBytes + kQBytes + kPs * kPBytes;
  static_assert(kTmemNeed <= 512, "TMEM budget");
};

constexpr int kPagedSite = LKV_SITE_WAIT_BASE + 300;  // wait sites of this kernel
enum PagedWaitSite { PW_EMPTY = 1, PW_RAW, PW_RAWFREE, PW_FULL, PW_VFULL, PW_KFREE, PW_SFREE, PW_QREADY, PW_PFULL, PW_OFREE, PW_SFULL, PW_ODONE, PW_VOTE, PW_XCHG, PW_FIN, PW_DRAIN };

template <int RW, int N, int NG, int NC, int FULL, int RD>
struct __align__(16) PagedSmem {
  uint64_t full[FULL], v_full[FULL], empty[FULL], k_free[3];  // of a stage's block; of a stage
  uint64_t raw_full[2 * RD], raw_free[RD];  // two a raw tile, for its uses in turn: a group may wait a use ahead of the other's
  uint64_t s_full[2], s_free[2], p_full[2], o_done[2];
  uint64_t vote_bar[2], xchg_bar[2];  // of a softmax group
  uint64_t q_ready, o_free, fin_bar, drain;
  alignas(16) float red[2][kPagedSoft][RW];  // [buffer][softmax warp][its row]
  alignas(16) float ref[kPagedSoft][RW];     // per softmax warp: its rows' references (log2 units)
  alignas(16) float fin_m[2][NG][N], fin_l[2][NG][N];  // [segment parity][group][row]: reference and sum at the segment's end
  alignas(16) float fac[kPagedSoft][NG][RW];  // per softmax warp: what the references rose by; then the groups' factors
  uint32_t vote[2][3];
  alignas(16) uint8_t state[RD][kPagedTile];  // of a raw tile's keys: PagedKeyState
  uint32_t tmem_base, abort;
  int tiles;  // of the range
  // Walk state of the warps that run out of registers first: read where it is needed.
  PagedCursor cur, walk[kPagedSoft + NC];  // NC: the converters, or the two warps that copy for them
  PagedSegment seg[kPagedSoft][2], conv_seg[NC];
};

// A key of a raw tile: a row that was copied, a token without a page, or behind the request's end; with the group's lowest
// bit above, which says where in the 16 bytes of scales the group's are.
enum PagedKeyState { PK_ROW = 0, PK_NO_PAGE = 1, PK_END = 2, PK_ODD_GROUP = 4 };

// The next segment of a warp's own walk, both in shared memory; the same answer in every lane.
__device__ __noinline__ bool paged_next(const PagedDecodeParams& p, int rows, PagedCursor& walk, PagedSegment& out, int lane) {
  int ok = 0;
  __syncwarp();
  if (lane == 0) ok = walk.next(p, rows, out);
  __syncwarp();
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// The wait on a phase that one test did not find complete.  It gives up after a limit, records the site and sets the
// block's abort flag; every later wait of the block then returns at once and its work runs on garbage, in bounds, to
// its end, which keeps a test of each wait's outcome out of the loops.
__device__ __noinline__ void paged_wait_slow(uint32_t bar, uint32_t parity, volatile uint32_t* abort, int* err, uint64_t limit_ns, int site) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1; !mbar_sleep_test(bar, parity); ++it) {
    if (*abort) return;
    if ((it & 15u) == 0 && globaltimer_ns() - t0 > limit_ns) {
      record_error(err, site);
      *abort = 1u;
    }
  }
}

// Key k's row in the value tile and in P^T where K is in TMEM: bits 1, 2, 3 of k move to 2, 3, 1.  The lanes that expand
// keys g and g + 8 then write different 16-byte columns of the swizzled rows.
__device__ __forceinline__ int paged_key_row(int k) { return (k & ~14) | ((k >> 2) & 2) | ((k & 6) << 1); }

// The raw tile's row of the key in TMEM lane k: where the converters read 128-byte rows of codes and of RoPE keys, bits 0, 1, 2,
// 3 of k move to 1, 0, 3, 2, so that eight neighbouring lanes read eight different 16-byte columns of the swizzled rows.
template <bool kWide>
__device__ __forceinline__ int paged_raw_row(int k) {
  return kWide ? (k & ~15) | ((k >> 1) & 5) | ((k << 1) & 10) : k;
}

template <int RW>
__device__ __forceinline__ void tmem_load_rows(uint32_t taddr, float (&v)[RW]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  static_assert(RW == 16 || RW == 8, "rows of a softmax warp");
  if constexpr (RW == 16) {
    tmem_ld16(taddr, reinterpret_cast<uint32_t(&)[16]>(*r));
  } else {
    tmem_ld8(taddr, reinterpret_cast<uint32_t(&)[8]>(*r));
  }
}
template <int RW>
__device__ __forceinline__ void tmem_store_rows(uint32_t taddr, const float (&v)[RW]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  if constexpr (RW == 16) {
    tmem_st16(taddr, reinterpret_cast<const uint32_t(&)[16]>(*r));
  } else {
    tmem_st8(taddr, reinterpret_cast<const uint32_t(&)[8]>(*r));
  }
}

// Sum RW values (rows) of every lane over the warp's lanes: lane l ends with row l % RW.
template <int RW>
__device__ __forceinline__ float paged_rows_sum(float (&v)[RW], int lane) {
#pragma unroll
  for (int s = RW / 2; s >= 1; s >>= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int j = 0; j < s; ++j) {
      const float got = __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j + s], s);
      v[j] = (up ? v[j + s] : v[j]) + got;
    }
  }
  float x = v[0];
#pragma unroll
  for (int s = RW; s < 32; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  return x;
}

// Loads at a constant offset.  Volatile: the compiler keeps them where they are, ahead of the waits that their
// latency is to overlap.
template <int kAt>
__device__ __forceinline__ uint4 ldg16(const uint8_t* ptr) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4+%5];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(ptr), "n"(kAt));
  return v;
}
__device__ __forceinline__ uint2 ldg8(const uint8_t* ptr) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(ptr));
  return v;
}
__device__ __forceinline__ void prefetch_l2(const uint8_t* ptr) { asm volatile("prefetch.global.L2 [%0];" ::"l"(ptr)); }

template <class F, int... I>
__device__ __forceinline__ void static_for_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int kN, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_of(f, std::make_integer_sequence<int, kN>{});
}

// ------------------------------------------------------------------------------------------
// The softmax warps' rare work, out of line: inlined, its registers spilled the loop's over every tile (a spill's
// reload misses an L1 that streams codes, and cost the loop more than half of its time).
// ------------------------------------------------------------------------------------------
// A segment's Q as the K-major B operand, rows behind the group's last as zeros.  The columns follow what the converters
// put into TMEM: register j of half h of a 128-column block is columns 32 (h + 2m) + 8e + 2i with j = 16m + 4e + i, of the
// RoPE key 8 (h + 2m) + 2i with j = 4m + i, and a 16-byte piece p holds j = 2p and 2p + 1, each for h = 0 and 1.
template <int D, int N, bool kTma>
__device__ __noinline__ void paged_load_q(const PagedDecodeParams& p, const PagedSegment& s, uint8_t* qsm, int first, int step) {
  constexpr int kC = (D + 64) / 8;
#pragma unroll 2
  for (int idx = first; idx < N * kC; idx += step) {
    const int row = idx / kC, piece = idx % kC;
    const int bx = piece >> 3, cc = piece & 7, g = s.row0 + row;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (g < p.R) {
      const int i = g >= p.hpg;
      const size_t qrow = (static_cast<size_t>(s.b) * p.s_q + i) * p.h_q + s.group * p.hpg + (g - i * p.hpg);
      const __nv_bfloat16* q = p.q + qrow * D;
      if (piece >= D / 8 && PagedCfg<D, N, kTma>::kKeyRaw) {
        x = __ldg(reinterpret_cast<const uint4*>(p.q_rope + qrow * 64) + cc);
      } else if (piece >= D / 8) {
        const uint32_t* k = reinterpret_cast<const uint32_t*>(p.q_rope + qrow * 64) + 8 * (cc >> 1) + 2 * (cc & 1);
        x = make_uint4(__ldg(k), __ldg(k + 4), __ldg(k + 1), __ldg(k + 5));
      } else if (PagedCfg<D, N, kTma>::kTS) {
        const int j = piece & 15;
        const uint32_t* k = reinterpret_cast<const uint32_t*>(q) + 64 * (piece >> 4) + 32 * (j >> 3) + 4 * ((j >> 1) & 3) + 2 * (j & 1);
        x = make_uint4(__ldg(k), __ldg(k + 16), __ldg(k + 1), __ldg(k + 17));
      } else {
        x = __ldg(reinterpret_cast<const uint4*>(q) + piece);
      }
    }
    *reinterpret_cast<uint4*>(qsm + bx * (N * 128) + row * 128 + ((cc ^ (row & 7)) << 4)) = x;
  }
  fence_proxy_async_smem();
}

// O^T after its rows' references rose by `up`.
template <int RW, int N, int kMB>
__device__ __noinline__ void paged_rescale(uint32_t tmem, const float* up) {
#pragma unroll 1
  for (int mb = 0; mb < kMB; ++mb) {
    float o[RW];
    tmem_load_rows<RW>(tmem + N * mb, o);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < RW; ++j) o[j] *= ex2_approx(-up[j]);
    tmem_store_rows<RW>(tmem + N * mb, o);
  }
  tmem_wait_st();
}

// The groups' O^T times their factors, summed: the result, or the range's partial.  tmem: the first of this warp's rows
// in group 0's accumulators; used: bit g set where group g had a tile; c: this thread's value column of an M block.
template <int D, int N, int RW>
__device__ __noinline__ void paged_store_out(const PagedDecodeParams& p, const PagedSegment& s, uint32_t tmem, const float* fac, int used,
                                             int rb, int c, size_t part) {
  const int n = min(RW, p.R - (s.row0 + rb));
  const size_t row0 = static_cast<size_t>(s.b) * p.s_q * p.h_q + s.group * p.hpg;
#pragma unroll 1
  for (int mb = 0; mb < D / 128; ++mb, c += 128) {
    float o[RW];
#pragma unroll
    for (int j = 0; j < RW; ++j) o[j] = 0.f;
#pragma unroll 1
    for (int g = 0; g < 2; ++g) {
      if (!(used >> g & 1)) continue;
      float v[RW];
      tmem_load_rows<RW>(tmem + N * (D / 128 * g + mb), v);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < RW; ++j) o[j] = fmaf(v[j], fac[RW * g + j], o[j]);
    }
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      if (j >= n) break;
      const int g = s.row0 + rb + j;
      if (s.slot < 0)
        p.out[(row0 + (g >= p.hpg ? p.h_q + g - p.hpg : g)) * D + c] = __float2bfloat16_rn(o[j]);
      else
        p.part_o[(part + rb + j) * D + c] = o[j];
    }
  }
}

template <int D, int N, bool kTma>
__global__ void __launch_bounds__(kPagedThreads, 1) paged_decode_kernel(const __grid_constant__ PagedDecodeParams p,
                                                                           const __grid_constant__ PagedMaps maps) {
  using Cfg = PagedCfg<D, N, kTma>;
  constexpr int TN = kPagedTile, ST = Cfg::kStages, BL = Cfg::kBlocks, SS = Cfg::kSBufs, PS = Cfg::kPs;
  constexpr int RW = Cfg::kRW, MB = Cfg::kMB, NG = Cfg::kGroups, GW = Cfg::kGW;
  constexpr int kBox = Cfg::kBox;
  constexpr uint32_t O0 = Cfg::kO0, K0 = Cfg::kK0;

  extern __shared__ __align__(1024) uint8_t paged_smem_raw[];
  constexpr int RD = Cfg::kRaws;
  __shared__ PagedSmem<RW, N, NG, kTma ? 2 : kPagedConv, ST * BL, RD> sm;
  static_assert(Cfg::kSmem + sizeof(sm) <= 232448, "shared memory budget");
  uint8_t* dsm = paged_smem_raw + ((1024u - (smem_u32(paged_smem_raw) & 1023u)) & 1023u);
  uint8_t* raw = dsm + ST * Cfg::kVStage;
  uint8_t* qsm = raw + RD * Cfg::kRawBytes;
  uint8_t* psm = qsm + Cfg::kQBytes;
  const uint32_t v_base = smem_u32(dsm), raw_base = smem_u32(raw), q_base = smem_u32(qsm), p_base = smem_u32(psm);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int range = blockIdx.x;

  if (tid == 0) {
    for (int s = 0; s < ST * BL; ++s) {
      mbar_init(smem_u32(&sm.full[s]), Cfg::kCW);
      mbar_init(smem_u32(&sm.v_full[s]), Cfg::kCW);
      mbar_init(smem_u32(&sm.empty[s]), 1);
    }
    for (int s = 0; s < RD; ++s) {
      mbar_init(smem_u32(&sm.raw_full[2 * s]), 2);  // the two copying warps
      mbar_init(smem_u32(&sm.raw_full[2 * s + 1]), 2);
      mbar_init(smem_u32(&sm.raw_free[s]), Cfg::kCW + Cfg::kKeyRaw);  // the converters' reads, and QK
    }
    for (int s = 0; s < 3; ++s) {
      mbar_init(smem_u32(&sm.k_free[s]), 1);
      sm.vote[0][s] = sm.vote[1][s] = 0;
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sm.s_full[b]), 1);
      mbar_init(smem_u32(&sm.s_free[b]), GW);
      mbar_init(smem_u32(&sm.p_full[b]), GW);
      mbar_init(smem_u32(&sm.o_done[b]), 1);
      mbar_init(smem_u32(&sm.vote_bar[b]), GW);
      mbar_init(smem_u32(&sm.xchg_bar[b]), GW);
    }
    mbar_init(smem_u32(&sm.q_ready), GW);
    mbar_init(smem_u32(&sm.o_free), GW);  // the warps of group 0, which store the result
    mbar_init(smem_u32(&sm.fin_bar), kPagedSoft);
    mbar_init(smem_u32(&sm.drain), 2);  // one commit from each issuer
    sm.abort = 0;
    p.seg_info[2 * range] = -1;
    p.seg_info[2 * range + 1] = -1;
    fence_mbar_init();
  }
  if (warp == 4) {
    PagedCursor c = paged_locate(p, range, lane);
    if (lane == 0) {
      sm.cur = c;
      PagedSegment s;
      int tiles = 0;
      while (c.next(p, N, s)) tiles += s.tile_hi - s.tile_lo;
      sm.tiles = tiles;
    }
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&sm.tmem_base), Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0) griddep_launch_dependents();  // the combine may start launching
  const uint32_t tbase = sm.tmem_base;
  auto wait = [&](uint64_t& bar, int phase, int site) {
    const uint32_t a = smem_u32(&bar), par = static_cast<uint32_t>(phase & 1);
    if (!mbar_test(a, par)) paged_wait_slow(a, par, &sm.abort, p.err, p.wait_limit_ns, kPagedSite + site);
  };
  auto raw_full = [&](int n) -> uint64_t& { return sm.raw_full[2 * (n % RD) + (n / RD & 1)]; };  // tile n's, in its phase n / 2RD
  auto warp_arrive = [&](uint64_t& bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bar));
  };

  if (warp < 2) {
    // ================================================================== MMA issuers
    if (elect_one()) {
      PagedCursor cur = sm.cur;
      PagedSegment sg;
      int n = 0, seg = 0;
      auto aborted = [&] { return *const_cast<volatile uint32_t*>(&sm.abort) != 0; };
      if (warp == 0) {
        // A = the key tile (the state in TMEM or, for D = 512, in shared memory, the RoPE key the other way about), B = Q
        const uint32_t id = idesc_bf16(128, N, 0, 0);
        const uint64_t qdesc = sdesc_sw128(q_base, 16, 1024);
        for (; cur.next(p, N, sg) && !aborted(); ++seg) {
          for (int t = sg.tile_lo; t < sg.tile_hi; ++t, ++n) {
            const int sb = n % SS, st = n % ST;
            wait(sm.full[st * BL], n / ST, PW_FULL);
            if (n >= SS) wait(sm.s_free[sb], n / SS - 1, PW_SFREE);
            if (t == sg.tile_lo) wait(sm.q_ready, seg, PW_QREADY);
            if (aborted()) break;
            tc_fence_after();
            const uint32_t ktm = tbase + K0 + st * Cfg::kKCols;
            const uint64_t kdesc = sdesc_sw128(v_base + st * Cfg::kVStage, 16, 1024);
            const int rw = n % RD;
            const uint64_t rdesc = sdesc_sw128(raw_base + rw * Cfg::kRawBytes, 16, 1024);
            if (Cfg::kKeyRaw) wait(raw_full(n), n / (2 * RD), PW_RAW);
#pragma unroll
            for (int ks = 0; ks < (D + 64) / 16; ++ks) {
              constexpr int kStep = D / 16 / BL;  // MMAs of a block
              if (BL > 1 && ks > 0 && ks < D / 16 && ks % kStep == 0) {
                wait(sm.full[st * BL + ks / kStep], n / ST, PW_FULL);
                tc_fence_after();
              }
              const uint64_t qd = desc_add(qdesc, (ks >> 2) * Cfg::kQBox + (ks & 3) * 32);
              if (ks < D / 16) {
                if (Cfg::kTS)
                  umma_ts(tbase + N * sb, ktm + 8 * ks, qd, id, ks ? 1u : 0u);
                else
                  umma_ss(tbase + N * sb, desc_add(kdesc, (ks >> 2) * kBox + (ks & 3) * 32), qd, id, ks ? 1u : 0u);
              } else if (Cfg::kKeyRaw) {
                umma_ss(tbase + N * sb, desc_add(rdesc, (ks & 3) * 32), qd, id, 1u);
              } else {
                umma_ts(tbase + N * sb, ktm + 8 * (Cfg::kTS ? ks : ks - D / 16), qd, id, 1u);
              }
            }
            if (Cfg::kKeyRaw) umma_commit(smem_u32(&sm.raw_free[rw]));
            if (Cfg::kSplit) umma_commit(smem_u32(&sm.k_free[st]));
            umma_commit(smem_u32(&sm.s_full[sb]));
          }
        }
      } else {
        // A = the value tile read MN-major (two 64-column boxes an M block, LBO between them), B = P^T, MN-major: 8-key
        // atoms of 8 * 2N bytes, swizzled over the 2N bytes of a key's rows.  The stage is free when PV is done.
        const uint32_t id = idesc_bf16(128, N, 1, 1);
        constexpr uint32_t atom = 16 * N;
        for (; cur.next(p, N, sg) && !aborted(); ++seg) {
          for (int t = sg.tile_lo; t < sg.tile_hi; ++t, ++n) {
            const int pb = n % PS, st = n % ST;
            const bool first = t - sg.tile_lo < NG;  // the group's first tile of the segment
            const uint32_t od = tbase + O0 + (n % NG) * (MB * N);
            wait(sm.p_full[pb], n / PS, PW_PFULL);
            if (t == sg.tile_lo && seg > 0) wait(sm.o_free, seg - 1, PW_OFREE);
            if (aborted()) break;
            tc_fence_after();
            const uint32_t paddr = p_base + pb * Cfg::kPBytes;
            const uint64_t pdesc = N == 64 ? sdesc_sw128(paddr, 16, atom) : N == 32 ? sdesc_sw64(paddr, 16, atom) : sdesc_sw32(paddr, 16, atom);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
              constexpr int kOf = MB / BL;  // M blocks of a stage's block
              if (Cfg::kSplit && mb % kOf == 0) {
                wait(sm.v_full[st * BL + mb / kOf], n / ST, PW_VFULL);
                tc_fence_after();
              }
              const uint64_t vdesc = sdesc_sw128(v_base + st * Cfg::kVStage + 2 * mb * kBox, kBox, 1024);
#pragma unroll
              for (int kk = 0; kk < TN / 16; ++kk)
                umma_ss(od + N * mb, desc_add(vdesc, kk * 2048), desc_add(pdesc, kk * 2 * atom), id, first && kk == 0 ? 0u : 1u);
              if (BL == MB && mb + 1 < MB) umma_commit(smem_u32(&sm.empty[st * BL + mb]));
            }
            umma_commit(smem_u32(&sm.o_done[pb]));
            umma_commit(smem_u32(&sm.empty[st * BL + BL - 1]));
          }
        }
      }
      // every MMA of this thread is complete before TMEM is released (both issuers arrive)
      umma_commit(smem_u32(&sm.drain));
      uint32_t zero = 0;
      const WaitCtl dc{&zero, p.err, p.wait_limit_ns};
      mbar_wait(smem_u32(&sm.drain), 0, dc, kPagedSite + PW_DRAIN);
    }
  } else if (warp < 4) {
    // ================================================================== copies
    // A tile's rows in boxes of box_rows within one page, a lane a box; a box that lies behind the request's end or has no
    // page is not copied.  Warp 2 copies the RoPE keys, warp 3 codes and scales: the copies of a warp's lanes are issued
    // one after the other, and their sum is on the way of every tile.
    if constexpr (kTma) {
      PagedCursor& walk = sm.walk[kPagedSoft + warp - 2];
      PagedSegment& seg = sm.conv_seg[warp - 2];
      if (lane == 0) walk = sm.cur;
      struct Tile {
        int t, L, group;  // t < 0: none
        const int* table;
      };
      int walk_t = 0, walk_hi = 0;
      auto next_tile = [&]() -> Tile {
        if (walk_t >= walk_hi) {
          if (!paged_next(p, N, walk, seg, lane)) return Tile{-1, 0, 0, nullptr};
          walk_t = seg.tile_lo;
          walk_hi = seg.tile_hi;
        }
        return Tile{walk_t++, seg.L, seg.group, p.pages.table + seg.b * p.pages.table_stride};
      };
      const int r = p.G * D, rows = p.box_rows, at = lane * rows;
      const int key_at = int4_rope_at(r);
      // the page of this lane's box of a tile, -1 where it holds no token or has none, and the box's slot there
      auto find = [&](const Tile& x, int& slot) -> int {
        const int key = x.t * TN + at;
        if (x.t < 0 || at >= TN || key >= x.L) return -1;
        const int k = p.pages.page_shift >= 0 ? key >> p.pages.page_shift : key / p.pages.page_size;
        slot = key - k * p.pages.page_size;
        return k < p.pages.max_pages ? __ldg(x.table + k) : -1;
      };
      int n = 0, slot = 0;
      Tile x = next_tile();
      int page = find(x, slot);
      for (; x.t >= 0; ++n) {
        // the next tile's pages are asked for ahead of this one's wait
        const Tile y = next_tile();
        int slot_y = 0;
        const int page_y = find(y, slot_y);
        const int rw = n % RD;
        const uint32_t bar = smem_u32(&raw_full(n)), dst = raw_base + rw * Cfg::kRawBytes;
        const int code_at = x.group * (D / 2), scale_at = r / 2 + (x.group * (D / 16) & ~15);
        if (page >= p.pages.n_pages) page = -1;
        const unsigned some = __ballot_sync(0xffffffffu, page >= 0);
        uint32_t states = 0;  // of four keys
        if (warp == 2) {
          if (page < 0 && at < TN && x.t * TN + at < x.L) record_error(p.err, LKV_SITE_BAD_ROW);
          const int state = (some >> (4 * lane / rows) & 1 ? PK_ROW : PK_NO_PAGE) | (x.group & 1 ? PK_ODD_GROUP : 0);
          const int left = x.L - x.t * TN - 4 * lane;
#pragma unroll
          for (int j = 0; j < 4; ++j) states |= static_cast<uint32_t>(j < left ? state : PK_END) << (8 * j);
        }
        if (n >= RD) wait(sm.raw_free[rw], n / RD - 1, PW_RAWFREE);
        if (__any_sync(0xffffffffu, *const_cast<volatile uint32_t*>(&sm.abort) != 0)) break;
        if (warp == 2) *reinterpret_cast<uint32_t*>(&sm.state[rw][4 * lane]) = states;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(some) * rows * (warp == 2 ? 128 : D / 2 + 16));
        __syncwarp();
        if (page >= 0) {
          if (warp == 2) {
            tma_load_3d(dst + at * 128, &maps.keys, bar, key_at, slot, page);
          } else {
            tma_load_3d(dst + kBox + at * (D / 2), &maps.codes, bar, code_at, slot, page);
            tma_load_3d(dst + kBox + Cfg::kCodeBytes + at * 16, &maps.scales, bar, scale_at, slot, page);
          }
        }
        x = y;
        page = page_y;
        slot = slot_y;
        // with a single raw tile its copies wait for the converters: the rows can come as far as L2 meanwhile (GLA-2 234 -> 229 us)
        if (RD == 1 && page >= 0 && page < p.pages.n_pages) {
          if (warp == 2) {
            tma_prefetch_3d(&maps.keys, key_at, slot, page);
          } else {
            tma_prefetch_3d(&maps.codes, x.group * (D / 2), slot, page);
            tma_prefetch_3d(&maps.scales, r / 2 + (x.group * (D / 16) & ~15), slot, page);
          }
        }
      }
      // no copy may still be on its way when the block exits
      uint32_t zero = 0;
      const WaitCtl dc{&zero, p.err, p.wait_limit_ns};
      for (int m = n > RD ? n - RD : 0; m < n; ++m) mbar_wait(smem_u32(&raw_full(m)), (m / (2 * RD)) & 1, dc, kPagedSite + PW_RAW);
    }
  } else if (warp >= 4 + kPagedSoft) {
    // ================================================================== converters
    // One group (kTurns = 1): warp w takes 16 keys of every tile, lanes 16 (w / 4) .. + 15 of the TMEM quadrant w % 4.  Two
    // groups (2): warp w takes the 32 keys of quadrant w % 4 of every second tile, from tile w / 4 on, as two times 16; a
    // tile's barriers then count the four warps of its group.  Of 16 keys thread 4g + 2h + b has key g + 8b and of it the
    // 32-column chunks h + 2m (m = 0, 1 in every 128 columns) and the 16-byte pieces h + 2m of the RoPE key, which is how
    // tcgen05.st 16x64b spreads a warp's registers; the K index of QK runs through the columns in that order, and Q is
    // stored to match.  Where they load for themselves, the next tile's loads are issued
    // when this one is converted; its rows were asked into L2 a tile earlier, and their page numbers one tile before.
    constexpr int kKeys = 16, kH = D / 128, kHalves = Cfg::kTurns;
    const int cw = warp - (4 + kPagedSoft), turn = kHalves == 2 ? cw >> 2 : 0, key0 = 32 * (cw & 3) + 16 * (kHalves == 2 ? 0 : cw >> 2);
    const int rr = (lane >> 2) + 8 * (lane & 1), hf = (lane >> 1) & 1;
    const int r = p.G * D;
    const uint8_t* pool = p.pages.pool;
    const int key_at = int4_rope_at(r);
    constexpr int kHL = kTma ? kH : 1;  // blocks of codes in registers: where they are loaded here, the next follows as one is used
    uint4 code[kHalves][kHL][2], key[4];
    const uint8_t* codes_at = nullptr;
    uint32_t scale[kHalves][2 * kH];  // of the chunks 2m and 2m + 1
    uint32_t mask = 0x000f000fu, magic = 0x43004300u;
    asm volatile("" : "+r"(mask), "+r"(magic));
    const uint32_t pick = hf ? 0x3232u : 0x1010u;  // this lane's scale of a pair, twice
    // (D = 512) V's rows are QK's too, so a key keeps its row, and the lanes take the keys of the codes in an order that writes
    // different columns of the swizzled rows (MLA 195 -> 183 us)
    const int rc = Cfg::kTS ? rr : 2 * (lane >> 2) + (lane & 1);
    const int vrow = key0 + (Cfg::kTS ? paged_key_row(rr) : rc);
    uint32_t at_word[4];  // where word e of this lane's chunk goes in the value tile
#pragma unroll
    for (int e = 0; e < 4; ++e) at_word[e] = vrow * 128 + (((4 * hf + e) ^ (vrow & 7)) << 4);
    const uint32_t tlane = tbase + K0 + (static_cast<uint32_t>(key0) << 16);
#pragma unroll
    for (int h = 0; h < kHL; ++h) code[0][h][0] = code[0][h][1] = make_uint4(0u, 0u, 0u, 0u);
    // one tile's registers to the value operand (V) and, where QK wants it there, to TMEM (K), in one pass or in two
    auto pass = [&](auto to_k, auto to_v, int n) {
      constexpr bool kK = decltype(to_k)::value, kV = decltype(to_v)::value;
      const int st = n % ST;
      uint8_t* stage = dsm + st * Cfg::kVStage;
      const uint32_t ktm = tlane + st * Cfg::kKCols;
      if (n >= ST) {
        if (kV)
          wait(sm.empty[st * BL], n / ST - 1, PW_EMPTY);
        else
          wait(sm.k_free[st], n / ST - 1, PW_KFREE);
      }
      tc_fence_after();
      if constexpr (kK && !Cfg::kKeyRaw) {
        uint32_t out[16];
#pragma unroll
        for (int m = 0; m < 4; ++m) out[4 * m] = key[m].x, out[4 * m + 1] = key[m].y, out[4 * m + 2] = key[m].z, out[4 * m + 3] = key[m].w;
        tmem_st_16x64_x16(ktm + (Cfg::kTS ? D / 2 : 0), out);
      }
#pragma unroll
      for (int u = 0; u < kHalves * kH; ++u) {
        const int h = u % kH, half = u / kH;  // 128 columns of 16 keys
        if (kV && BL > 1 && h > 0 && n >= ST) {
          wait(sm.empty[st * BL + h], n / ST - 1, PW_EMPTY);
          tc_fence_after();
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t out[16];
          const uint32_t s2 = __byte_perm(scale[half][2 * h + m], 0, pick);
          const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&s2);
          const __nv_bfloat162 o = __hmul2(s, __float2bfloat162_rn(-136.f));
          const uint4 c = code[half][h % kHL][m];
          const uint32_t word[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4 x = int4_expand(word[e], mask, magic, s, o);
            if (kV) *reinterpret_cast<uint4*>(stage + at_word[e] + half * 2048 + (2 * h + m) * kBox) = x;
            out[4 * e] = x.x;
            out[4 * e + 1] = x.y;
            out[4 * e + 2] = x.z;
            out[4 * e + 3] = x.w;
          }
          if (kK && Cfg::kTS) tmem_st_16x64_x16(ktm + (half << 20) + 64 * h + 32 * m, out);
        }
        if (BL > 1 || u == kHalves * kH - 1) {
          if (kK && (Cfg::kTS || h == 0)) tmem_wait_st();
          if (kV) fence_proxy_async_smem();  // ahead of the next global loads: its memory barrier would wait for them
          tc_fence_before();
          warp_arrive((kK ? sm.full : sm.v_full)[st * BL + (BL > 1 ? h : 0)]);
        }
        if (kHL < kH && h + kHL < kH && codes_at) {
          code[half][h % kHL][0] = ldg16<0>(codes_at + 64 * (h + kHL));
          code[half][h % kHL][1] = ldg16<32>(codes_at + 64 * (h + kHL));
        }
      }
    };
    auto convert = [&](int n) {
      if constexpr (Cfg::kSplit) {
        pass(std::true_type{}, std::false_type{}, n);
        // opaque to the compiler, which would keep the first pass's values for the second one, in local memory
#pragma unroll
        for (int u = 0; u < kHalves * kHL * 2; ++u) {
          uint4& c = code[u / (2 * kHL)][u / 2 % kHL][u & 1];
          asm volatile("" : "+r"(c.x), "+r"(c.y), "+r"(c.z), "+r"(c.w));
        }
        pass(std::false_type{}, std::true_type{}, n);
      } else {
        pass(std::true_type{}, std::true_type{}, n);
      }
    };
    if constexpr (kTma) {
      const int tiles = sm.tiles;
      const int raw_row = key0 + paged_raw_row<Cfg::kWide>(rr), x8 = Cfg::kWide ? raw_row & 7 : 0;
      for (int n = turn; n < tiles; n += Cfg::kTurns) {
        const int rw = n % RD;
        uint8_t* tile = raw + rw * Cfg::kRawBytes;
        wait(raw_full(n), n / (2 * RD), PW_RAW);
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
          const int row = raw_row + 16 * half;
          uint8_t* key_row = tile + row * 128;
          const uint8_t* cp = tile + kBox + row * (D / 2);
          const uint8_t* sp = tile + kBox + Cfg::kCodeBytes + row * 16;
          const int state = sm.state[rw][row];
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            code[half][h][0] = *reinterpret_cast<const uint4*>(cp + (((4 * h + hf) ^ x8) << 4));
            code[half][h][1] = *reinterpret_cast<const uint4*>(cp + (((4 * h + 2 + hf) ^ x8) << 4));
          }
          if constexpr (D == 128) {
            const uint2 v = *reinterpret_cast<const uint2*>(sp + (state & PK_ODD_GROUP ? 8 : 0));
            scale[half][0] = v.x, scale[half][1] = v.y;
          } else {
            const uint4 v = *reinterpret_cast<const uint4*>(sp);
            scale[half][0] = v.x, scale[half][1] = v.y, scale[half][2] = v.z, scale[half][3] = v.w;
          }
          if constexpr (!Cfg::kKeyRaw) {
#pragma unroll
            for (int m = 0; m < 4; ++m) key[m] = *reinterpret_cast<const uint4*>(key_row + (((hf + 2 * m) ^ x8) << 4));
          }
          if (state & (PK_NO_PAGE | PK_END)) {  // scales of 0 make any codes zeros; behind the end the scores are not looked at
#pragma unroll
            for (int m = 0; m < 2 * kH; ++m) scale[half][m] = 0;
            if (state & PK_NO_PAGE) {
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                if constexpr (Cfg::kKeyRaw)
                  *reinterpret_cast<uint4*>(key_row + 64 * hf + 16 * m) = make_uint4(0u, 0u, 0u, 0u);
                else
                  key[m] = make_uint4(0u, 0u, 0u, 0u);
              }
              if constexpr (Cfg::kKeyRaw) fence_proxy_async_smem();
            }
          }
        }
        warp_arrive(sm.raw_free[rw]);
        convert(n);
      }
    } else {
      struct Tile {
        int b, t, L, group;  // t < 0: none
      };
      PagedCursor& walk = sm.walk[kPagedSoft + cw];
      PagedSegment& seg = sm.conv_seg[cw];
      if (lane == 0) walk = sm.cur;
      int walk_t = 0, walk_hi = 0;
      auto next_tile = [&]() -> Tile {
        if (walk_t >= walk_hi) {
          if (!paged_next(p, N, walk, seg, lane)) return Tile{0, -1, 0, 0};
          walk_t = seg.tile_lo;
          walk_hi = seg.tile_hi;
        }
        return Tile{seg.b, walk_t++, seg.L, seg.group};
      };
      // this lane's key of a tile (lanes 0 .. 15): the page is asked for here, used a tile later
      int page = -1, slot = 0;
      bool key_live = false;
      auto ask_page = [&](const Tile& x) {
        const int key = x.t * TN + key0 + lane;
        key_live = x.t >= 0 && lane < kKeys && key < x.L;
        page = -1;
        if (key_live) {
          const int k = p.pages.page_shift >= 0 ? key >> p.pages.page_shift : key / p.pages.page_size;
          slot = key - k * p.pages.page_size;
          if (k < p.pages.max_pages) page = __ldg(p.pages.table + x.b * p.pages.table_stride + k);
        }
      };
      auto row_of_page = [&](const Tile& x) -> long long {
        if (!key_live) return -1;
        if (page < 0 || page >= p.pages.n_pages) {
          record_error(p.err, LKV_SITE_BAD_ROW);
          return -1;
        }
        const long long off = page * p.pages.page_stride + slot * p.pages.row_stride;
        const uint8_t* row = pool + off;
        prefetch_l2(row + x.group * (D / 2));
        if (D == 512) prefetch_l2(row + x.group * (D / 2) + 128);
        prefetch_l2(row + key_at);
        return off;
      };
      auto load_rows = [&](long long off, int group) {
        const long long at = __shfl_sync(0xffffffffu, off, rc), key_from = Cfg::kTS ? at : __shfl_sync(0xffffffffu, off, rr);
        const uint8_t* cp = pool + at + (16 * hf + group * (D / 2));
        const uint8_t* sp = pool + at + (r / 2 + group * (D / 16));
        const uint8_t* kp = pool + key_from + (16 * hf + key_at);
        const bool whole = __all_sync(0xffffffffu, at >= 0 && key_from >= 0);
        if (whole || at >= 0) {
          codes_at = cp;
          static_for<kHL>([&](auto h) {
            code[0][h][0] = ldg16<64 * h>(cp);
            code[0][h][1] = ldg16<64 * h + 32>(cp);
          });
          if constexpr (D == 128) {
            const uint2 v = ldg8(sp);
            scale[0][0] = v.x, scale[0][1] = v.y;
          } else {
            static_for<kH / 2>([&](auto h) {
              const uint4 v = ldg16<16 * h>(sp);
              scale[0][4 * h] = v.x, scale[0][4 * h + 1] = v.y, scale[0][4 * h + 2] = v.z, scale[0][4 * h + 3] = v.w;
            });
          }
        } else {  // no token: scales of 0 make any codes zeros, and the key is zeros
          codes_at = nullptr;
#pragma unroll
          for (int m = 0; m < 2 * kH; ++m) scale[0][m] = 0;
        }
        if (whole || key_from >= 0) {
          static_for<4>([&](auto m) { key[m] = ldg16<32 * m>(kp); });
        } else {
#pragma unroll
          for (int m = 0; m < 4; ++m) key[m] = make_uint4(0u, 0u, 0u, 0u);
        }
      };
      Tile now = next_tile();
      ask_page(now);
      long long off_then = row_of_page(now);
      Tile then = Tile{0, -1, 0, 0};
      if (now.t >= 0) {
        load_rows(off_then, now.group);
        then = next_tile();
      }
      ask_page(then);
      off_then = row_of_page(then);
      Tile later = then.t >= 0 ? next_tile() : then;
      ask_page(later);
      for (int n = 0; now.t >= 0; ++n) {
        convert(n);
        if (then.t >= 0) load_rows(off_then, then.group);
        now = then;
        then = later;
        off_then = row_of_page(then);
        if (then.t >= 0) later = next_tile();
        ask_page(later);
      }
    }
  } else if (warp >= 4) {
    // ================================================================== softmax / epilogue
    const int sw = warp - 4;
    const int q4 = warp & 3;                     // TMEM lane quadrant
    const int set = sw >> 2;
    const int grp = NG == 2 ? set >> 1 : 0;                // this warp's group
    const int rb = RW * (NG == 2 ? set & 1 : set);         // rows rb .. rb + RW - 1 of the unit
    const int k = q4 * 32 + lane;                          // key of the tile; value column (of an M block) of O^T
    const int rl = lane % RW;                              // this lane's row, rb + rl, after a reduction over lanes
    const uint32_t tlane = tbase + (static_cast<uint32_t>(q4 * 32) << 16) + rb;
    int xc = 0, vc = 0;
    // every warp posts one value per row (lanes 0 .. RW - 1) and reads the posts of the four warps with its rows
    auto exchange = [&](float v, float (&all)[4]) {
      const int b = xc & 1;
      if (lane < RW) sm.red[b][sw][lane] = v;
      warp_arrive(sm.xchg_bar[grp]);
      wait(sm.xchg_bar[grp], xc, PW_XCHG);
#pragma unroll
      for (int w = 0; w < 4; ++w) all[w] = sm.red[b][4 * set + w][rl];
      ++xc;
    };
    auto load_q = [&](const PagedSegment& s) {
      paged_load_q<D, N, kTma>(p, s, qsm, (sw % GW) * 32 + lane, 32 * GW);
      warp_arrive(sm.q_ready);
    };

    // idle requests: no tile is walked for them
    for (int b = range; b < p.B; b += p.P) {
      if (__ldg(p.pages.seq_lens + b) > 0) continue;
      const size_t rows = static_cast<size_t>(p.s_q) * p.h_q;
      uint4* o = reinterpret_cast<uint4*>(p.out + b * rows * D);
      for (size_t e = sw * 32 + lane; e < rows * D / 8; e += 32 * kPagedSoft) o[e] = make_uint4(0u, 0u, 0u, 0u);
      for (size_t e = sw * 32 + lane; e < rows; e += 32 * kPagedSoft) p.lse[b * rows + e] = -INFINITY;
    }

    // where this key's weights go: 2N bytes a key, 16-byte chunk c at c ^ the swizzle of that width
    const int krow = Cfg::kTS ? paged_key_row(k) : k;
    const int x8 = N == 64 ? (krow & 7) : N == 32 ? ((krow >> 1) & 3) : ((krow >> 2) & 1);
    uint8_t* prow0 = psm + krow * (2 * N);
    PagedCursor& walk = sm.walk[sw];
    if (lane == 0) walk = sm.cur;
    int n0 = 0, seg = 0;  // the tile count at the segment's start
    float l[RW];          // this key lane's share of each row's sum of weights
    bool have = paged_next(p, N, walk, sm.seg[sw][0], lane);
    if (have && grp == 0) load_q(sm.seg[sw][0]);
    for (; have; ++seg) {
      const PagedSegment& sg = sm.seg[sw][seg & 1];
      PagedSegment& nx = sm.seg[sw][(seg + 1) & 1];
      const int tiles = sg.tile_hi - sg.tile_lo;
      const int key = paged_raw_row<Cfg::kWide>(k);
      const int lim0 = sg.L - p.s_q - sg.tile_lo * TN - key;  // query i sees this thread's key of tile j where 128 j <= lim0 + i
      const int whole = lim0 + key - (TN - 1);                // 128 j <= whole: every query sees all keys of the tile
      const int newest = p.hpg - (sg.row0 + rb);            // rows from here on are query 1's (or padding)
      float m_run = 0.f;                                    // reference of row rb + rl (log2 units)
#pragma unroll
      for (int j = 0; j < RW; ++j) l[j] = 0.f;
      const int j0 = NG == 2 ? (n0 ^ grp) & 1 : 0;
      for (int j = j0; j < tiles; j += NG) {
        const int n = n0 + j, sb = n % SS, pb = n % PS;
        const bool first = j == j0;
        wait(sm.s_full[sb], n / SS, PW_SFULL);
        tc_fence_after();
        // the tile's scores, -inf where the row does not see the key
        float x[RW];
        tmem_load_rows<RW>(tlane + N * sb, x);
        tmem_wait_ld();
        tc_fence_before();
        warp_arrive(sm.s_free[sb]);
        if (TN * j > whole) {
          const int ahead = TN * j - lim0;
#pragma unroll
          for (int i = 0; i < RW; ++i)
            if (ahead > (i >= newest ? 1 : 0)) x[i] = -INFINITY;
        }
        bool raise = first;
        if (first) {
#pragma unroll
          for (int i = 0; i < RW; ++i) x[i] *= p.sl2;
        } else {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < RW; i += 4) {
            const float4 r4 = *reinterpret_cast<const float4*>(&sm.ref[sw][i]);
            x[i] = fmaf(x[i], p.sl2, -r4.x);
            x[i + 1] = fmaf(x[i + 1], p.sl2, -r4.y);
            x[i + 2] = fmaf(x[i + 2], p.sl2, -r4.z);
            x[i + 3] = fmaf(x[i + 3], p.sl2, -r4.w);
            top = fmaxf(top, fmaxf(fmaxf(x[i], x[i + 1]), fmaxf(x[i + 2], x[i + 3])));
          }
          // The flag of vote vc is one of three words: it is cleared after vote vc + 1, when every warp has read
          // it, and set again for vote vc + 3 by warps that passed vote vc + 2, which this warp joins after clearing.
          volatile uint32_t* flag = sm.vote[grp];
          if (__any_sync(0xffffffffu, top > kPagedRaise) && lane == 0) flag[vc % 3] = 1u;
          warp_arrive(sm.vote_bar[grp]);
          wait(sm.vote_bar[grp], vc, PW_VOTE);
          raise = flag[vc % 3] != 0;  // the same for all the group's warps
          if (sw % GW == 0 && lane == 0) flag[(vc + 2) % 3] = 0u;
          ++vc;
        }
        if (raise) {
          // the rows' maxima over the tile's keys, above the references (the first tile's references are 0)
          float mw = -INFINITY;
#pragma unroll
          for (int i = 0; i < RW; ++i) {
            const float v = warp_max(x[i]);
            if (rl == i) mw = v;
          }
          float all[4];
          exchange(mw, all);
          const float mt = fmaxf(fmaxf(all[0], all[1]), fmaxf(all[2], all[3])) + kPagedShift;
          // a row that sees no key of the group's first tile sees none of its later ones: its reference stays 0
          const float up = first ? (mt == -INFINITY ? 0.f : mt) : fmaxf(mt, 0.f);
          m_run = first ? up : m_run + up;
          if (lane < RW) {
            sm.ref[sw][lane] = m_run;
            sm.fac[sw][0][lane] = up;
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < RW; ++i) {
            const float u = *const_cast<volatile float*>(&sm.fac[sw][0][i]);
            x[i] -= u;
            l[i] = first ? 0.f : l[i] * ex2_approx(-u);
          }
        }
        uint32_t pw[RW / 2];
#pragma unroll
        for (int i = 0; i < RW / 2; ++i) {
          const float e0 = ex2_approx(x[2 * i]), e1 = ex2_approx(x[2 * i + 1]);
          l[2 * i] += e0;
          l[2 * i + 1] += e1;
          pw[i] = pack_bf16x2(e0, e1);
        }
        // P buffer pb was last read by PV(n - PS), the group's previous tile where the groups take turns
        if (n >= PS) wait(sm.o_done[pb], n / PS - 1, PW_ODONE);
        uint8_t* prow = prow0 + pb * Cfg::kPBytes;
#pragma unroll
        for (int c = 0; c < RW / 8; ++c)
          *reinterpret_cast<uint4*>(prow + ((((rb / 8) + c) ^ x8) << 4)) =
              make_uint4(pw[4 * c], pw[4 * c + 1], pw[4 * c + 2], pw[4 * c + 3]);
        fence_proxy_async_smem();
        if (raise && !first) {
          // O^T holds the group's tiles up to the one before
          if (NG == 1) wait(sm.o_done[(n - 1) % PS], (n - 1) / PS, PW_ODONE);
          tc_fence_after();
          paged_rescale<RW, N, MB>(tlane + O0 + grp * (MB * N), sm.fac[sw][0]);
        }
        tc_fence_before();
        warp_arrive(sm.p_full[pb]);
      }
      // ---------------------------------------------------------------- the segment's end
      const int n_last = n0 + tiles - 1;
      const bool have_nx = paged_next(p, N, walk, nx, lane);
      // the group with the last tile loads Q: that tile's QK, the unit's last, is done
      if (have_nx && grp == (NG == 2 ? n_last & 1 : 0)) load_q(nx);
      float lt[4];
      exchange(paged_rows_sum<RW>(l, lane), lt);
      const int f = seg & 1;
      if (q4 == 0 && lane < RW) {
        sm.fin_m[f][grp][rb + lane] = m_run;
        sm.fin_l[f][grp][rb + lane] = (lt[0] + lt[1]) + (lt[2] + lt[3]);
      }
      warp_arrive(sm.fin_bar);
      wait(sm.fin_bar, seg, PW_FIN);
      if (grp == 0) {
        // out = sum_g 2^(m_g - m) O_g / sum_g 2^(m_g - m) l_g over the groups that saw a key
        const int row = rb + rl;
        const float l0 = sm.fin_l[f][0][row], l1 = NG == 2 ? sm.fin_l[f][NG - 1][row] : 0.f;
        const float m0 = l0 == 0.f ? -INFINITY : sm.fin_m[f][0][row];
        const float m1 = l1 == 0.f ? -INFINITY : sm.fin_m[f][NG - 1][row];
        const float m = fmaxf(m0, m1);
        const float w0 = l0 == 0.f ? 0.f : ex2_approx(m0 - m), w1 = l1 == 0.f ? 0.f : ex2_approx(m1 - m);
        const float sum = w0 * l0 + w1 * l1;  // a NaN stays one in both results
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (lane < RW) {
          sm.fac[sw][0][lane] = w0 * inv;
          if (NG == 2) sm.fac[sw][NG - 1][lane] = w1 * inv;
          const int g = sg.row0 + row;
          if (q4 == 0 && g < p.R) {
            const float lse = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994531f;
            const int i = g >= p.hpg;
            if (sg.slot < 0)
              p.lse[(static_cast<size_t>(sg.b) * p.s_q + i) * p.h_q + sg.group * p.hpg + (g - i * p.hpg)] = lse;
            else
              p.part_lse[static_cast<size_t>(2 * range + sg.slot) * N + row] = lse;
          }
        }
        __syncwarp();
        wait(sm.o_done[n_last % PS], n_last / PS, PW_ODONE);  // the commit covers the MMAs before it too
        tc_fence_after();
        const int used = NG == 1 ? 1 : tiles > 1 ? 3 : 1 << (n_last & 1);
        paged_store_out<D, N, RW>(p, sg, tlane + O0, &sm.fac[sw][0][0], used, rb, k,
                                  static_cast<size_t>(2 * range + (sg.slot < 0 ? 0 : sg.slot)) * N);
        if (sg.slot >= 0 && sw == 0 && lane == 0) p.seg_info[2 * range + sg.slot] = 4 * sg.unit + sg.first + 2 * sg.last;
        tc_fence_before();
        warp_arrive(sm.o_free);
      }
      n0 += tiles;
      have = have_nx;
    }
  }
  // ---------------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tbase, Cfg::kTmemCols);
  }
}

// ------------------------------------------------------------------------------------------
// Join the partials of the units that ranges share.  Block (p, y): if range p holds the first tile of such a
// unit, its pieces are that slot and slot 0 of the following ranges (of the same lockstep unit) up to the one
// with the last tile; a warp joins one row,
//   lse = ln sum_k exp(lse_k),  out = sum_k exp(lse_k - lse) o_k,  in range order.
// ------------------------------------------------------------------------------------------
constexpr int kPagedCombineWarps = 8;
constexpr int kPagedMaxRanges = 1024;

template <int D, int N>
__global__ void __launch_bounds__(kPagedCombineWarps * 32) paged_combine_kernel(const __grid_constant__ PagedDecodeParams p) {
  __shared__ int info[2 * kPagedMaxRanges], piece[kPagedMaxRanges];
  __shared__ int n_pieces, unit;
  griddep_wait();  // a programmatic dependent of the decode kernel: its writes first
  const int range = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const int2 own = *reinterpret_cast<const int2*>(p.seg_info + 2 * range);
  const bool in0 = own.x >= 0 && (own.x & 3) == 1, in1 = own.y >= 0 && (own.y & 3) == 1;
  if (!in0 && !in1) return;
  // every range's entry at once: a walk from range to range would wait for each load in turn
  for (int i = 2 * range + tid; i < 2 * p.P; i += blockDim.x) info[i] = p.seg_info[i];
  __syncthreads();
  if (tid == 0) {
    const int slot = in1 ? 1 : 0;
    unit = (slot ? own.y : own.x) >> 2;
    piece[0] = 2 * range + slot;
    int n = 1;
    const int step = p.lockstep ? p.U : 1;
    for (int q = range + step; q < p.P; q += step) {
      const int v = info[2 * q];
      if (v < 0) continue;  // a range without tiles
      if ((v >> 2) != unit) break;
      piece[n++] = 2 * q;
      if (v & 2) break;
    }
    n_pieces = n;
  }
  __syncthreads();
  const int n = n_pieces;
  const int row = blockIdx.y * kPagedCombineWarps + (tid >> 5);
  const int b = unit / p.U, u = unit - b * p.U, group = u / p.RB;
  const int g = (u - group * p.RB) * N + row;
  if (row >= N || g >= p.R) return;
  float mx = -INFINITY;
  for (int k = lane; k < n; k += 32) mx = fmaxf(mx, p.part_lse[static_cast<size_t>(piece[k]) * N + row]);
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float top = mx == -INFINITY ? 0.f : mx;
  float tot = 0.f;
  float4 acc[D / 128];
#pragma unroll
  for (int c = 0; c < D / 128; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < n; k0 += 32) {
    // 0 for a piece whose keys the row does not see
    const float wl = k0 + lane < n ? expf(p.part_lse[static_cast<size_t>(piece[k0 + lane]) * N + row] - top) : 0.f;
    const int m = min(32, n - k0);
#pragma unroll 4
    for (int k = 0; k < m; ++k) {
      const float w = __shfl_sync(0xffffffffu, wl, k);
      const float* part = p.part_o + (static_cast<size_t>(piece[k0 + k]) * N + row) * D;
      tot += w;
#pragma unroll
      for (int c = 0; c < D / 128; ++c) {
        const float4 o = *reinterpret_cast<const float4*>(part + 128 * c + 4 * lane);
        acc[c].x = fmaf(w, o.x, acc[c].x);
        acc[c].y = fmaf(w, o.y, acc[c].y);
        acc[c].z = fmaf(w, o.z, acc[c].z);
        acc[c].w = fmaf(w, o.w, acc[c].w);
      }
    }
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  const int i = g >= p.hpg;
  const size_t orow = (static_cast<size_t>(b) * p.s_q + i) * p.h_q + group * p.hpg + (g - i * p.hpg);
#pragma unroll
  for (int c = 0; c < D / 128; ++c) {
    uint2 v;
    v.x = pack_bf16x2(acc[c].x * inv, acc[c].y * inv);
    v.y = pack_bf16x2(acc[c].z * inv, acc[c].w * inv);
    *reinterpret_cast<uint2*>(p.out + orow * D + 128 * c + 4 * lane) = v;
  }
  if (lane == 0) p.lse[orow] = tot == 0.f ? -INFINITY : top + logf(tot);
}

}  // namespace lkv
