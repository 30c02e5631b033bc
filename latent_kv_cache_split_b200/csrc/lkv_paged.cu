// Host side of the paged 4-bit cache (include/lkv.h): rotary positions, the append that rotates and
// quantises, and decode attention over the pool.  Argument checks make no CUDA call.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/lkv.h"
#include "lkv_int4.cuh"
#include "lkv_paged_decode.cuh"
#include "lkv_rope.cuh"
#include "lkv_tma_host.h"

lkv_status lkv_internal_device_info(int** err, int* num_sms, unsigned long long* wait_ns);  // lkv_api.cu

namespace {

using namespace lkv;

constexpr int kMaxDevices = 64;

inline bool al(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline bool finite_positive(float v) { return std::isfinite(v) && v > 0.f; }

lkv_status launched() {
  const cudaError_t e = cudaGetLastError();  // a launch error is not sticky; this clears it for the caller
  return e == cudaSuccess ? LKV_OK : LKV_ERR_CUDA;
}

size_t row_bytes_of(int r, int d_rope) {
  if (r <= 0 || r % kInt4Block || r > kInt4MaxLatent || d_rope < 0 || d_rope % 8 || d_rope > 2 * kRopeMaxPairs) return 0;
  return static_cast<size_t>(int4_rope_at(r)) + 2 * static_cast<size_t>(d_rope);
}

// Checks of a pool and its table, and the kernels' view of them.
lkv_status check_pool(Paged* g, const void* pool, int64_t page_stride, int64_t row_stride, int64_t n_pages, int page_size,
                      const int32_t* table, int64_t table_stride, int max_pages, const int32_t* seq_lens, int batch,
                      int r, int d_rope) {
  const size_t rb = row_bytes_of(r, d_rope);
  if (!pool || !table || !seq_lens || rb == 0 || batch <= 0 || n_pages <= 0 || page_size <= 0 || max_pages <= 0)
    return LKV_ERR_INVALID_ARG;
  if (!al(pool, 16) || !al(table, 4) || !al(seq_lens, 4) || page_stride % 16 || row_stride % 16 || row_stride < static_cast<int64_t>(rb) ||
      table_stride < max_pages)
    return LKV_ERR_INVALID_ARG;
  // pages do not overlap: whole pages apart, or their rows interleaved with others' (a view of a wider pool)
  if (n_pages > 1 && page_stride < static_cast<int64_t>(rb)) return LKV_ERR_INVALID_ARG;
  g->pool = static_cast<uint8_t*>(const_cast<void*>(pool));
  g->page_stride = page_stride;
  g->row_stride = row_stride;
  g->n_pages = n_pages;
  g->page_size = page_size;
  g->page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (page_size == 1 << i) g->page_shift = i;
  g->table = table;
  g->table_stride = table_stride;
  g->max_pages = max_pages;
  g->seq_lens = seq_lens;
  return LKV_OK;
}

// Whether two of the rows of d elements at token * ts + head * hs share one.
bool rows_overlap(int64_t ts, int64_t n_tok, int64_t hs, int64_t heads, int64_t d) {
  ts = ts < 0 ? -ts : ts;  // a sign mirrors the rows' order
  hs = hs < 0 ? -hs : hs;
  if ((n_tok > 1 && ts < d) || (heads > 1 && hs < d)) return true;
  if (n_tok == 1 || heads == 1) return false;
  if ((hs - d) / ts >= n_tok - 1 || (ts - d) / hs >= heads - 1) return false;  // one kind of rows lies within the other's steps
  for (int64_t h = 1; h < heads; ++h) {  // interleaved: the tokens nearest to h heads' distance
    const int64_t t = h * hs / ts, past = h * hs - t * ts;
    if ((past < d && t < n_tok) || (ts - past < d && t + 1 < n_tok)) return true;
  }
  return false;
}

template <typename T, int V>
void launch_rope(const RopeParams& p, bool interleaved, dim3 blocks, dim3 threads, cudaStream_t s) {
  if (interleaved)
    rope_kernel<T, V, true><<<blocks, threads, 0, s>>>(p);
  else
    rope_kernel<T, V, false><<<blocks, threads, 0, s>>>(p);
}

// Rows of a unit (the MMA's N): the smallest of 16, 32, 64 that holds a group's rows, so that small groups
// spend no softmax on padding; 64 at most, and a group of more rows is several units that read the same tiles.
// 64 x 8192 tokens, 8 groups of 128: 16 rows 222 us as units of 16 and 248 us as units of 32, 32 rows 252 us
// as units of 32 and 370 us as units of 64.
int paged_rows(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : 64; }

struct PagedPlan {
  int N, RB, U, P, lockstep;
  size_t seg, lse, o, total;  // workspace offsets and size
};

void paged_plan(PagedPlan* w, int s_q, int h_q, int groups, int d, int num_sms) {
  const int R = s_q * (h_q / groups);
  w->N = paged_rows(R);
  w->RB = (R + w->N - 1) / w->N;
  w->U = groups * w->RB;
  // Units in lockstep share a request's RoPE keys and scales through L2 (64 x 8192 tokens, 8 groups of 32 rows: 252 us
  // against 278 us); not where that leaves more than a tenth of the SMs without a range, nor for so few units that
  // there is little to share.
  const int sms = num_sms < kPagedMaxRanges ? num_sms : kPagedMaxRanges;
  const int whole = w->U <= sms ? sms / w->U * w->U : 0;
  w->lockstep = w->U >= 4 && 10 * whole >= 9 * sms;
  w->P = w->lockstep ? whole : sms;
  auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  const size_t slots = 2 * static_cast<size_t>(w->P);
  w->seg = 0;
  w->lse = up(slots * sizeof(int));
  w->o = w->lse + up(slots * w->N * sizeof(float));
  w->total = w->o + up(slots * w->N * d * sizeof(float));
}

// A kernel's dynamic shared memory is an attribute, set on each device once.
template <class Kernel>
lkv_status allow_smem(Kernel k, size_t bytes, bool (&ready)[kMaxDevices]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return LKV_ERR_CUDA;
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess) {
      cudaGetLastError();
      return LKV_ERR_CUDA;
    }
    ready[dev] = true;
  }
  return LKV_OK;
}

// The decode kernel, then the combine as its programmatic dependent: its launch overlaps the decode, and its
// blocks wait for the decode's completion before they read the partials.
template <int D, int N, bool kTma>
lkv_status launch_decode(const PagedDecodeParams& p, cudaStream_t s) {
  using Cfg = PagedCfg<D, N, kTma>;
  static bool ready[kMaxDevices];
  lkv_status st;
  if ((st = allow_smem(paged_decode_kernel<D, N, kTma>, Cfg::kSmem, ready)) != LKV_OK) return st;
  PagedMaps maps = {};
  if (kTma) {
    const Paged& g = p.pages;
    const uint64_t rb = row_bytes_of(p.G * D, 64), ps = g.n_pages > 1 ? g.page_stride : g.row_stride * g.page_size;
    auto map = [&](CUtensorMap* m, uint32_t bytes, CUtensorMapSwizzle sw) {
      return make_tmap_u8_3d(m, g.pool, rb, g.page_size, g.n_pages, g.row_stride, ps, bytes, p.box_rows, sw);
    };
    if (!map(&maps.codes, D / 2, Cfg::kWide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !map(&maps.scales, 16, CU_TENSOR_MAP_SWIZZLE_NONE) || !map(&maps.keys, 128, CU_TENSOR_MAP_SWIZZLE_128B))
      return LKV_ERR_UNSUPPORTED;  // strides past what a tensor map holds
  }
  paged_decode_kernel<D, N, kTma><<<p.P, kPagedThreads, Cfg::kSmem, s>>>(p, maps);
  if ((st = launched()) != LKV_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.P, (N + kPagedCombineWarps - 1) / kPagedCombineWarps);
  cfg.blockDim = dim3(kPagedCombineWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_combine_kernel<D, N>, p);
  st = launched();
  return e == cudaSuccess ? st : LKV_ERR_CUDA;
}

// Tiles come by TMA where pages hold runs of 16 rows: a copy costs about as much as 25 of its rows.  64 x 8192 tokens, by TMA
// against loaded by the converters: 8 groups of 128, 32 rows, pages of 64 252 against 339 us, of 16 318 against 357 us; 2 groups
// of 256, 64 rows, pages of 64 142 against 223 us, of 16 161 against 224 us; 4 groups, 32 rows, pages of 16 260 against 265
// us, of 8 367 against 263 us.
template <int D>
lkv_status launch_decode_of(const PagedDecodeParams& p, int N, cudaStream_t s) {
  if constexpr (D <= 256) {
    if (p.box_rows >= 16)
      return N == 16 ? launch_decode<D, 16, true>(p, s) : N == 32 ? launch_decode<D, 32, true>(p, s) : launch_decode<D, 64, true>(p, s);
  }
  return N == 16 ? launch_decode<D, 16, false>(p, s) : N == 32 ? launch_decode<D, 32, false>(p, s) : launch_decode<D, 64, false>(p, s);
}

lkv_status launch_decode_for(const PagedDecodeParams& p, int d, int N, cudaStream_t s) {
  return d == 128 ? launch_decode_of<128>(p, N, s) : d == 256 ? launch_decode_of<256>(p, N, s) : launch_decode_of<512>(p, N, s);
}

}  // namespace

extern "C" {

lkv_status lkv_rope_rotate(const void* x, int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
                           const double* freqs, int64_t n_tok, int heads, int d, int first, int rot, int interleaved,
                           int inverse, float gain, int dtype, void* out, int64_t out_token_stride,
                           int64_t out_head_stride, lkv_stream_t stream) {
  if (!x || !positions || !freqs || !out || n_tok < 0 || heads <= 0 || d <= 0) return LKV_ERR_INVALID_ARG;
  if (first < 0 || rot <= 0 || rot % 2 || rot > d - first || !finite_positive(gain)) return LKV_ERR_INVALID_ARG;
  if (dtype != LKV_BF16 && dtype != LKV_FP32) return LKV_ERR_INVALID_ARG;
  if (x == out && (x_token_stride != out_token_stride || x_head_stride != out_head_stride)) return LKV_ERR_INVALID_ARG;
  if (rot / 2 > kRopeMaxPairs || heads > 1 << 20) return LKV_ERR_UNSUPPORTED;
  const int size = dtype == LKV_BF16 ? 2 : 4, wide = 16 / size;
  if (!al(x, size) || !al(out, size) || !al(positions, 4) || !al(freqs, 8)) return LKV_ERR_INVALID_ARG;
  if (n_tok == 0) return LKV_OK;
  if (rows_overlap(out_token_stride, n_tok, out_head_stride, heads, d)) return LKV_ERR_INVALID_ARG;
  RopeParams p;
  p.x = x;
  p.out = out;
  p.x_ts = x_token_stride;
  p.x_hs = x_head_stride;
  p.o_ts = out_token_stride;
  p.o_hs = out_head_stride;
  p.pos = positions;
  p.freqs = freqs;
  p.n_tok = n_tok;
  p.heads = heads;
  p.d = d;
  p.first = first;
  p.rot = rot;
  p.inverse = inverse != 0;
  p.gain = gain;
  p.copy = x != out;
  // 16-byte accesses where every row, and every run of columns in it, starts and ends on 16 bytes
  const bool vec = al(x, 16) && al(out, 16) && x_token_stride % wide == 0 && x_head_stride % wide == 0 &&
                   out_token_stride % wide == 0 && out_head_stride % wide == 0 && first % wide == 0 && d % wide == 0 &&
                   (interleaved ? rot : rot / 2) % wide == 0;
  const int v = vec ? wide : 1;
  const int items = (interleaved ? rot / (vec ? wide : 2) : rot / 2 / v) + (p.copy ? (d - rot) / v : 0);
  const int bx = items < kRopeThreads ? items : kRopeThreads, by = kRopeThreads / bx;
  // A block takes several tokens where one token's heads do not fill it, else the heads of one token: up to 16 for each
  // row of threads, fewer where that leaves less than 2048 blocks.
  p.tok_block = 1;
  p.head_block = heads;
  if (heads <= by) {
    const int most = kRopeTable / (rot / 2);
    p.tok_block = by / heads < most ? by / heads : most;
  } else {
    int loads = 16;
    while (loads > 1 && n_tok * ((heads + loads * by - 1) / (loads * by)) < 2048) --loads;
    const int most = 65535, chunks = std::min((heads + loads * by - 1) / (loads * by), most);  // a grid's second dimension
    p.head_block = (heads + chunks - 1) / chunks;
  }
  const int64_t nx = (n_tok + p.tok_block - 1) / p.tok_block;
  const int ny = (heads + p.head_block - 1) / p.head_block;
  if (nx > INT_MAX || ny > 65535) return LKV_ERR_UNSUPPORTED;
  const dim3 blocks(static_cast<unsigned>(nx), ny), threads(bx, by);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == LKV_BF16) {
    if (vec)
      launch_rope<__nv_bfloat16, 8>(p, interleaved, blocks, threads, s);
    else
      launch_rope<__nv_bfloat16, 1>(p, interleaved, blocks, threads, s);
  } else {
    if (vec)
      launch_rope<float, 4>(p, interleaved, blocks, threads, s);
    else
      launch_rope<float, 1>(p, interleaved, blocks, threads, s);
  }
  return launched();
}

size_t lkv_int4_cache_row_bytes(int r, int d_rope) { return row_bytes_of(r, d_rope); }

lkv_status lkv_paged_append_int4(const void* new_rows, int64_t new_row_stride, int64_t n_new, void* pool,
                                 int64_t page_stride_bytes, int64_t row_stride_bytes, int64_t n_pages, int page_size,
                                 const int32_t* block_table, int64_t table_stride, int max_pages,
                                 const int32_t* seq_lens, const int32_t* cu_new, int batch, int r, int d_rope,
                                 const double* freqs, int interleaved, float gain, void* rows_out,
                                 int64_t rows_out_stride, lkv_stream_t stream) {
  AppendParams p;
  lkv_status st = check_pool(&p.pages, pool, page_stride_bytes, row_stride_bytes, n_pages, page_size, block_table,
                             table_stride, max_pages, seq_lens, batch, r, d_rope);
  if (st != LKV_OK) return st;
  if (!new_rows || n_new < 0 || !al(new_rows, 16) || new_row_stride % 8 || new_row_stride < r + d_rope) return LKV_ERR_INVALID_ARG;
  if (cu_new ? !al(cu_new, 4) : n_new % batch != 0) return LKV_ERR_INVALID_ARG;
  if (freqs && (!al(freqs, 8) || !finite_positive(gain))) return LKV_ERR_INVALID_ARG;
  if (rows_out && (!al(rows_out, 16) || rows_out_stride % 8 || rows_out_stride < r + d_rope)) return LKV_ERR_INVALID_ARG;
  if (rows_out == new_rows && rows_out_stride != new_row_stride) return LKV_ERR_INVALID_ARG;
  if (n_new >= INT_MAX / 2) return LKV_ERR_UNSUPPORTED;
  if (n_new == 0) return LKV_OK;
  int num_sms;
  unsigned long long wait_ns;
  if ((st = lkv_internal_device_info(&p.err, &num_sms, &wait_ns)) != LKV_OK) return st;
  p.rows = static_cast<const __nv_bfloat16*>(new_rows);
  p.row_stride = new_row_stride;
  p.n_new = n_new;
  p.cu_new = cu_new;
  p.batch = batch;
  p.per = cu_new ? 0 : static_cast<int>(n_new / batch);
  p.r = r;
  p.d_rope = d_rope;
  p.freqs = freqs;
  p.interleaved = interleaved != 0;
  p.gain = gain;
  p.held = static_cast<__nv_bfloat16*>(rows_out);
  p.held_stride = rows_out_stride;
  constexpr int per_block = kAppendThreads / 32;
  append_int4_kernel<<<static_cast<unsigned>((n_new + per_block - 1) / per_block), kAppendThreads, 0,
                       reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return launched();
}

size_t lkv_paged_decode_workspace_size(int batch, int s_q, int h_q, int groups, int d, int num_sms) {
  if (batch <= 0 || s_q <= 0 || h_q <= 0 || groups <= 0 || h_q % groups || num_sms <= 0) return 0;
  if ((d != 128 && d != 256 && d != 512) || static_cast<long long>(s_q) * (h_q / groups) > 256) return 0;
  PagedPlan w;
  paged_plan(&w, s_q, h_q, groups, d, num_sms);
  return w.total;
}

lkv_status lkv_paged_decode_int4(const void* q, const void* q_rope, const void* pool, int64_t page_stride_bytes,
                                 int64_t row_stride_bytes, int64_t n_pages, int page_size, const int32_t* block_table,
                                 int64_t table_stride, int max_pages, const int32_t* seq_lens, int batch, int s_q,
                                 int h_q, int groups, int d, int d_rope, float scale, void* out, float* lse,
                                 void* workspace, size_t workspace_bytes, lkv_stream_t stream) {
  PagedDecodeParams p;
  if (!q || !q_rope || !out || !lse || h_q <= 0 || groups <= 0 || d <= 0 || h_q % groups || !finite_positive(scale))
    return LKV_ERR_INVALID_ARG;
  if (!al(q, 16) || !al(q_rope, 16) || !al(out, 16) || !al(lse, 4)) return LKV_ERR_INVALID_ARG;
  if (s_q != 1 && s_q != 2) return LKV_ERR_UNSUPPORTED;
  if ((d != 128 && d != 256 && d != 512) || d_rope != 64 || s_q * static_cast<long long>(h_q / groups) > 256)
    return LKV_ERR_UNSUPPORTED;
  if (static_cast<long long>(groups) * d > kInt4MaxLatent) return LKV_ERR_UNSUPPORTED;
  lkv_status st = check_pool(&p.pages, pool, page_stride_bytes, row_stride_bytes, n_pages, page_size, block_table,
                             table_stride, max_pages, seq_lens, batch, groups * d, d_rope);
  if (st != LKV_OK) return st;
  if (static_cast<long long>(batch) * s_q * h_q >= (1LL << 28)) return LKV_ERR_UNSUPPORTED;
  int num_sms;
  if ((st = lkv_internal_device_info(&p.err, &num_sms, &p.wait_limit_ns)) != LKV_OK) return st;
  PagedPlan w;
  paged_plan(&w, s_q, h_q, groups, d, num_sms);
  if (!workspace || !al(workspace, 16) || workspace_bytes < w.total) return LKV_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_rope = static_cast<const __nv_bfloat16*>(q_rope);
  p.B = batch;
  p.s_q = s_q;
  p.h_q = h_q;
  p.G = groups;
  p.hpg = h_q / groups;
  p.R = s_q * p.hpg;
  p.RB = w.RB;
  p.U = w.U;
  p.P = w.P;
  p.lockstep = w.lockstep;
  // What a unit's start and end take in tiles (its pipeline fills and drains).  32 requests of 64 .. 20000 tokens, 2 groups of
  // 64 rows, d = 128: 71 us without this term, 46 us with 3, 41 us with 6, 42 us with 10; 40 of 64 .. 16000 at d = 256: 109,
  // 72, 59 and 60 us; 24 of 0 .. 2500, groups of 8 rows: 24, 17, 18.6 and 20 us; 40 of 64 .. 6000 at d = 512: 80 us with 3,
  // 83 us with 6.
  p.unit_cost = d == 512 || w.N == 16 ? 3 : 6;
  p.sl2 = scale * 1.4426950408889634f;
  p.box_rows = 1;
  while (p.box_rows < kPagedTile && page_size % (2 * p.box_rows) == 0) p.box_rows *= 2;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.seg_info = reinterpret_cast<int*>(ws + w.seg);
  p.part_lse = reinterpret_cast<float*>(ws + w.lse);
  p.part_o = reinterpret_cast<float*>(ws + w.o);
  return launch_decode_for(p, d, w.N, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
