// Host side of kv_attend: checks, the units of the call and the choice of the
// kernel.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <functional>
#include <queue>
#include <climits>
#include <cmath>
#include <new>
#include <vector>

#include "kvq_attend.h"
#include "kvq_host.h"

namespace kvq {
namespace {

// ---- merge of partials -----------------------------------------------------
// out = sum_p O_p 2^(m_p - M) / sum_p l_p 2^(m_p - M); a warp per row (a lane four
// channels): the parts' m and l at once, a part per lane, then their O by eights.
// Bound by the partials' bytes, which are still in L2.
constexpr int kMergeRows = 8;
__global__ void __launch_bounds__(32 * kMergeRows) attend_merge_kernel(AttArgs A, const AttUnit* __restrict__ units,
                                                                       const AttMerge* __restrict__ merges,
                                                                       const float* __restrict__ part, int part_rows) {
  const AttMerge D = merges[blockIdx.y];
  const int i = blockIdx.x * kMergeRows + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= D.rows) return;
  const AttUnit u = units[D.unit];
  const size_t step = (size_t)D.stride * part_rows * kAttPart;
  const float* base = part + ((size_t)D.part0 * part_rows + i) * kAttPart;
  float M = -INFINITY;
  for (int p0 = 0; p0 < D.n_parts; p0 += 32)
    if (p0 + lane < D.n_parts) M = fmaxf(M, base[(size_t)(p0 + lane) * step + kHeadDim]);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float L = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int p0 = 0; p0 < D.n_parts; p0 += 32) {
    float f = 0.0f;
    if (p0 + lane < D.n_parts) {
      const float2 ml = *reinterpret_cast<const float2*>(base + (size_t)(p0 + lane) * step + kHeadDim);
      // a part that saw nothing (m = -inf, l = 0) adds nothing; one with a NaN sum keeps it
      f = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : exp2f(ml.x - M);
      L = fmaf(ml.y, f, L);
    }
    const int n = min(32, D.n_parts - p0);
    for (int p = 0; p < n; p += 8) {
      float4 a[8];
#pragma unroll
      for (int y = 0; y < 8; ++y)
        a[y] = *reinterpret_cast<const float4*>(base + (size_t)(p0 + min(p + y, n - 1)) * step + 4 * lane);
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const float w = __shfl_sync(0xFFFFFFFFu, f, (p + y) & 31);
        if (p + y < n && w != 0.0f) {
          o.x = fmaf(a[y].x, w, o.x); o.y = fmaf(a[y].y, w, o.y); o.z = fmaf(a[y].z, w, o.z); o.w = fmaf(a[y].w, w, o.w);
        }
      }
    }
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, x);
  const float inv = row_inverse(M, L);
  const float r[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
  bool bad = false;
  const int g = A.hq / A.hkv, row = D.row0 + i;
  uint16_t* op = A.out + ((size_t)(u.tok0 + row / g) * A.hq + (size_t)u.kvh * g + row % g) * kHeadDim + 4 * lane;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (!(fabsf(r[k]) < INFINITY)) bad = true;
    op[k] = __bfloat16_as_ushort(__float2bfloat16_rn(r[k]));
  }
  if (bad) atomicOr(A.status, kStatusRange);
}

// The same for parts of many rows, which hold 128 rows as [channels / 4][row][4] and
// then (m, l) [row]: a row per lane, four channels per warp, so that loads are whole
// lines; 32 results of 128 channels then cross over through shared memory.
constexpr int kTallRows = 128, kTallWarps = kHeadDim / 4;
__global__ void __launch_bounds__(32 * kTallWarps) attend_merge_tall_kernel(AttArgs A, const AttUnit* __restrict__ units,
                                                                            const AttMerge* __restrict__ merges,
                                                                            const float* __restrict__ part) {
  __shared__ uint2 done[32][kTallWarps + 1];
  const AttMerge D = merges[blockIdx.y];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r0 = 32 * (int)blockIdx.x;
  if (r0 >= D.rows) return;
  const size_t step = (size_t)D.stride * kTallRows * kAttPart;
  const int i = min(r0 + lane, D.rows - 1);   // rows past the end repeat the last one
  const float* base = part + (size_t)D.part0 * kTallRows * kAttPart;
  const float2* ml = reinterpret_cast<const float2*>(base + kTallRows * kHeadDim) + i;
  const float4* ov = reinterpret_cast<const float4*>(base) + (size_t)warp * kTallRows + i;
  constexpr int kAhead = 8;
  float M = -INFINITY, L = 0.0f;
  for (int p = 0; p < D.n_parts; p += kAhead)
#pragma unroll
    for (int y = 0; y < kAhead; ++y)
      if (p + y < D.n_parts) M = fmaxf(M, ml[(size_t)(p + y) * (step / 2)].x);
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int p = 0; p < D.n_parts; p += kAhead) {
    float4 a[kAhead];
    float2 b[kAhead];
#pragma unroll
    for (int y = 0; y < kAhead; ++y)
      if (p + y < D.n_parts) {
        a[y] = ov[(size_t)(p + y) * (step / 4)];
        b[y] = ml[(size_t)(p + y) * (step / 2)];
      }
#pragma unroll
    for (int y = 0; y < kAhead; ++y)
      if (p + y < D.n_parts) {
        // a part that saw nothing (m = -inf, l = 0) adds nothing; one with a NaN sum keeps it
        const float f = b[y].x == -INFINITY ? (b[y].y == 0.0f ? 0.0f : 1.0f) : exp2f(b[y].x - M);
        L = fmaf(b[y].y, f, L);
        if (f != 0.0f) {
          o.x = fmaf(a[y].x, f, o.x); o.y = fmaf(a[y].y, f, o.y); o.z = fmaf(a[y].z, f, o.z); o.w = fmaf(a[y].w, f, o.w);
        }
      }
  }
  const float inv = row_inverse(M, L);
  const float r[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
  bool bad = false;
  uint32_t h[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (!(fabsf(r[k]) < INFINITY)) bad = true;
    h[k] = __bfloat16_as_ushort(__float2bfloat16_rn(r[k]));
  }
  done[lane][warp] = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  if (bad) atomicOr(A.status, kStatusRange);
  __syncthreads();
  if (r0 + warp < D.rows) {
    const AttUnit u = units[D.unit];
    const int g = A.hq / A.hkv, row = D.row0 + r0 + warp;
    uint16_t* op = A.out + ((size_t)(u.tok0 + row / g) * A.hq + (size_t)u.kvh * g + row % g) * kHeadDim + 4 * lane;
    const uint2 w = done[warp][lane];
    if (((uintptr_t)A.out & 7) == 0) {
      *reinterpret_cast<uint2*>(op) = w;
    } else {
      op[0] = (uint16_t)w.x;
      op[1] = (uint16_t)(w.x >> 16);
      op[2] = (uint16_t)w.y;
      op[3] = (uint16_t)(w.y >> 16);
    }
  }
}

cudaError_t launch_attend_merge(kv_pool* P, const AttArgs& A, const AttUnit* d_units, const AttMerge* d_merges,
                                int n_merges, int max_rows, const float* d_part, int part_rows, cudaStream_t s) {
  const bool tall = part_rows == kTallRows;
  const int per = tall ? 32 : kMergeRows;
  for (int a = 0; a < n_merges; a += 65535) {
    ++P->launches;
    const dim3 grid((unsigned)((max_rows + per - 1) / per), (unsigned)std::min(65535, n_merges - a));
    if (tall)
      attend_merge_tall_kernel<<<grid, 32 * kTallWarps, 0, s>>>(A, d_units, d_merges + a, d_part);
    else
      attend_merge_kernel<<<grid, 32 * kMergeRows, 0, s>>>(A, d_units, d_merges + a, d_part, part_rows);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// ---- work plan ---------------------------------------------------------
struct AttPlan {
  std::vector<AttItem> items;
  std::vector<int32_t> cta_item;   // per pass: first item of every CTA, and the end
  std::vector<AttMerge> merges;
  int64_t n_parts = 0;
  int merge_rows = 0;
};

// Key tiles of the block of rows [row0, row0 + rows) of a unit.
int block_tiles(const AttUnit& u, int g, int row0, int rows, bool kv, bool tree) {
  const int t_last = (row0 + rows - 1) / g;
  return (u.n_pages + 3) / 4 + (u.n_fp + 127) / 128 + (kv ? (tree ? u.T - 1 : t_last) / 128 + 1 : 0);
}

// Blocks of kWideRows rows of units [u0, u1).  An item costs its tiles (3700 cycles
// each) and kWideItem more (20,000 for its rows, the first and last steps).  Whole
// blocks, those with the most tiles first, go to the least loaded CTA while they fit
// into an equal share; the blocks that are left are cut to fill up the shares, and
// their pieces merged.  So most items are whole blocks, and the blocks of a unit, which
// start together, read each tile at about the same time: it comes from L2 once it has
// been read.  (One line of blocks cut into equal runs took 1006 us for four chunks of
// 300 to 512 tokens over 15K to 32K, 850 us with every tile in L2; 761 us so.)
// by_cta[c] gets the items of CTA c.
constexpr int kWideRows = 256;
constexpr double kWideItem = 5.4;
void plan_wide(const std::vector<AttUnit>& units, int u0, int u1, int g, bool kv, bool tree, int ctas,
               std::vector<std::vector<AttItem>>& by_cta, AttPlan& out) {
  struct Block {
    int unit, row0, rows, tiles;
  };
  std::vector<Block> blocks, rest;
  double total = kWideItem * ctas;   // about one cut per CTA
  for (int x = u0; x < u1; ++x) {
    const int rows = units[(size_t)x].T * g;
    for (int r = 0; r < rows; r += kWideRows) {
      const int n = std::min(kWideRows, rows - r);
      const Block b{x, r, n, block_tiles(units[(size_t)x], g, r, n, kv, tree)};
      blocks.push_back(b);
      total += b.tiles + kWideItem;
    }
  }
  std::stable_sort(blocks.begin(), blocks.end(), [](const Block& a, const Block& b) { return a.tiles > b.tiles; });
  const double share = total / ctas;
  std::vector<double> load((size_t)ctas, 0.0);
  std::vector<std::pair<int, size_t>> pieces;   // (CTA, index) of a block's items
  auto give = [&](int cta, const Block& b, int t0, int t1) {
    pieces.emplace_back(cta, by_cta[(size_t)cta].size());
    by_cta[(size_t)cta].push_back(AttItem{b.unit, b.row0, t0, t1, -1, {0, 0, 0}});
  };
  auto join = [&](const Block& b) {   // partials of a block, if it needs any
    const int n = (int)pieces.size();
    if (n == 1) return;
    const int32_t p0 = (int32_t)out.n_parts;
    for (int y = 0; y < n; ++y) by_cta[(size_t)pieces[(size_t)y].first][pieces[(size_t)y].second].part = p0 + 2 * y;
    out.n_parts += 2 * n;
    out.merges.push_back(AttMerge{b.unit, b.row0, std::min(128, b.rows), p0, n, 2});
    if (b.rows > 128) out.merges.push_back(AttMerge{b.unit, b.row0 + 128, b.rows - 128, p0 + 1, n, 2});
    out.merge_rows = std::max(out.merge_rows, std::min(128, b.rows));
  };
  std::priority_queue<std::pair<double, int>, std::vector<std::pair<double, int>>, std::greater<>> least;
  for (int c = 0; c < ctas; ++c) least.emplace(0.0, c);
  for (const Block& b : blocks) {
    const double cost = b.tiles + kWideItem;
    const auto [l, c] = least.top();
    if (l + cost > share) {
      rest.push_back(b);
      continue;
    }
    least.pop();
    least.emplace(load[(size_t)c] = l + cost, c);
    pieces.clear();
    give(c, b, 0, b.tiles);
    join(b);
  }
  int cta = 0;
  double room = share - load[0];   // of the CTAs up to this one
  for (const Block& b : rest) {
    pieces.clear();
    int t = 0;
    do {
      int take = b.tiles - t;
      if (cta < ctas - 1) {
        const int fit = (int)(room - kWideItem + 0.5);
        if (fit < std::min(2, take)) {   // nothing worth starting fits: the next CTA
          ++cta;
          room += share - load[(size_t)cta];
          continue;
        }
        if (fit + 1 < take) take = fit;
      }
      give(cta, b, t, t + take);
      room -= take + kWideItem;
      t += take;
    } while (t < b.tiles);
    join(b);
  }
}

// Which kernel.  Per key tile (cycles of a CTA) the few-row kernel unpacks for every
// block of up to 64 rows, the other once and then works through blocks of 256; that one
// also costs a launch more and a longer first and last step.  Up to kFewRows rows the
// first is faster whatever the size (128 rows of 8 requests x 8 kv heads over 16K: 212 us
// against 259), above kFewMost the second (512 rows: 783 against 390); between them the
// call's tiles decide (256 rows: 405 against 271, but 42 against 58 for one request
// over 4K).
constexpr int kFewRows = 128, kFewMost = 384;
constexpr int64_t kFewBlock = 3400, kWideTile = 3900, kWideBlock = 3900, kWideStart = 38000;
int64_t wide_gain(int rows, int64_t tiles) {
  return tiles * (kFewBlock * ((rows + 63) / 64) - kWideTile - kWideBlock * ((rows + 255) / 256));
}

// Few rows per unit: blocks of R rows, all key tiles of all blocks in one line, cut
// into equal runs.  A tile costs 1 (its unpacking, whatever R), an item 3 more (its
// rows, the first and last steps).
void plan_few(const std::vector<AttUnit>& units, int g, int R, bool kv, bool tree, int sms, AttPlan& out) {
  double total = 0.0;
  int64_t tiles = 0;
  for (const AttUnit& u : units)
    for (int r = 0; r < u.T * g; r += R) {
      const int t = block_tiles(u, g, r, std::min(R, u.T * g - r), kv, tree);
      tiles += t;
      total += t + 3.0;
    }
  const int ctas = (int)std::max<int64_t>(1, std::min<int64_t>(sms, tiles));
  const double share = (total + 3.0 * (ctas - 1)) / ctas;
  double done = 0.0;
  int cta = 0;
  out.cta_item.push_back(0);
  for (int x = 0; x < (int)units.size(); ++x) {
    const AttUnit& u = units[(size_t)x];
    for (int r = 0; r < u.T * g; r += R) {
      const int rows = std::min(R, u.T * g - r), n = block_tiles(u, g, r, rows, kv, tree);
      const size_t first = out.items.size();
      int t = 0;
      do {
        int take = n - t;
        if (cta < ctas - 1) {
          const int fit = (int)((cta + 1) * share - done - 2.5);
          if (fit < std::min(1, take)) {
            out.cta_item.push_back((int32_t)out.items.size());
            ++cta;
            continue;
          }
          take = std::min(take, fit);
        }
        out.items.push_back(AttItem{x, r, t, t + take, -1, {0, 0, 0}});
        done += take + 3.0;
        t += take;
      } while (t < n);
      const int pieces = (int)(out.items.size() - first);
      if (pieces == 1) continue;
      for (int y = 0; y < pieces; ++y) out.items[first + (size_t)y].part = (int32_t)out.n_parts + y;
      out.merges.push_back(AttMerge{x, r, rows, (int32_t)out.n_parts, pieces, 1});
      out.n_parts += pieces;
      out.merge_rows = std::max(out.merge_rows, rows);
    }
  }
  out.cta_item.push_back((int32_t)out.items.size());
}

// A pass holds the operand tiles of as many units as fit into this many.
constexpr int64_t kTilesPerPass = 1 << 16;   // 4.3 GB

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" kv_status_t kv_attend(kv_pool_t* P, const void* q, const void* k, const void* v, const uint64_t* tree,
                                 const int32_t* req_ids, const int32_t* n_new, int32_t n_req, int32_t hq,
                                 float softmax_scale, void* out, void* stream) try {
  if (!P) return fail(KV_ERR_INVALID_ARG, "kv_attend: null pool");
  if (!req_ids || !n_new || n_req < 1) return fail(KV_ERR_INVALID_ARG, "kv_attend: null pointer or n_req < 1");
  if ((k == nullptr) != (v == nullptr)) return fail(KV_ERR_INVALID_ARG, "kv_attend: k and v come together");
  if (tree && !k) return fail(KV_ERR_INVALID_ARG, "kv_attend: a tree needs k and v");
  const int hkv = P->cfg.num_kv_heads;
  if (hq < hkv || hq % hkv != 0 || hq / hkv > 8)
    return fail(KV_ERR_INVALID_ARG, "kv_attend: num_q_heads %d must be a multiple of %d with ratio <= 8", hq, hkv);
  if (!std::isfinite(softmax_scale)) return fail(KV_ERR_INVALID_ARG, "kv_attend: softmax_scale must be finite");
  if ((int64_t)n_req * hkv > 65535) return fail(KV_ERR_INVALID_ARG, "kv_attend: n_req x num_kv_heads must be <= 65535");
  const int g = hq / hkv;
  int64_t total = 0;
  int32_t max_new = 0;
  for (int32_t b = 0; b < n_req; ++b) {
    if (!req_ok(P, req_ids[b])) return fail(KV_ERR_INVALID_ARG, "kv_attend: request %d not open", req_ids[b]);
    if (n_new[b] < 0 || n_new[b] > kMaxNewTokens)
      return fail(KV_ERR_INVALID_ARG, "kv_attend: n_new[%d] = %d is not in [0, %d]", b, n_new[b], kMaxNewTokens);
    if (tree && n_new[b] > 64) return fail(KV_ERR_INVALID_ARG, "kv_attend: a tree holds at most 64 tokens of a request");
    total += n_new[b];
    max_new = std::max(max_new, n_new[b]);
  }
  if (total == 0) return KV_OK;
  if (total > kMaxRows / hq)
    return fail(KV_ERR_INVALID_ARG, "kv_attend: more than %lld rows (tokens x num_q_heads)", (long long)kMaxRows);
  if (!q || !out) return fail(KV_ERR_INVALID_ARG, "kv_attend: null pointer");
  DeviceGuard dg(P->cfg.device);
  cudaStream_t s = (cudaStream_t)stream;
  kv_status_t st = refuse_capture("kv_attend", s);
  if (st != KV_OK) return st;
  if ((st = order_after_previous(P, s)) != KV_OK) return st;

  AttArgs A;
  A.pool = P->d_pool;
  A.int4_off = P->int4_offset;
  A.int3_off = P->int3_offset;
  A.fp4_off = P->fp4_offset;
  A.n2 = P->cfg.n_int2_pages;
  A.n3b = A.n2 + P->cfg.n_int4_pages;
  A.nfb = A.n3b + P->cfg.n_int3_pages;
  A.table = P->d_table;
  A.hdead = P->hdead.empty() ? nullptr : P->d_hdead;
  A.fpk = P->d_fpk;
  A.fpv = P->d_fpv;
  A.q = (const uint16_t*)q;
  A.k = (const uint16_t*)k;
  A.v = (const uint16_t*)v;
  A.tree = tree;
  A.out = (uint16_t*)out;
  A.status = P->d_status;
  A.scale_log2 = softmax_scale * 1.4426950408889634f;
  A.max_pages = P->cfg.max_pages_per_request;
  A.hkv = hkv;
  A.hq = hq;
  A.fp_cap = P->fp_cap;

  const bool simt = P->decode_impl == KV_DECODE_SIMT;
  std::vector<AttUnit> units, few;   // many rows (or all, on the CUDA cores) and few rows per unit
  const bool kv = k != nullptr, tr = tree != nullptr;
  auto unit = [&](int32_t b, int h, int64_t tok0) {
    const int32_t r = req_ids[b];
    return AttUnit{r, h, n_new[b], (int32_t)P->reqs[r].table.size(), P->n_fp.empty() ? 0 : P->n_fp[r], 0, tok0};
  };
  int few_most = kFewMost;   // rows of a unit that the few-row kernel takes
  int64_t gain = -kWideStart * P->sm_count;
  for (int32_t b = 0; b < n_req; ++b) {
    const int rows = n_new[b] * g;
    if (rows > kFewMost) gain += kWideStart * P->sm_count;   // the other kernel runs anyway
    if (rows > kFewRows && rows <= kFewMost) gain += hkv * wide_gain(rows, block_tiles(unit(b, 0, 0), g, 0, rows, kv, tr));
  }
  if (gain > 0) few_most = kFewRows;
  int few_rows = 0;
  int64_t tok0 = 0;
  for (int32_t b = 0; b < n_req; ++b) {
    const bool is_few = !simt && n_new[b] * g <= few_most;
    if (n_new[b] > 0)
      for (int h = 0; h < hkv; ++h) (is_few ? few : units).push_back(unit(b, h, tok0));
    if (is_few) few_rows = std::max(few_rows, n_new[b] * g);
    tok0 += n_new[b];
  }
  if (simt) {
    Upload u;
    u.add(units.data(), units.size() * sizeof(AttUnit));
    if ((st = ensure(P->attend, u.size)) != KV_OK) return st;
    if ((st = h2d(P, P->attend.ptr, u, s)) != KV_OK) return st;
    KV_CUDA(launch_attend_simt(P, A, (const AttUnit*)P->attend.ptr, (int)units.size(), max_new * g, s));
    return KV_OK;
  }
  AttPlan pf, pl;
  const int R = few_rows <= 16 ? 16 : (few_rows <= 32 ? 32 : 64);
  if (!few.empty()) plan_few(few, g, R, kv, tr, P->sm_count, pf);
  struct Pass {
    int u0, u1, max_tiles, cta0;
  };
  std::vector<Pass> passes;
  std::vector<std::vector<AttItem>> by_cta((size_t)P->sm_count);
  int64_t most = 0, n = 0;
  int u0 = 0, max_tiles = 0;
  auto end_pass = [&](int x) {
    passes.push_back(Pass{u0, x, max_tiles, (int)pl.cta_item.size()});
    plan_wide(units, u0, x, g, kv, tr, P->sm_count, by_cta, pl);
    for (auto& c : by_cta) {
      pl.cta_item.push_back((int32_t)pl.items.size());
      pl.items.insert(pl.items.end(), c.begin(), c.end());
      c.clear();
    }
    pl.cta_item.push_back((int32_t)pl.items.size());
    most = std::max(most, n);
    u0 = x;
    n = 0;
    max_tiles = 0;
  };
  if (!units.empty()) {
    for (int x = 0; x < (int)units.size(); ++x) {
      const int t = block_tiles(units[(size_t)x], g, 0, units[(size_t)x].T * g, kv, tr);
      if (x > u0 && n + t > kTilesPerPass) end_pass(x);
      units[(size_t)x].tile_base = (int32_t)n;
      n += t;
      max_tiles = std::max(max_tiles, t);
    }
    end_pass((int)units.size());
  }
  struct Placed {   // a plan's arrays in the upload, its partials behind
    size_t units, items, ctas, merges, parts;
  };
  Upload u;
  auto place = [&](const std::vector<AttUnit>& un, const AttPlan& p) {
    Placed x;
    x.units = u.add(un.data(), un.size() * sizeof(AttUnit));
    x.items = u.add(p.items.data(), p.items.size() * sizeof(AttItem));
    x.ctas = u.add(p.cta_item.data(), p.cta_item.size() * sizeof(int32_t));
    x.merges = u.add(p.merges.data(), p.merges.size() * sizeof(AttMerge));
    return x;
  };
  Placed xf = place(few, pf), xl = place(units, pl);
  xf.parts = (u.size + 255) & ~size_t(255);
  xl.parts = xf.parts + (size_t)pf.n_parts * R * kAttPart * sizeof(float);
  if ((st = ensure(P->attend, xl.parts + (size_t)pl.n_parts * 128 * kAttPart * sizeof(float))) != KV_OK) return st;
  if ((st = ensure(P->attend_tiles, (size_t)most * (kAttTileBytes + 16), (size_t)kTilesPerPass * (kAttTileBytes + 16))) !=
      KV_OK)
    return st;
  if ((st = h2d(P, P->attend.ptr, u, s)) != KV_OK) return st;
  uint8_t* base = (uint8_t*)P->attend.ptr;
  auto merge = [&](const Placed& x, const AttPlan& p, int part_rows) -> cudaError_t {
    if (p.merges.empty()) return cudaSuccess;
    return launch_attend_merge(P, A, (const AttUnit*)(base + x.units), (const AttMerge*)(base + x.merges),
                               (int)p.merges.size(), p.merge_rows, (const float*)(base + x.parts), part_rows, s);
  };
  if (!few.empty()) {
    KV_CUDA(launch_attend_few(P, R, A, (const AttUnit*)(base + xf.units), (const AttItem*)(base + xf.items),
                              (const int32_t*)(base + xf.ctas), (int)pf.cta_item.size() - 1, (float*)(base + xf.parts), s));
    KV_CUDA(merge(xf, pf, R));
  }
  const AttUnit* du = (const AttUnit*)(base + xl.units);
  uint32_t* d_live = (uint32_t*)((uint8_t*)P->attend_tiles.ptr + (size_t)most * kAttTileBytes);
  for (const Pass& G : passes) {
    KV_CUDA(launch_attend_tiles(P, A, du + G.u0, G.u1 - G.u0, G.max_tiles, P->attend_tiles.ptr, d_live, s));
    KV_CUDA(launch_attend_wide(P, A, du, (const AttItem*)(base + xl.items), (const int32_t*)(base + xl.ctas) + G.cta0,
                               P->sm_count, P->attend_tiles.ptr, d_live, (float*)(base + xl.parts), s));
  }
  KV_CUDA(merge(xl, pl, 128));
  return KV_OK;
} catch (const std::bad_alloc&) {
  return fail(KV_ERR_OOM, "kv_attend: host allocation failed");
}
