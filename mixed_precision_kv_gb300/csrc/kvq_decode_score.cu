// The decode step that also accumulates attention weight per cached token
// (kv_decode_attn_scored).
//
// For every live slot t of kv head h of a request, with the logits s_jt (base
// 2) of the g q heads j of h and their softmax statistics (M_j, L_j):
//     score_t <- decay * score_t + sum_j 2^(s_jt - M_j) / L_j.
// The weights need M_j and L_j of the whole row, which exist only after the
// scan, so the scan keeps its logits and a second kernel turns them into
// weights once the merge has (M_j, 1 / L_j).  Reading K again instead would
// cost the scan's unpacking a second time (the scan is bound by instruction
// issue, and K is about half of it); the logits cost 8 g bytes per slot and kv
// head of traffic (written and read once), and most of that stays below the
// scan's own bound.
#include <algorithm>
#include <cmath>
#include <new>

#include "kvq_host.h"
#include "kvq_scan_mma.cuh"

namespace kvq {
namespace {

constexpr int kScoreWarps = 4;
constexpr int kScorePages = 4;   // pages in flight per warp

// Warp = a run of kScorePages table entries of one unit, lane = slot.  Bound
// by memory: 128 g bytes of logits, 128 bytes of positions (shared by the kv
// heads, so mostly from L2) and 256 bytes of scores per page and kv head.  The
// logits' loads come first: they need no table entry, and the chain entry ->
// position -> score runs behind them (80 us for 16 requests of 100K slots and 8
// kv heads of 8 q heads, 6.5 TB/s; 110 us with them behind the entries).  Slots
// of a page hold tokens in order of arrival, so the scattered scores of a page
// fall into one or two runs.
template <int G>
__global__ void __launch_bounds__(32 * kScoreWarps) score_add_kernel(
    const Unit* __restrict__ units, const float2* __restrict__ ml, const float* __restrict__ logits,
    const Entry* __restrict__ table, int max_pages, const int32_t* __restrict__ ntab,
    const uint32_t* __restrict__ hdead, const int32_t* __restrict__ pos, int hkv, float decay,
    float* __restrict__ scores, int64_t stride) {
  const Unit u = units[blockIdx.y];
  // A unit without page splits had an empty table when it was planned, and still has one (a table that gains
  // its first page is planned again).  ntab and table are written by appends only: under a request id that
  // was closed and opened again they hold the earlier request's until then.
  if (u.n_splits == 0) return;
  const int lane = threadIdx.x & 31;
  const int n = ntab[u.req];
  const int p0 = (blockIdx.x * kScoreWarps + (threadIdx.x >> 5)) * kScorePages;
  if (p0 >= n) return;
  const Entry* tab = table + (size_t)u.req * max_pages;
  float* sc = scores + ((size_t)u.b * hkv + u.kvh) * stride;
  float M[G], inv[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const float2 v = ml[(size_t)blockIdx.y * G + h];
    M[h] = v.x;
    inv[h] = v.y;
  }
  bool live[kScorePages];
  int32_t at[kScorePages];
  float lg[kScorePages][G], old[kScorePages];
#pragma unroll
  for (int x = 0; x < kScorePages; ++x) {   // (past the end: the last page's again, not used)
    const float* lp = logits + ((size_t)(uint32_t)u.pad + min(p0 + x, n - 1)) * (G * kPage) + lane;
#pragma unroll
    for (int h = 0; h < G; ++h) lg[x][h] = __ldcs(lp + h * kPage);
  }
#pragma unroll
  for (int x = 0; x < kScorePages; ++x) {
    live[x] = false;
    if (p0 + x < n) {
      const Entry e = tab[p0 + x];
      const uint32_t m = hdead ? e.live & ~hdead[(size_t)e.id * hkv + u.kvh] : e.live;
      live[x] = (m >> lane) & 1u;
      if (live[x]) at[x] = pos[(size_t)e.id * kPage + lane];
    }
  }
#pragma unroll
  for (int x = 0; x < kScorePages; ++x)
    if (live[x]) old[x] = sc[at[x]];
#pragma unroll
  for (int x = 0; x < kScorePages; ++x)
    if (live[x]) {
      float w = 0.0f;
#pragma unroll
      for (int h = 0; h < G; ++h) w = fmaf(ex2(lg[x][h] - M[h]), inv[h], w);
      sc[at[x]] = fmaf(decay, old[x], w);
    }
}

template <int G>
cudaError_t launch_scored_g(kv_pool* P, const void* q, int32_t hq, float scale_log2, const Unit* d_units, int n_units,
                            const Split* d_splits, const int32_t* d_wsplit, int n_workers, void* d_frags,
                            float* d_part, float* logits, cudaStream_t s) {
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(attr_set.load() >> dev & 1u)) {
    cudaError_t e = set_scan_attributes<G, true, false, false, true>();
    if (e == cudaSuccess) e = set_scan_attributes<G, true, false, true, true>();
    if (e != cudaSuccess) return e;
    attr_set.fetch_or(uint64_t(1) << dev);
  }
  if (n_workers <= 0 || n_units <= 0) return cudaSuccess;
  const uint32_t* smax = P->d_status + 1;
  P->launches += 2;
  cudaError_t e = launch_pdl(frag_kernel<G>, dim3((unsigned)n_units), dim3(256), 0, s, (const __nv_bfloat16*)q,
                             (int)hq, scale_log2, d_units, smax, (UnitFrag*)d_frags, (const GroupPool*)nullptr);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((n_workers + kWarps - 1) / kWarps);
  auto* kernel = P->cfg.n_int3_pages > 0 || P->cfg.n_fp4_pages > 0 ? decode_mma_kernel<G, true, false, true, true>
                                                                   : decode_mma_kernel<G, true, false, false, true>;
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), (size_t)kScanSmem, s, (const uint8_t*)P->d_pool,
                    P->int4_offset, (int64_t)P->cfg.n_int2_pages, P->cfg.num_kv_heads, P->cfg.max_pages_per_request,
                    (const Entry*)P->d_table, (const UnitFrag*)d_frags, d_splits, d_wsplit, n_workers,
                    (const int32_t*)P->d_ntab, (const uint32_t*)(P->hdead.empty() ? nullptr : P->d_hdead), d_part, smax,
                    P->d_status, P->first_wait_spins < 0 ? kSpinLimit : (uint32_t)P->first_wait_spins,
                    (const GroupPool*)nullptr, P->int3_offset, (int64_t)(P->cfg.n_int2_pages + P->cfg.n_int4_pages),
                    P->fp4_offset, (int64_t)(P->cfg.n_int2_pages + P->cfg.n_int4_pages + P->cfg.n_int3_pages), logits);
}

template <int G>
cudaError_t launch_score_add(kv_pool* P, const Unit* d_units, int n_units, int max_len, const float2* ml,
                             const float* logits, float decay, float* scores, int64_t stride, cudaStream_t s) {
  ++P->launches;
  const dim3 grid((unsigned)((max_len + kScoreWarps * kScorePages - 1) / (kScoreWarps * kScorePages)), (unsigned)n_units);
  score_add_kernel<G><<<grid, 32 * kScoreWarps, 0, s>>>(
      d_units, ml, logits, P->d_table, P->cfg.max_pages_per_request, P->d_ntab, P->hdead.empty() ? nullptr : P->d_hdead,
      P->d_pos, P->cfg.num_kv_heads, decay, scores, stride);
  return cudaGetLastError();
}

#define KVQ_BY_GROUP(g, call)                \
  switch (g) {                               \
    case 1: { constexpr int G = 1; call; }   \
    case 2: { constexpr int G = 2; call; }   \
    case 3: { constexpr int G = 3; call; }   \
    case 4: { constexpr int G = 4; call; }   \
    case 5: { constexpr int G = 5; call; }   \
    case 6: { constexpr int G = 6; call; }   \
    case 7: { constexpr int G = 7; call; }   \
    case 8: { constexpr int G = 8; call; }   \
    default: return cudaErrorInvalidValue;   \
  }

cudaError_t launch_score_add_any(int g, kv_pool* P, const Unit* d_units, int n_units, int max_len, const float2* ml,
                                 const float* logits, float decay, float* scores, int64_t stride, cudaStream_t s) {
  KVQ_BY_GROUP(g, return launch_score_add<G>(P, d_units, n_units, max_len, ml, logits, decay, scores, stride, s))
}

cudaError_t launch_scored_any(int g, kv_pool* P, const void* q, int32_t hq, float scale_log2, const Unit* d_units,
                              int n_units, const Split* d_splits, const int32_t* d_wsplit, int n_workers, void* d_frags,
                              float* d_part, float* logits, cudaStream_t s) {
  KVQ_BY_GROUP(g, return launch_scored_g<G>(P, q, hq, scale_log2, d_units, n_units, d_splits, d_wsplit, n_workers,
                                            d_frags, d_part, logits, s))
}

}  // namespace

cudaError_t launch_decode_mma_scored(kv_pool* P, const void* q, int32_t hq, float scale_log2, const Unit* d_units,
                                     int n_units, const Split* d_splits, const int32_t* d_wsplit, int n_workers,
                                     void* d_frags, float* d_part, float* out, float* logits, float2* ml,
                                     cudaStream_t s) {
  const int g = hq / P->cfg.num_kv_heads;
  cudaError_t e = launch_scored_any(g, P, q, hq, scale_log2, d_units, n_units, d_splits, d_wsplit, n_workers, d_frags,
                                    d_part, logits, s);
  if (e != cudaSuccess) return e;
  if ((e = launch_fp_pending(P, q, hq, scale_log2, d_units, d_part, s)) != cudaSuccess) return e;
  return launch_merge(P, g, d_units, n_units, d_part, hq, out, s, ml);
}

}  // namespace kvq

using namespace kvq;

extern "C" kv_status_t kv_decode_attn_scored(kv_pool_t* P, const void* q, const int32_t* req_ids, int32_t batch,
                                             int32_t hq, float softmax_scale, float decay, float* scores,
                                             int64_t score_stride, float* out, void* stream) try {
  if (!P) return fail(KV_ERR_INVALID_ARG, "kv_decode_attn_scored: null pool");
  if (!q || !out || !req_ids || !scores || batch < 1)
    return fail(KV_ERR_INVALID_ARG, "kv_decode_attn_scored: null pointer or batch < 1");
  const int hkv = P->cfg.num_kv_heads;
  if (hq < hkv || hq % hkv != 0 || hq / hkv > 8)
    return fail(KV_ERR_INVALID_ARG, "kv_decode_attn_scored: num_q_heads %d must be a multiple of %d with ratio <= 8", hq,
                hkv);
  if (!std::isfinite(softmax_scale) || !std::isfinite(decay))
    return fail(KV_ERR_INVALID_ARG, "kv_decode_attn_scored: softmax_scale and decay must be finite");
  if ((int64_t)batch * hkv > 65535)
    return fail(KV_ERR_INVALID_ARG, "kv_decode_attn_scored: batch x num_kv_heads must be <= 65535");
  int32_t max_len = 0;
  for (int32_t b = 0; b < batch; ++b) {
    if (!req_ok(P, req_ids[b])) return fail(KV_ERR_INVALID_ARG, "kv_decode_attn_scored: request %d not open", req_ids[b]);
    const Request& R = P->reqs[req_ids[b]];
    if ((int64_t)R.loc.size() > score_stride)
      return fail(KV_ERR_INVALID_ARG, "kv_decode_attn_scored: request %d has %lld positions, the rows of scores hold %lld",
                  req_ids[b], (long long)R.loc.size(), (long long)score_stride);
    max_len = std::max(max_len, (int32_t)R.table.size());
  }
  DeviceGuard dg(P->cfg.device);
  cudaStream_t s = (cudaStream_t)stream;
  kv_status_t st = refuse_capture("kv_decode_attn_scored", s);
  if (st != KV_OK) return st;
  if ((st = order_after_previous(P, s)) != KV_OK) return st;
  if ((st = build_plan(P, req_ids, batch, hq, KV_DECODE_MMA, s)) != KV_OK) return st;
  if (P->plan_rows > INT32_MAX)
    return fail(KV_ERR_INVALID_ARG, "kv_decode_attn_scored: the batch holds more than 2^31 - 1 (page, kv head) pairs");
  if ((st = sync_positions(P, s)) != KV_OK) return st;
  const int g = hq / hkv;
  const size_t ml_off = ((size_t)P->plan_rows * g * kPage * sizeof(float) + 255) & ~size_t(255);
  if ((st = ensure(P->logits, ml_off + (size_t)P->n_units * g * sizeof(float2))) != KV_OK) return st;
  if ((st = ensure(P->partials, (size_t)std::max(P->n_splits, 1) * g * (kHeadDim + 4) * sizeof(float))) != KV_OK)
    return st;
  if ((st = ensure(P->frags, (size_t)std::max(P->n_units, 1) * decode_mma_frag_bytes())) != KV_OK) return st;
  const uint8_t* base = (const uint8_t*)P->plan.ptr;
  const Unit* du = (const Unit*)(base + P->plan_units_off);
  const Split* dsp = (const Split*)(base + P->plan_splits_off);
  float* logits = (float*)P->logits.ptr;
  float2* ml = (float2*)((uint8_t*)P->logits.ptr + ml_off);
  P->merge_event = nullptr;
  P->fp_pending = FpLaunch{dsp + P->n_page_splits, (const int32_t*)(base + P->plan_fpw_off), P->n_fpw, P->n_page_splits};
  KV_CUDA(launch_decode_mma_scored(P, q, hq, softmax_scale * 1.4426950408889634f, du, P->n_units, dsp,
                                   (const int32_t*)(base + P->plan_cta_off), P->n_ctas, P->frags.ptr,
                                   (float*)P->partials.ptr, out, logits, ml, s));
  if (max_len > 0)
    KV_CUDA(launch_score_add_any(g, P, du, P->n_units, max_len, ml, logits, decay, scores, score_stride, s));
  P->stat_req.assign(req_ids, req_ids + batch);
  P->stat_hq = hq;
  P->stat_skip_dead = true;   // as the scan does
  return KV_OK;
} catch (const std::bad_alloc&) {
  return fail(KV_ERR_OOM, "kv_decode_attn_scored: host allocation failed");
}
