// Host side of kv_attend: checks, the units of the call and the choice of the
// kernel.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <vector>

#include "kvq_attend.h"
#include "kvq_host.h"

using namespace kvq;

extern "C" kv_status_t kv_attend(kv_pool_t* P, const void* q, const void* k, const void* v, const uint64_t* tree,
                                 const int32_t* req_ids, const int32_t* n_new, int32_t n_req, int32_t hq,
                                 float softmax_scale, void* out, void* stream) {
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

  std::vector<AttUnit> units;
  units.reserve((size_t)n_req * hkv);
  int64_t tok0 = 0;
  for (int32_t b = 0; b < n_req; ++b) {
    const int32_t r = req_ids[b];
    if (n_new[b] > 0)
      for (int h = 0; h < hkv; ++h)
        units.push_back(AttUnit{r, h, n_new[b], (int32_t)P->reqs[r].table.size(), P->n_fp.empty() ? 0 : P->n_fp[r], 0, tok0});
    tok0 += n_new[b];
  }
  Upload u;
  const size_t ou = u.add(units.data(), units.size() * sizeof(AttUnit));
  if ((st = ensure(P->attend, u.size)) != KV_OK) return st;
  if ((st = h2d(P, P->attend.ptr, u, s)) != KV_OK) return st;
  const AttUnit* du = (const AttUnit*)((const uint8_t*)P->attend.ptr + ou);
  KV_CUDA(launch_attend_simt(P, A, du, (int)units.size(), max_new * g, s));
  return KV_OK;
}
