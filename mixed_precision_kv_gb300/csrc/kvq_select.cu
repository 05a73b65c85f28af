// Selection of the cached tokens with the lowest score (kv_select_lowest), and
// the positions of the slots on the device, which it and the scored decode
// read.
//
// Per row (a request, or a request and kv head): among the positions that are
// live and older than the protected window, the n of least key, a tie going to
// the lower position; listed in ascending order.  Keys are the scores' bits
// mapped to unsigned integers of the same order (-0 as +0, NaN last), so the
// choice is exact whatever the order of the work.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <vector>

#include "kvq_host.h"

namespace kvq {
namespace {

// ---- positions -------------------------------------------------------------
struct PosRow {
  int32_t pos[kPage];
};
constexpr size_t kPosChunk = 1 << 16;   // page rows per upload

__global__ void pos_scatter_kernel(const int32_t* __restrict__ ids, const PosRow* __restrict__ rows, int n,
                                   int32_t* __restrict__ d_pos) {
  const int x = blockIdx.x * blockDim.x + threadIdx.x;
  if (x < n * kPage) d_pos[(size_t)ids[x / kPage] * kPage + x % kPage] = rows[x / kPage].pos[x % kPage];
}

// ---- selection -------------------------------------------------------------
// One row of the selection.
struct SelRow {
  int32_t b;        // index into the caller's requests
  int32_t req;
  int32_t limit;    // positions [0, limit) may be chosen
  int32_t want;     // how many
};

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);   // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Eligible positions as bits, one row of words per request (rows_per = 1) or
// per request and kv head (rows_per = hkv).  Warp = a page, lane = slot.
__global__ void __launch_bounds__(256) eligible_kernel(const SelRow* __restrict__ rows, const Entry* __restrict__ table,
                                                       int max_pages, const int32_t* __restrict__ ntab,
                                                       const uint32_t* __restrict__ hdead,
                                                       const int32_t* __restrict__ pos, int hkv, int rows_per,
                                                       int words, uint32_t* __restrict__ bits) {
  const SelRow r = rows[blockIdx.y];
  const int lane = threadIdx.x & 31;
  const int p = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (p >= ntab[r.req]) return;
  const Entry e = table[(size_t)r.req * max_pages + p];
  const int32_t at = pos[(size_t)e.id * kPage + lane];
  for (int h = 0; h < rows_per; ++h) {
    uint32_t live = e.live;
    if (hdead) {
      if (rows_per > 1) {
        live &= ~hdead[(size_t)e.id * hkv + h];
      } else {   // all heads together: a slot that some head still reads
        uint32_t any = 0u;
        for (int x = 0; x < hkv; ++x) any |= ~hdead[(size_t)e.id * hkv + x];
        live &= any;
      }
    }
    const bool can = ((live >> lane) & 1u) && at < r.limit;
    if (can) atomicOr(&bits[((size_t)blockIdx.y * rows_per + h) * words + (at >> 5)], 1u << (at & 31));
  }
}

// Keys of the rows that sum their kv heads: the sum in 64 bits, rounded once.
__global__ void __launch_bounds__(256) sum_key_kernel(const SelRow* __restrict__ rows, const float* __restrict__ scores,
                                                      int64_t stride, int hkv, int max_len, uint32_t* __restrict__ keys) {
  const SelRow r = rows[blockIdx.y];
  const int x = blockIdx.x * 256 + threadIdx.x;
  if (x >= r.limit) return;
  double sum = 0.0;
  for (int h = 0; h < hkv; ++h) sum += (double)scores[((size_t)r.b * hkv + h) * stride + x];
  keys[(size_t)blockIdx.y * max_len + x] = order_key((float)sum);
}

// One CTA per row: radix selection by 8-bit digits, then an ordered listing.
__global__ void __launch_bounds__(1024) select_kernel(const SelRow* __restrict__ rows, const uint32_t* __restrict__ bits,
                                                      int bit_rows_per, int words, const float* __restrict__ scores,
                                                      int64_t stride, int hkv, const uint32_t* __restrict__ keys,
                                                      int max_len, int rows_per, int32_t* __restrict__ out,
                                                      int64_t out_stride) {
  __shared__ uint32_t hist[256], warp_n[32], warp_t[32];
  __shared__ uint32_t s_prefix, s_left;
  const int row = blockIdx.x / rows_per, h = blockIdx.x - row * rows_per;
  const SelRow r = rows[row];
  const uint32_t* bw = bits + ((size_t)row * bit_rows_per + (bit_rows_per > 1 ? h : 0)) * words;
  const float* sc = scores + ((size_t)r.b * hkv + h) * stride;
  const uint32_t* ky = keys ? keys + (size_t)row * max_len : nullptr;
  int32_t* o = out + ((size_t)r.b * rows_per + h) * out_stride;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  auto key_at = [&](int x) { return ky ? ky[x] : order_key(sc[x]); };
  auto can = [&](int x) { return x < r.limit && ((bw[x >> 5] >> (x & 31)) & 1u); };
  uint32_t prefix = 0u, left = (uint32_t)r.want;
  bool all = false;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0u;
    __syncthreads();
    for (int x = tid; x < r.limit; x += 1024)
      if (can(x)) {
        const uint32_t k = key_at(x);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
    __syncthreads();
    if (tid == 0) {
      uint32_t n = left;
      int d = 0;
      while (d < 256 && hist[d] < n) n -= hist[d++];
      s_prefix = d < 256 ? (prefix | ((uint32_t)d << shift)) : 0xFFFFFFFFu;
      s_left = d < 256 ? n : 0xFFFFFFFFu;   // fewer eligible positions than wanted: all of them
    }
    __syncthreads();
    if (s_left == 0xFFFFFFFFu) {
      all = true;
      break;
    }
    prefix = s_prefix;
    left = s_left;
    __syncthreads();
  }
  // take keys below prefix and the first `left` that equal it
  uint32_t base = 0u, ties = 0u;
  for (int x0 = 0; x0 < r.limit; x0 += 1024) {
    const int x = x0 + tid;
    const bool c = can(x);
    const uint32_t k = c ? key_at(x) : 0u;
    const bool below = c && (all || k < prefix), tie = c && !all && k == prefix;
    const uint32_t tb = __ballot_sync(0xFFFFFFFFu, tie);
    if (lane == 0) warp_t[w] = __popc(tb);
    __syncthreads();
    uint32_t before = ties, total_t = 0u;
    for (int y = 0; y < 32; ++y) {
      if (y < w) before += warp_t[y];
      total_t += warp_t[y];
    }
    before += __popc(tb & ((1u << lane) - 1u));
    const bool take = below || (tie && before < left);
    const uint32_t nb = __ballot_sync(0xFFFFFFFFu, take);
    if (lane == 0) warp_n[w] = __popc(nb);
    __syncthreads();
    uint32_t at = base, total = 0u;
    for (int y = 0; y < 32; ++y) {
      if (y < w) at += warp_n[y];
      total += warp_n[y];
    }
    at += __popc(nb & ((1u << lane) - 1u));
    if (take) o[at] = x;
    base += total;
    ties += total_t;
    __syncthreads();
  }
  for (int64_t x = base + tid; x < out_stride; x += 1024) o[x] = -1;
}

}  // namespace

kv_status_t refuse_capture(const char* what, cudaStream_t s) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  KV_CUDA(cudaStreamIsCapturing(s, &cs));
  if (cs != cudaStreamCaptureStatusNone)
    return fail(KV_ERR_STATE, "%s: the call plans on the host and cannot be captured into a graph", what);
  return KV_OK;
}

kv_status_t sync_positions(kv_pool* P, cudaStream_t s) {
  std::vector<int32_t>& ids = P->pos_dirty;
  if (!P->d_pos) {
    const size_t n = P->fill.size() * (size_t)kPage;
    if (cudaMalloc(&P->d_pos, n * sizeof(int32_t)) != cudaSuccess) {
      cudaGetLastError();
      P->d_pos = nullptr;
      return fail(KV_ERR_OOM, "cannot allocate the positions of %zu slots", n);
    }
    ids.clear();
    for (const Request& R : P->reqs) ids.insert(ids.end(), R.table.begin(), R.table.end());
  }
  if (ids.empty()) return KV_OK;
  std::sort(ids.begin(), ids.end());
  ids.erase(std::unique(ids.begin(), ids.end()), ids.end());
  std::vector<PosRow> rows;
  for (size_t a = 0; a < ids.size(); a += kPosChunk) {
    const size_t n = std::min(kPosChunk, ids.size() - a);
    rows.resize(n);
    for (size_t x = 0; x < n; ++x)
      std::copy_n(&P->pos[(size_t)ids[a + x] * kPage], kPage, rows[x].pos);
    Upload u;
    const size_t oi = u.add(ids.data() + a, n * sizeof(int32_t)), orow = u.add(rows.data(), n * sizeof(PosRow));
    const kv_status_t st = upload(P, u, s);
    if (st != KV_OK) return st;
    const uint8_t* base = (const uint8_t*)P->upload.ptr;
    ++P->launches;
    pos_scatter_kernel<<<(unsigned)((n * kPage + 255) / 256), 256, 0, s>>>((const int32_t*)(base + oi),
                                                                           (const PosRow*)(base + orow), (int)n, P->d_pos);
    KV_CUDA(cudaGetLastError());
  }
  ids.clear();
  return KV_OK;
}

}  // namespace kvq

using namespace kvq;

extern "C" kv_status_t kv_select_lowest(kv_pool_t* P, const float* scores, int64_t score_stride, const int32_t* req_ids,
                                        const int32_t* n_select, int32_t n_req, int64_t protect, int32_t per_head,
                                        int32_t* out, int64_t out_stride, void* stream) {
  if (!P) return fail(KV_ERR_INVALID_ARG, "kv_select_lowest: null pool");
  if (!scores || !req_ids || !n_select || n_req < 1 || protect < 0 || out_stride < 0 || (out_stride > 0 && !out))
    return fail(KV_ERR_INVALID_ARG, "kv_select_lowest: bad arguments");
  const int hkv = P->cfg.num_kv_heads, rows_per = per_head ? hkv : 1;
  if (n_req > 65535) return fail(KV_ERR_INVALID_ARG, "kv_select_lowest: at most 65535 requests");
  std::vector<SelRow> rows((size_t)n_req);
  int32_t max_len = 0, max_pages = 0;
  for (int32_t b = 0; b < n_req; ++b) {
    if (!req_ok(P, req_ids[b])) return fail(KV_ERR_INVALID_ARG, "kv_select_lowest: request %d not open", req_ids[b]);
    const Request& R = P->reqs[req_ids[b]];
    const int64_t n = (int64_t)R.loc.size();
    if (n > score_stride)
      return fail(KV_ERR_INVALID_ARG, "kv_select_lowest: request %d has %lld positions, the rows of scores hold %lld",
                  req_ids[b], (long long)n, (long long)score_stride);
    if (n_select[b] < 0 || n_select[b] > out_stride)
      return fail(KV_ERR_INVALID_ARG, "kv_select_lowest: n_select[%d] = %d is not in [0, out_stride]", b, n_select[b]);
    rows[(size_t)b] = SelRow{b, req_ids[b], (int32_t)std::max<int64_t>(0, n - protect), n_select[b]};
    max_len = std::max(max_len, rows[(size_t)b].limit);
    max_pages = std::max(max_pages, (int32_t)R.table.size());
  }
  if (out_stride == 0) return KV_OK;
  DeviceGuard dg(P->cfg.device);
  cudaStream_t s = (cudaStream_t)stream;
  kv_status_t st = refuse_capture("kv_select_lowest", s);
  if (st != KV_OK) return st;
  if ((st = order_after_previous(P, s)) != KV_OK) return st;
  if ((st = sync_positions(P, s)) != KV_OK) return st;
  const bool hd = !P->hdead.empty();
  const int bit_rows_per = per_head && hd ? hkv : 1;
  const int words = std::max(1, (max_len + 31) / 32);
  const size_t bit_bytes = (size_t)n_req * bit_rows_per * words * sizeof(uint32_t);
  const size_t rows_off = (bit_bytes + 255) & ~size_t(255);
  const size_t key_off = (rows_off + (size_t)n_req * sizeof(SelRow) + 255) & ~size_t(255);
  const size_t key_bytes = per_head ? 0 : (size_t)n_req * std::max(1, max_len) * sizeof(uint32_t);
  if ((st = ensure(P->select, key_off + key_bytes)) != KV_OK) return st;
  uint8_t* base = (uint8_t*)P->select.ptr;
  uint32_t* bits = (uint32_t*)base;
  const SelRow* d_rows = (const SelRow*)(base + rows_off);
  uint32_t* keys = per_head ? nullptr : (uint32_t*)(base + key_off);
  Upload u;
  u.add(rows.data(), rows.size() * sizeof(SelRow));
  if ((st = h2d(P, base + rows_off, u, s)) != KV_OK) return st;
  KV_CUDA(cudaMemsetAsync(bits, 0, bit_bytes, s));
  if (max_pages > 0 && max_len > 0) {
    ++P->launches;
    eligible_kernel<<<dim3((unsigned)((max_pages + 7) / 8), (unsigned)n_req), 256, 0, s>>>(
        d_rows, P->d_table, P->cfg.max_pages_per_request, P->d_ntab, hd ? P->d_hdead : nullptr, P->d_pos, hkv,
        bit_rows_per, words, bits);
    KV_CUDA(cudaGetLastError());
    if (!per_head) {
      ++P->launches;
      sum_key_kernel<<<dim3((unsigned)((max_len + 255) / 256), (unsigned)n_req), 256, 0, s>>>(
          d_rows, scores, score_stride, hkv, max_len, keys);
      KV_CUDA(cudaGetLastError());
    }
  }
  ++P->launches;
  select_kernel<<<(unsigned)(n_req * rows_per), 1024, 0, s>>>(d_rows, bits, bit_rows_per, words, scores, score_stride,
                                                             hkv, keys, max_len, rows_per, out, out_stride);
  KV_CUDA(cudaGetLastError());
  return KV_OK;
}
