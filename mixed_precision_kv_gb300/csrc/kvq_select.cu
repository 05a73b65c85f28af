// Selection of the cached tokens with the lowest score (kv_select_lowest), and
// the positions of the slots on the device, which it and the scored decode
// read.
//
// Per row (a request, or a request and kv head): among the positions that are
// live and older than the protected window, the n of least key, a tie going to
// the lower position; listed in ascending order.  Keys are the scores' bits
// mapped to unsigned integers of the same order (-0 as +0, NaN last), so the
// choice is exact whatever the order of the work.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <new>
#include <vector>

#include "kvq_host.h"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

// ---- positions -------------------------------------------------------------
struct PosRow {
  int32_t pos[kPage];
};
constexpr size_t kPosChunk = 1 << 11;   // page rows per upload: one copy runs while the next is gathered

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
  if (x != x) return 0xFFFFFFFEu;   // 0xFFFFFFFF marks a position that may not be chosen
  const uint32_t u = __float_as_uint(x + 0.0f);   // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The rows of a call, by value while they fit the parameters.
constexpr int kRowsByValue = 128;
struct SelRows {
  SelRow r[kRowsByValue];
};

// Which of a page's slots may be chosen (bits): live, for the row's head or for any.
__device__ __forceinline__ uint32_t eligible_slots(const Entry& e, const uint32_t* hdead, int hkv, int h, bool per_head) {
  uint32_t live = e.live;
  if (hdead) {
    if (per_head) {
      live &= ~hdead[(size_t)e.id * hkv + h];
    } else {   // all heads together: a slot that some head still reads
      uint32_t any = 0u;
      for (int x = 0; x < hkv; ++x) any |= ~hdead[(size_t)e.id * hkv + x];
      live &= any;
    }
  }
  return live;
}
// Key of a position: the head's score, or the heads' sum taken in fp64, head after head,
// and rounded once.  fp64 runs at 1/64 of the fp32 rate here, so the sum is carried as an
// unevaluated pair of fp32 first:
//   hi + f = t + e exactly (e: the two-sum's error), hi <- t, lo <- fl(lo + e).
// With u = 2^-24, n heads and m >= sum |f|, every |e| <= u m, so |lo| <= n u m.
//   - Every f is a multiple of q = ulp(least |f| above 0) > u least |f|.  Where n u m <= least
//     |f|, lo and the fp64 sums are multiples of q below 2^24 q and 2^53 q: both sums are
//     exact, and hi + lo rounds once.  So it is for scores of one scale (0 of 10^6 sums of 2
//     to 16 lognormal scores, of sigma 2, fail this).
//   - Else lo's n roundings add up to n^2 u^2 m at most, and the fp64 sum is within n 2^-53 m of
//     the exact one, so it lies within 2^-47 n^2 m of hi + lo; where both ends of that range
//     round to the same fp32, so does it.
//   - Else (next to the middle of two fp32 values, where terms cancel, or not finite) it is
//     taken again in fp64.
__device__ __noinline__ float sum_wide(const float* sc, int64_t stride, int hkv, int x) {
  double sum = 0.0;
  for (int y = 0; y < hkv; ++y) sum += (double)__ldg(sc + (size_t)y * stride + x);
  return (float)sum;
}
__device__ __forceinline__ uint32_t key_of(const float* sc, int64_t stride, int hkv, int h, bool per_head, int x) {
  if (per_head) return order_key(__ldg(sc + (size_t)h * stride + x));
  float hi = 0.0f, lo = 0.0f, m = 0.0f;
  uint32_t least = 0xFFFFFFFFu;   // 2 |f|'s bits - 1: a zero is no least
  auto add = [&](float f) {
    const float t = __fadd_rn(hi, f), b = __fsub_rn(t, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(f, b)));
    hi = t;
    m = __fadd_ru(m, fabsf(f));
    least = min(least, (__float_as_uint(f) << 1) - 1u);
  };
  const float* p = sc + x;
  int y = 0;
  for (; y + 8 <= hkv; y += 8, p += 8 * stride) {
    float f[8];
#pragma unroll
    for (int z = 0; z < 8; ++z) f[z] = __ldg(p + z * stride);
#pragma unroll
    for (int z = 0; z < 8; ++z) add(f[z]);
  }
  for (; y < hkv; ++y, p += stride) add(__ldg(p));
  const float sum = __fadd_rn(hi, lo);
  bool sure = __fmul_ru(m, (float)hkv * 0x1p-24f) <= __uint_as_float((least + 1u) >> 1);
  if (!sure) {
    const float b = __fsub_rn(sum, hi), rest = __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, b)), __fsub_rn(lo, b));   // hi + lo = sum + rest
    const float most = __fmul_ru(m, (float)(hkv * hkv) * 0x1p-47f);
    sure = __fadd_rn(sum, __fadd_ru(rest, most)) == sum && __fadd_rn(sum, __fadd_rd(rest, -most)) == sum;
  }
  sure = sure && fabsf(sum) < INFINITY;   // an overflow on the way leaves an infinity or a NaN behind
  return order_key(sure ? sum : sum_wide(sc, stride, hkv, x));
}
// Inclusive sum over the block's 512 threads; `total` is the whole sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sum, uint32_t& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[w] = x;
  __syncthreads();
  uint32_t t = warp_sum[lane & 15];   // lanes 16 .. 31: the same, not read below
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, t, o);
    if (lane >= o) t += y;
  }
  total = __shfl_sync(0xFFFFFFFFu, t, 15);
  const uint32_t before = w ? __shfl_sync(0xFFFFFFFFu, t, w - 1) : 0u;
  __syncthreads();
  return before + x;
}

// *p |= v in CTA `rank` of the cluster, without waiting for the old value (a call alone
// on 16 rows of 100K: 83.5 us, 87.7 with an atomicOr through the mapped pointer).
__device__ __forceinline__ void or_in_cluster(uint32_t* p, uint32_t rank, uint32_t v) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// A cluster of CTAs per row; CTA c holds the keys of positions [c per, (c + 1) per)
// in shared memory, so the scores are read once and the rest stays on the SMs:
//   the table's pages, a share per CTA, set the eligible positions' bits where they
//   belong (a page's slots are one or two runs of positions, so a warp sends one or
//   two words); keys; radix selection by digits of 11 bits, the CTAs' histograms
//   added up through distributed shared memory; an ordered listing.
// Bound by the scores' bytes for long rows, by a dozen barriers for short ones.
// 16 x 100K positions, 8 heads summed: 66 us, of which the eligible positions and the
// keys take a third each; 380 with one CTA per row that reads its keys once per digit.
constexpr int kSelThreads = 512;            // (1024, and no limit of two CTAs per SM below: 64 rows of 20K to 32K 73 us, 38 so)
constexpr int kSelStored = 48 * 1024;      // positions per CTA whose keys fit its shared memory
constexpr int kSelMost = 3 * 512 * 1024;   // ... whose bits do
constexpr int sel_smem(int per) { return (per <= kSelStored ? per * 4 : 0) + per / 8; }
constexpr int kBins = 2048;                // digits of 11, 11 and 10 bits
static_assert(kBins == 4 * kSelThreads, "four bins per thread");
struct SelShared {
  alignas(16) uint32_t hist[3][kBins];
  uint32_t warp_sum[32];
  uint32_t below, ties;      // of this CTA
  uint32_t digit, left;
};
template <bool kStored>
__global__ void __launch_bounds__(kSelThreads) select_kernel(
    SelRows by_value, const SelRow* __restrict__ rows, const Entry* __restrict__ table, int max_pages,
    const int32_t* __restrict__ ntab, const uint32_t* __restrict__ hdead, const int32_t* __restrict__ pos, int hkv,
    int per_head, const float* __restrict__ scores, int64_t stride, int per, int32_t* __restrict__ out,
    int64_t out_stride) {
  extern __shared__ __align__(16) uint32_t keys[];   // kStored: per keys; then per / 32 words of bits
  __shared__ SelShared S;
  cg::cluster_group cl = cg::this_cluster();
  const int n_cta = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int rows_per = per_head ? hkv : 1;
  const int idx = (int)(blockIdx.x / n_cta), row = idx / rows_per, h = idx - row * rows_per;
  const SelRow r = rows ? rows[row] : by_value.r[row];
  const float* sc = scores + (size_t)r.b * hkv * stride;
  int32_t* o = out + (size_t)idx * out_stride;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  uint32_t* bits = keys + (kStored ? per : 0);
  const int words = per >> 5;
  const int n_pages = r.limit > 0 ? ntab[r.req] : 0;   // (a request that was never appended to has no length there)
  for (int x = tid; x < words; x += kSelThreads) bits[x] = 0u;
  for (int x = tid; x < 3 * kBins; x += kSelThreads) (&S.hist[0][0])[x] = 0u;
  if (tid == 0) S.below = S.ties = 0u;
  cl.sync();
  // ---- eligible positions: a warp takes up to 32 pages, their entries at once, their positions by eights
  const Entry* tab = table + (size_t)r.req * max_pages;
  constexpr int kWarps = kSelThreads / 32;
  const float inv_words = 1.0f / (float)words;
  const int warps = n_cta * kWarps, share = min(32, max(1, (n_pages + warps - 1) / warps));
  for (int p0 = (rank * kWarps + w) * share; p0 < n_pages; p0 += warps * share) {
    const int n = min(share, n_pages - p0);
    Entry e{-1, 0u};
    uint32_t can = 0u;
    if (lane < n) {
      e = tab[p0 + lane];
      if (e.id >= 0) can = eligible_slots(e, hdead, hkv, h, per_head);
    }
    for (int y0 = 0; y0 < n; y0 += 8) {
      uint32_t m[8];
      int32_t at[8];
#pragma unroll
      for (int y = 0; y < 8; ++y) {   // y0 + y <= 31; lanes from n on have no slots
        m[y] = __shfl_sync(0xFFFFFFFFu, can, y0 + y);
        const int32_t id = __shfl_sync(0xFFFFFFFFu, e.id, y0 + y);
        at[y] = m[y] ? pos[(size_t)id * kPage + lane] : 0;
      }
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        if (m[y] == 0u) continue;   // the same for the whole warp
        const bool take = ((m[y] >> lane) & 1u) && (uint32_t)at[y] < (uint32_t)r.limit;
        const int word = take ? at[y] >> 5 : -1;
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, word);
        if (take) {
          const uint32_t set = __reduce_or_sync(peers, 1u << (at[y] & 31));
          if (lane == __ffs(peers) - 1) {
            // word / words: exact, as (word + 1/2) / words is at least 1 / (2 words) > 8 2^-22 from an integer
            const int cta = (int)(((float)word + 0.5f) * inv_words);
            or_in_cluster(bits + (word - cta * words), (uint32_t)cta, set);
          }
        }
      }
    }
  }
  cl.sync();
  // ---- keys of this CTA's positions
  const int x0 = rank * per, mine = max(0, min(per, r.limit - x0));
  auto fresh = [&](int x) {
    return (bits[x >> 5] >> (x & 31)) & 1u ? key_of(sc, stride, hkv, h, per_head, x0 + x) : 0xFFFFFFFFu;
  };
  if constexpr (kStored) {
#pragma unroll 4
    for (int x = tid; x < mine; x += kSelThreads) keys[x] = fresh(x);
    __syncthreads();
  }
  auto key = [&](int x) { return kStored ? keys[x] : fresh(x); };
  // ---- the n-th least key, digit by digit
  uint32_t prefix = 0u, left = (uint32_t)r.want;
  bool all = false;
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0);
    const uint32_t mask = d == 2 ? 1023u : 2047u;
    const uint32_t high = d == 0 ? 0u : (d == 1 ? 0xFFE00000u : 0xFFFFFC00u);   // the bits settled so far
    for (int y = tid; y < ((mine + 127) >> 7) << 5; y += kSelThreads) {   // whole warps, four positions a thread
      uint32_t b[4];
      if constexpr (kStored) {
        const uint4 k = 4 * y < per ? reinterpret_cast<const uint4*>(keys)[y] : make_uint4(0u, 0u, 0u, 0u);
        b[0] = k.x; b[1] = k.y; b[2] = k.z; b[3] = k.w;
      }
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int x = 4 * y + z;
        const uint32_t k = x >= mine ? 0xFFFFFFFFu : (kStored ? b[z] : fresh(x));
        b[z] = k != 0xFFFFFFFFu && ((k ^ prefix) & high) == 0u ? (k >> shift) & mask : 0xFFFFFFFFu;
      }
      const uint32_t f = __shfl_sync(0xFFFFFFFFu, b[0], 0);
      if (__all_sync(0xFFFFFFFFu, b[0] == f && b[1] == f && b[2] == f && b[3] == f)) {   // scores crowd into few digits
        if (f != 0xFFFFFFFFu && lane == 0) atomicAdd(&S.hist[d][f], 128u);
      } else {
#pragma unroll
        for (int z = 0; z < 4; ++z)
          if (b[z] != 0xFFFFFFFFu) atomicAdd(&S.hist[d][b[z]], 1u);
      }
    }
    if (tid == 0) S.digit = 0xFFFFFFFFu;
    cl.sync();
    {
      // bins 4 tid .. 4 tid + 3 over all CTAs, then the first whose running sum reaches `left`
      uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll 8
      for (int y = 0; y < n_cta; ++y) {
        const uint4 q = reinterpret_cast<const uint4*>(cl.map_shared_rank(&S.hist[d][0], y))[tid];
        v[0] += q.x; v[1] += q.y; v[2] += q.z; v[3] += q.w;
      }
      uint32_t total;
      uint32_t run = block_scan(v[0] + v[1] + v[2] + v[3], S.warp_sum, total) - (v[0] + v[1] + v[2] + v[3]);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        if (run < left && run + v[y] >= left) {   // one bin at most, none if there are too few (or left is 0)
          S.digit = 4u * tid + y;
          S.left = left - run;
        }
        run += v[y];
      }
    }
    __syncthreads();
    if (S.digit == 0xFFFFFFFFu) {   // fewer eligible positions than wanted: all of them (or none wanted)
      all = left > 0u;
      break;
    }
    prefix |= S.digit << shift;
    left = S.left;
    __syncthreads();
  }
  const bool none = r.want == 0;
  // ---- counts per CTA, then the listing: a thread takes a run of positions (an odd number of them)
  const int run = ((per + kSelThreads - 1) / kSelThreads) | 1;
  const int a = min(mine, tid * run), e = min(mine, a + run);
  uint32_t nb = 0u, nt = 0u;
  for (int x = a; x < e; ++x) {
    const uint32_t k = key(x);
    if (k == 0xFFFFFFFFu) continue;
    nb += (all || k < prefix) ? 1u : 0u;
    nt += (!all && k == prefix) ? 1u : 0u;
  }
  if (none) nb = nt = 0u;
  uint32_t tb, tt;
  const uint32_t sb = block_scan(nb, S.warp_sum, tb), st = block_scan(nt, S.warp_sum, tt);
  if (tid == 0) {
    S.below = tb;
    S.ties = tt;
  }
  cl.sync();
  // every CTA's counts, one per lane
  uint32_t yb = 0u, yt = 0u;
  if (lane < n_cta) {
    const SelShared* q = cl.map_shared_rank(&S, lane);
    yb = q->below;
    yt = q->ties;
  }
  uint32_t off = 0u, ties_before = 0u, count = 0u, tie_all = 0u;
  for (int y = 0; y < n_cta; ++y) {
    const uint32_t cb = __shfl_sync(0xFFFFFFFFu, yb, y), ct = __shfl_sync(0xFFFFFFFFu, yt, y);
    const uint32_t took = cb + min(ct, left - min(left, tie_all));
    if (y < rank) {
      off += took;
      ties_before += ct;
    }
    count += took;
    tie_all += ct;
  }
  uint32_t t = ties_before + st - nt;   // ties before this thread's run; those before `left` are taken
  off += sb - nb + (min(t, max(left, ties_before)) - ties_before);
  if (!none)
    for (int x = a; x < e; ++x) {
      const uint32_t k = key(x);
      if (k == 0xFFFFFFFFu) continue;
      bool take = all || k < prefix;
      if (!all && k == prefix) take = t++ < left;
      if (take) o[off++] = x0 + x;
    }
  for (int64_t x = count + (int64_t)rank * kSelThreads + tid; x < out_stride; x += (int64_t)n_cta * kSelThreads) o[x] = -1;
  cl.sync();   // the shared memory of every CTA is still read above
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
  const bool first = !P->d_pos;
  if (first) {
    ids.clear();
    for (const Request& R : P->reqs) ids.insert(ids.end(), R.table.begin(), R.table.end());
    const size_t n = P->fill.size() * (size_t)kPage;
    if (cudaMalloc(&P->d_pos, n * sizeof(int32_t)) != cudaSuccess) {
      cudaGetLastError();
      P->d_pos = nullptr;
      return fail(KV_ERR_OOM, "cannot allocate the positions of %zu slots", n);
    }
  }
  if (ids.empty()) return KV_OK;
  if (!first) {   // (a page is in one table, once)
    std::sort(ids.begin(), ids.end());
    ids.erase(std::unique(ids.begin(), ids.end()), ids.end());
  }
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
                                        int32_t* out, int64_t out_stride, void* stream) try {
  if (!P) return fail(KV_ERR_INVALID_ARG, "kv_select_lowest: null pool");
  if (!scores || !req_ids || !n_select || n_req < 1 || protect < 0 || out_stride < 0 || (out_stride > 0 && !out))
    return fail(KV_ERR_INVALID_ARG, "kv_select_lowest: bad arguments");
  const int hkv = P->cfg.num_kv_heads, rows_per = per_head ? hkv : 1;
  if (n_req > 65535) return fail(KV_ERR_INVALID_ARG, "kv_select_lowest: at most 65535 requests");
  std::vector<SelRow> rows((size_t)n_req);
  int32_t max_len = 0;
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
  }
  if (out_stride == 0) return KV_OK;
  DeviceGuard dg(P->cfg.device);
  cudaStream_t s = (cudaStream_t)stream;
  kv_status_t st = refuse_capture("kv_select_lowest", s);
  if (st != KV_OK) return st;
  if ((st = order_after_previous(P, s)) != KV_OK) return st;
  if ((st = sync_positions(P, s)) != KV_OK) return st;
  const bool hd = !P->hdead.empty();
  // CTAs per row: at most two per SM over all rows (more would wait for a place: 64 rows of 20-32K
  // positions took 52 us with 256 CTAs and 72 us with 512), 2,048 positions or more each, and as many
  // as the row's keys need; clusters of 16 were slower than of 8 (16 rows of 100K: 117 and 62 us).
  const int n_rows = n_req * rows_per;
  int n_cta = 1;
  while (n_cta < 8 && max_len > 2048 * n_cta && (int64_t)n_rows * n_cta * 2 <= 2 * P->sm_count) n_cta *= 2;
  while (n_cta < 8 && max_len > kSelStored * n_cta) n_cta *= 2;
  if (max_len > kSelMost * n_cta)
    return fail(KV_ERR_INVALID_ARG, "kv_select_lowest: a request holds more than %d positions", 8 * kSelMost);
  const int per = std::max(32, ((max_len + n_cta - 1) / n_cta + 31) & ~31);
  auto* kernel = per <= kSelStored ? select_kernel<true> : select_kernel<false>;   // longer rows read their keys again
  static std::atomic<uint64_t> attr_set{0};
  if (!(attr_set.load() >> (P->cfg.device & 63) & 1u)) {
    KV_CUDA(cudaFuncSetAttribute(select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, sel_smem(kSelStored)));
    KV_CUDA(cudaFuncSetAttribute(select_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, sel_smem(kSelMost)));
    attr_set.fetch_or(uint64_t(1) << (P->cfg.device & 63));
  }
  SelRows by_value;
  const SelRow* d_rows = nullptr;
  if (n_req <= kRowsByValue) {
    std::copy(rows.begin(), rows.end(), by_value.r);
  } else {
    Upload u;
    u.add(rows.data(), rows.size() * sizeof(SelRow));
    if ((st = ensure(P->select, u.size)) != KV_OK) return st;
    if ((st = h2d(P, P->select.ptr, u, s)) != KV_OK) return st;
    d_rows = (const SelRow*)P->select.ptr;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)n_cta;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n_rows * n_cta));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = (size_t)sel_smem(per);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ++P->launches;
  KV_CUDA(cudaLaunchKernelEx(&cfg, kernel, by_value, d_rows, (const Entry*)P->d_table,
                             (int)P->cfg.max_pages_per_request, (const int32_t*)P->d_ntab,
                             (const uint32_t*)(hd ? P->d_hdead : nullptr), (const int32_t*)P->d_pos, hkv,
                             (int)(per_head ? 1 : 0), scores, score_stride, per, out, out_stride));
  return KV_OK;
} catch (const std::bad_alloc&) {
  return fail(KV_ERR_OOM, "kv_select_lowest: host allocation failed");
}
