// kv_read_tokens: cached tokens' values, dequantized, by token position.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <new>
#include <vector>

#include "kvq_attend.h"
#include "kvq_host.h"

namespace kvq {
namespace {

// One request of a call: positions [first, first + n) go to rows row0 .. of the outputs.
struct ReadRow {
  int32_t req, n_pages;
  int32_t first, n;
  int64_t row0;
};
constexpr int kReadByValue = 64;
struct ReadRows {
  ReadRow r[kReadByValue];
};

struct ReadArgs {
  const uint8_t* pool;
  size_t int4_off, int3_off, fp4_off;
  int64_t n2, n3b, nfb;
  const Entry* table;
  const uint32_t* hdead;
  const int32_t* pos;
  void *k, *v;           // either may be null
  int32_t max_pages, hkv;
};

constexpr int kReadThreads = 128;

__device__ __forceinline__ float half_lo(uint32_t w) { return __half2float(__ushort_as_half((uint16_t)w)); }
__device__ __forceinline__ float half_hi(uint32_t w) { return __half2float(__ushort_as_half((uint16_t)(w >> 16))); }
__device__ __forceinline__ float half_of(const uint8_t* p) { return __half2float(*reinterpret_cast<const __half*>(p)); }

// 8 values of a row, rounded once to bf16 or kept
template <bool kF32>
__device__ __forceinline__ void put8(void* out, size_t at, const float (&x)[8]) {
  if constexpr (kF32) {
    float4* p = reinterpret_cast<float4*>((float*)out + at);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(x[2 * k + 1]), "f"(x[2 * k]));
    *reinterpret_cast<uint4*>((uint16_t*)out + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// K: channels 8 c8 .. 8 c8 + 7 of slot t.
__device__ __forceinline__ void k_values(const uint8_t* b, int cls, int t, int c8, float (&x)[8]) {
  const int gr = c8 >> 2, i = c8 & 3;
  if (cls == kClsInt2) {
    const uint32_t w = __ldg(reinterpret_cast<const uint16_t*>(b + kI2KCodes + 32 * t + 2 * c8));
    // channel 8 c8 + n is in pair (gr, i >> 1, 4 (n >> 2) + (n & 3)), the half by i & 1 (the first pair swapped)
    const uint4* p = reinterpret_cast<const uint4*>(b + kI2KMeta + 4 * ((gr * 2 + (i >> 1)) * 8));
    const uint4 s0 = __ldg(p), s1 = __ldg(p + 1), z0 = __ldg(p + 16), z1 = __ldg(p + 17);
    const uint32_t s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    const uint32_t z[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const bool hi = ((i & 1) != 0) != (n == 0);
      x[n] = fmaf((float)((w >> (2 * n)) & 3u), hi ? half_hi(s[n]) : half_lo(s[n]), hi ? half_hi(z[n]) : half_lo(z[n]));
    }
  } else if (cls == kClsInt4) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(b + kI4KCodes + 64 * t + 16 * i + 4 * gr));
    const uint32_t m = __ldg(reinterpret_cast<const uint32_t*>(b + kI4KMeta + 16 * t + 4 * gr));
    const float s = half_lo(m), z = half_hi(m);
#pragma unroll
    for (int n = 0; n < 8; ++n) x[n] = fmaf((float)((w >> (4 * n)) & 15u), s, z);
  } else if (cls == kClsInt3) {
    const uint32_t m = __ldg(reinterpret_cast<const uint32_t*>(b + kI3KMeta + 16 * t + 4 * gr));
    const float s = half_lo(m), z = half_hi(m);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int c = 8 * c8 + n;
      const uint32_t code = (((uint32_t)b[i3k_lo_byte(t, c)] >> i3k_lo_shift(c)) & 3u) |
                            ((((uint32_t)b[i3k_hi_byte(t, c)] >> i3k_hi_shift(c)) & 1u) << 2);
      x[n] = fmaf((float)code, s, z);
    }
  } else {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(b + kF4KCodes + 64 * t + 16 * i + 4 * gr));
    const float s = half_of(b + kF4KScale + 8 * t + 2 * gr);
#pragma unroll
    for (int n = 0; n < 8; ++n) x[n] = e2m1_value((w >> (8 * (n & 3) + 4 * (n >> 2))) & 15u) * s;
  }
}

// V: the code words of channels 8 o .. 8 o + 7, slots 8 j .. 8 j + 7, and the slots' scales and zeros.
struct VBlock {
  uint32_t w[8];
  uint4 s, z;
};
__device__ __forceinline__ void v_load(const uint8_t* b, int cls, int j, int o, VBlock& B) {
  const int m = o >> 1, e = o & 1, gr = o >> 2;
#pragma unroll
  for (int r = 0; r < 8; ++r)
    B.w[r] = cls == kClsInt2 ? __ldg(reinterpret_cast<const uint32_t*>(b + kI2VCodes + 16 * (32 * (m >> 2) + 4 * r + j) + 4 * (m & 3)))
             : cls == kClsInt3 ? 0u
                               : __ldg(reinterpret_cast<const uint32_t*>(b + kI4VCodes + 16 * (32 * (m >> 1) + 4 * r + j) + 4 * (2 * (m & 1) + e)));
  const int meta = cls == kClsInt2 ? kI2VMeta : (cls == kClsInt4 ? kI4VMeta : (cls == kClsInt3 ? kI3VMeta : kF4VScale));
  B.s = __ldg(reinterpret_cast<const uint4*>(b + meta + 64 * gr + 16 * j));
  B.z = cls == kClsFp4 ? make_uint4(0u, 0u, 0u, 0u) : __ldg(reinterpret_cast<const uint4*>(b + meta + 256 + 64 * gr + 16 * j));
}
// The row of slot 8 j + k.
__device__ __forceinline__ void v_values(const VBlock& B, const uint8_t* b, int cls, int j, int o, int k, float (&x)[8]) {
  // slots k and k + 4 share a word of scales
  const uint32_t sw = (k & 3) == 0 ? B.s.x : ((k & 3) == 1 ? B.s.y : ((k & 3) == 2 ? B.s.z : B.s.w));
  const uint32_t zw = (k & 3) == 0 ? B.z.x : ((k & 3) == 1 ? B.z.y : ((k & 3) == 2 ? B.z.z : B.z.w));
  const float s = k < 4 ? half_lo(sw) : half_hi(sw), z = k < 4 ? half_lo(zw) : half_hi(zw);
  const int e = o & 1;
  if (cls == kClsInt2) {
    const int half = (k >> 2) ^ ((e == 0 && (k & 3) == 0) ? 1 : 0), sh = 8 * e + 16 * half + 2 * (k & 3);
#pragma unroll
    for (int r = 0; r < 8; ++r) x[r] = fmaf((float)((B.w[r] >> sh) & 3u), s, z);
  } else if (cls == kClsInt4) {
#pragma unroll
    for (int r = 0; r < 8; ++r) x[r] = fmaf((float)((B.w[r] >> (4 * k)) & 15u), s, z);
  } else if (cls == kClsInt3) {
    const int t = 8 * j + k;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int c = 8 * o + r;
      const uint32_t code = (((uint32_t)b[i3v_lo_byte(t, c)] >> i3v_lo_shift(t)) & 3u) |
                            ((((uint32_t)b[i3v_hi_byte(t, c)] >> i3v_hi_shift(t, c)) & 1u) << 2);
      x[r] = fmaf((float)code, s, z);
    }
  } else {
#pragma unroll
    for (int r = 0; r < 8; ++r) x[r] = e2m1_value((B.w[r] >> (8 * (k & 3) + 4 * (k >> 2))) & 15u) * s;
  }
}

// A CTA per (page, request, kv head): warps 0 and 1 take K, a run of 8 channels of a
// slot per lane at a time (16 lanes write a row); warps 2 and 3 V, whose codes lie by
// channel: a lane takes 8 channels x 8 slots, a code word per channel, and gives 8
// rows 16 bytes each.  Bound by the rows written.
template <bool kF32>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadArgs A,
                                                            const __grid_constant__ ReadRows by_value,
                                                            const ReadRow* __restrict__ d_rows) {
  const ReadRow R = d_rows ? d_rows[blockIdx.y] : by_value.r[blockIdx.y];
  if ((int)blockIdx.x >= R.n_pages) return;
  const int h = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Entry e = A.table[(size_t)R.req * A.max_pages + blockIdx.x];
  // this lane's slot: its place in the range (-1: none, or outside)
  const int p = A.pos[(size_t)e.id * kPage + lane];
  const int mine = p >= R.first && p - R.first < R.n ? p - R.first : -1;
  if (!__any_sync(0xFFFFFFFFu, mine >= 0)) return;
  const uint32_t live = A.hdead ? e.live & ~A.hdead[(size_t)e.id * A.hkv + h] : e.live;
  AttArgs T;
  T.pool = A.pool; T.int4_off = A.int4_off; T.int3_off = A.int3_off; T.fp4_off = A.fp4_off;
  T.n2 = A.n2; T.n3b = A.n3b; T.nfb = A.nfb; T.hkv = A.hkv;
  const uint8_t* b;
  const int cls = att_page(T, e.id, h, b);
  const size_t step = (size_t)A.hkv * kHeadDim, base = (size_t)R.row0 * step + (size_t)h * kHeadDim;
  if (warp < 2) {
    if (!A.k) return;
    const int c8 = lane & 15;
#pragma unroll 4
    for (int y = 0; y < 8; ++y) {
      const int t = 4 * y + 2 * warp + (lane >> 4);
      const int row = __shfl_sync(0xFFFFFFFFu, mine, t);
      float x[8];
      if (row >= 0) {
        if ((live >> t) & 1u) {
          k_values(b, cls, t, c8, x);
        } else {
#pragma unroll
          for (int n = 0; n < 8; ++n) x[n] = 0.0f;
        }
        put8<kF32>(A.k, base + (size_t)row * step + 8 * c8, x);
      }
    }
  } else {
    if (!A.v) return;
    const int o = (lane & 7) + 8 * (warp & 1), j = lane >> 3;   // 8 lanes: half a row
    VBlock B;
    v_load(b, cls, j, o, B);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int t = 8 * j + k;
      const int row = __shfl_sync(0xFFFFFFFFu, mine, t);
      float x[8];
      if (row >= 0) {
        if ((live >> t) & 1u) {
          v_values(B, b, cls, j, o, k, x);
        } else {
#pragma unroll
          for (int n = 0; n < 8; ++n) x[n] = 0.0f;
        }
        put8<kF32>(A.v, base + (size_t)row * step + 8 * o, x);
      }
    }
  }
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" kv_status_t kv_read_tokens(kv_pool_t* P, const int32_t* req_ids, const int64_t* first, const int64_t* n_tok,
                                      int32_t n_req, int32_t fp32, void* k, void* v, void* stream) try {
  if (!P) return fail(KV_ERR_INVALID_ARG, "kv_read_tokens: null pool");
  if (n_req < 0 || (n_req > 0 && (!req_ids || !first || !n_tok))) return fail(KV_ERR_INVALID_ARG, "kv_read_tokens: bad arguments");
  if (n_req > 65535) return fail(KV_ERR_INVALID_ARG, "kv_read_tokens: at most 65535 requests");
  std::vector<ReadRow> rows;
  int64_t total = 0;
  int32_t max_pages = 0;
  bool dropped = false;
  for (int32_t b = 0; b < n_req; ++b) {
    if (!req_ok(P, req_ids[b])) return fail(KV_ERR_INVALID_ARG, "kv_read_tokens: request %d not open", req_ids[b]);
    const Request& R = P->reqs[req_ids[b]];
    const int64_t have = (int64_t)R.loc.size();
    if (first[b] < 0 || n_tok[b] < 0 || first[b] > have || n_tok[b] > have - first[b])
      return fail(KV_ERR_INVALID_ARG, "kv_read_tokens: request %d holds %lld positions, [%lld, + %lld) asked for", req_ids[b],
                  (long long)have, (long long)first[b], (long long)n_tok[b]);
    if (n_tok[b] > 0) {
      rows.push_back(ReadRow{req_ids[b], (int32_t)R.table.size(), (int32_t)first[b], (int32_t)n_tok[b], total});
      max_pages = std::max(max_pages, (int32_t)R.table.size());
      dropped = dropped || R.dropped;
    }
    total += n_tok[b];
  }
  if (total == 0 || (!k && !v)) return KV_OK;
  if (((uintptr_t)k | (uintptr_t)v) % 16 != 0) return fail(KV_ERR_INVALID_ARG, "kv_read_tokens: k and v need 16-byte alignment");
  DeviceGuard dg(P->cfg.device);
  cudaStream_t s = (cudaStream_t)stream;
  kv_status_t st = refuse_capture("kv_read_tokens", s);
  if (st != KV_OK) return st;
  if ((st = order_after_previous(P, s)) != KV_OK) return st;
  if ((st = sync_positions(P, s)) != KV_OK) return st;
  const int hkv = P->cfg.num_kv_heads;
  if (dropped) {   // positions of dropped pages are in no page any more
    const size_t bytes = (size_t)total * hkv * kHeadDim * (fp32 ? 4 : 2);
    if (k) KV_CUDA(cudaMemsetAsync(k, 0, bytes, s));
    if (v) KV_CUDA(cudaMemsetAsync(v, 0, bytes, s));
    if (max_pages == 0) return KV_OK;
  }
  ReadRows by_value;
  const ReadRow* d_rows = nullptr;
  if (rows.size() <= (size_t)kReadByValue) {
    std::copy(rows.begin(), rows.end(), by_value.r);
  } else {
    Upload u;
    u.add(rows.data(), rows.size() * sizeof(ReadRow));
    if ((st = ensure(P->read, u.size)) != KV_OK) return st;
    if ((st = h2d(P, P->read.ptr, u, s)) != KV_OK) return st;
    d_rows = (const ReadRow*)P->read.ptr;
  }
  ReadArgs A;
  A.pool = P->d_pool;
  A.int4_off = P->int4_offset;
  A.int3_off = P->int3_offset;
  A.fp4_off = P->fp4_offset;
  A.n2 = P->cfg.n_int2_pages;
  A.n3b = A.n2 + P->cfg.n_int4_pages;
  A.nfb = A.n3b + P->cfg.n_int3_pages;
  A.table = P->d_table;
  A.hdead = P->hdead.empty() ? nullptr : P->d_hdead;
  A.pos = P->d_pos;
  A.k = k;
  A.v = v;
  A.max_pages = P->cfg.max_pages_per_request;
  A.hkv = hkv;
  const dim3 grid((unsigned)max_pages, (unsigned)rows.size(), (unsigned)hkv);
  ++P->launches;
  if (fp32)
    read_kernel<true><<<grid, kReadThreads, 0, s>>>(A, by_value, d_rows);
  else
    read_kernel<false><<<grid, kReadThreads, 0, s>>>(A, by_value, d_rows);
  KV_CUDA(cudaGetLastError());
  return KV_OK;
} catch (const std::bad_alloc&) {
  return fail(KV_ERR_OOM, "kv_read_tokens: host allocation failed");
}
