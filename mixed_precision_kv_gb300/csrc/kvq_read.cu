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

constexpr int kReadThreads = 256;

__device__ __forceinline__ float half_lo(uint32_t w) { return __half2float(__ushort_as_half((uint16_t)w)); }
__device__ __forceinline__ float half_hi(uint32_t w) { return __half2float(__ushort_as_half((uint16_t)(w >> 16))); }
__device__ __forceinline__ float half_of(const uint8_t* p) { return __half2float(*reinterpret_cast<const __half*>(p)); }

// The code in the bits `mask` of w, at bit p, as the float code * 2^p (p <= 19), exactly: or-ed into the
// mantissa of 2^23, and 2^23 taken off.  Conversions of integers run at a quarter of the rate.  With the
// scale times 2^-p (exact) one fused multiply-add then gives code * scale + zero, rounded once.
__device__ __forceinline__ float code_at(uint32_t w, uint32_t mask) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "r"(mask), "n"(0x4B000000));
  return __uint_as_float(d);
}
// (a0, a1) * (s0, s1) + (z0, z1) of two codes from code_at
__device__ __forceinline__ void value2(float& x0, float& x1, float a0, float a1, float s0, float s1, float z0, float z1) {
  asm("{.reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%8, %8};\n add.rn.f32x2 a, a, b;\n"
      " mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;}"
      : "=f"(x0), "=f"(x1) : "f"(a0), "f"(a1), "f"(s0), "f"(s1), "f"(z0), "f"(z1), "f"(-8388608.0f));
}

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

// INT3 and FP4 pages: channels c0 .. c0 + 7 of slot t of K or V, code by code.
struct Eight {
  float x[8];
};
__device__ __noinline__ Eight other_values(const uint8_t* b, int cls, bool is_k, int t, int c0) {
  Eight r;
  const int gr = c0 >> 5, mi = v_meta_index(t, gr);
  if (cls == kClsInt3) {
    const uint8_t* m = is_k ? b + kI3KMeta + 16 * t + 4 * gr : b + kI3VMeta + 2 * mi;
    const float s = half_of(m), z = half_of(m + (is_k ? 2 : 256));
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int c = c0 + n;
      const uint32_t code = is_k ? (((uint32_t)b[i3k_lo_byte(t, c)] >> i3k_lo_shift(c)) & 3u) |
                                       ((((uint32_t)b[i3k_hi_byte(t, c)] >> i3k_hi_shift(c)) & 1u) << 2)
                                 : (((uint32_t)b[i3v_lo_byte(t, c)] >> i3v_lo_shift(t)) & 3u) |
                                       ((((uint32_t)b[i3v_hi_byte(t, c)] >> i3v_hi_shift(t, c)) & 1u) << 2);
      r.x[n] = fmaf((float)code, s, z);
    }
  } else {
    const float s = half_of(is_k ? b + kF4KScale + 8 * t + 2 * gr : b + kF4VScale + 2 * mi);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int c = c0 + n;
      const uint32_t code = is_k ? (uint32_t)b[f4k_byte(t, c)] >> f4k_shift(c) : (uint32_t)b[f4v_byte(t, c)] >> f4v_shift(t);
      r.x[n] = e2m1_value(code & 15u) * s;
    }
  }
  return r;
}

// A CTA per (page, request): warps 2 x and 2 x + 1 take K and V of heads x, x + 4, ..  K: a lane takes a run
// of 8 channels of a slot at a time, 16 lanes a row, so an INT2 page's scales, which go by channel, stay in
// registers over the page.  V, whose codes lie by channel: 8 channels x 8 slots at a time, a code word per
// channel, which give 8 rows 16 bytes each (8 lanes: 128 bytes of a row).
// Bound by the rows written, 3.2 (INT4) to 5.3 (INT2) bytes of bf16 for each one read:
// 8 requests, 20K to 32K tokens, 8 kv heads (1.0 GB) in 174 us, 0.90 of the copy rate.
// With a conversion per code and no values by pairs it was bound by issue: 291 us.
// INT3 and FP4 pages, code by code, take five times as long as INT2 pages (65K tokens x
// 8 heads: 273 and 291 us against 58).
template <bool kF32>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadArgs A,
                                                            const __grid_constant__ ReadRows by_value,
                                                            const ReadRow* __restrict__ d_rows) {
  const ReadRow R = d_rows ? d_rows[blockIdx.y] : by_value.r[blockIdx.y];
  if ((int)blockIdx.x >= R.n_pages) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_k = (warp & 1) == 0;
  void* const out = is_k ? A.k : A.v;
  if (!out) return;
  const Entry e = A.table[(size_t)R.req * A.max_pages + blockIdx.x];
  // this lane's slot: its place in the range (-1: none, or outside)
  const int p = A.pos[(size_t)e.id * kPage + lane];
  const int mine = p >= R.first && p - R.first < R.n ? p - R.first : -1;
  if (!__any_sync(0xFFFFFFFFu, mine >= 0)) return;
  AttArgs T;
  T.pool = A.pool; T.int4_off = A.int4_off; T.int3_off = A.int3_off; T.fp4_off = A.fp4_off;
  T.n2 = A.n2; T.n3b = A.n3b; T.nfb = A.nfb; T.hkv = A.hkv;
  const size_t step = (size_t)A.hkv * kHeadDim;
#pragma unroll 1
  for (int h = warp >> 1; h < A.hkv; h += kReadThreads / 64) {
    const uint32_t live = A.hdead ? e.live & ~A.hdead[(size_t)e.id * A.hkv + h] : e.live;
    const uint8_t* b;
    const int cls = att_page(T, e.id, h, b);
    const size_t base = (size_t)R.row0 * step + (size_t)h * kHeadDim;
    // row of slot t: values x, or zeros where the slot is dead; rows outside the range are left
    auto store = [&](int t, int c0, float (&x)[8]) {
      const int row = __shfl_sync(0xFFFFFFFFu, mine, t);
      if (!((live >> t) & 1u)) {
#pragma unroll
        for (int n = 0; n < 8; ++n) x[n] = 0.0f;
      }
      if (row >= 0) put8<kF32>(out, base + (size_t)row * step + c0, x);
    };
    if (cls > kClsInt4) {
#pragma unroll 1
      for (int y = 0; y < 16; ++y) {
        const int t = 2 * y + (lane >> 4), c0 = 8 * (lane & 15);
        Eight v = other_values(b, cls, is_k, t, c0);
        store(t, c0, v.x);
      }
    } else if (is_k) {
      const int c8 = lane & 15, hi = lane >> 4, gr = c8 >> 2, i = c8 & 3;
      if (cls == kClsInt2) {
        // channel 8 c8 + n is in pair (gr, i >> 1, n), the half by i & 1 (the first pair swapped)
        float s[8], z[8];
        {
          const uint4* m = reinterpret_cast<const uint4*>(b + kI2KMeta + 4 * ((gr * 2 + (i >> 1)) * 8));
          const uint4 s0 = __ldg(m), s1 = __ldg(m + 1), z0 = __ldg(m + 16), z1 = __ldg(m + 17);
          const uint32_t sw[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
          const uint32_t zw[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const uint32_t sh = ((i & 1) != 0) != (n == 0) ? 16u : 0u;
            s[n] = half_lo(sw[n] >> sh) * (1.0f / (float)(1 << (2 * n)));
            z[n] = half_lo(zw[n] >> sh);
          }
        }
#pragma unroll 1
        for (int y0 = 0; y0 < 16; y0 += 8) {
          uint32_t w[8];
#pragma unroll
          for (int y = 0; y < 8; ++y)
            w[y] = __ldg(reinterpret_cast<const uint16_t*>(b + kI2KCodes + 32 * (2 * (y0 + y) + hi) + 2 * c8));
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            float x[8];
#pragma unroll
            for (int n = 0; n < 8; n += 2)
              value2(x[n], x[n + 1], code_at(w[y], 3u << (2 * n)), code_at(w[y], 12u << (2 * n)), s[n], s[n + 1], z[n], z[n + 1]);
            store(2 * (y0 + y) + hi, 8 * c8, x);
          }
        }
      } else {
#pragma unroll 1
        for (int y0 = 0; y0 < 16; y0 += 8) {
          uint32_t w[8], m[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int t = 2 * (y0 + y) + hi;
            w[y] = __ldg(reinterpret_cast<const uint32_t*>(b + kI4KCodes + 64 * t + 16 * i + 4 * gr));
            m[y] = __ldg(reinterpret_cast<const uint32_t*>(b + kI4KMeta + 16 * t + 4 * gr));
          }
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const float s = half_lo(m[y]), z = half_hi(m[y]);
            float x[8];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const float sp = s * (1.0f / (float)(1 << (4 * n)));
              value2(x[n], x[n + 4], code_at(w[y], 15u << (4 * n)), code_at(w[y] >> 16, 15u << (4 * n)), sp, sp, z, z);
            }
            store(2 * (y0 + y) + hi, 8 * c8, x);
          }
        }
      }
    } else {
      const int j = lane >> 3;
#pragma unroll 1
      for (int o = lane & 7; o < 16; o += 8) {   // channels 8 o .. 8 o + 7
        const int mt = o >> 1, ev = o & 1, gr = o >> 2;
        const int meta = cls == kClsInt2 ? kI2VMeta : kI4VMeta;
        const uint8_t* cw = cls == kClsInt2 ? b + kI2VCodes + 16 * (32 * (mt >> 2) + j) + 4 * (mt & 3)
                                            : b + kI4VCodes + 16 * (32 * (mt >> 1) + j) + 4 * (2 * (mt & 1) + ev);
        uint32_t w[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) w[r] = __ldg(reinterpret_cast<const uint32_t*>(cw + 64 * r));
        const uint4 s4 = __ldg(reinterpret_cast<const uint4*>(b + meta + 64 * gr + 16 * j));
        const uint4 z4 = __ldg(reinterpret_cast<const uint4*>(b + meta + 256 + 64 * gr + 16 * j));
        const uint32_t sw[4] = {s4.x, s4.y, s4.z, s4.w}, zw[4] = {z4.x, z4.y, z4.z, z4.w};   // slots k and k + 4
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float s = half_lo(sw[k & 3] >> (k < 4 ? 0 : 16)), z = half_lo(zw[k & 3] >> (k < 4 ? 0 : 16));
          // INT2: byte ev (slots 0..3) or ev + 2 (4..7) of a word, slot 8 j and 8 j + 4 the other way round for ev 0
          const uint32_t sh = cls == kClsInt2 ? 8u * ev + 2u * (k & 3) + (((k >> 2) != 0) != (ev == 0 && (k & 3) == 0) ? 16u : 0u)
                                              : 4u * k;
          const uint32_t mask = cls == kClsInt2 ? 3u : 15u;
          float x[8];
#pragma unroll
          for (int r = 0; r < 8; r += 2)
            value2(x[r], x[r + 1], code_at(w[r] >> sh, mask), code_at(w[r + 1] >> sh, mask), s, s, z, z);
          store(8 * j + k, 8 * o, x);
        }
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
  const dim3 grid((unsigned)max_pages, (unsigned)rows.size());
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
