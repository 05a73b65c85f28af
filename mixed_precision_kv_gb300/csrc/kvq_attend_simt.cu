// CUDA-core form of kv_attend: the plain statement of the operator that the
// tensor-core kernels are compared with, chosen by
// kv_set_decode_impl(KV_DECODE_SIMT).
//
// Row i of a unit (new token t, q head j) takes, over the request's live
// cached slots, its full-precision list and the new tokens its mask allows,
//     o_i = sum_x p_ix v_x / sum_x p_ix,   p_ix = 2^(s_ix - m_i),
//     s_ix = softmax_scale * log2(e) * q_i . k_x,
// in one pass with the running maximum m_i and sum; a row that sees nothing is
// 0.  One CTA of 8 warps takes 32 rows (4 per warp): 32 keys at a time are
// dequantized to fp32 in shared memory, a lane holds a key for the logits and
// four channels for P.V.  Bound by instruction issue and latency (a CTA takes a
// whole cache: 850 us for one new token over 2K tokens, 6 TFLOP/s on a chunk of
// 2048 over 32K).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_values.cuh"

namespace kvq {
namespace {

constexpr int kRows = 32;            // rows per CTA
constexpr int kPer = 4;              // rows per warp
constexpr int kKs = kHeadDim + 4;    // K row stride in floats: 16-byte reads of 8 lanes hit distinct banks

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
// a new or list token's value: NaN, Inf and |x| > 65504 are reported and used as 0
__device__ __forceinline__ float new_value(uint16_t x, uint32_t* status) {
  const float f = bf(x);
  if (fabsf(f) <= 65504.0f) return f;
  atomicOr(status, kStatusRange);
  return 0.0f;
}

__global__ void __launch_bounds__(256) attend_simt_kernel(AttArgs A, const AttUnit* __restrict__ units) {
  __shared__ float qs[kRows][kHeadDim];
  __shared__ __align__(16) float ks[kPage][kKs];
  __shared__ __align__(16) float vs[kPage][kHeadDim];
  const AttUnit u = units[blockIdx.y];
  const int g = A.hq / A.hkv, rows = u.T * g, r0 = blockIdx.x * kRows;
  if (r0 >= rows) return;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  auto row_at = [&](int i) { return ((size_t)(u.tok0 + i / g) * A.hq + (size_t)u.kvh * g + i % g) * kHeadDim; };
  for (int x = tid; x < kRows * kHeadDim; x += 256) {
    const int i = r0 + x / kHeadDim;
    qs[x / kHeadDim][x % kHeadDim] = i < rows ? bf(A.q[row_at(i) + x % kHeadDim]) : 0.0f;
  }
  float m[kPer], l[kPer], o[kPer][4];
  bool seen[kPer];   // this lane's keys so far: any that the row sees
#pragma unroll
  for (int y = 0; y < kPer; ++y) {
    m[y] = -INFINITY;
    l[y] = 0.0f;
    seen[y] = false;
    o[y][0] = o[y][1] = o[y][2] = o[y][3] = 0.0f;
  }
  // the 32 keys in shared memory; may(y): whether this lane's key is seen by row r0 + kPer w + y
  auto keys = [&](auto&& may) {
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
      const float* qr = qs[kPer * w + y];
      float s = 0.0f;
      for (int c = 0; c < kHeadDim; c += 4) {
        const float4 kv = *reinterpret_cast<const float4*>(&ks[lane][c]);
        const float4 qv = *reinterpret_cast<const float4*>(&qr[c]);
        s = fmaf(qv.x, kv.x, s); s = fmaf(qv.y, kv.y, s); s = fmaf(qv.z, kv.z, s); s = fmaf(qv.w, kv.w, s);
      }
      const bool see = may(y), whole = fabsf(s) < INFINITY;
      s = see ? s * A.scale_log2 : -INFINITY;
      // A row whose greatest logit is past fp32's range, above or below, is not a number, nor is one with a sum
      // that is not finite.
      if (__any_sync(0xFFFFFFFFu, see && !(whole && s < INFINITY))) l[y] = __int_as_float(0x7FFFFFFF);
      if (see) seen[y] = true;
      s = whole && s < INFINITY ? s : -INFINITY;
      float mx = s;
#pragma unroll
      for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
      const float mn = fmaxf(m[y], mx);
      if (mn == -INFINITY) continue;   // nothing seen yet (warp-uniform)
      const float corr = exp2f(m[y] - mn);
      const float p = exp2f(s - mn);
      float ps = p;
#pragma unroll
      for (int off = 16; off; off >>= 1) ps += __shfl_xor_sync(0xFFFFFFFFu, ps, off);
      l[y] = l[y] * corr + ps;
      m[y] = mn;
#pragma unroll
      for (int a = 0; a < 4; ++a) o[y][a] *= corr;
      for (int t = 0; t < kPage; ++t) {
        const float pt = __shfl_sync(0xFFFFFFFFu, p, t);
        const float4 vv = *reinterpret_cast<const float4*>(&vs[t][4 * lane]);
        o[y][0] = fmaf(pt, vv.x, o[y][0]); o[y][1] = fmaf(pt, vv.y, o[y][1]);
        o[y][2] = fmaf(pt, vv.z, o[y][2]); o[y][3] = fmaf(pt, vv.w, o[y][3]);
      }
    }
  };
  // ---- cached pages
  const Entry* tab = A.table + (size_t)u.req * A.max_pages;
  for (int p = 0; p < u.n_pages; ++p) {
    const Entry e = tab[p];
    const uint32_t live = A.hdead ? e.live & ~A.hdead[(size_t)e.id * A.hkv + u.kvh] : e.live;
    if (live == 0u) continue;
    const uint8_t* blk;
    const int cls = att_page(A, e.id, u.kvh, blk);
    __syncthreads();
    for (int x = tid; x < kPage * kHeadDim; x += 256) {
      const int t = x / kHeadDim, c = x % kHeadDim;
      const bool on = (live >> t) & 1u;   // slots never written hold no values
      ks[t][c] = on ? k_value(blk, cls, t, c) : 0.0f;
      vs[t][c] = on ? v_value(blk, cls, t, c) : 0.0f;
    }
    __syncthreads();
    keys([&](int) { return (live >> lane) & 1u; });
  }
  // ---- full-precision list
  const size_t fp0 = ((size_t)u.req * A.hkv + u.kvh) * A.fp_cap * kHeadDim;
  for (int j0 = 0; j0 < u.n_fp; j0 += kPage) {
    __syncthreads();
    for (int x = tid; x < kPage * kHeadDim; x += 256) {
      const int t = x / kHeadDim, c = x % kHeadDim;
      const bool on = j0 + t < u.n_fp;
      ks[t][c] = on ? new_value(A.fpk[fp0 + (size_t)(j0 + t) * kHeadDim + att_list_at(j0 + t, c)], A.status) : 0.0f;
      vs[t][c] = on ? new_value(A.fpv[fp0 + (size_t)(j0 + t) * kHeadDim + att_list_at(j0 + t, c)], A.status) : 0.0f;
    }
    __syncthreads();
    keys([&](int) { return j0 + lane < u.n_fp; });
  }
  // ---- new tokens
  const int r_last = min(rows, r0 + kRows) - 1;
  const int n_new = !A.k ? 0 : (A.tree ? u.T : r_last / g + 1);
  for (int j0 = 0; j0 < n_new; j0 += kPage) {
    __syncthreads();
    for (int x = tid; x < kPage * kHeadDim; x += 256) {
      const int t = x / kHeadDim, c = x % kHeadDim;
      const bool on = j0 + t < n_new;
      const size_t at = ((size_t)(u.tok0 + j0 + t) * A.hkv + u.kvh) * kHeadDim + c;
      ks[t][c] = on ? new_value(A.k[at], A.status) : 0.0f;
      vs[t][c] = on ? new_value(A.v[at], A.status) : 0.0f;
    }
    __syncthreads();
    keys([&](int y) {
      const int i = r0 + kPer * w + y, t = i / g, j = j0 + lane;
      if (i >= rows || j >= n_new) return false;
      return A.tree ? ((A.tree[u.tok0 + t] >> j) & 1ull) != 0ull : j <= t;
    });
  }
  bool bad = false;
#pragma unroll
  for (int y = 0; y < kPer; ++y) {
    const int i = r0 + kPer * w + y;
    if (i >= rows) continue;   // (warp-uniform)
    if (__any_sync(0xFFFFFFFFu, seen[y]) && m[y] == -INFINITY) l[y] = __int_as_float(0x7FFFFFFF);
    const float inv = l[y] > 0.0f ? 1.0f / l[y] : (l[y] == 0.0f ? 0.0f : l[y]);   // a NaN sum stays NaN
    uint16_t* op = A.out + row_at(i) + 4 * lane;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float v = o[y][a] * inv;
      if (!(fabsf(v) < INFINITY)) bad = true;
      op[a] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
  }
  if (bad) atomicOr(A.status, kStatusRange);
}

}  // namespace

cudaError_t launch_attend_simt(kv_pool* P, const AttArgs& A, const AttUnit* d_units, int n_units, int max_rows,
                               cudaStream_t s) {
  if (n_units <= 0 || max_rows <= 0) return cudaSuccess;
  ++P->launches;
  attend_simt_kernel<<<dim3((unsigned)((max_rows + kRows - 1) / kRows), (unsigned)n_units), 256, 0, s>>>(A, d_units);
  return cudaGetLastError();
}

}  // namespace kvq
