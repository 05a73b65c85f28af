// kv_rotate (rotary positions on rows of q and k) and the entry of
// kv_append_rotated, whose kernels are those of kv_append_quant (kvq_quant.cu).
#include <cuda_runtime.h>

#include <algorithm>
#include <new>

#include "kvq_host.h"

namespace kvq {
namespace {

// One tensor of a call.
struct RotTensor {
  const uint16_t* x;
  uint16_t* y;
  int64_t xs, ys;   // elements from a token's rows to the next token's
  int32_t heads;    // 0: none
};

constexpr int kRotThreads = 256;

__device__ __forceinline__ uint4 row_load(const uint16_t* p, bool aligned) {
  if (aligned) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = (uint32_t)p[2 * k] | ((uint32_t)p[2 * k + 1] << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void row_store(uint16_t* p, const uint4& v, bool aligned) {
  if (aligned) {
    *reinterpret_cast<uint4*>(p) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    p[2 * k] = (uint16_t)w[k];
    p[2 * k + 1] = (uint16_t)(w[k] >> 16);
  }
}

// A thread takes item i of a row (kvq_rope.h) of one token, its factors once and
// then every `lines`-th head of q and k together; 256 / (8 lines) tokens a CTA.
// Rows are read and written once, 16 bytes a thread at a time, a row's 8 threads
// side by side.  Bound by HBM: 16384 tokens x 72 heads (612 MB) in 92.7 us, 0.97 of
// the copy rate.  Three heads in flight at four CTAs an SM: two 107 us, one 106
// (longer lines, eight heads a thread 141), four 92 to 95.
template <bool kAligned>
__global__ void __launch_bounds__(kRotThreads, 4) rotate_kernel(const __grid_constant__ RopeArgs R,
                                                             const __grid_constant__ RotTensor Q,
                                                             const __grid_constant__ RotTensor K, int64_t n, int lines,
                                                             uint32_t* __restrict__ status) {
  const int i = threadIdx.x & 7, line = ((int)threadIdx.x >> 3) & (lines - 1);
  const int per = kRotThreads / 8 / lines;
  const int64_t t = (int64_t)blockIdx.x * per + (int)threadIdx.x / (8 * lines);
  if (t >= n) return;
  int a, b;
  rope_item(R, i, a, b);
  const bool turn = 8 * i < R.half;
  bool bad = false;
  float c[8], s[8];
  if (turn) {
    rope_factors<8>(R, t, 8 * i, c, s, bad);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) c[k] = s[k] = 0.0f;
  }
  const uint16_t* qx = Q.x + (size_t)t * (size_t)Q.xs;
  const uint16_t* kx = K.x + (size_t)t * (size_t)K.xs;
  uint16_t* qy = Q.y + (size_t)t * (size_t)Q.ys;
  uint16_t* ky = K.y + (size_t)t * (size_t)K.ys;
  const int all = Q.heads + K.heads;
  constexpr int kAhead = 3;
  for (int h0 = line; h0 < all; h0 += kAhead * lines) {
    uint4 x[kAhead], z[kAhead];
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      const int h = h0 + y * lines;
      if (h >= all) break;
      const uint16_t* p = h < Q.heads ? qx + (size_t)h * kHeadDim : kx + (size_t)(h - Q.heads) * kHeadDim;
      x[y] = row_load(p + 8 * a, kAligned);
      z[y] = row_load(p + 8 * b, kAligned);
    }
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      const int h = h0 + y * lines;
      if (h >= all) break;
      if (turn) rope_turn(R, x[y], z[y], c, s);
      uint16_t* p = h < Q.heads ? qy + (size_t)h * kHeadDim : ky + (size_t)(h - Q.heads) * kHeadDim;
      row_store(p + 8 * a, x[y], kAligned);
      row_store(p + 8 * b, z[y], kAligned);
    }
  }
  if (bad) atomicOr(status, kStatusRange);
}

// The checks of a rotation that both entries make.
kv_status_t rope_args(const char* what, const kv_rope_t* rope, const int32_t* pos, int64_t pos_stride, int64_t n_tok,
                      RopeArgs& R) {
  if (!rope || !rope->cos_sin || !pos) return fail(KV_ERR_INVALID_ARG, "%s: null rotation, table or positions", what);
  if (rope->rot_dim < 16 || rope->rot_dim > kHeadDim || rope->rot_dim % 16 != 0)
    return fail(KV_ERR_INVALID_ARG, "%s: rot_dim %d is not a multiple of 16 in [16, 128]", what, rope->rot_dim);
  if (rope->rows < 1 || rope->rows > INT32_MAX)
    return fail(KV_ERR_INVALID_ARG, "%s: a table of %lld positions", what, (long long)rope->rows);
  if (rope->n_axes < 1 || rope->n_axes > kMaxAxes)
    return fail(KV_ERR_INVALID_ARG, "%s: n_axes %d is not in [1, %d]", what, rope->n_axes, kMaxAxes);
  if (rope->n_axes > 1 && !rope->axis) return fail(KV_ERR_INVALID_ARG, "%s: several axes need the frequencies' axes", what);
  if ((uintptr_t)rope->cos_sin % 16 != 0 || (uintptr_t)pos % 4 != 0)
    return fail(KV_ERR_INVALID_ARG, "%s: the table needs 16-byte and the positions 4-byte alignment", what);
  if (rope->n_axes > 1 && pos_stride < n_tok)
    return fail(KV_ERR_INVALID_ARG, "%s: pos_stride %lld holds fewer than %lld positions", what, (long long)pos_stride,
                (long long)n_tok);
  R = RopeArgs{};
  R.table = rope->cos_sin;
  R.pos = pos;
  R.pos_stride = pos_stride;
  R.rows = (int32_t)rope->rows;
  R.half = rope->rot_dim / 2;
  R.pairs = rope->interleaved ? 1 : 0;
  R.n_axes = rope->n_axes;
  R.minus0 = -0.0f;
  for (int f = 0; rope->axis && f < R.half; ++f) {
    if (rope->axis[f] >= rope->n_axes)
      return fail(KV_ERR_INVALID_ARG, "%s: frequency %d has axis %d of %d", what, f, rope->axis[f], rope->n_axes);
    R.axis[f >> 4] |= (uint32_t)rope->axis[f] << (2 * (f & 15));
  }
  return KV_OK;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" kv_status_t kv_rotate(kv_pool_t* P, const kv_rope_t* rope, const int32_t* pos, int64_t pos_stride, int64_t n_tok,
                                 const void* q, int32_t q_heads, int64_t q_stride, void* q_out, int64_t q_out_stride,
                                 const void* k, int32_t k_heads, int64_t k_stride, void* k_out, int64_t k_out_stride,
                                 void* stream) {
  if (!P) return fail(KV_ERR_INVALID_ARG, "kv_rotate: null pool");
  if (n_tok < 0 || n_tok > INT32_MAX) return fail(KV_ERR_INVALID_ARG, "kv_rotate: bad n_tok %lld", (long long)n_tok);
  if (q_heads < 0 || k_heads < 0 || q_heads > 65535 || k_heads > 65535)
    return fail(KV_ERR_INVALID_ARG, "kv_rotate: heads must be in [0, 65535]");
  if (n_tok == 0 || q_heads + k_heads == 0) return KV_OK;
  RotTensor T[2] = {{(const uint16_t*)q, (uint16_t*)q_out, q_stride, q_out_stride, q_heads},
                    {(const uint16_t*)k, (uint16_t*)k_out, k_stride, k_out_stride, k_heads}};
  bool aligned = true;
  for (RotTensor& x : T) {
    if (x.heads == 0) {
      x = RotTensor{};
      continue;
    }
    if (!x.x || !x.y) return fail(KV_ERR_INVALID_ARG, "kv_rotate: null pointer");
    if (((uintptr_t)x.x | (uintptr_t)x.y) % 2 != 0) return fail(KV_ERR_INVALID_ARG, "kv_rotate: rows need 2-byte alignment");
    if (x.xs < 0 || x.ys < 0 || (n_tok > 1 && x.ys < (int64_t)x.heads * kHeadDim))
      return fail(KV_ERR_INVALID_ARG, "kv_rotate: a stride is negative, or an output's tokens overlap");
    aligned = aligned && ((uintptr_t)x.x | (uintptr_t)x.y) % 16 == 0 && x.xs % 8 == 0 && x.ys % 8 == 0;
  }
  RopeArgs R;
  const kv_status_t st = rope_args("kv_rotate", rope, pos, pos_stride, n_tok, R);
  if (st != KV_OK) return st;
  DeviceGuard dg(P->cfg.device);
  // Lines of heads side by side: 3 to 6 heads a thread (4 to 8: 96.5 us for 16384 x 72 heads against 92.7), fewer
  // while the call's tokens do not fill the SMs, down to a head each: a call of one token is one round of loads.
  int lines = 1;
  while (lines < kRotThreads / 8 && (lines * 6 < q_heads + k_heads || n_tok * lines * 8 < (int64_t)P->sm_count * 512)) lines *= 2;
  const int per = kRotThreads / 8 / lines;
  const unsigned grid = (unsigned)((n_tok + per - 1) / per);
  ++P->launches;
  if (aligned)
    rotate_kernel<true><<<grid, kRotThreads, 0, (cudaStream_t)stream>>>(R, T[0], T[1], n_tok, lines, P->d_status);
  else
    rotate_kernel<false><<<grid, kRotThreads, 0, (cudaStream_t)stream>>>(R, T[0], T[1], n_tok, lines, P->d_status);
  KV_CUDA(cudaGetLastError());
  return KV_OK;
}

extern "C" kv_status_t kv_append_rotated(kv_pool_t* P, const kv_rope_t* rope, const int32_t* pos, int64_t pos_stride,
                                         const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                         const int32_t* req_ids, const uint8_t* bits, int64_t n_tok, void* stream) try {
  if (!P) return fail(KV_ERR_INVALID_ARG, "kv_append_rotated: null pool");
  if (n_tok < 0 || n_tok > INT32_MAX) return fail(KV_ERR_INVALID_ARG, "kv_append_rotated: bad n_tok %lld", (long long)n_tok);
  if (n_tok == 0) return KV_OK;
  if (k_stride < 0 || v_stride < 0 || k_stride % 4 != 0 || v_stride % 4 != 0 || ((uintptr_t)k | (uintptr_t)v) % 8 != 0)
    return fail(KV_ERR_INVALID_ARG, "kv_append_rotated: k and v need 8-byte alignment and strides that are multiples of 4");
  RopeArgs R;
  const kv_status_t st = rope_args("kv_append_rotated", rope, pos, pos_stride, n_tok, R);
  if (st != KV_OK) return st;
  R.k_stride = k_stride;
  R.v_stride = v_stride;
  struct Running {
    kv_pool* P;
    ~Running() { P->rope = nullptr; }
  } running{P};
  P->rope = &R;
  return append_tokens(P, "kv_append_rotated", k, v, req_ids, bits, n_tok, stream);
} catch (const std::bad_alloc&) {
  return fail(KV_ERR_OOM, "kv_append_rotated: host allocation failed");
}
