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

#include "kvq_host.h"
#include "kvq_values.cuh"

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

// Rows with a shared prefix: the parts of the request's own unit and those of the
// prefix unit, each in the layout of the kernel that made it.  A warp takes two
// rows, a lane 4 channels of each half of one: parts by channel hold neighbouring
// rows side by side, so whole sectors are read (64 requests over 100K with 64 q
// heads: the call 317 us, 326 with a row per warp).  Bound by the partials' latency:
// they are still in L2, and a row has few of them.
struct PartRow {
  const float *o, *ml;   // this lane's first channels of part 0, the row's m and l
  size_t step;
  int half;              // from channel 0 to channel 64
  int n;
  float head;            // what its maxima lack of the attention kernels' (kAttHead or 0)
};
__device__ __forceinline__ PartRow part_row(const AttSrc& S, const float* part, int r, int c, bool tall) {
  const float* p = part + S.off;
  return tall ? PartRow{p + (size_t)c * (4 * kTallRows) + 4 * r, p + kTallRows * kHeadDim + 2 * r, (size_t)S.step,
                        64 * kTallRows, S.n_parts, 0.0f}
              : PartRow{p + (size_t)r * kAttPart + 4 * c, p + (size_t)r * kAttPart + kHeadDim, (size_t)S.step, 64, S.n_parts, 0.0f};
}
// Reductions over the 16 lanes of a row.
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int o = 16; o > 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 16; o > 1; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}
__device__ __forceinline__ float part_max(const PartRow& R, int c) {
  float M = -INFINITY;
  for (int p = c; p < R.n; p += 16) M = fmaxf(M, R.ml[(size_t)p * R.step]);
  return row_max(M) + R.head;
}
// Adds a row's parts, relative to the maximum M: L per lane (to be summed), o: 4 channels of each half.
__device__ __forceinline__ void part_add(const PartRow& R, int lane, float M, float& L, float4 (&o)[2]) {
  const int c = lane >> 1, rr = lane & 1;
  const int most = max(R.n, __shfl_xor_sync(0xFFFFFFFFu, R.n, 1));
  for (int p0 = 0; p0 < most; p0 += 16) {
    float f = 0.0f;
    if (p0 + c < R.n) {
      const float2 ml = *reinterpret_cast<const float2*>(R.ml + (size_t)(p0 + c) * R.step);
      // a part that saw nothing (m = -inf, l = 0) adds nothing; one with a NaN sum keeps it
      f = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : exp2f(ml.x + R.head - M);
      L = fmaf(ml.y, f, L);
    }
    for (int p = 0; p < min(16, most - p0); p += 4) {
      float4 a[4][2];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float* q = R.o + (size_t)(p0 + p + y) * R.step;
        const bool is = p0 + p + y < R.n;
        a[y][0] = is ? *reinterpret_cast<const float4*>(q) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        a[y][1] = is ? *reinterpret_cast<const float4*>(q + R.half) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float w = __shfl_sync(0xFFFFFFFFu, f, 2 * (p + y) + rr);
        if (w != 0.0f)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            o[x].x = fmaf(a[y][x].x, w, o[x].x); o[x].y = fmaf(a[y][x].y, w, o[x].y);
            o[x].z = fmaf(a[y][x].z, w, o[x].z); o[x].w = fmaf(a[y][x].w, w, o[x].w);
          }
      }
    }
  }
}
__device__ __forceinline__ bool finite4(const float4& o) {
  return fabsf(o.x) < INFINITY && fabsf(o.y) < INFINITY && fabsf(o.z) < INFINITY && fabsf(o.w) < INFINITY;
}

// A row over its request's pages, plainly (as the CUDA-core kernel): where the scan's parts do not say it.  A
// warp: a slot per lane for the logits, four channels for the sums.
struct PlainRow {
  float m, l;
  float4 o;
};
__device__ __noinline__ PlainRow plain_row(const AttArgs& A, const uint16_t* q, int req, int kvh, int n_pages) {
  const int lane = threadIdx.x & 31;
  PlainRow R{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  bool seen = false, wild = false;
  // rows past 2^60 are taken 2^64 smaller and their logits 2^64 larger, both exact, so that q . k stays in fp32
  // where the logit does (the scale is within 2^40 of one here)
  float mx_q = 0.0f;
#pragma unroll
  for (int c = 0; c < 4; ++c) mx_q = fmaxf(mx_q, fabsf(__uint_as_float((uint32_t)q[4 * lane + c] << 16)));
#pragma unroll
  for (int o = 16; o; o >>= 1) mx_q = fmaxf(mx_q, __shfl_xor_sync(0xFFFFFFFFu, mx_q, o));
  const bool large = mx_q > 0x1p60f;
  const float down = large ? 0x1p-64f : 1.0f, scale = large ? A.scale_log2 * 0x1p64f : A.scale_log2;
  // the next page with a live slot: the entries of 32 pages at a time.  A row that is not a number stays one.
  int p0 = -32;
  Entry e{0, 0u};        // lane's entry, its slots that are live for the head
  uint32_t todo = 0u;    // pages of the 32 that are left
  while (!wild) {
    if (todo == 0u) {
      p0 += 32;
      if (p0 >= n_pages) break;
      e = Entry{0, 0u};
      if (p0 + lane < n_pages) e = A.table[(size_t)req * A.max_pages + p0 + lane];
      if (A.hdead && e.live) e.live &= ~A.hdead[(size_t)e.id * A.hkv + kvh];
      todo = __ballot_sync(0xFFFFFFFFu, e.live != 0u);
      continue;
    }
    const int at = __ffs(todo) - 1;
    todo &= todo - 1u;
    const int32_t id = __shfl_sync(0xFFFFFFFFu, e.id, at);
    const uint32_t live = __shfl_sync(0xFFFFFFFFu, e.live, at);
    seen = true;
    const uint8_t* b;
    const int cls = att_page(A, id, kvh, b);
    const bool on = (live >> lane) & 1u;
    float s = 0.0f;
    for (int c = 0; on && c < kHeadDim; ++c) s = fmaf(__uint_as_float((uint32_t)q[c] << 16) * down, k_value(b, cls, lane, c), s);
    const bool whole = fabsf(s) < INFINITY;
    s *= scale;
    // past fp32's range, above or below: the row is not a number
    if (__any_sync(0xFFFFFFFFu, on && !(whole && s < INFINITY))) wild = true;
    s = on && whole && s < INFINITY ? s : -INFINITY;
    float mx = s;
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    const float mn = fmaxf(R.m, mx);
    if (mn == -INFINITY) continue;
    const float corr = exp2f(R.m - mn), w = exp2f(s - mn);
    float ws = w;
#pragma unroll
    for (int o = 16; o; o >>= 1) ws += __shfl_xor_sync(0xFFFFFFFFu, ws, o);
    R.l = R.l * corr + ws;
    R.m = mn;
    R.o.x *= corr; R.o.y *= corr; R.o.z *= corr; R.o.w *= corr;
    for (int t = 0; t < kPage; ++t) {
      const float wt = __shfl_sync(0xFFFFFFFFu, w, t);
      if (!((live >> t) & 1u)) continue;   // slots never written hold no values
      R.o.x = fmaf(wt, v_value(b, cls, t, 4 * lane), R.o.x);
      R.o.y = fmaf(wt, v_value(b, cls, t, 4 * lane + 1), R.o.y);
      R.o.z = fmaf(wt, v_value(b, cls, t, 4 * lane + 2), R.o.z);
      R.o.w = fmaf(wt, v_value(b, cls, t, 4 * lane + 3), R.o.w);
    }
  }
  if (wild || (seen && R.m == -INFINITY)) R.l = __int_as_float(0x7FFFFFFF);
  return R;
}

// The decode scan gives a dead slot the logit kSentinel and the value 0.  Above kSentinel + 160 a maximum leaves it
// no weight (2^-160 is 0), as here; a row below that, or one that is not finite, is taken plainly.
constexpr float kSentinel = -1.0e4f * 1.4426950408889634f + kAttHead;

__global__ void __launch_bounds__(32 * kMergeRows) attend_join_kernel(AttArgs A, const AttJoin* __restrict__ joins,
                                                                      const AttSrc* __restrict__ srcs,
                                                                      const float* __restrict__ part,
                                                                      const Unit* __restrict__ scan_units,
                                                                      const float* __restrict__ scan_part) {
  const AttJoin J = joins[blockIdx.y];
  wait_for_grid(part, scan_part);   // (the plans were there before the kernels that this one follows)
  const int lane = threadIdx.x & 31, c = lane >> 1;
  const int i0 = 2 * (blockIdx.x * kMergeRows + (int)(threadIdx.x >> 5));
  if (i0 >= J.rows) return;
  const bool mine = i0 + (lane & 1) < J.rows;   // (an odd last row: both halves of the warp take it)
  const int i = mine ? i0 + (lane & 1) : i0;
  const int g = A.hq / A.hkv;
  const size_t at = ((size_t)(J.tok0 + i / g) * A.hq + (size_t)J.kvh * g + i % g) * kHeadDim;
  const bool scan = (J.flags & kJoinScan) != 0;
  PartRow own, pre{nullptr, nullptr, 0, 0, 0, 0.0f};
  if (scan) {
    const Unit u = scan_units[J.own0];
    const float* p = scan_part + ((size_t)u.split_begin * g + i) * kAttPart;
    own = PartRow{p + 4 * c, p + kHeadDim, (size_t)g * kAttPart, 64, u.n_splits, kAttHead};
  } else {
    own = part_row(srcs[J.own0 + (i >> J.own_shift)], part, i & ((1 << J.own_shift) - 1), c, (J.flags & kJoinOwnTall) != 0);
  }
  if (J.pre0 >= 0) {
    const int ip = J.pre_row + i;
    pre = part_row(srcs[J.pre0 + (ip >> J.pre_shift)], part, ip & ((1 << J.pre_shift) - 1), c, (J.flags & kJoinPreTall) != 0);
  }
  const float mo = part_max(own, c), mp = part_max(pre, c);
  float L = 0.0f, M = fmaxf(mo, mp);
  float4 o[2] = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  part_add(own, lane, M, L, o);
  if (scan && J.n_pages > 0) {
    const uint32_t unsure = __ballot_sync(0xFFFFFFFFu, !(mo > kSentinel + 160.0f && finite4(o[0]) && finite4(o[1]) && L < INFINITY));
#pragma unroll 1
    for (int y = 0; y < 2; ++y) {
      if (!(unsure & (0x55555555u << y))) continue;
      const PlainRow R = plain_row(A, A.q + __shfl_sync(0xFFFFFFFFu, (unsigned long long)at, y), J.req, J.kvh, J.n_pages);
      const float x[4] = {R.o.x, R.o.y, R.o.z, R.o.w};
      float lo[4], hi[4];   // channels 4 c .. and 64 + 4 c ..
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        lo[k] = __shfl_sync(0xFFFFFFFFu, x[k], c);
        hi[k] = __shfl_sync(0xFFFFFFFFu, x[k], 16 + c);
      }
      if ((lane & 1) != y) continue;
      const float m = R.m + kAttHead;
      M = fmaxf(m, mp);
      const float f = R.m == -INFINITY ? (R.l == 0.0f ? 0.0f : 1.0f) : exp2f(m - M);
      L = c == 0 ? R.l * f : 0.0f;
      o[0] = make_float4(lo[0] * f, lo[1] * f, lo[2] * f, lo[3] * f);
      o[1] = make_float4(hi[0] * f, hi[1] * f, hi[2] * f, hi[3] * f);
    }
    __syncwarp();
  }
  part_add(pre, lane, M, L, o);
  L = row_sum(L);
  const float inv = row_inverse(M, L);
  bool bad = false;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const float r[4] = {o[x].x * inv, o[x].y * inv, o[x].z * inv, o[x].w * inv};
    uint16_t* op = A.out + at + 64 * x + 4 * c;
    uint32_t h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!(fabsf(r[k]) < INFINITY)) bad = true;
      h[k] = __bfloat16_as_ushort(__float2bfloat16_rn(r[k]));
    }
    if (!mine) continue;
    if (((uintptr_t)A.out & 7) == 0) {
      *reinterpret_cast<uint2*>(op) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) op[k] = (uint16_t)h[k];
    }
  }
  if (bad) atomicOr(A.status, kStatusRange);
}

cudaError_t launch_attend_join(kv_pool* P, const AttArgs& A, const AttJoin* d_joins, int n_joins, int max_rows,
                               const AttSrc* d_srcs, const float* d_part, const Unit* scan_units, const float* scan_part,
                               cudaStream_t s) {
  if (n_joins == 0) return cudaSuccess;
  ++P->launches;   // (a join per request and kv head: at most 65535)
  return launch_pdl(attend_join_kernel, dim3((unsigned)((max_rows + 2 * kMergeRows - 1) / (2 * kMergeRows)), (unsigned)n_joins),
                    dim3(32 * kMergeRows), 0, s, A, d_joins, d_srcs, d_part, scan_units, scan_part);
}

// ---- work plan ---------------------------------------------------------
struct AttPlan {
  std::vector<AttItem> items;
  std::vector<int32_t> cta_item;   // per pass: first item of every CTA, and the end
  std::vector<AttMerge> merges;
  int64_t n_parts = 0;
  int merge_rows = 0;
  std::vector<AttSrc> srcs;        // joined units: the blocks' parts (off, step: parts), and a unit's first block
  std::vector<int32_t> src0;
};

// Key tiles of the block of rows [row0, row0 + rows) of a unit.
int block_tiles(const AttUnit& u, int g, int row0, int rows, bool tree) {
  const int t_last = (row0 + rows - 1) / g;
  return (u.n_pages + 3) / 4 + (u.n_fp + 127) / 128 + (u.n_own ? (tree ? u.T - 1 : t_last) / 128 + 1 : 0);
}
// Room for the blocks of joined units [u0, u1), blocks of `rows` rows.
void make_srcs(const std::vector<AttUnit>& units, int u0, int u1, int g, int rows, AttPlan& out) {
  out.src0.resize(units.size(), -1);
  for (int x = u0; x < u1; ++x) {
    if (!units[(size_t)x].joined) continue;
    out.src0[(size_t)x] = (int32_t)out.srcs.size();
    out.srcs.resize(out.srcs.size() + (size_t)((units[(size_t)x].T * g + rows - 1) / rows));
  }
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
void plan_wide(const std::vector<AttUnit>& units, int u0, int u1, int g, bool tree, int ctas,
               std::vector<std::vector<AttItem>>& by_cta, AttPlan& out) {
  struct Block {
    int unit, row0, rows, tiles;
  };
  std::vector<Block> blocks, rest;
  double total = kWideItem * ctas;   // about one cut per CTA
  make_srcs(units, u0, u1, g, 128, out);
  for (int x = u0; x < u1; ++x) {
    const int rows = units[(size_t)x].T * g;
    for (int r = 0; r < rows; r += kWideRows) {
      const int n = std::min(kWideRows, rows - r);
      const Block b{x, r, n, block_tiles(units[(size_t)x], g, r, n, tree)};
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
    const bool joined = units[(size_t)b.unit].joined;
    if (n == 1 && !joined) return;
    const int32_t p0 = (int32_t)out.n_parts;
    for (int y = 0; y < n; ++y) by_cta[(size_t)pieces[(size_t)y].first][pieces[(size_t)y].second].part = p0 + 2 * y;
    out.n_parts += 2 * n;
    if (joined) {
      AttSrc* s = &out.srcs[(size_t)(out.src0[(size_t)b.unit] + b.row0 / 128)];
      s[0] = AttSrc{p0, n, 2};
      if (b.rows > 128) s[1] = AttSrc{p0 + 1, n, 2};
      return;
    }
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
void plan_few(const std::vector<AttUnit>& units, int g, int R, bool tree, int sms, AttPlan& out) {
  double total = 0.0;
  make_srcs(units, 0, (int)units.size(), g, R, out);
  int64_t tiles = 0;
  for (const AttUnit& u : units)
    for (int r = 0; r < u.T * g; r += R) {
      const int t = block_tiles(u, g, r, std::min(R, u.T * g - r), tree);
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
      const int rows = std::min(R, u.T * g - r), n = block_tiles(u, g, r, rows, tree);
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
      if (pieces == 1 && !u.joined) continue;
      for (int y = 0; y < pieces; ++y) out.items[first + (size_t)y].part = (int32_t)out.n_parts + y;
      if (u.joined) {
        out.srcs[(size_t)(out.src0[(size_t)x] + r / R)] = AttSrc{out.n_parts, pieces, 1};
      } else {
        out.merges.push_back(AttMerge{x, r, rows, (int32_t)out.n_parts, pieces, 1});
        out.merge_rows = std::max(out.merge_rows, rows);
      }
      out.n_parts += pieces;
    }
  }
  out.cta_item.push_back((int32_t)out.items.size());
}

// A pass holds the operand tiles of as many units as fit into this many.
constexpr int64_t kTilesPerPass = 1 << 16;   // 4.3 GB

// The units of a call that run one after the other in the same way, shared out to the two kernels and planned.
struct AttSet {
  std::vector<AttUnit> few, wide;   // few and many rows per unit
  struct Where {
    int32_t wide, index;
  };
  std::vector<Where> where;         // of every unit that plan() was given
  AttPlan pf, pl;
  int R = 16;                       // rows of the first kernel's blocks
  struct Pass {
    int u0, u1, max_tiles, cta0;
  };
  std::vector<Pass> passes;         // of the second kernel
  int64_t most = 0;                 // operand tiles of a pass
  struct Placed {                   // a plan's arrays in the upload, its partials behind
    size_t units, items, ctas, merges, parts;
  } xf, xl;

  // units: hkv of every request (or prefix), kv head by kv head
  void plan(const std::vector<AttUnit>& units, int g, int hkv, bool tree, int sms) {
    int few_most = kFewMost;        // rows of a unit that the few-row kernel takes
    int64_t gain = -kWideStart * sms;
    for (size_t x = 0; x < units.size(); x += (size_t)hkv) {
      const int rows = units[x].T * g;
      if (rows > kFewMost) gain += kWideStart * sms;   // the other kernel runs anyway
      if (rows > kFewRows && rows <= kFewMost) gain += hkv * wide_gain(rows, block_tiles(units[x], g, 0, rows, tree));
    }
    if (gain > 0) few_most = kFewRows;
    int few_rows = 0;
    for (const AttUnit& u : units) {
      const bool many = u.T * g > few_most;
      where.push_back(Where{many, (int32_t)(many ? wide : few).size()});
      if (many) {
        wide.push_back(u);
      } else {
        few.push_back(u);
        few_rows = std::max(few_rows, u.T * g);
      }
    }
    R = few_rows <= 16 ? 16 : (few_rows <= 32 ? 32 : 64);
    if (!few.empty()) plan_few(few, g, R, tree, sms, pf);
    std::vector<std::vector<AttItem>> by_cta((size_t)sms);
    int64_t n = 0;
    int u0 = 0, max_tiles = 0;
    auto end_pass = [&](int x) {
      passes.push_back(Pass{u0, x, max_tiles, (int)pl.cta_item.size()});
      plan_wide(wide, u0, x, g, tree, sms, by_cta, pl);
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
    for (int x = 0; x < (int)wide.size(); ++x) {
      const int t = block_tiles(wide[(size_t)x], g, 0, wide[(size_t)x].T * g, tree);
      if (x > u0 && n + t > kTilesPerPass) end_pass(x);
      wide[(size_t)x].tile_base = (int32_t)n;
      n += t;
      max_tiles = std::max(max_tiles, t);
    }
    if (!wide.empty()) end_pass((int)wide.size());
  }
  void place(Upload& u) {
    auto one = [&](const std::vector<AttUnit>& un, const AttPlan& p, Placed& x) {
      x.units = u.add(un.data(), un.size() * sizeof(AttUnit));
      x.items = u.add(p.items.data(), p.items.size() * sizeof(AttItem));
      x.ctas = u.add(p.cta_item.data(), p.cta_item.size() * sizeof(int32_t));
      x.merges = u.add(p.merges.data(), p.merges.size() * sizeof(AttMerge));
    };
    if (!few.empty()) one(few, pf, xf);
    if (!wide.empty()) one(wide, pl, xl);
  }
  // partials from byte `at` on; returns the end
  size_t place_parts(size_t at) {
    xf.parts = at;
    xl.parts = at + (size_t)pf.n_parts * R * kAttPart * sizeof(float);
    return xl.parts + (size_t)pl.n_parts * 128 * kAttPart * sizeof(float);
  }
  // the joined units' blocks, in floats from byte `from` of the workspace; the first block of a unit of
  // each kind is src0[unit] + the index that comes back
  std::pair<int32_t, int32_t> add_srcs(size_t from, std::vector<AttSrc>& out) const {
    std::pair<int32_t, int32_t> at;
    auto add = [&](const AttPlan& p, size_t parts, int rows) {
      const int32_t first = (int32_t)out.size();
      for (AttSrc s : p.srcs) {
        s.off = (int64_t)((parts - from) / sizeof(float)) + s.off * rows * kAttPart;
        s.step *= rows * kAttPart;
        out.push_back(s);
      }
      return first;
    };
    at.first = add(pf, xf.parts, R);
    at.second = add(pl, xl.parts, 128);
    return at;
  }
  // chain: as launch_attend_few, where the set is one launch of that kernel
  bool one_launch() const { return wide.empty() && !few.empty() && pf.merges.empty(); }
  kv_status_t launch(kv_pool* P, const AttArgs& A, int64_t tiles, cudaStream_t s, int chain = 0) const {
    uint8_t* base = (uint8_t*)P->attend.ptr;
    auto merge = [&](const Placed& x, const AttPlan& p, int part_rows) -> cudaError_t {
      if (p.merges.empty()) return cudaSuccess;
      return launch_attend_merge(P, A, (const AttUnit*)(base + x.units), (const AttMerge*)(base + x.merges),
                                 (int)p.merges.size(), p.merge_rows, (const float*)(base + x.parts), part_rows, s);
    };
    if (!few.empty()) {
      KV_CUDA(launch_attend_few(P, R, A, (const AttUnit*)(base + xf.units), (const AttItem*)(base + xf.items),
                                (const int32_t*)(base + xf.ctas), (int)pf.cta_item.size() - 1, (float*)(base + xf.parts), s,
                                chain));
      KV_CUDA(merge(xf, pf, R));
    }
    if (wide.empty()) return KV_OK;
    const AttUnit* du = (const AttUnit*)(base + xl.units);
    uint32_t* d_live = (uint32_t*)((uint8_t*)P->attend_tiles.ptr + (size_t)tiles * kAttTileBytes);
    for (const Pass& G : passes) {
      KV_CUDA(launch_attend_tiles(P, A, du + G.u0, G.u1 - G.u0, G.max_tiles, P->attend_tiles.ptr, d_live, s));
      KV_CUDA(launch_attend_wide(P, A, du, (const AttItem*)(base + xl.items), (const int32_t*)(base + xl.ctas) + G.cta0,
                                 P->sm_count, P->attend_tiles.ptr, d_live, (float*)(base + xl.parts), s));
    }
    KV_CUDA(merge(xl, pl, 128));
    return KV_OK;
  }
};

// Workspaces of a call, grown: `bytes` of plan and partials, `tiles` operand tiles.
kv_status_t attend_room(kv_pool* P, size_t bytes, int64_t tiles) {
  const kv_status_t st = ensure(P->attend, bytes);
  if (st != KV_OK) return st;
  return ensure(P->attend_tiles, (size_t)tiles * (kAttTileBytes + 16), (size_t)kTilesPerPass * (kAttTileBytes + 16));
}

// The checks that both entries make; total: new tokens.
kv_status_t attend_check(const char* what, kv_pool* P, const void* q, const void* k, const void* v, const uint64_t* tree,
                         const int32_t* req_ids, const int32_t* n_new, int32_t n_req, int32_t hq, float softmax_scale,
                         const void* out, int64_t& total, int32_t& max_new) {
  if (!P) return fail(KV_ERR_INVALID_ARG, "%s: null pool", what);
  if (!req_ids || !n_new || n_req < 1) return fail(KV_ERR_INVALID_ARG, "%s: null pointer or n_req < 1", what);
  if ((k == nullptr) != (v == nullptr)) return fail(KV_ERR_INVALID_ARG, "%s: k and v come together", what);
  if (tree && !k) return fail(KV_ERR_INVALID_ARG, "%s: a tree needs k and v", what);
  const int hkv = P->cfg.num_kv_heads;
  if (hq < hkv || hq % hkv != 0 || hq / hkv > 8)
    return fail(KV_ERR_INVALID_ARG, "%s: num_q_heads %d must be a multiple of %d with ratio <= 8", what, hq, hkv);
  if (!std::isfinite(softmax_scale)) return fail(KV_ERR_INVALID_ARG, "%s: softmax_scale must be finite", what);
  if ((int64_t)n_req * hkv > 65535) return fail(KV_ERR_INVALID_ARG, "%s: n_req x num_kv_heads must be <= 65535", what);
  total = 0;
  max_new = 0;
  for (int32_t b = 0; b < n_req; ++b) {
    if (!req_ok(P, req_ids[b])) return fail(KV_ERR_INVALID_ARG, "%s: request %d not open", what, req_ids[b]);
    if (n_new[b] < 0 || n_new[b] > kMaxNewTokens)
      return fail(KV_ERR_INVALID_ARG, "%s: n_new[%d] = %d is not in [0, %d]", what, b, n_new[b], kMaxNewTokens);
    if (tree && n_new[b] > 64) return fail(KV_ERR_INVALID_ARG, "%s: a tree holds at most 64 tokens of a request", what);
    total += n_new[b];
    max_new = std::max(max_new, n_new[b]);
  }
  if (total == 0) return KV_OK;
  if (total > kMaxRows / hq)
    return fail(KV_ERR_INVALID_ARG, "%s: more than %lld rows (tokens x num_q_heads)", what, (long long)kMaxRows);
  if (!q || !out) return fail(KV_ERR_INVALID_ARG, "%s: null pointer", what);
  return KV_OK;
}

AttArgs attend_args(const kv_pool* P, const void* q, const void* k, const void* v, const uint64_t* tree, int32_t hq,
                    float softmax_scale, void* out) {
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
  A.tok_map = nullptr;
  A.out = (uint16_t*)out;
  A.status = P->d_status;
  A.scale_log2 = softmax_scale * 1.4426950408889634f;
  A.max_pages = P->cfg.max_pages_per_request;
  A.hkv = P->cfg.num_kv_heads;
  A.hq = hq;
  A.fp_cap = P->fp_cap;
  return A;
}

AttUnit attend_unit(const kv_pool* P, int32_t r, int h, int32_t T, bool kv, int64_t tok0) {
  return AttUnit{r, h, T, (int32_t)P->reqs[r].table.size(), P->n_fp.empty() ? 0 : P->n_fp[r], 0, tok0, -1, kv ? T : 0, 0, 0};
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" kv_status_t kv_attend(kv_pool_t* P, const void* q, const void* k, const void* v, const uint64_t* tree,
                                 const int32_t* req_ids, const int32_t* n_new, int32_t n_req, int32_t hq,
                                 float softmax_scale, void* out, void* stream) try {
  int64_t total;
  int32_t max_new;
  kv_status_t st = attend_check("kv_attend", P, q, k, v, tree, req_ids, n_new, n_req, hq, softmax_scale, out, total, max_new);
  if (st != KV_OK || total == 0) return st;
  DeviceGuard dg(P->cfg.device);
  cudaStream_t s = (cudaStream_t)stream;
  if ((st = refuse_capture("kv_attend", s)) != KV_OK) return st;
  if ((st = order_after_previous(P, s)) != KV_OK) return st;
  const AttArgs A = attend_args(P, q, k, v, tree, hq, softmax_scale, out);
  const int hkv = A.hkv, g = hq / hkv;
  std::vector<AttUnit> units;
  int64_t tok0 = 0;
  for (int32_t b = 0; b < n_req; ++b) {
    if (n_new[b] > 0)
      for (int h = 0; h < hkv; ++h) units.push_back(attend_unit(P, req_ids[b], h, n_new[b], k != nullptr, tok0));
    tok0 += n_new[b];
  }
  Upload u;
  if (P->decode_impl == KV_DECODE_SIMT) {
    u.add(units.data(), units.size() * sizeof(AttUnit));
    if ((st = ensure(P->attend, u.size)) != KV_OK) return st;
    if ((st = h2d(P, P->attend.ptr, u, s)) != KV_OK) return st;
    KV_CUDA(launch_attend_simt(P, A, (const AttUnit*)P->attend.ptr, (int)units.size(), max_new * g, s));
    return KV_OK;
  }
  AttSet S;
  S.plan(units, g, hkv, tree != nullptr, P->sm_count);
  S.place(u);
  const size_t end = S.place_parts((u.size + 255) & ~size_t(255));
  if ((st = attend_room(P, end, S.most)) != KV_OK) return st;
  if ((st = h2d(P, P->attend.ptr, u, s)) != KV_OK) return st;
  return S.launch(P, A, S.most, s);
} catch (const std::bad_alloc&) {
  return fail(KV_ERR_OOM, "kv_attend: host allocation failed");
}

// The rows of every request with a prefix are in two units: the prefix's, which reads its keys once for all of
// them, and the request's own.  Both give partials, joined at the end.
extern "C" kv_status_t kv_attend_shared(kv_pool_t* P, const void* q, const void* k, const void* v, const uint64_t* tree,
                                        const int32_t* req_ids, const int32_t* prefix_ids, const int32_t* n_new,
                                        int32_t n_req, int32_t hq, float softmax_scale, void* out, void* stream) try {
  int64_t total;
  int32_t max_new;
  kv_status_t st =
      attend_check("kv_attend_shared", P, q, k, v, tree, req_ids, n_new, n_req, hq, softmax_scale, out, total, max_new);
  if (st != KV_OK) return st;
  if (!prefix_ids) return fail(KV_ERR_INVALID_ARG, "kv_attend_shared: null prefix_ids");
  // prefixes in the order of their first request, each with its requests
  std::vector<int32_t> group_of((size_t)n_req, -1), pre_id;
  std::vector<int64_t> pre_tok((size_t)n_req, 0), tok0((size_t)n_req, 0), group_T;
  {
    std::vector<int32_t> at((size_t)P->cfg.max_requests, -1);
    int64_t t = 0;
    for (int32_t b = 0; b < n_req; ++b) {
      const int32_t p = prefix_ids[b];
      tok0[(size_t)b] = t;
      t += n_new[b];
      if (p == -1) continue;
      if (!req_ok(P, p)) return fail(KV_ERR_INVALID_ARG, "kv_attend_shared: prefix %d not open", p);
      if (p == req_ids[b]) return fail(KV_ERR_INVALID_ARG, "kv_attend_shared: request %d is its own prefix", p);
      if (n_new[b] == 0) continue;
      int32_t& x = at[(size_t)p];
      if (x < 0) {
        x = (int32_t)pre_id.size();
        pre_id.push_back(p);
        group_T.push_back(0);
      }
      group_of[(size_t)b] = x;
      pre_tok[(size_t)b] = group_T[(size_t)x];
      if ((group_T[(size_t)x] += n_new[b]) > kMaxNewTokens)
        return fail(KV_ERR_INVALID_ARG, "kv_attend_shared: more than %d new tokens share prefix %d", kMaxNewTokens, p);
    }
  }
  if (total == 0) return KV_OK;
  DeviceGuard dg(P->cfg.device);
  cudaStream_t s = (cudaStream_t)stream;
  if ((st = refuse_capture("kv_attend_shared", s)) != KV_OK) return st;
  if ((st = order_after_previous(P, s)) != KV_OK) return st;
  AttArgs A = attend_args(P, q, k, v, tree, hq, softmax_scale, out);
  const int hkv = A.hkv, g = hq / hkv;

  // ---- the prefixes' units: tokens that lie together by their first row, others by a list
  std::vector<AttUnit> pre, own;
  std::vector<int32_t> tok_map;
  {
    const size_t n = pre_id.size();
    std::vector<int64_t> first(n, -1);
    std::vector<uint8_t> apart(n, 0);
    for (int32_t b = 0; b < n_req; ++b) {
      const int32_t x = group_of[(size_t)b];
      if (x < 0) continue;
      if (first[(size_t)x] < 0) first[(size_t)x] = tok0[(size_t)b];
      if (tok0[(size_t)b] != first[(size_t)x] + pre_tok[(size_t)b]) apart[(size_t)x] = 1;
    }
    std::vector<int32_t> map(n, -1);
    for (size_t x = 0; x < n; ++x)
      if (apart[x]) {
        map[x] = (int32_t)tok_map.size();
        tok_map.resize(tok_map.size() + (size_t)group_T[x]);
      }
    for (int32_t b = 0; b < n_req; ++b) {
      const int32_t x = group_of[(size_t)b];
      if (x < 0 || map[(size_t)x] < 0) continue;
      for (int32_t t = 0; t < n_new[b]; ++t)
        tok_map[(size_t)(map[(size_t)x] + pre_tok[(size_t)b] + t)] = (int32_t)(tok0[(size_t)b] + t);
    }
    for (size_t x = 0; x < n; ++x)
      for (int h = 0; h < hkv; ++h) {
        AttUnit w = attend_unit(P, pre_id[x], h, (int32_t)group_T[x], false, map[x] < 0 ? first[x] : 0);
        w.map = map[x];
        w.joined = 1;
        pre.push_back(w);
      }
  }
  for (int32_t b = 0; b < n_req; ++b)
    for (int h = 0; h < hkv && n_new[b] > 0; ++h) {
      AttUnit w = attend_unit(P, req_ids[b], h, n_new[b], k != nullptr, tok0[(size_t)b]);
      // (few rows without a prefix too, so that one kernel ends the call; more of them would be partials of 528 bytes
      // a row, written and read again: 4096 tokens x 64 q heads beside one token with a prefix took 561 us that way,
      // 391 without)
      w.joined = group_of[(size_t)b] >= 0 || (!pre.empty() && n_new[b] * g <= kFewRows);
      own.push_back(w);
    }
  // One launch for both kinds where their rows go by blocks of one size, or where there is so little
  // work that a launch and a plan more count for more than the larger blocks (4 requests over 2K tokens of
  // 2 kv heads: 20 us of the host's time a call, 34 apart).
  auto size_of = [&](const std::vector<AttUnit>& units, int64_t& tiles) {
    int rows = 0;
    tiles = 0;
    for (const AttUnit& w : units) {
      rows = std::max(rows, w.T * g);
      tiles += block_tiles(w, g, 0, w.T * g, tree != nullptr);
    }
    return rows;
  };
  int64_t pre_tiles, own_tiles;
  const int pre_rows = size_of(pre, pre_tiles), own_rows = size_of(own, own_tiles);
  auto block_of = [](int rows) { return rows <= 16 ? 16 : (rows <= 32 ? 32 : 64); };
  const bool little = pre_tiles + own_tiles <= 2 * (int64_t)P->sm_count;
  // A decode step (a token per request, nothing but caches): the decode's scan reads the own caches faster than the
  // few-row kernel, whose blocks such rows fill to a quarter or half: 32 x 1050 tokens, 32 q and 8 kv heads, 19 us
  // against 32; 64 x 1000, 64 and 8 heads, 29 against 58.  It costs two launches and a plan more, so not for few tiles.
  // The scan scales rows of q to binary16 by 2^-100 to 2^100: enough for every row whose logits are neither all
  // near 0 nor past fp32, if the softmax's scale is within 2^40 of one.
  const float abs_scale = std::fabs(softmax_scale);
  bool scan = !k && !little && own_tiles > 4 * (int64_t)P->sm_count && abs_scale >= 0x1p-40f && abs_scale <= 0x1p40f;
  for (int32_t b = 0; b < n_req && scan; ++b)
    scan = n_new[b] == 1 && (P->n_fp.empty() || P->n_fp[req_ids[b]] == 0);
  const bool together = !scan && !pre.empty() && std::max(pre_rows, own_rows) <= kFewRows &&
                        (block_of(pre_rows) == block_of(own_rows) || little);
  const size_t n_pre = pre.size();
  AttSet SP, SO;   // together: SO holds the prefixes' units too, first
  if (together) {
    std::vector<AttUnit> all(pre);
    all.insert(all.end(), own.begin(), own.end());
    SO.plan(all, g, hkv, tree != nullptr, P->sm_count);
  } else {
    SP.plan(pre, g, hkv, tree != nullptr, P->sm_count);
    if (!scan) SO.plan(own, g, hkv, tree != nullptr, P->sm_count);
  }
  const size_t o0 = together ? n_pre : 0;   // the first own unit of SO

  // ---- joins; where a unit's blocks are: units go to a set's two lists in order
  std::vector<AttJoin> joins;
  std::vector<AttSrc> srcs;
  int32_t join_rows = 0;
  Upload u;
  SP.place(u);
  SO.place(u);
  const size_t o_map = u.add(tok_map.data(), tok_map.size() * sizeof(int32_t));
  // the partials lie behind everything that is uploaded: sizes first
  const size_t n_src = SP.pf.srcs.size() + SP.pl.srcs.size() + SO.pf.srcs.size() + SO.pl.srcs.size();
  size_t n_joins = 0;
  for (const AttUnit& w : own) n_joins += scan || w.joined ? 1 : 0;
  joins.reserve(n_joins);
  srcs.reserve(n_src);
  const size_t o_joins = u.add(joins.data(), n_joins * sizeof(AttJoin));
  const size_t o_srcs = u.add(srcs.data(), n_src * sizeof(AttSrc));
  const size_t end = SO.place_parts(SP.place_parts((u.size + 255) & ~size_t(255)));
  const auto ps0 = SP.add_srcs(0, srcs), os = SO.add_srcs(0, srcs);
  const auto ps = together ? os : ps0;
  const AttSet& PS = together ? SO : SP;   // where the prefixes' units are
  auto log2i = [](int x) { int n = 0; while ((1 << n) < x) ++n; return n; };
  size_t x = 0;
  for (int32_t b = 0; b < n_req; ++b)
    for (int h = 0; h < hkv && n_new[b] > 0; ++h, ++x) {
      if (!scan && !own[x].joined) continue;
      AttJoin J{};
      J.tok0 = own[x].tok0;
      J.kvh = h;
      J.rows = n_new[b] * g;
      J.req = own[x].req;
      J.n_pages = own[x].n_pages;
      if (scan) {
        J.own0 = (int32_t)x;   // the decode plan's units are in this order
        J.flags = kJoinScan;
      } else {
        const AttSet::Where o = SO.where[o0 + x];
        J.own0 = o.wide ? os.second + SO.pl.src0[(size_t)o.index] : os.first + SO.pf.src0[(size_t)o.index];
        J.own_shift = o.wide ? 7 : log2i(SO.R);
        J.flags = o.wide ? kJoinOwnTall : 0;
      }
      J.pre0 = -1;
      if (group_of[(size_t)b] >= 0) {
        const AttSet::Where p = PS.where[(size_t)group_of[(size_t)b] * hkv + h];
        J.pre0 = p.wide ? ps.second + PS.pl.src0[(size_t)p.index] : ps.first + PS.pf.src0[(size_t)p.index];
        J.pre_shift = p.wide ? 7 : log2i(PS.R);
        J.pre_row = (int32_t)pre_tok[(size_t)b] * g;
        J.flags |= p.wide ? kJoinPreTall : 0;
      }
      joins.push_back(J);
      join_rows = std::max(join_rows, J.rows);
    }
  const int64_t tiles = std::max(SP.most, SO.most);
  if ((st = attend_room(P, end, tiles)) != KV_OK) return st;
  DecodePlan& D = P->shared_plan;
  if (scan) {
    if ((st = build_plan(P, D, req_ids, n_req, hq, KV_DECODE_MMA, s)) != KV_OK) return st;
    if ((st = ensure(P->shared_partials, (size_t)std::max(D.n_splits, 1) * g * kAttPart * sizeof(float))) != KV_OK) return st;
    if ((st = ensure(P->shared_frags, (size_t)std::max(D.n_units, 1) * decode_mma_frag_bytes())) != KV_OK) return st;
  }
  if ((st = h2d(P, P->attend.ptr, u, s)) != KV_OK) return st;
  uint8_t* base = (uint8_t*)P->attend.ptr;
  A.tok_map = (const int32_t*)(base + o_map);
  // The second attention launch starts as CTAs of the first leave, the joins as those of the second do.  A scan of
  // the own caches starts when the first launch is done: only its q operands are prepared meanwhile.
  const bool chained = SP.one_launch() && (scan || SO.one_launch());
  if ((st = SP.launch(P, A, tiles, s, chained ? kChainNext : 0)) != KV_OK) return st;
  const uint8_t* plan = (const uint8_t*)D.buf.ptr;
  const Unit* scan_units = scan ? (const Unit*)(plan + D.units_off) : nullptr;
  if (scan)
    KV_CUDA(launch_scan_mma(P, q, hq, A.scale_log2, scan_units, D.n_units, (const Split*)(plan + D.splits_off),
                            (const int32_t*)(plan + D.cta_off), D.n_ctas, P->shared_frags.ptr, (float*)P->shared_partials.ptr, s));
  else if ((st = SO.launch(P, A, tiles, s, SO.one_launch() ? kChainNext | (chained ? kChainPrev : 0) : 0)) != KV_OK)
    return st;
  KV_CUDA(launch_attend_join(P, A, (const AttJoin*)(base + o_joins), (int)joins.size(), join_rows,
                             (const AttSrc*)(base + o_srcs), (const float*)base, scan_units, (const float*)P->shared_partials.ptr, s));
  return KV_OK;
} catch (const std::bad_alloc&) {
  return fail(KV_ERR_OOM, "kv_attend_shared: host allocation failed");
}
