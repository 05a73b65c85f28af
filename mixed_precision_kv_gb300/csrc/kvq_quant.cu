// Quantize-on-append (INT4 tail / staging pages), INT2 repack and table
// scatter kernels.
//
// Quantization follows TriAxialKV, key design 3 (asymmetric group
// quantization, G = 32): for a group with minimum mn and maximum mx,
//   scale = half_rn((mx - mn) / (2^b - 1)),  zero = half_rn(mn),
//   code  = clamp(rint((x - zero) / scale), 0, 2^b - 1)   (0 when scale == 0),
// with IEEE fp32 subtraction and division (no fast-math, no FTZ) and binary16
// round-to-nearest-even storage.  INT4 K and V are per token (32 consecutive
// channels); the INT2 repack dequantizes a full 32-token staging page with
// fmaf(code, scale, zero) and requantizes K per channel (across the 32 tokens)
// and V per token.
#include <cuda_fp16.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 128;

// Every kernel that reads K rows comes in two forms: as they are, or rotated on the
// way (kRope: RopeArgs, which also gives the distance between tokens' rows).
struct NoRope {};
template <bool kRope>
using RopeParam = std::conditional_t<kRope, RopeArgs, NoRope>;
// elements from a token's K (V) rows to the next token's
template <bool kRope>
__device__ __forceinline__ size_t k_step(const RopeParam<kRope>& R, int hkv) {
  if constexpr (kRope) return (size_t)R.k_stride;
  else return (size_t)hkv * kHeadDim;
}
template <bool kRope>
__device__ __forceinline__ size_t v_step(const RopeParam<kRope>& R, int hkv) {
  if constexpr (kRope) return (size_t)R.v_stride;
  else return (size_t)hkv * kHeadDim;
}

__device__ __forceinline__ bool out_of_range(float x) { return !(fabsf(x) <= 65504.0f); }

struct GroupMeta {
  __half s, z;
  float sf, zf;
  bool nz;
};

__device__ __forceinline__ GroupMeta make_meta(float mn, float mx, float qmax) {
  GroupMeta m;
  const float s32 = __fdiv_rn(__fsub_rn(mx, mn), qmax);
  m.s = __float2half_rn(s32);
  m.z = __float2half_rn(mn);
  m.sf = __half2float(m.s);
  m.zf = __half2float(m.z);
  m.nz = (__half_as_ushort(m.s) & 0x7FFFu) != 0;
  return m;
}

// code = clamp(rint(fl((x - zero) / scale)), 0, qmax) (0 when scale == 0),
// without a division in the common case.  rs = approximate
// reciprocal of m.sf (relative error < 2^-22), so q0 = u * rs lies within
// 4e-6 of the correctly rounded quotient fl(u / s) for |u / s| < 64 (here
// |u / s| <= qmax + 1).  When q0 is more than 1e-5 from every half-integer,
// fl(u / s) rounds to the same integer; otherwise the quotient is computed
// exactly.  Same result as the division form, bit for bit.
__device__ __forceinline__ float approx_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t qcode_fast(float x, const GroupMeta& m, float rs, float qmax) {
  if (!m.nz) return 0u;
  const float u = __fsub_rn(x, m.zf);
  const float q0 = u * rs;
  float c = rintf(q0);
  if (!(fabsf(fabsf(q0 - c) - 0.5f) > 1e-5f)) c = rintf(__fdiv_rn(u, m.sf));
  return (uint32_t)fminf(fmaxf(c, 0.0f), qmax);
}

// min / max over the 8 lanes of one 32-channel group (lanes 8*gr .. 8*gr + 7)
__device__ __forceinline__ void group8_minmax(float& mn, float& mx) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  }
}

__device__ __forceinline__ void st_half(uint8_t* img, int byte_off, __half h) {
  *reinterpret_cast<__half*>(img + byte_off) = h;
}

__device__ __forceinline__ void or_bits(uint8_t* img, int byte_off, int shift, uint32_t val) {
  atomicOr(reinterpret_cast<uint32_t*>(img) + (byte_off >> 2), val << (8 * (byte_off & 3) + shift));
}

// Quantize one token (a warp: lane = channels 4*lane .. 4*lane+3) into slot
// `slot` of an INT4 block image `img` (shared or global memory).  V nibbles
// are OR-ed in: the block's unfilled slots hold zeros.
// With vcodes (shared memory, [slot][channel] bytes) the V codes go there
// for a later word-wise packing (pack_i4v) instead of being OR-ed into img.
// vmax: the warp's running maximum of V scales (one atomic per warp at the
// end instead of one per token on the pool's single maximum word).
// A token's K and V rows of one kv head, as each lane holds them (4 bf16
// channels 4*lane .. 4*lane+3 of each).
struct RawRows {
  uint2 kr, vr;
};
// With kRope they come with the lane's factors, and turned() gives K rotated (rounded
// to bf16, as a key that came rotated would be).
template <bool kRope>
struct Rows {
  RawRows raw;
  std::conditional_t<kRope, RopeLane, NoRope> lane;
};
template <bool kRope>
__device__ __forceinline__ Rows<kRope> load_rows(const RopeParam<kRope>& R, const __nv_bfloat16* __restrict__ k,
                                                 const __nv_bfloat16* __restrict__ v, int t, int h, int hkv, bool& bad) {
  const size_t at = (size_t)h * kHeadDim + 4 * (threadIdx.x & 31);
  Rows<kRope> r;
  r.raw = RawRows{*reinterpret_cast<const uint2*>(k + (size_t)t * k_step<kRope>(R, hkv) + at),
                  *reinterpret_cast<const uint2*>(v + (size_t)t * v_step<kRope>(R, hkv) + at)};
  if constexpr (kRope) r.lane = rope_lane(R, t, bad);
  return r;
}
template <bool kRope>
__device__ __forceinline__ RawRows turned(const RopeParam<kRope>& R, const Rows<kRope>& r) {
  if constexpr (kRope) return RawRows{rope_lane_turn(R, r.raw.kr, r.lane), r.raw.vr};
  else return r.raw;
}

__device__ __forceinline__ bool quantize_rows(uint8_t* img, const RawRows& rr, int slot, float& vmax,
                                              uint8_t* vcodes = nullptr) {
  const int lane = threadIdx.x & 31, gr = lane >> 3;
  const uint2 kr = rr.kr, vr = rr.vr;
  float xk[4], xv[4];
  xk[0] = __uint_as_float(kr.x << 16); xk[1] = __uint_as_float(kr.x & 0xFFFF0000u);
  xk[2] = __uint_as_float(kr.y << 16); xk[3] = __uint_as_float(kr.y & 0xFFFF0000u);
  xv[0] = __uint_as_float(vr.x << 16); xv[1] = __uint_as_float(vr.x & 0xFFFF0000u);
  xv[2] = __uint_as_float(vr.y << 16); xv[3] = __uint_as_float(vr.y & 0xFFFF0000u);
  bool bad = false;
  float kmn = xk[0], kmx = xk[0], vmn = xv[0], vmx = xv[0];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    bad |= out_of_range(xk[a]) | out_of_range(xv[a]);
    kmn = fminf(kmn, xk[a]); kmx = fmaxf(kmx, xk[a]);
    vmn = fminf(vmn, xv[a]); vmx = fmaxf(vmx, xv[a]);
  }
  group8_minmax(kmn, kmx);
  group8_minmax(vmn, vmx);
  const GroupMeta km = make_meta(kmn, kmx, 15.0f);
  const GroupMeta vm = make_meta(vmn, vmx, 15.0f);
  uint32_t ck[4], cv[4];
  const float krs = approx_rcp(km.sf), vrs = approx_rcp(vm.sf);
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    ck[a] = qcode_fast(xk[a], km, krs, 15.0f);
    cv[a] = qcode_fast(xv[a], vm, vrs, 15.0f);
  }
  // K: channels 4*lane .. 4*lane+3 are nibbles 0..3 or 4..7 of one word -> 2 bytes
  const int kb = i4k_byte(slot, 4 * lane);
  *reinterpret_cast<uint16_t*>(img + kb) = (uint16_t)(ck[0] | (ck[1] << 4) | (ck[2] << 8) | (ck[3] << 12));
  // V: channel-major, one nibble per channel
  if (vcodes) {
    *reinterpret_cast<uint32_t*>(vcodes + kHeadDim * slot + 4 * lane) = cv[0] | (cv[1] << 8) | (cv[2] << 16) | (cv[3] << 24);
  } else {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int c = 4 * lane + a;
      or_bits(img, i4v_byte(slot, c), i4v_shift(slot), cv[a]);
    }
  }
  vmax = fmaxf(vmax, vm.sf);   // per lane; reduced over the warp by flush_vmax
  if ((lane & 7) == 0) {
    st_half(img, kI4KMeta + 16 * slot + 4 * gr, km.s);
    st_half(img, kI4KMeta + 16 * slot + 4 * gr + 2, km.z);
    st_half(img, kI4VMeta + 2 * v_meta_index(slot, gr), vm.s);
    st_half(img, kI4VMeta + 256 + 2 * v_meta_index(slot, gr), vm.z);
  }
  return bad;
}

// The tokens j = warp, warp + W, ... < n of a job (W = warps per CTA), each
// into slot first + j: their indices are read at once (lane q holds the q-th)
// and the next token's rows are loaded while the current one is quantized.
template <int W, bool kRope>
__device__ __forceinline__ bool quantize_tokens(const RopeParam<kRope>& R, uint8_t* img, const __nv_bfloat16* __restrict__ k,
                                                const __nv_bfloat16* __restrict__ v,
                                                const int32_t* __restrict__ tk, int n, int first, int h, int hkv,
                                                float& vmax, uint8_t* vcodes) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = n > warp ? (n - warp + W - 1) / W : 0;   // <= 32 / W
  const int t_l = lane < mine ? tk[warp + W * lane] : 0;
  bool bad = false;
  if (mine == 0) return bad;
  Rows<kRope> cur = load_rows<kRope>(R, k, v, __shfl_sync(0xFFFFFFFFu, t_l, 0), h, hkv, bad);
  for (int q = 0; q < mine; ++q) {
    Rows<kRope> nxt = cur;
    if (q + 1 < mine) nxt = load_rows<kRope>(R, k, v, __shfl_sync(0xFFFFFFFFu, t_l, q + 1), h, hkv, bad);
    bad |= quantize_rows(img, turned<kRope>(R, cur), first + warp + W * q, vmax, vcodes);
    cur = nxt;
  }
  return bad;
}

// One atomic per warp for the pool's running maximum of V scales
// (non-negative floats order as their bits).
__device__ __forceinline__ void flush_vmax(float vmax, uint32_t* __restrict__ status) {
#pragma unroll
  for (int o = 16; o; o >>= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xFFFFFFFFu, vmax, o));
  if ((threadIdx.x & 31) == 0 && vmax > 0.0f) atomicMax(status + 2, __float_as_uint(vmax));
}

// INT4 V words from [slot][channel] code bytes: word (channel c, slot chunk j)
// holds slots 8j .. 8j+7 in nibbles 0..7; every word is built by one thread.
__device__ __forceinline__ void pack_i4v(uint8_t* __restrict__ img, const uint8_t* __restrict__ vcodes) {
  for (int x = threadIdx.x; x < kHeadDim * (kPage / 8); x += kThreads) {
    const int c = x & (kHeadDim - 1), j = x >> 7;
    uint32_t w = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) w |= (uint32_t)vcodes[kHeadDim * (8 * j + k) + c] << (4 * k);
    *reinterpret_cast<uint32_t*>(img + i4v_byte(8 * j, c)) = w;
  }
}

// Positions of a page's slots first .. first + n - 1 (a new page's others: -1, no token), by one CTA: tp, or
// the tokens' indices and a constant.
__device__ __forceinline__ void write_positions(int32_t* __restrict__ pos, int32_t page, const int32_t* tp,
                                                const int32_t* __restrict__ tk, int32_t pos0, int first, int n) {
  const int t = threadIdx.x;
  if (t >= kPage || t < first) return;
  if (t < first + n)
    pos[(size_t)page * kPage + t] = tp ? tp[t - first] : pos0 + tk[t - first];
  else if (first == 0)
    pos[(size_t)page * kPage + t] = -1;
}

// One CTA per (job, kv head), a warp per token.  A new page (job starting at
// slot 0) is built as an image in shared memory from zeros and written whole,
// so its unfilled slots read as code 0, scale 0, zero 0; a page that already
// holds tokens gets only its new slots written in place (the V words by
// atomic OR).  The kv-head-0 CTA also writes the page's table entry and the
// request's table length, so an append that only fills or adds tail pages
// needs no separate table update.
template <bool kByValue, bool kRope>
__global__ void __launch_bounds__(kThreads) append_int4_kernel(
    uint8_t* __restrict__ pool, size_t int4_off, int64_t n2, int hkv, const __nv_bfloat16* __restrict__ k,
    const __nv_bfloat16* __restrict__ v, const AppendJob* __restrict__ jobs, const int32_t* __restrict__ toks,
    Entry* __restrict__ table, int32_t* __restrict__ ntab, uint32_t* __restrict__ status,
    const __grid_constant__ SmallAppend small, int32_t* __restrict__ pos, const int32_t* __restrict__ tok_pos,
    const __grid_constant__ RopeParam<kRope> rope) {
  __shared__ __align__(16) uint8_t img[kInt4Block];
  __shared__ __align__(16) uint8_t vcodes[kPage * kHeadDim];   // V codes of a new page, packed after
  wait_for_grid(k, v);   // earlier work on the stream (the previous decode) is done
  asm volatile("griddepcontrol.launch_dependents;");
  const AppendJob job = kByValue ? small.jobs[blockIdx.x] : jobs[blockIdx.x];
  const int32_t* tk = kByValue ? small.toks : toks;
  const int h = blockIdx.y;
  uint8_t* blk = pool + int4_off + ((size_t)(job.page - n2) * hkv + h) * kInt4Block;
  const bool fresh = job.first_slot == 0;
  bool bad = false;
  float vmax = 0.0f;
  if (fresh) {
    uint4* img4 = reinterpret_cast<uint4*>(img);
    for (int i = threadIdx.x; i < kInt4Block / 16; i += kThreads) img4[i] = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < kPage * kHeadDim / 16; i += kThreads)
      reinterpret_cast<uint4*>(vcodes)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    bad |= quantize_tokens<kThreads / 32, kRope>(rope, img, k, v, tk + job.tok_off, job.n_slots, job.first_slot, h, hkv,
                                                 vmax, vcodes);
    __syncthreads();
    pack_i4v(img, vcodes);
    __syncthreads();
    uint4* out4 = reinterpret_cast<uint4*>(blk);
    for (int i = threadIdx.x; i < kInt4Block / 16; i += kThreads) out4[i] = img4[i];
  } else {
    bad |= quantize_tokens<kThreads / 32, kRope>(rope, blk, k, v, tk + job.tok_off, job.n_slots, job.first_slot, h, hkv,
                                                 vmax, nullptr);
  }
  if (pos && h == 0) {
    const int32_t* tp = kByValue ? small.pos : tok_pos;
    write_positions(pos, job.page, tp ? tp + job.tok_off : nullptr, tk + job.tok_off, job.pos0, job.first_slot, job.n_slots);
  }
  flush_vmax(vmax, status);
  if (bad) atomicOr(status, kStatusRange);
  if (h == 0 && threadIdx.x == 0) {
    if (job.tab_index >= 0) table[job.tab_index] = Entry{job.page, job.live};
    if (job.ntab_req >= 0) ntab[job.ntab_req] = job.ntab_len;
  }
}

// ---- INT3 pages (TriAxialKV, limitations and outlook: INT3 as a further
// width): the INT4 per-token rule with 2^3 - 1 levels, codes stored as a
// 2-bit low plane and a 1-bit high plane.  A warp quantizes one token of one
// kv head, lane = channels 4*lane .. 4*lane+3 (one group per 8 lanes).
// K: a lane's four low-bit fields are one byte of the token's low plane and
// its four high bits one nibble of the high plane, whose byte it shares with
// the lane of the neighbouring group (lane ^ 8): the even group's lane writes
// the byte.  V (channel-major) goes to vcodes for a fresh page (packed by
// pack_i3v), else its bits are OR-ed into the block.
__device__ __forceinline__ bool quantize_rows3(uint8_t* img, const RawRows& rr, int slot, float& vmax,
                                               uint8_t* vcodes) {
  const int lane = threadIdx.x & 31, gr = lane >> 3;
  const uint2 kr = rr.kr, vr = rr.vr;
  float xk[4], xv[4];
  xk[0] = __uint_as_float(kr.x << 16); xk[1] = __uint_as_float(kr.x & 0xFFFF0000u);
  xk[2] = __uint_as_float(kr.y << 16); xk[3] = __uint_as_float(kr.y & 0xFFFF0000u);
  xv[0] = __uint_as_float(vr.x << 16); xv[1] = __uint_as_float(vr.x & 0xFFFF0000u);
  xv[2] = __uint_as_float(vr.y << 16); xv[3] = __uint_as_float(vr.y & 0xFFFF0000u);
  bool bad = false;
  float kmn = xk[0], kmx = xk[0], vmn = xv[0], vmx = xv[0];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    bad |= out_of_range(xk[a]) | out_of_range(xv[a]);
    kmn = fminf(kmn, xk[a]); kmx = fmaxf(kmx, xk[a]);
    vmn = fminf(vmn, xv[a]); vmx = fmaxf(vmx, xv[a]);
  }
  group8_minmax(kmn, kmx);
  group8_minmax(vmn, vmx);
  const GroupMeta km = make_meta(kmn, kmx, 7.0f);
  const GroupMeta vm = make_meta(vmn, vmx, 7.0f);
  uint32_t ck[4], cv[4];
  const float krs = approx_rcp(km.sf), vrs = approx_rcp(vm.sf);
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    ck[a] = qcode_fast(xk[a], km, krs, 7.0f);
    cv[a] = qcode_fast(xv[a], vm, vrs, 7.0f);
  }
  const int c0 = 4 * lane;
  img[i3k_lo_byte(slot, c0)] = (uint8_t)((ck[0] & 3u) | ((ck[1] & 3u) << 2) | ((ck[2] & 3u) << 4) | ((ck[3] & 3u) << 6));
  const uint32_t hi = (ck[0] >> 2) | ((ck[1] >> 2) << 1) | ((ck[2] >> 2) << 2) | ((ck[3] >> 2) << 3);
  const uint32_t hi_odd = __shfl_xor_sync(0xFFFFFFFFu, hi, 8);
  if ((gr & 1) == 0) img[i3k_hi_byte(slot, c0)] = (uint8_t)(hi | (hi_odd << 4));
  if (vcodes) {
    *reinterpret_cast<uint32_t*>(vcodes + kHeadDim * slot + c0) = cv[0] | (cv[1] << 8) | (cv[2] << 16) | (cv[3] << 24);
  } else {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int c = c0 + a;
      or_bits(img, i3v_lo_byte(slot, c), i3v_lo_shift(slot), cv[a] & 3u);
      or_bits(img, i3v_hi_byte(slot, c), i3v_hi_shift(slot, c), cv[a] >> 2);
    }
  }
  vmax = fmaxf(vmax, vm.sf);
  if ((lane & 7) == 0) {
    st_half(img, kI3KMeta + 16 * slot + 4 * gr, km.s);
    st_half(img, kI3KMeta + 16 * slot + 4 * gr + 2, km.z);
    st_half(img, kI3VMeta + 2 * v_meta_index(slot, gr), vm.s);
    st_half(img, kI3VMeta + 256 + 2 * v_meta_index(slot, gr), vm.z);
  }
  return bad;
}

// INT3 V planes from [slot][channel] code bytes, every word by one thread:
// low-plane word (chunk X, h) and high-plane word X of the layout.
__device__ __forceinline__ void pack_i3v(uint8_t* __restrict__ img, const uint8_t* __restrict__ vcodes) {
  for (int x = threadIdx.x; x < 3 * 128; x += kThreads) {
    const int X = x < 256 ? x >> 1 : x - 256;
    const int mh = X >> 5, r = (X >> 2) & 7, j = X & 3;   // chunk X = 32 (m >> 1) + 4 r + j
    uint32_t w = 0u;
    if (x < 256) {
      const int h = x & 1, m = 2 * mh + h;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          w |= ((uint32_t)vcodes[kHeadDim * (8 * j + k) + 16 * m + 8 * e + r] & 3u) << (8 * e + 2 * (k & 3) + 16 * (k >> 2));
      *reinterpret_cast<uint32_t*>(img + kI3VCodes + 8 * X + 4 * h) = w;
    } else {
#pragma unroll
      for (int wd = 0; wd < 4; ++wd) {
        const int m = 2 * mh + (wd >> 1), e = wd & 1;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          w |= ((uint32_t)vcodes[kHeadDim * (8 * j + k) + 16 * m + 8 * e + r] >> 2) << (4 * wd + (k & 3) + 16 * (k >> 2));
      }
      *reinterpret_cast<uint32_t*>(img + kI3VHigh + 4 * X) = w;
    }
  }
}

// One CTA per (job, kv head) of INT3 tail pages, a warp per token; a new page
// is built in shared memory from zeros and written whole, a page that
// already holds tokens gets its new slots in place (V bits by atomic OR).
// Table entry and length as in append_int4_kernel.
template <bool kRope>
__global__ void __launch_bounds__(kThreads) append_int3_kernel(
    uint8_t* __restrict__ pool, size_t int3_off, int64_t n3b, int hkv, const __nv_bfloat16* __restrict__ k,
    const __nv_bfloat16* __restrict__ v, const AppendJob* __restrict__ jobs, const int32_t* __restrict__ toks,
    Entry* __restrict__ table, int32_t* __restrict__ ntab, uint32_t* __restrict__ status,
    const __grid_constant__ RopeParam<kRope> rope) {
  __shared__ __align__(16) uint8_t img[kInt3Block];
  __shared__ __align__(16) uint8_t vcodes[kPage * kHeadDim];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const AppendJob job = jobs[blockIdx.x];
  const int h = blockIdx.y;
  uint8_t* blk = pool + int3_off + ((size_t)(job.page - n3b) * hkv + h) * kInt3Block;
  const bool fresh = job.first_slot == 0;
  uint8_t* dst = fresh ? img : blk;
  if (fresh) {
    for (int i = threadIdx.x; i < kInt3Block / 16; i += kThreads) reinterpret_cast<uint4*>(img)[i] = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < kPage * kHeadDim / 16; i += kThreads)
      reinterpret_cast<uint4*>(vcodes)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  const int warp = threadIdx.x >> 5;
  const int32_t* tk = toks + job.tok_off;
  bool bad = false;
  float vmax = 0.0f;
  for (int q = warp; q < job.n_slots; q += kThreads / 32)
    bad |= quantize_rows3(dst, turned<kRope>(rope, load_rows<kRope>(rope, k, v, tk[q], h, hkv, bad)), job.first_slot + q,
                         vmax, fresh ? vcodes : nullptr);
  if (fresh) {
    __syncthreads();
    pack_i3v(img, vcodes);
    __syncthreads();
    for (int i = threadIdx.x; i < kInt3Block / 16; i += kThreads)
      reinterpret_cast<uint4*>(blk)[i] = reinterpret_cast<const uint4*>(img)[i];
  }
  flush_vmax(vmax, status);
  if (bad) atomicOr(status, kStatusRange);
  if (h == 0 && threadIdx.x == 0) {
    if (job.tab_index >= 0) table[job.tab_index] = Entry{job.page, job.live};
    if (job.ntab_req >= 0) ntab[job.ntab_req] = job.ntab_len;
  }
}

// ---- FP4 pages (TriAxialKV, limitations and outlook: non-uniform FP
// formats; HyQuant background: s = max|X| / c_B with c_B = 6 for E2M1):
// per token and 32-channel group s = half_rn(max|x| / 6), code = the E2M1
// value nearest to x / s (IEEE fp32 quotient), ties to the even mantissa,
// saturating at 6, zero coded +0; s = 0 codes everything 0.  The midpoints of
// the E2M1 grid are exact in fp32, so comparisons decide the rounding.
__device__ __forceinline__ uint32_t e2m1_code(float x, float sf, bool nz) {
  if (!nz) return 0u;
  const float u = __fdiv_rn(x, sf);
  const float a = fabsf(u);
  const uint32_t m = a <= 0.25f ? 0u : a < 0.75f ? 1u : a <= 1.25f ? 2u : a < 1.75f ? 3u
                   : a <= 2.5f  ? 4u : a < 3.5f  ? 5u : a <= 5.0f  ? 6u : 7u;
  return m == 0u ? 0u : ((u < 0.0f ? 8u : 0u) | m);
}

// A warp quantizes one token of one kv head (lane = channels 4*lane ..
// 4*lane+3).  K: a lane's four codes are the low (lane even) or high (lane
// odd) nibbles of one word; the even lane writes the word with its
// neighbour's nibbles.  V as in quantize_rows3.
__device__ __forceinline__ bool quantize_rows_fp4(uint8_t* img, const RawRows& rr, int slot, float& vmax,
                                                  uint8_t* vcodes) {
  const int lane = threadIdx.x & 31, gr = lane >> 3;
  const uint2 kr = rr.kr, vr = rr.vr;
  float xk[4], xv[4];
  xk[0] = __uint_as_float(kr.x << 16); xk[1] = __uint_as_float(kr.x & 0xFFFF0000u);
  xk[2] = __uint_as_float(kr.y << 16); xk[3] = __uint_as_float(kr.y & 0xFFFF0000u);
  xv[0] = __uint_as_float(vr.x << 16); xv[1] = __uint_as_float(vr.x & 0xFFFF0000u);
  xv[2] = __uint_as_float(vr.y << 16); xv[3] = __uint_as_float(vr.y & 0xFFFF0000u);
  bool bad = false;
  float kmn = xk[0], kmx = xk[0], vmn = xv[0], vmx = xv[0];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    bad |= out_of_range(xk[a]) | out_of_range(xv[a]);
    kmn = fminf(kmn, xk[a]); kmx = fmaxf(kmx, xk[a]);
    vmn = fminf(vmn, xv[a]); vmx = fmaxf(vmx, xv[a]);
  }
  group8_minmax(kmn, kmx);
  group8_minmax(vmn, vmx);
  const __half ks = __float2half_rn(__fdiv_rn(fmaxf(-kmn, kmx), 6.0f));
  const __half vs = __float2half_rn(__fdiv_rn(fmaxf(-vmn, vmx), 6.0f));
  const float ksf = __half2float(ks), vsf = __half2float(vs);
  const bool knz = (__half_as_ushort(ks) & 0x7FFFu) != 0, vnz = (__half_as_ushort(vs) & 0x7FFFu) != 0;
  uint32_t ck[4], cv[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    ck[a] = e2m1_code(xk[a], ksf, knz);
    cv[a] = e2m1_code(xv[a], vsf, vnz);
  }
  const int c0 = 4 * lane;
  const uint32_t kw = ck[0] | (ck[1] << 8) | (ck[2] << 16) | (ck[3] << 24);
  const uint32_t kw_odd = __shfl_xor_sync(0xFFFFFFFFu, kw, 1);
  if ((lane & 1) == 0) *reinterpret_cast<uint32_t*>(img + f4k_byte(slot, c0)) = kw | (kw_odd << 4);
  if (vcodes) {
    *reinterpret_cast<uint32_t*>(vcodes + kHeadDim * slot + c0) = cv[0] | (cv[1] << 8) | (cv[2] << 16) | (cv[3] << 24);
  } else {
#pragma unroll
    for (int a = 0; a < 4; ++a) or_bits(img, f4v_byte(slot, c0 + a), f4v_shift(slot), cv[a]);
  }
  vmax = fmaxf(vmax, vsf);
  if ((lane & 7) == 0) {
    st_half(img, kF4KScale + 8 * slot + 2 * gr, ks);
    st_half(img, kF4VScale + 2 * v_meta_index(slot, gr), vs);
  }
  return bad;
}

// FP4 V words from [slot][channel] code bytes, each word by one thread.
__device__ __forceinline__ void pack_f4v(uint8_t* __restrict__ img, const uint8_t* __restrict__ vcodes) {
  for (int x = threadIdx.x; x < 512; x += kThreads) {
    const int X = x >> 2, w = x & 3;
    const int m = 2 * (X >> 5) + (w >> 1), e = w & 1, r = (X >> 2) & 7, j = X & 3;
    const int c = 16 * m + 8 * e + r;
    uint32_t v = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) v |= (uint32_t)vcodes[kHeadDim * (8 * j + k) + c] << (8 * (k & 3) + 4 * (k >> 2));
    *reinterpret_cast<uint32_t*>(img + kF4VCodes + 16 * X + 4 * w) = v;
  }
}

// One CTA per (job, kv head) of FP4 tail pages, a warp per token (as
// append_int3_kernel).
template <bool kRope>
__global__ void __launch_bounds__(kThreads) append_fp4_kernel(
    uint8_t* __restrict__ pool, size_t fp4_off, int64_t nfb, int hkv, const __nv_bfloat16* __restrict__ k,
    const __nv_bfloat16* __restrict__ v, const AppendJob* __restrict__ jobs, const int32_t* __restrict__ toks,
    Entry* __restrict__ table, int32_t* __restrict__ ntab, uint32_t* __restrict__ status,
    const __grid_constant__ RopeParam<kRope> rope) {
  __shared__ __align__(16) uint8_t img[kFp4Block];
  __shared__ __align__(16) uint8_t vcodes[kPage * kHeadDim];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const AppendJob job = jobs[blockIdx.x];
  const int h = blockIdx.y;
  uint8_t* blk = pool + fp4_off + ((size_t)(job.page - nfb) * hkv + h) * kFp4Block;
  const bool fresh = job.first_slot == 0;
  uint8_t* dst = fresh ? img : blk;
  if (fresh) {
    for (int i = threadIdx.x; i < kFp4Block / 16; i += kThreads) reinterpret_cast<uint4*>(img)[i] = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < kPage * kHeadDim / 16; i += kThreads)
      reinterpret_cast<uint4*>(vcodes)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  const int warp = threadIdx.x >> 5;
  const int32_t* tk = toks + job.tok_off;
  bool bad = false;
  float vmax = 0.0f;
  for (int q = warp; q < job.n_slots; q += kThreads / 32)
    bad |= quantize_rows_fp4(dst, turned<kRope>(rope, load_rows<kRope>(rope, k, v, tk[q], h, hkv, bad)), job.first_slot + q,
                            vmax, fresh ? vcodes : nullptr);
  if (fresh) {
    __syncthreads();
    pack_f4v(img, vcodes);
    __syncthreads();
    for (int i = threadIdx.x; i < kFp4Block / 16; i += kThreads)
      reinterpret_cast<uint4*>(blk)[i] = reinterpret_cast<const uint4*>(img)[i];
  }
  flush_vmax(vmax, status);
  if (bad) atomicOr(status, kStatusRange);
  if (h == 0 && threadIdx.x == 0) {
    if (job.tab_index >= 0) table[job.tab_index] = Entry{job.page, job.live};
    if (job.ntab_req >= 0) ntab[job.ntab_req] = job.ntab_len;
  }
}

// Requantize a 32-token INT4 block image (shared memory) into an INT2 block
// image (shared memory): K per channel across the 32 tokens, V per token and
// group, both from the INT4-dequantized values fmaf(code, scale, zero); tracks
// the largest INT2 K and V scales.  The codes go through `codes` ([slot]
// [channel] bytes, shared memory) and are packed so that every output byte is
// written by one thread.  128 threads.
__device__ __forceinline__ void repack_image(const uint8_t* __restrict__ src, uint8_t* __restrict__ dst,
                                             uint32_t* __restrict__ smax_bits, uint8_t* __restrict__ codes) {
  // K: thread c owns channel c; its group is the 32 tokens of the page.
  {
    const int c = threadIdx.x;
    const int gr = c >> 5;
    float x[kPage];
    float mn, mx;
#pragma unroll
    for (int t = 0; t < kPage; ++t) {
      const uint32_t code = (src[i4k_byte(t, c)] >> i4k_shift(c)) & 15u;
      const float sf = __half2float(*reinterpret_cast<const __half*>(src + kI4KMeta + 16 * t + 4 * gr));
      const float zf = __half2float(*reinterpret_cast<const __half*>(src + kI4KMeta + 16 * t + 4 * gr + 2));
      x[t] = __fmaf_rn((float)code, sf, zf);
      mn = t ? fminf(mn, x[t]) : x[t];
      mx = t ? fmaxf(mx, x[t]) : x[t];
    }
    const GroupMeta m = make_meta(mn, mx, 3.0f);
    const float rs = approx_rcp(m.sf);
#pragma unroll
    for (int t = 0; t < kPage; ++t) codes[kHeadDim * t + c] = (uint8_t)qcode_fast(x[t], m, rs, 3.0f);
    st_half(dst, kI2KMeta + 2 * i2k_meta_index(c), m.s);
    st_half(dst, kI2KMeta + 256 + 2 * i2k_meta_index(c), m.z);
    // running maximum of INT2 K scales (non-negative floats order as their bits)
    float smx = m.sf;
#pragma unroll
    for (int o = 16; o; o >>= 1) smx = fmaxf(smx, __shfl_xor_sync(0xFFFFFFFFu, smx, o));
    if ((threadIdx.x & 31) == 0) atomicMax(smax_bits, __float_as_uint(smx));
  }
  __syncthreads();
  // K codes: byte (slot t, b) holds channels 4b .. 4b+3
  for (int x = threadIdx.x; x < kPage * (kHeadDim / 4); x += kThreads) {
    const int t = x >> 5, b = x & 31;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + kHeadDim * t + 4 * b);
    dst[i2k_byte(t, 4 * b)] = (uint8_t)((w & 3u) | ((w >> 6) & 0xCu) | ((w >> 12) & 0x30u) | ((w >> 18) & 0xC0u));
  }
  __syncthreads();
  // V: thread -> (slot t, group gr), 32 channels each.
  {
    const int t = threadIdx.x >> 2, gr = threadIdx.x & 3;
    const int mi = v_meta_index(t, gr);
    const float sf = __half2float(*reinterpret_cast<const __half*>(src + kI4VMeta + 2 * mi));
    const float zf = __half2float(*reinterpret_cast<const __half*>(src + kI4VMeta + 256 + 2 * mi));
    float x[kGroup];
    float mn, mx;
#pragma unroll
    for (int cc = 0; cc < kGroup; ++cc) {
      const int c = kGroup * gr + cc;
      const uint32_t code = (src[i4v_byte(t, c)] >> i4v_shift(t)) & 15u;
      x[cc] = __fmaf_rn((float)code, sf, zf);
      mn = cc ? fminf(mn, x[cc]) : x[cc];
      mx = cc ? fmaxf(mx, x[cc]) : x[cc];
    }
    const GroupMeta m = make_meta(mn, mx, 3.0f);
    const float rs = approx_rcp(m.sf);
#pragma unroll
    for (int cc = 0; cc < kGroup; ++cc) codes[kHeadDim * t + kGroup * gr + cc] = (uint8_t)qcode_fast(x[cc], m, rs, 3.0f);
    st_half(dst, kI2VMeta + 2 * mi, m.s);
    st_half(dst, kI2VMeta + 256 + 2 * mi, m.z);
    float vmx = m.sf;
#pragma unroll
    for (int o = 16; o; o >>= 1) vmx = fmaxf(vmx, __shfl_xor_sync(0xFFFFFFFFu, vmx, o));
    if ((threadIdx.x & 31) == 0) atomicMax(smax_bits + 1, __float_as_uint(vmx));
  }
  __syncthreads();
  // V codes: the 8 slots of chunk i of channel c fill two bytes (4 slots each)
  for (int x = threadIdx.x; x < kHeadDim * (kPage / 8); x += kThreads) {
    const int c = x & (kHeadDim - 1), i = x >> 7;
    const int b0 = i2v_byte(8 * i, c);
    int b1 = b0;
    uint32_t v0 = 0u, v1 = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int t = 8 * i + k, b = i2v_byte(t, c);
      const uint32_t code = (uint32_t)codes[kHeadDim * t + c] << i2v_shift(t);
      if (b == b0) {
        v0 |= code;
      } else {
        v1 |= code;
        b1 = b;
      }
    }
    dst[b0] = (uint8_t)v0;
    dst[b1] = (uint8_t)v1;
  }
}

// One CTA per (repack job, kv head): INT4 staging block -> INT2 block.
__global__ void __launch_bounds__(kThreads) repack_int2_kernel(uint8_t* __restrict__ pool, size_t int4_off,
                                                              int64_t n2, int hkv,
                                                              const RepackJob* __restrict__ jobs,
                                                              uint32_t* __restrict__ smax_bits) {
  __shared__ __align__(16) uint8_t src[kInt4Block];
  __shared__ __align__(16) uint8_t dst[kInt2Block];
  __shared__ __align__(16) uint8_t codes[kPage * kHeadDim];
  const RepackJob job = jobs[blockIdx.x];
  const int h = blockIdx.y;
  const uint8_t* sblk = pool + int4_off + ((size_t)(job.src - n2) * hkv + h) * kInt4Block;
  uint8_t* dblk = pool + ((size_t)job.dst * hkv + h) * kInt2Block;
  for (int i = threadIdx.x; i < kInt4Block / 16; i += kThreads)
    reinterpret_cast<uint4*>(src)[i] = reinterpret_cast<const uint4*>(sblk)[i];
  for (int i = threadIdx.x; i < kInt2Block / 16; i += kThreads)
    reinterpret_cast<uint4*>(dst)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  repack_image(src, dst, smax_bits, codes);
  __syncthreads();
  for (int i = threadIdx.x; i < kInt2Block / 16; i += kThreads)
    reinterpret_cast<uint4*>(dblk)[i] = reinterpret_cast<const uint4*>(dst)[i];
}

// One CTA per (direct job, kv head): 32 tokens that fill a fresh staging page
// within one call.  The staging page's INT4 image is built in shared memory
// exactly as the append kernel builds a new page (a warp per token), then
// requantized to INT2 as the repack kernel does; only the INT2 block is
// written to memory.  Launched as a programmatic dependent of the append
// kernel, which signals after its own wait: the earlier work on the stream
// (the previous decode, the uploads) is complete when this grid starts, and
// it touches nothing the append kernel writes, so the two run side by side.
// Every thread waits for the append grid before it exits, so the kernels
// that follow in stream order (the repack reads staging pages the append
// kernel fills) see both.
template <bool kRope>
__global__ void __launch_bounds__(kThreads) direct_int2_kernel(
    uint8_t* __restrict__ pool, int hkv, const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
    const DirectJob* __restrict__ jobs, const int32_t* __restrict__ toks, uint32_t* __restrict__ status,
    int32_t* __restrict__ pos, const __grid_constant__ RopeParam<kRope> rope) {
  __shared__ __align__(16) uint8_t img[kInt4Block];
  __shared__ __align__(16) uint8_t dst[kInt2Block];
  __shared__ __align__(16) uint8_t codes[kPage * kHeadDim];
  const DirectJob job = jobs[blockIdx.x];
  const int h = blockIdx.y;
  bool bad = false;
  float vmax = 0.0f;
  if (pos && h == 0 && job.pos0 != kNoPos) write_positions(pos, job.dst, nullptr, toks + job.tok_off, job.pos0, 0, kPage);
  // every slot is written: no zeroing
  bad |= quantize_tokens<kThreads / 32, kRope>(rope, img, k, v, toks + job.tok_off, kPage, 0, h, hkv, vmax, codes);
  flush_vmax(vmax, status);
  if (bad) atomicOr(status, kStatusRange);
  __syncthreads();
  pack_i4v(img, codes);
  __syncthreads();
  repack_image(img, dst, status + 1, codes);
  __syncthreads();
  uint8_t* dblk = pool + ((size_t)job.dst * hkv + h) * kInt2Block;
  for (int i = threadIdx.x; i < kInt2Block / 16; i += kThreads)
    reinterpret_cast<uint4*>(dblk)[i] = reinterpret_cast<const uint4*>(dst)[i];
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---- bulk kernels: a CTA of 4 warps per (page, kv head), warp gr = the
// 32-channel group gr, lane t = slot t.  The page's K and V rows come to shared
// memory first (V while K is worked on; K rotated on the way where the call asks
// for it), and a lane reads its token's 32 channels of the group from there, 8 at a
// time.  A token's group is quantized without any cross-lane step; INT4 metadata
// comes from packed bf16 min / max, per-channel INT2 K statistics from warp
// reductions across the 32 tokens.  The results are those of make_meta and
// qcode_fast, bit for bit.
//
// What bounds them: nothing alone.  65K tokens x 8 kv heads as they are: INT4 pages 97
// us, INT2 171, issue active 72 and 70 % of the cycles; rotated 135 and 185, at 59 and
// 70 %.  The first stalls are waits for memory (per issue 2.0 and 2.6, rotated 4.7 and
// 2.6: job, token, position, table row and K row are loads that depend on one another
// at the start of every CTA, and nothing of a next page is in flight), then the barrier
// after the rotation (2.0).  In mixed calls, half and 0.6 of the tokens INT2: 65K of
// each width 136 and 194 us; 106K and 156K, rotated, 215 and 427.  Rows through
// registers and a step per value took 145 and 277, rotated 222 and 670; rows fetched
// by the lane that reads them, half sectors, 155 and 210.  A page's heads side by
// side in the grid change nothing.  The loops over the 8-channel pieces are kept
// as loops and the rare exact divisions out of line: with everything unrolled the
// INT2 kernel was 105 KB of code, and a third of its stalls were waits for
// instructions.
constexpr int kBulkThreads = 128;
constexpr float kRound = 12582912.0f;    // 1.5 * 2^23: x + kRound - kRound is x rounded to an integer, ties to even

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf2_min(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf2_max(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float redux_min(float x) {
  float d;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ float redux_max(float x) {
  float d;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(x));
  return d;
}

struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("{.reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("{.reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("{.reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// Codes of two values, negated (the steps then need no sign changes): with f = 1 / (QMAX s), approximately,
//     q = sat((x - z) f),   code = rint(QMAX q),
// so the clamp to [0, QMAX] costs nothing.  negz = -z, f = 0 where the scale is 0: code 0.  f is off by
// less than 2^-21.2 of itself and QMAX q by less than 1e-5 from the exact quotient's value; far: the
// largest distance of QMAX q from its integer so far.  Past kTie the exact quotient could round the
// other way, and the caller takes the 8 codes again, divided.
constexpr float kTie = 0.49999f;
__device__ __forceinline__ float mul_sat(float a, float b) {
  float d;
  asm("mul.rn.sat.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
template <int QMAX>
__device__ __forceinline__ F2 codes2(F2 x, F2 negz, F2 f, float& far) {
  constexpr float Q = (float)QMAX;
  const F2 u = add2(x, negz);
  const F2 q{mul_sat(u.x, f.x), mul_sat(u.y, f.y)};
  const F2 c = add2(fma2(q, F2{-Q, -Q}, F2{-kRound, -kRound}), F2{kRound, kRound});
  const F2 d = fma2(q, F2{Q, Q}, c);
  far = fmaxf(fmaxf(far, fabsf(d.x)), fabsf(d.y));
  return c;
}
__device__ __forceinline__ float code_divided(float x, float z, float s, float qmax) {
  return s == 0.0f ? 0.0f : fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x, z), s)), 0.0f), qmax);
}
// 8 codes, divided: of bf16 values, and (INT2 K) of the INT4 values of a code word, channel by channel
__device__ __noinline__ uint32_t divided_nib8(uint4 v, float z, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t d = 0u;
#pragma unroll 1
  for (int n = 0; n < 4; ++n) {
    const uint32_t x = n == 0 ? w[0] : (n == 1 ? w[1] : (n == 2 ? w[2] : w[3]));
    d |= (uint32_t)code_divided(bf_lo(x), z, s, 15.0f) << (8 * n);
    d |= (uint32_t)code_divided(bf_hi(x), z, s, 15.0f) << (8 * n + 4);
  }
  return d;
}
__device__ __noinline__ uint32_t divided_crumb8(uint32_t cw, float s4, float z4, const float* z, const float* s) {
  uint32_t d = 0u;
#pragma unroll 1
  for (int n = 0; n < 8; ++n)
    d |= (uint32_t)code_divided(__fmaf_rn((float)((cw >> (4 * n)) & 15u), s4, z4), z[n], s[n], 3.0f) << (2 * n);
  return d;
}
__device__ __noinline__ float divided_one(float x, float z, float s, float qmax) { return code_divided(x, z, s, qmax); }

// A page's 32 K rows, rotated, in shared memory (rows 272 bytes apart, so that the
// reads of a group by 32 lanes hit distinct banks).  The channels that a rotation
// pairs lie in two groups, so the rows are rotated before a lane takes its token's
// group: an item of a row (8 pairs) per thread at a time, loads by whole rows.
struct RopeTile {
  uint4 row[kPage][17];
};
__device__ __forceinline__ void rotate_page(RopeTile& K, const RopeArgs& R, const __nv_bfloat16* __restrict__ k,
                                            const int32_t* __restrict__ toks, int h, bool& bad) {
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int t = (int)(threadIdx.x >> 3) + 16 * y, i = threadIdx.x & 7;
    const int T = __ldg(toks + t);
    const uint4* p = reinterpret_cast<const uint4*>(k + (size_t)T * (size_t)R.k_stride + (size_t)h * kHeadDim);
    int a, b;
    rope_item(R, i, a, b);
    uint4 x = __ldg(p + a), z = __ldg(p + b);
    if (8 * i < R.half) {
      float c[8], s[8];
      rope_factors<8>(R, T, 8 * i, c, s, bad);
      rope_turn(R, x, z, c, s);
    }
    K.row[t][a] = x;
    K.row[t][b] = z;
  }
}
// The warp's group of K or V as it is, asynchronously: 4 lanes take a token's 64 bytes, whole sectors, so that
// the warp that reads them fetches them and needs no CTA-wide barrier.  T: token of slot t, this lane.
__device__ __forceinline__ void fetch_group(RopeTile& X, const __nv_bfloat16* __restrict__ src, int T, int t, int h, size_t step,
                                            int gr) {
  const __nv_bfloat16* p = src + (size_t)h * kHeadDim + 32 * gr + 8 * (t & 3);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int y = 8 * q + (t >> 2);
    const int Ty = __shfl_sync(0xFFFFFFFFu, T, y);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(&X.row[y][4 * gr + (t & 3)])), "l"(p + (size_t)Ty * step) : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// The rows of a page: K's in shared memory, V's on their way.
template <bool kRope>
__device__ __forceinline__ void start_page(RopeTile& K, RopeTile& V, const RopeParam<kRope>& R,
                                           const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                                           const int32_t* __restrict__ toks, int T, int t, int h, int hkv, int gr, bool& bad) {
  if constexpr (!kRope) fetch_group(K, k, T, t, h, k_step<kRope>(R, hkv), gr);
  fetch_group(V, v, T, t, h, v_step<kRope>(R, hkv), gr);
  if constexpr (kRope) {
    rotate_page(K, R, k, toks, h, bad);
    __syncthreads();
  } else {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
  }
}
__device__ __forceinline__ void v_ready() {
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
}

// Metadata of a token's group at row (4 pieces of 8 bf16 channels): min / max exactly, NaN
// carried so that the range check sees it (NaN, Inf or |x| > 65504 sets `bad`).
__device__ __forceinline__ GroupMeta meta_i4(const uint4* row, bool& bad, float& mn, float& mx) {
  uint32_t lo = 0u, hi = 0u;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 v = row[q];
    const uint32_t a = bf2_min(bf2_min(v.x, v.y), bf2_min(v.z, v.w)), b = bf2_max(bf2_max(v.x, v.y), bf2_max(v.z, v.w));
    lo = q ? bf2_min(lo, a) : a;
    hi = q ? bf2_max(hi, b) : b;
  }
  const float a = bf_lo(lo), b = bf_hi(lo), c = bf_lo(hi), d = bf_hi(hi);
  bad |= out_of_range(a) | out_of_range(b) | out_of_range(c) | out_of_range(d);
  mn = fminf(a, b);
  mx = fmaxf(c, d);
  return make_meta(mn, mx, 15.0f);
}
template <int QMAX>
__device__ __forceinline__ float factor_of(const GroupMeta& m) { return m.nz ? approx_rcp(m.sf) * (1.0f / QMAX) : 0.0f; }

// INT4 codes of 8 channels as nibbles; c: the codes as floats, negated, pairs (2 j, 2 j + 1).
__device__ __forceinline__ uint32_t quant_i4_8(uint4 v, const GroupMeta& m, float f, F2 (&c)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float far = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = codes2<15>(F2{bf_lo(w[j]), bf_hi(w[j])}, F2{-m.zf, -m.zf}, F2{f, f}, far);
  if (far > kTie) {
    const uint32_t d = divided_nib8(v, m.zf, m.sf);
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = F2{-(float)((d >> (8 * j)) & 15u), -(float)((d >> (8 * j + 4)) & 15u)};
  }
  // exact: integers below 2^16, read off after adding 2^23
  const F2 a = fma2(c[1], F2{256.0f, 256.0f}, c[0]), b = fma2(c[3], F2{256.0f, 256.0f}, c[2]);
  const uint32_t l = __float_as_uint(8388608.0f - fmaf(a.y, 16.0f, a.x)), h = __float_as_uint(8388608.0f - fmaf(b.y, 16.0f, b.x));
  return __byte_perm(l, h, 0x5410u);
}
// 8 codes 0..3, negated, pairs (2 j, 2 j + 1), as 2-bit fields
__device__ __forceinline__ uint32_t pack_crumb8(const F2 (&c)[4]) {
  F2 a = fma2(c[1], F2{16.0f, 16.0f}, c[0]);
  a = fma2(c[2], F2{256.0f, 256.0f}, a);
  a = fma2(c[3], F2{4096.0f, 4096.0f}, a);
  return __float_as_uint(8388608.0f - fmaf(a.y, 4.0f, a.x)) & 0xFFFFu;
}

// Transpose of an 8 x 8 matrix of nibbles held in 8 words (word k = row k,
// nibble n = column n): on return word n holds column n (nibble k = row k).
__device__ __forceinline__ void transpose_nib8x8(uint32_t (&r)[8]) {
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const uint32_t t = ((r[k] >> 4) ^ r[k + 1]) & 0x0F0F0F0Fu;
    r[k + 1] ^= t;
    r[k] ^= t << 4;
  }
#pragma unroll
  for (int k = 0; k < 8; k += 4)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t x = r[k + q], y = r[k + q + 2];
      r[k + q] = __byte_perm(x, y, 0x6240u);
      r[k + q + 2] = __byte_perm(x, y, 0x7351u);
    }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t x = r[q], y = r[q + 4];
    r[q] = __byte_perm(x, y, 0x5410u);
    r[q + 4] = __byte_perm(x, y, 0x7632u);
  }
}

// INT4 V codes of one group into the block image: word (channel, slot chunk j) gets
// slots 8j .. 8j + 7 in nibbles 0..7.  `wbuf`: 128 words of the warp's own shared
// memory, [o][slot] the codes of channels 32gr + 8o + n as nibbles.
__device__ __forceinline__ void store_i4v_group(uint8_t* img, int gr, const uint32_t* wbuf) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  if (lane < 16) {
    const int o = lane >> 2, j = lane & 3;
    const uint4 a = *reinterpret_cast<const uint4*>(wbuf + 32 * o + 8 * j);
    const uint4 b = *reinterpret_cast<const uint4*>(wbuf + 32 * o + 8 * j + 4);
    uint32_t r[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};   // row k = slot 8j + k
    transpose_nib8x8(r);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *reinterpret_cast<uint32_t*>(img + i4v_byte(8 * j, 32 * gr + 8 * o + k)) = r[k];
  }
  __syncwarp();
}

// Fresh INT4 pages filled with 32 tokens within one call.  Grid (jobs, kv heads).
template <bool kRope>
__global__ void __launch_bounds__(kBulkThreads, 8) bulk_int4_kernel(
    uint8_t* __restrict__ pool, size_t int4_off, int64_t n2, int hkv, const __nv_bfloat16* __restrict__ k,
    const __nv_bfloat16* __restrict__ v, const AppendJob* __restrict__ jobs, const int32_t* __restrict__ toks,
    Entry* __restrict__ table, int32_t* __restrict__ ntab, uint32_t* __restrict__ status,
    int32_t* __restrict__ pos, const int32_t* __restrict__ tok_pos, const __grid_constant__ RopeParam<kRope> rope) {
  __shared__ __align__(16) uint8_t img[kInt4Block];
  __shared__ __align__(16) uint32_t wbuf[4][128];
  __shared__ RopeTile kt, vt;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // token lists and earlier stream work are done
  asm volatile("griddepcontrol.launch_dependents;");
  const AppendJob job = jobs[blockIdx.x];
  const int h = blockIdx.y, gr = threadIdx.x >> 5, t = threadIdx.x & 31;
  const int T = toks[job.tok_off + t];
  bool bad = false;
  start_page<kRope>(kt, vt, rope, k, v, toks + job.tok_off, T, t, h, hkv, gr, bad);
  float vmax = 0.0f;
#pragma unroll 1
  for (int kv = 0; kv < 2; ++kv) {   // K, then V: the same code
    if (kv) v_ready();
    const uint4* row = &(kv ? vt : kt).row[t][4 * gr];
    float mn, mx;
    const GroupMeta m = meta_i4(row, bad, mn, mx);
    const float f = factor_of<15>(m);
    // K: words (i, gr), i = 0..3, hold channels 32gr + 8i + n of slot t in nibble n; V: to be transposed
    uint32_t* to = kv ? wbuf[gr] + t : reinterpret_cast<uint32_t*>(img + kI4KCodes + 64 * t + 4 * gr);
    const int by = kv ? 32 : 4;
#pragma unroll 2
    for (int q = 0; q < 4; ++q) {
      F2 c[4];
      to[by * q] = quant_i4_8(row[q], m, f, c);
    }
    if (!kv) {
      *reinterpret_cast<uint32_t*>(img + kI4KMeta + 16 * t + 4 * gr) =
          (uint32_t)__half_as_ushort(m.s) | ((uint32_t)__half_as_ushort(m.z) << 16);
    } else {
      store_i4v_group(img, gr, wbuf[gr]);
      st_half(img, kI4VMeta + 2 * v_meta_index(t, gr), m.s);
      st_half(img, kI4VMeta + 256 + 2 * v_meta_index(t, gr), m.z);
      vmax = m.sf;
    }
  }
  flush_vmax(vmax, status);
  if (__any_sync(0xFFFFFFFFu, bad) && t == 0) atomicOr(status, kStatusRange);
  if (pos && h == 0 && gr == 0) pos[(size_t)job.page * kPage + t] = tok_pos ? tok_pos[job.tok_off + t] : job.pos0 + T;
  __syncthreads();
  uint4* out4 = reinterpret_cast<uint4*>(pool + int4_off + ((size_t)(job.page - n2) * hkv + h) * kInt4Block);
  const uint4* img4 = reinterpret_cast<const uint4*>(img);
  for (int x = threadIdx.x; x < kInt4Block / 16; x += kBulkThreads) out4[x] = img4[x];
  if (h == 0 && threadIdx.x == 0) {
    if (job.tab_index >= 0) table[job.tab_index] = Entry{job.page, job.live};
    if (job.ntab_req >= 0) ntab[job.ntab_req] = job.ntab_len;
  }
}

// Direct INT2 groups: 32 tokens that fill a staging page within one call,
// quantized to INT4 (per token and group), dequantized with fmaf(code, scale,
// zero) and requantized to INT2: K per channel across the 32 tokens, V per
// token and group.  Only the INT2 block is written.  Grid (jobs, kv heads).
// Launched as a programmatic dependent of the INT4 kernels, as the
// warp-per-token direct kernel is (it touches nothing they write).
//
// V: both quantizations go by (token, group), so the INT2 code of a value is a
// function of its INT4 code alone, 16 entries per lane, looked up by byte permutes.
// The least and greatest INT4 value are those of the codes of the least and
// greatest channel, since every step is monotone.
template <bool kRope>
__global__ void __launch_bounds__(kBulkThreads, 8) bulk_int2_kernel(
    uint8_t* __restrict__ pool, int hkv, const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
    const DirectJob* __restrict__ jobs, const int32_t* __restrict__ toks, uint32_t* __restrict__ status,
    int32_t* __restrict__ pos, const __grid_constant__ RopeParam<kRope> rope) {
  __shared__ __align__(16) uint8_t img[kInt2Block];
  __shared__ RopeTile kt, vt;
  __shared__ uint32_t kcw[4][4][32];                     // INT4 K codes [group][8-channel piece][slot]
  __shared__ __align__(16) float kz[4][32], kr[4][32], ks[4][32];   // per channel of the warp's group: -zero, 1 / (3 scale), scale
  __shared__ uint32_t vbuf[4][2][33];                    // INT2 V codes [group][channels 0..15, 16..31][slot]
  const DirectJob job = jobs[blockIdx.x];
  const int h = blockIdx.y, gr = threadIdx.x >> 5, t = threadIdx.x & 31;
  const int T = toks[job.tok_off + t];
  bool bad = false;
  start_page<kRope>(kt, vt, rope, k, v, toks + job.tok_off, T, t, h, hkv, gr, bad);
  // ---- K: INT4 per token, dequantized, then INT2 per channel across the 32 slots
  {
    const uint4* row = &kt.row[t][4 * gr];
    float mn, mx;
    const GroupMeta m = meta_i4(row, bad, mn, mx);
    const float f = factor_of<15>(m);
    float my_mn = 0.0f, my_mx = 0.0f;   // channel t of the group: min / max over the 32 slots
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      F2 c[4];
      kcw[gr][q][t] = quant_i4_8(row[q], m, f, c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 y = fma2(c[j], F2{-m.sf, -m.sf}, F2{m.zf, m.zf});
        const float a0 = redux_min(y.x), b0 = redux_max(y.x), a1 = redux_min(y.y), b1 = redux_max(y.y);
        if (t == 8 * q + 2 * j) my_mn = a0, my_mx = b0;
        if (t == 8 * q + 2 * j + 1) my_mn = a1, my_mx = b1;
      }
    }
    const GroupMeta m2 = make_meta(my_mn, my_mx, 3.0f);
    kz[gr][t] = -m2.zf;
    kr[gr][t] = factor_of<3>(m2);
    ks[gr][t] = m2.sf;
    const int ch = 32 * gr + t;
    st_half(img, kI2KMeta + 2 * i2k_meta_index(ch), m2.s);
    st_half(img, kI2KMeta + 256 + 2 * i2k_meta_index(ch), m2.z);
    const float smx = redux_max(m2.sf);   // running maximum of INT2 K scales
    if (t == 0) atomicMax(status + 1, __float_as_uint(smx));
    __syncwarp();
    // slot t's codes, channel c with channel c's metadata: channel c at byte c >> 2, bits 2 (c & 3) of its row
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      const uint32_t cw = kcw[gr][q][t];
      F2 c2[4];
      float far = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // codes 2 j and 2 j + 1 times 16^(2 (j & 1)) and 16 times that, in the mantissa of 2^23 (exact)
        const uint32_t w = j < 2 ? cw : cw >> 16;
        const int p = 8 * (j & 1);
        const F2 c = add2(F2{__uint_as_float((w & (15u << p)) | 0x4B000000u), __uint_as_float((w & (240u << p)) | 0x4B000000u)},
                          F2{-8388608.0f, -8388608.0f});
        const F2 y = fma2(c, F2{m.sf * (1.0f / (1 << p)), m.sf * (1.0f / (16 << p))}, F2{m.zf, m.zf});
        const float2 z = *reinterpret_cast<const float2*>(&kz[gr][8 * q + 2 * j]), r = *reinterpret_cast<const float2*>(&kr[gr][8 * q + 2 * j]);
        c2[j] = codes2<3>(y, F2{z.x, z.y}, F2{r.x, r.y}, far);
      }
      uint32_t d = pack_crumb8(c2);
      if (far > kTie) {
        float z[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) z[n] = -kz[gr][8 * q + n];
        d = divided_crumb8(cw, m.sf, m.zf, z, &ks[gr][8 * q]);
      }
      *reinterpret_cast<uint16_t*>(img + kI2KCodes + 32 * t + 8 * gr + 2 * q) = (uint16_t)d;
    }
  }
  // ---- V: INT4 per token, then INT2 per token on the dequantized values
  v_ready();
  {
    const uint4* row = &vt.row[t][4 * gr];
    float mn, mx;
    const GroupMeta m = meta_i4(row, bad, mn, mx);
    const float f = factor_of<15>(m);
    flush_vmax(m.sf, status);   // the INT4 V scales count toward the pool's V-scale maximum too
    const float c_lo = divided_one(mn, m.zf, m.sf, 15.0f), c_hi = divided_one(mx, m.zf, m.sf, 15.0f);
    const GroupMeta m2 = make_meta(__fmaf_rn(c_lo, m.sf, m.zf), __fmaf_rn(c_hi, m.sf, m.zf), 3.0f);
    const float f2 = factor_of<3>(m2);
    st_half(img, kI2VMeta + 2 * v_meta_index(t, gr), m2.s);
    st_half(img, kI2VMeta + 256 + 2 * v_meta_index(t, gr), m2.z);
    const float vmx = redux_max(m2.sf);
    if (t == 0) atomicMax(status + 2, __float_as_uint(vmx));
    // the INT2 code of every INT4 code, a byte each
    uint32_t tab[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      float far = 0.0f;
      F2 c[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float n = (float)(4 * y + 2 * j);
        c[j] = codes2<3>(fma2(F2{n, n + 1.0f}, F2{m.sf, m.sf}, F2{m.zf, m.zf}), F2{-m2.zf, -m2.zf}, F2{f2, f2}, far);
      }
      if (far > kTie) {
#pragma unroll 1
        for (int n = 0; n < 4; ++n) {
          const float x = -divided_one(__fmaf_rn((float)(4 * y + n), m.sf, m.zf), m2.zf, m2.sf, 3.0f);
          if (n == 0) c[0].x = x;
          else if (n == 1) c[0].y = x;
          else if (n == 2) c[1].x = x;
          else c[1].y = x;
        }
      }
      // below 2^24: two bytes at a time
      const uint32_t l = __float_as_uint(8388608.0f - fmaf(c[0].y, 256.0f, c[0].x)), u = __float_as_uint(8388608.0f - fmaf(c[1].y, 256.0f, c[1].x));
      tab[y] = __byte_perm(l, u, 0x5410u);
    }
    uint32_t half[2] = {0u, 0u};   // channels 0..15 and 16..31 as 2-bit fields
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      F2 c[4];
      const uint32_t cw = quant_i4_8(row[q], m, f, c);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t sel = cw >> (16 * y);
        const uint32_t lo = __byte_perm(tab[0], tab[1], sel & 0x7777u), hi = __byte_perm(tab[2], tab[3], sel & 0x7777u);
        const uint32_t up = __byte_perm(0x0000FF00u, 0u, (sel >> 3) & 0x1111u);   // bytes whose code is 8 or more
        const uint32_t b = (lo & ~up) | (hi & up);
        // bytes of 2 bits -> the top byte of the product (no carries)
        half[q >> 1] |= ((b * 0x01041040u) >> 24) << (16 * (q & 1) + 8 * y);
      }
    }
    vbuf[gr][0][t] = half[0];
    vbuf[gr][1][t] = half[1];
  }
  __syncwarp();
  // INT2 V words: lane = (r, i); word (r, m, i) of m = 2 gr and 2 gr + 1 (channels 16 m + r and 16 m + r + 8, slots 8 i .. + 7)
  {
    const int r = t >> 2, i = t & 3;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      uint32_t p[2] = {0u, 0u};   // slots 0..3 and 4..7: channel r in the low half, r + 8 in the high one
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) p[kk >> 2] |= ((vbuf[gr][y][8 * i + kk] >> (2 * r)) & 0x00030003u) << (2 * (kk & 3));
      uint32_t w = __byte_perm(p[0], p[1], 0x6420u);
      const uint32_t x = (w ^ (w >> 16)) & 3u;   // channel r: slots 8 i and 8 i + 4 the other way round
      w ^= x | (x << 16);
      const int mm = 2 * gr + y;
      *reinterpret_cast<uint32_t*>(img + kI2VCodes + 16 * (32 * (mm >> 2) + 4 * r + i) + 4 * (mm & 3)) = w;
    }
  }
  if (__any_sync(0xFFFFFFFFu, bad) && t == 0) atomicOr(status, kStatusRange);
  if (pos && h == 0 && gr == 0 && job.pos0 != kNoPos) pos[(size_t)job.dst * kPage + t] = job.pos0 + T;
  __syncthreads();
  uint4* out4 = reinterpret_cast<uint4*>(pool + ((size_t)job.dst * hkv + h) * kInt2Block);
  const uint4* img4 = reinterpret_cast<const uint4*>(img);
  for (int x = threadIdx.x; x < kInt2Block / 16; x += kBulkThreads) out4[x] = img4[x];
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__global__ void scatter_kernel(Entry* __restrict__ table, int32_t* __restrict__ ntab, uint32_t* __restrict__ hdead,
                               int hkv, const TableUpd* __restrict__ upd, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const TableUpd u = upd[i];
  if (u.kind == 0) table[u.index] = Entry{u.a, u.b};
  else if (u.kind == 1) ntab[u.index] = u.a;
  else if (hdead) hdead[(size_t)u.index * hkv + u.a] = u.b;   // kind 2: per-head exclusion word
}

}  // namespace

// with(std::bool_constant<kRope>, RopeParam<kRope>): the form of the running append
template <class F>
static cudaError_t with_rope(const kv_pool* P, F&& with) {
  return P->rope ? with(std::true_type{}, *P->rope) : with(std::false_type{}, NoRope{});
}

cudaError_t launch_append(kv_pool* P, const void* k, const void* v, const AppendJob* d_jobs, int n_jobs,
                          const int32_t* d_toks, const SmallAppend* small, cudaStream_t s) {
  if (n_jobs <= 0) return cudaSuccess;
  dim3 grid((unsigned)n_jobs, (unsigned)P->cfg.num_kv_heads);
  ++P->launches;
  return with_rope(P, [&](auto is, const auto& rope) {
    constexpr bool kRope = decltype(is)::value;
    const AppendJob* no_jobs = nullptr;
    const int32_t* no_toks = nullptr;
    if (small)
      return launch_pdl(append_int4_kernel<true, kRope>, grid, dim3(kThreads), 0, s, P->d_pool, P->int4_offset,
                        P->cfg.n_int2_pages, P->cfg.num_kv_heads, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v,
                        no_jobs, no_toks, P->d_table, P->d_ntab, P->d_status, *small, P->job_pos, P->tok_pos, rope);
    static const SmallAppend none{};
    return launch_pdl(append_int4_kernel<false, kRope>, grid, dim3(kThreads), 0, s, P->d_pool, P->int4_offset,
                      P->cfg.n_int2_pages, P->cfg.num_kv_heads, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v,
                      d_jobs, d_toks, P->d_table, P->d_ntab, P->d_status, none, P->job_pos, P->tok_pos, rope);
  });
}

cudaError_t launch_append_int3(kv_pool* P, const void* k, const void* v, const AppendJob* d_jobs, int n_jobs,
                               const int32_t* d_toks, cudaStream_t s) {
  if (n_jobs <= 0) return cudaSuccess;
  ++P->launches;
  return with_rope(P, [&](auto is, const auto& rope) {
    return launch_pdl(append_int3_kernel<decltype(is)::value>, dim3((unsigned)n_jobs, (unsigned)P->cfg.num_kv_heads),
                      dim3(kThreads), 0, s, P->d_pool, P->int3_offset,
                      (int64_t)(P->cfg.n_int2_pages + P->cfg.n_int4_pages), P->cfg.num_kv_heads, (const __nv_bfloat16*)k,
                      (const __nv_bfloat16*)v, d_jobs, d_toks, P->d_table, P->d_ntab, P->d_status, rope);
  });
}

cudaError_t launch_append_fp4(kv_pool* P, const void* k, const void* v, const AppendJob* d_jobs, int n_jobs,
                              const int32_t* d_toks, cudaStream_t s) {
  if (n_jobs <= 0) return cudaSuccess;
  ++P->launches;
  return with_rope(P, [&](auto is, const auto& rope) {
    return launch_pdl(append_fp4_kernel<decltype(is)::value>, dim3((unsigned)n_jobs, (unsigned)P->cfg.num_kv_heads),
                      dim3(kThreads), 0, s, P->d_pool, P->fp4_offset,
                      (int64_t)(P->cfg.n_int2_pages + P->cfg.n_int4_pages + P->cfg.n_int3_pages), P->cfg.num_kv_heads,
                      (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, d_jobs, d_toks, P->d_table, P->d_ntab,
                      P->d_status, rope);
  });
}

cudaError_t launch_bulk_int4(kv_pool* P, const void* k, const void* v, const AppendJob* d_jobs, int n_jobs,
                             const int32_t* d_toks, cudaStream_t s) {
  if (n_jobs <= 0) return cudaSuccess;
  ++P->launches;
  return with_rope(P, [&](auto is, const auto& rope) {
    return launch_pdl(bulk_int4_kernel<decltype(is)::value>, dim3((unsigned)n_jobs, (unsigned)P->cfg.num_kv_heads),
                      dim3(kBulkThreads), 0, s, P->d_pool, P->int4_offset, P->cfg.n_int2_pages, P->cfg.num_kv_heads,
                      (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, d_jobs, d_toks, P->d_table, P->d_ntab,
                      P->d_status, P->job_pos, P->tok_pos, rope);
  });
}

cudaError_t launch_bulk_int2(kv_pool* P, const void* k, const void* v, const DirectJob* d_jobs, int n_jobs,
                             const int32_t* d_toks, cudaStream_t s) {
  if (n_jobs <= 0) return cudaSuccess;
  ++P->launches;
  return with_rope(P, [&](auto is, const auto& rope) {
    return launch_pdl(bulk_int2_kernel<decltype(is)::value>, dim3((unsigned)n_jobs, (unsigned)P->cfg.num_kv_heads),
                      dim3(kBulkThreads), 0, s, P->d_pool, P->cfg.num_kv_heads, (const __nv_bfloat16*)k,
                      (const __nv_bfloat16*)v, d_jobs, d_toks, P->d_status, P->job_pos, rope);
  });
}

cudaError_t launch_repack(kv_pool* P, const RepackJob* d_jobs, int n_jobs, cudaStream_t s) {
  if (n_jobs <= 0) return cudaSuccess;
  dim3 grid((unsigned)n_jobs, (unsigned)P->cfg.num_kv_heads);
  ++P->launches;
  repack_int2_kernel<<<grid, kThreads, 0, s>>>(P->d_pool, P->int4_offset, P->cfg.n_int2_pages,
                                               P->cfg.num_kv_heads, d_jobs, P->d_status + 1);
  return cudaGetLastError();
}

cudaError_t launch_direct_int2(kv_pool* P, const void* k, const void* v, const DirectJob* d_jobs, int n_jobs,
                               const int32_t* d_toks, cudaStream_t s) {
  if (n_jobs <= 0) return cudaSuccess;
  dim3 grid((unsigned)n_jobs, (unsigned)P->cfg.num_kv_heads);
  ++P->launches;
  return with_rope(P, [&](auto is, const auto& rope) {
    return launch_pdl(direct_int2_kernel<decltype(is)::value>, grid, dim3(kThreads), 0, s, P->d_pool,
                      P->cfg.num_kv_heads, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, d_jobs, d_toks,
                      P->d_status, P->job_pos, rope);
  });
}

cudaError_t launch_scatter(kv_pool* P, const TableUpd* d_upd, int n, cudaStream_t s) {
  if (n <= 0) return cudaSuccess;
  ++P->launches;
  scatter_kernel<<<(n + 255) / 256, 256, 0, s>>>(P->d_table, P->d_ntab, P->d_hdead, P->cfg.num_kv_heads, d_upd, n);
  return cudaGetLastError();
}

}  // namespace kvq
