// Rotary positions: what the host hands to the kernels that rotate, and the
// rotation itself.
//
// Frequency f (of half = rot_dim / 2) turns one pair of channels, (f, f + half) or
// (2 f, 2 f + 1), at the token's position on f's axis:
//     u = a cos - b sin,   v = b cos + a sin,
// each product and the sum rounded to fp32 (no fused multiply-add), then once to
// bf16.  The cosines and sines are the caller's table, so that any schedule of
// frequencies (scaled, interpolated) is the caller's to choose and a far position
// loses nothing to an angle in fp32; and the arithmetic has one order, so a key
// rotated on its way into a page is the key that kv_rotate returns, bit for bit.
#pragma once
#include <stdint.h>

namespace kvq {

constexpr int kMaxAxes = 4;

struct RopeArgs {
  const float* table;    // [rows][2 * half]: cosines, then sines
  const int32_t* pos;    // [n_axes][pos_stride]
  int64_t pos_stride;
  int32_t rows, half;
  int32_t pairs;         // 1: neighbouring channels
  int32_t n_axes;
  float minus0;          // -0: see rope_uv2
  uint32_t axis[4];      // axis of frequency f: 2 bits at 2 (f & 15) of word f >> 4
  int64_t k_stride, v_stride;   // appends: elements from a token's rows to the next token's
};

#ifdef __CUDACC__
// The table row of token t on an axis; a position outside the table is reported and takes row 0.
__device__ __forceinline__ int rope_row(const RopeArgs& R, int axis, int64_t t, bool& bad) {
  int p = __ldg(R.pos + (size_t)axis * R.pos_stride + t);
  if ((uint32_t)p >= (uint32_t)R.rows) {
    bad = true;
    p = 0;
  }
  return p;
}
// Cosines and sines of frequencies f0 .. f0 + N - 1 (f0 a multiple of N; N 4 or 8) of token t.
template <int N>
__device__ __forceinline__ void rope_factors(const RopeArgs& R, int64_t t, int f0, float (&c)[N], float (&s)[N], bool& bad) {
  if (R.n_axes == 1) {
    const float4* p = reinterpret_cast<const float4*>(R.table + (size_t)rope_row(R, 0, t, bad) * 2 * R.half + f0);
    const int to_sin = R.half >> 2;
#pragma unroll
    for (int y = 0; y < N / 4; ++y) {
      const float4 a = __ldg(p + y), b = __ldg(p + to_sin + y);
      c[4 * y] = a.x; c[4 * y + 1] = a.y; c[4 * y + 2] = a.z; c[4 * y + 3] = a.w;
      s[4 * y] = b.x; s[4 * y + 1] = b.y; s[4 * y + 2] = b.z; s[4 * y + 3] = b.w;
    }
  } else {
    int row[kMaxAxes];
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) row[a] = a < R.n_axes ? rope_row(R, a, t, bad) : 0;
    // the N axis fields are N adjacent 2-bit fields of one word
    const uint32_t ax = R.axis[f0 >> 4] >> (2 * (f0 & 15));
#pragma unroll
    for (int y = 0; y < N; ++y) {
      const uint32_t a = (ax >> (2 * y)) & 3u;
      const int r = a == 0u ? row[0] : (a == 1u ? row[1] : (a == 2u ? row[2] : row[3]));
      const float* p = R.table + (size_t)r * 2 * R.half + f0 + y;
      c[y] = __ldg(p);
      s[y] = __ldg(p + R.half);
    }
  }
}
__device__ __forceinline__ float rope_u(float a, float b, float c, float s) { return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)); }
__device__ __forceinline__ float rope_v(float a, float b, float c, float s) { return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)); }
__device__ __forceinline__ uint32_t rope_bf2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float rope_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float rope_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The same of two pairs at once: (u, v) = (a c - b s, b c + a s), each step rounded as above.  The products
// are multiply-adds of R.minus0, which the compiler does not know: it merges a packed product and a sum into
// one rounding, whatever their modifiers.
__device__ __forceinline__ void rope_uv2(const RopeArgs& R, float2 a, float2 b, float2 c, float2 s, float2& u, float2& v) {
  asm("{.reg .b64 a, b, c, s, n, x, y, o;\n mov.b64 a, {%4, %5};\n mov.b64 b, {%6, %7};\n mov.b64 c, {%8, %9};\n"
      " mov.b64 s, {%10, %11};\n mov.b64 n, {%12, %13};\n mov.b64 o, {%14, %14};\n"
      " fma.rn.f32x2 x, a, c, o;\n fma.rn.f32x2 y, b, n, o;\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n"
      " fma.rn.f32x2 x, b, c, o;\n fma.rn.f32x2 y, a, s, o;\n add.rn.f32x2 x, x, y;\n mov.b64 {%2, %3}, x;}"
      : "=f"(u.x), "=f"(u.y), "=f"(v.x), "=f"(v.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(s.x), "f"(s.y), "f"(-s.x), "f"(-s.y), "f"(R.minus0));
}

// A row of 128 channels is 16 chunks of 8; item i of a row takes two of them: for i < rot_dim / 16 those of
// frequencies 8 i .. 8 i + 7, else two that pass.
__device__ __forceinline__ void rope_item(const RopeArgs& R, int i, int& a, int& b) {
  const int h = R.half >> 3;
  a = R.pairs ? 2 * i : (i < h ? i : 2 * i);
  b = R.pairs ? a + 1 : (i < h ? i + h : 2 * i + 1);
}
// Rotates an item's chunks.
__device__ __forceinline__ void rope_turn(const RopeArgs& R, uint4& x, uint4& y, const float (&c)[8], const float (&s)[8]) {
  uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
  float2 u, v;
  if (!R.pairs) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      rope_uv2(R, make_float2(rope_lo(a[k]), rope_hi(a[k])), make_float2(rope_lo(b[k]), rope_hi(b[k])),
               make_float2(c[2 * k], c[2 * k + 1]), make_float2(s[2 * k], s[2 * k + 1]), u, v);
      a[k] = rope_bf2(u.x, u.y);
      b[k] = rope_bf2(v.x, v.y);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      rope_uv2(R, make_float2(rope_lo(a[k]), rope_lo(a[k + 1])), make_float2(rope_hi(a[k]), rope_hi(a[k + 1])),
               make_float2(c[k], c[k + 1]), make_float2(s[k], s[k + 1]), u, v);
      a[k] = rope_bf2(u.x, v.x);
      a[k + 1] = rope_bf2(u.y, v.y);
      rope_uv2(R, make_float2(rope_lo(b[k]), rope_lo(b[k + 1])), make_float2(rope_hi(b[k]), rope_hi(b[k + 1])),
               make_float2(c[4 + k], c[5 + k]), make_float2(s[4 + k], s[5 + k]), u, v);
      b[k] = rope_bf2(u.x, v.x);
      b[k + 1] = rope_bf2(u.y, v.y);
    }
  }
  x = make_uint4(a[0], a[1], a[2], a[3]);
  y = make_uint4(b[0], b[1], b[2], b[3]);
}

// The form for a warp per row, a lane holding channels 4 lane .. 4 lane + 3: the lane's factors
// (neighbouring channels: two of them), then the row, whose other halves of pairs come from
// lane +- half / 4.
struct RopeLane {
  float c[4], s[4];
};
__device__ __forceinline__ RopeLane rope_lane(const RopeArgs& R, int64_t t, bool& bad) {
  const int lane = threadIdx.x & 31;
  RopeLane L;
#pragma unroll
  for (int y = 0; y < 4; ++y) L.c[y] = L.s[y] = 0.0f;
  if (4 * lane >= 2 * R.half) return L;
  if (R.pairs) {
    rope_factors<4>(R, t, (2 * lane) & ~3, L.c, L.s, bad);
    if (lane & 1) {
      L.c[0] = L.c[2]; L.c[1] = L.c[3];
      L.s[0] = L.s[2]; L.s[1] = L.s[3];
    }
  } else {
    rope_factors<4>(R, t, 4 * lane < R.half ? 4 * lane : 4 * lane - R.half, L.c, L.s, bad);
  }
  return L;
}
__device__ __forceinline__ uint2 rope_lane_turn(const RopeArgs& R, uint2 x, const RopeLane& L) {
  const int lane = threadIdx.x & 31, q = R.half >> 2;
  const float a[4] = {rope_lo(x.x), rope_hi(x.x), rope_lo(x.y), rope_hi(x.y)};
  float r[4];
  if (R.pairs) {   // (uniform)
    r[0] = rope_u(a[0], a[1], L.c[0], L.s[0]);
    r[1] = rope_v(a[0], a[1], L.c[0], L.s[0]);
    r[2] = rope_u(a[2], a[3], L.c[1], L.s[1]);
    r[3] = rope_v(a[2], a[3], L.c[1], L.s[1]);
  } else {
    const int from = lane < q ? lane + q : (lane < 2 * q ? lane - q : lane);
    const uint32_t o0 = __shfl_sync(0xFFFFFFFFu, x.x, from), o1 = __shfl_sync(0xFFFFFFFFu, x.y, from);
    const float o[4] = {rope_lo(o0), rope_hi(o0), rope_lo(o1), rope_hi(o1)};
#pragma unroll
    for (int y = 0; y < 4; ++y)
      r[y] = lane < q ? rope_u(a[y], o[y], L.c[y], L.s[y]) : rope_v(o[y], a[y], L.c[y], L.s[y]);
  }
  return 4 * lane < 2 * R.half ? make_uint2(rope_bf2(r[0], r[1]), rope_bf2(r[2], r[3])) : x;
}
#endif

}  // namespace kvq
