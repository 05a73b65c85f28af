// kv_attend for many rows per unit (chunks of a prompt): the cache is
// dequantized once per call into operand tiles, then tcgen05 attention runs over
// the tiles.
//
// attend_tiles_kernel turns every 128 keys of a (request, kv head) unit (four
// pages, or bf16 rows of the list or of the new tokens) into one K and one V
// operand tile, 32 KB each, in the very layout that the MMAs read from shared
// memory (V transposed), and the keys' live bits into four words.  Every block of
// 256 rows reads the tiles again, most of them from L2 (the plan starts a unit's
// blocks together), so this costs one pass over the pages for any number of blocks.
// Dequantizing inside the attention kernel instead cost eight warps' issue slots per
// block: 2.72 ms for 2048 tokens of 64 heads over 32K, 1.77 ms so.
//
// attend_wide_kernel: a CTA takes an item: a block of up to 256 rows of a unit
// and a run of its tiles.  Per tile
//     S_x = Q_x K^T          (x = 0, 1: 128 rows each; 128 x 128 x 128)
//     P_x = 2^(S_x rf - m)   (rf: softmax scale, log2 e and the row's power of two)
//     O_x += P_x V           (P_x read from TMEM)
// with the running maximum m and sum of each row; O_x stays in TMEM over the
// item and is rescaled only when a row's maximum has grown by more than 2^8
// (the sums are fp32 and P is binary16 with 2^7 of headroom below 65504, so a
// stale maximum loses nothing).
//
// Roles: two warpgroups hold one row per thread of S_0 / S_1; one thread per x
// issues the MMAs of S_x and O_x; one thread streams tiles through a ring of
// five.  While one warpgroup works on its S, the tensor cores work for the other;
// two issuing threads, because the waits and commits between runs of MMAs cost one
// thread 600 of every 1650 cycles.  (Even and odd tiles of a last block of at most 128
// rows given to the two warpgroups took 3350 cycles per tile, as they are 3700.)
//
// What bounds it: 3700 cycles per tile of 256 rows, of which the tensor cores work
// 2048 (their operand reads of shared memory 1536, the exponentials 1024): a half's
// MMAs wait for its softmax (TMEM to registers, maximum, exponentials, back), about
// 2700 cycles, and the other half's fill only part of that; S, P and O of both halves
// are all of TMEM, and Q and five tiles all of shared memory.  An item costs 20,000
// cycles more.  2048 tokens of 64 q on 8 kv heads over 32K: 1.77 ms, 1.28 PFLOP/s.
// Slower: P V in two halves as P arrives (1.88 ms), 16 softmax warps (2.06 ms).
#include <algorithm>
#include <atomic>

#include "kvq_attend_mma.cuh"

namespace kvq {
namespace {

constexpr int kRing = 5;                        // K and V tiles in flight
constexpr int kWarps = 12;                      // the last one idle
constexpr int kThreads = 32 * kWarps;
constexpr int kTileBytes = 128 * 128 * 2;
constexpr float kHead = 7.0f;                   // P = 2^(x - m + 7)
constexpr float kGrow = 8.0f;                   // a maximum may be stale by this much (base 2)
constexpr float kNever = -3.0e38f;              // S of a key that is not seen
constexpr float kLowest = 0.9f * kNever;        // logits below it count as it

struct alignas(1024) WideSmem {
  uint8_t q[2][kTileBytes], kv[kRing][kTileBytes];
  uint64_t full[kRing], empty[kRing];
  uint64_t q_full, s_full[2], p_full[2], o_full, turn[2], drain[2];
  uint32_t tmem, gave_up;
};
static_assert(sizeof(WideSmem) <= 232448, "one CTA's shared memory");

struct Tiles {   // an item's tiles: [0, pages), [pages, lists), [lists, all) by kind
  int pages, lists, all, rows;
};
__device__ __forceinline__ Tiles tiles_of(const AttArgs& A, const AttUnit& u, int row0, int rows) {
  Tiles t;
  const int g = A.hq / A.hkv;
  t.rows = min(rows, u.T * g - row0);
  t.pages = (u.n_pages + 3) >> 2;
  t.lists = t.pages + ((u.n_fp + 127) >> 7);
  t.all = t.lists + (!A.k ? 0 : (((A.tree ? u.T - 1 : (row0 + t.rows - 1) / g) >> 7) + 1));
  return t;
}

// One CTA of eight warps per tile: the four page blocks go to shared memory in
// 16-byte pieces, then warp p dequantizes K of page (or 32 rows) p and warp 4 + p
// its V.  Bound by memory: 64 KB written per 12 to 20 KB read.
__global__ void __launch_bounds__(256) attend_tiles_kernel(AttArgs A, const AttUnit* __restrict__ units,
                                                           uint8_t* __restrict__ tiles, uint32_t* __restrict__ live) {
  __shared__ __align__(16) uint8_t raw[4][kInt4Block];
  const AttUnit u = units[blockIdx.y];
  const Tiles T = tiles_of(A, u, 0, 1 << 30);
  const int tile = blockIdx.x;
  if (tile >= T.all) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_k = warp < 4;
  const int p = warp & 3;
  uint8_t* const dst = tiles + ((size_t)(u.tile_base + tile) * 2 + (is_k ? 0 : 1)) * kTileBytes;
  uint32_t bad = 0u;
  const int rk = lane >> 2, rv = rk, i = lane & 3;   // slots r of runs i
  if (tile < T.pages) {
    const int pi = 4 * tile + p;
    Entry e{-1, 0u};
    int cls = -1;
    const uint8_t* blk = nullptr;
    if (pi < u.n_pages) {
      e = A.table[(size_t)u.req * A.max_pages + pi];
      if (A.hdead) e.live &= ~A.hdead[(size_t)e.id * A.hkv + u.kvh];
      if (e.live) cls = att_page(A, e.id, u.kvh, blk);
    }
    if (cls >= 0) {   // the two warps of a page copy half of it each
      const int n16 = (cls == kClsInt2 ? kInt2Block : (cls == kClsInt4 ? kInt4Block : (cls == kClsInt3 ? kInt3Block : kFp4Block))) / 16;
      uint4 w[5];
#pragma unroll
      for (int y = 0; y < 5; ++y) {
        const int c = 64 * y + 32 * (is_k ? 0 : 1) + lane;
        if (c < n16) w[y] = __ldcs(reinterpret_cast<const uint4*>(blk) + c);
      }
#pragma unroll
      for (int y = 0; y < 5; ++y) {
        const int c = 64 * y + 32 * (is_k ? 0 : 1) + lane;
        if (c < n16) reinterpret_cast<uint4*>(raw[p])[c] = w[y];
      }
      blk = raw[p];
    }
    __syncthreads();
    if (is_k && lane == 0) live[(size_t)(u.tile_base + tile) * 4 + p] = order_bits(e.live);
    {
          if (is_k) {
            if (cls == kClsInt2) {
#pragma unroll 1
              for (int gr = 0; gr < 4; ++gr) {
                uint32_t sc[4], z[4];
                k_scales2(blk, gr, i, sc, z);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                  uint32_t y[4];
                  k_run2(blk, 8 * b + rk, gr, i, sc, z, y);
                  *reinterpret_cast<uint4*>(dst + tile_off(128, 32 * p + 8 * b + order8(rk), 4 * gr + i)) =
                      make_uint4(y[0], y[1], y[2], y[3]);
                }
              }
            } else {
#pragma unroll 2
              for (int y = 0; y < 8; ++y) {
                const int t = 8 * (y >> 1) + rk, half = y & 1;
                uint32_t w[2][4];
                if (cls == kClsInt4) {
                  k_slot4(blk, t, i, half, w);
                } else if (cls == kClsInt3) {
                  k_slot3(blk, t, i, half, w);
                } else if (cls == kClsFp4) {
                  k_slotf(blk, t, i, half, w);
                } else {
#pragma unroll
                  for (int x = 0; x < 8; ++x) w[x >> 2][x & 3] = 0u;
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
                  *reinterpret_cast<uint4*>(dst + tile_off(128, 32 * p + (t & ~7) + order8(rk), 4 * (2 * half + x) + i)) =
                      make_uint4(w[x][0], w[x][1], w[x][2], w[x][3]);
              }
            }
          } else {
            auto put = [&](int gr, const uint32_t (&w)[4][4]) {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                *reinterpret_cast<uint4*>(dst + tile_off(128, 32 * gr + 8 * x + rv, 4 * p + i)) =
                    make_uint4(w[x][0], w[x][1], w[x][2], w[x][3]);
            };
            uint32_t w[4][4];
            if (cls == kClsInt2) {
#pragma unroll 1
              for (int gr = 0; gr < 4; ++gr) {
                v_group2(blk, gr, rv, i, w);
                put(gr, w);
              }
            } else if (cls == kClsInt4) {
#pragma unroll 1
              for (int gr = 0; gr < 4; ++gr) {
                v_group4(blk, gr, rv, i, w);
                put(gr, w);
              }
            } else {
#pragma unroll 1
              for (int gr = 0; gr < 4; ++gr) {
                if (cls == kClsInt3) {
                  v_group3(blk, gr, rv, i, w);
                } else if (cls == kClsFp4) {
                  v_groupf(blk, gr, rv, i, w);
                } else {
#pragma unroll
                  for (int x = 0; x < 16; ++x) w[x >> 2][x & 3] = 0u;
                }
                put(gr, w);
              }
            }
          }
    }
  } else {
    const bool kal = (((uintptr_t)A.k | (uintptr_t)A.v) & 15) == 0;
    const bool val = (((uintptr_t)A.k | (uintptr_t)A.v) & 3) == 0;
    {
          // ---- 32 bf16 rows: list tokens or new tokens
          const bool list = tile < T.lists;
          const int j0 = 128 * (tile - (list ? T.pages : T.lists)) + 32 * p;   // first row of this warp
          const int n = list ? u.n_fp : u.T;
          const size_t stride = list ? kHeadDim : (size_t)A.hkv * kHeadDim;
          const uint16_t* src =
              list ? (is_k ? A.fpk : A.fpv) + ((size_t)u.req * A.hkv + u.kvh) * (size_t)A.fp_cap * kHeadDim
                   : (is_k ? A.k : A.v) + ((size_t)u.tok0 * A.hkv + u.kvh) * kHeadDim;
          // rows past the end: the last row is loaded and used as 0 (loads without branches stay in flight together)
          if (is_k) {
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
              const int j = j0 + 8 * b + rk, jc = min(j, n - 1), nn = 32 * p + 8 * b + order8(rk);
              uint4 y[4];
#pragma unroll
              for (int gr = 0; gr < 4; ++gr) {
                const int ch = 4 * gr + i;
                y[gr] = load8(src + (size_t)jc * stride + 8 * (list ? ch ^ (jc & 7) : ch), list || kal);
              }
#pragma unroll
              for (int gr = 0; gr < 4; ++gr) {
                uint32_t w[4];
                if (j >= n) y[gr] = make_uint4(0u, 0u, 0u, 0u);
                order8_f16(y[gr], 1.0f, w, bad);
                *reinterpret_cast<uint4*>(dst + tile_off(128, nn, 4 * gr + i)) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          } else {
            // a lane takes channels (2 cp, 2 cp + 1) of 8 rows at a time
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
              uint32_t y[2][8];
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                  const int jc = min(j0 + 8 * b + s, n - 1), c = 2 * (lane + 32 * x);
                  const uint16_t* q = src + (size_t)jc * stride + (list ? att_list_at(jc, c) : c);
                  y[x][s] = list || val ? __ldg(reinterpret_cast<const uint32_t*>(q))
                                        : (uint32_t)__ldg(q) | ((uint32_t)__ldg(q + 1) << 16);
                }
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int c = 2 * (lane + 32 * x);
                float lo[8], hi[8];
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                  const uint32_t w = j0 + 8 * b + s < n ? y[x][s] : 0u;
                  lo[s] = in_range(bf_f(w & 0xFFFFu), bad);
                  hi[s] = in_range(__uint_as_float(w & 0xFFFF0000u), bad);
                }
                *reinterpret_cast<uint4*>(dst + tile_off(128, c, 4 * p + b)) =
                    make_uint4(f16x2(lo[0], lo[4]), f16x2(lo[1], lo[5]), f16x2(lo[2], lo[6]), f16x2(lo[3], lo[7]));
                *reinterpret_cast<uint4*>(dst + tile_off(128, c + 1, 4 * p + b)) =
                    make_uint4(f16x2(hi[0], hi[4]), f16x2(hi[1], hi[5]), f16x2(hi[2], hi[6]), f16x2(hi[3], hi[7]));
              }
            }
          }
    }
  }
  if (bad) atomicOr(A.status, kStatusRange);
}

__global__ void __launch_bounds__(kThreads, 1) attend_wide_kernel(
    AttArgs A, const AttUnit* __restrict__ units, const AttItem* __restrict__ items, const int32_t* __restrict__ cta_item,
    const uint8_t* __restrict__ tiles, const uint32_t* __restrict__ live, float* __restrict__ part,
    uint32_t first_spins) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  WideSmem& S = *reinterpret_cast<WideSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i0 = cta_item[blockIdx.x], i1 = cta_item[blockIdx.x + 1];
  volatile uint32_t* gave_up = &S.gave_up;
  if (tid == 0) {
    for (int x = 0; x < kRing; ++x) {
      mb_init(&S.full[x], 1);
      mb_init(&S.empty[x], 2);
    }
    for (int x = 0; x < 2; ++x) {
      mb_init(&S.s_full[x], 1);
      mb_init(&S.p_full[x], 4);
      mb_init(&S.drain[x], 1);
      mb_init(&S.turn[x], 1);
    }
    mb_init(&S.q_full, 8);
    mb_init(&S.o_full, 2);
    S.gave_up = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) tm_alloc(&S.tmem, 512);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tmem = S.tmem;
  const int g = A.hq / A.hkv;

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    const int x = warp >> 2;                               // S / P / O of this warpgroup
    const int rt = tid & 127;
    const uint32_t tl = tmem + ((uint32_t)(warp & 3) << 21);   // the warp's 32 TMEM lanes
    const uint32_t ts = tl + 128u * x, to = tl + 256u + 128u * x;
    uint32_t s_phase = 0, o_phase = 0, bad = 0u;
    bool ok = true;
    const bool qal = ((uintptr_t)A.q & 15) == 0, oal = ((uintptr_t)A.out & 15) == 0;
    const RowMap rows(g);
    for (int it = i0; it < i1 && ok; ++it) {
      const AttItem I = items[it];
      const AttUnit u = units[I.unit];
      const Tiles T = tiles_of(A, u, I.row0, 256);
      const int rl = 128 * x + rt;                         // row in the block
      const bool valid = rl < T.rows;
      const int t = rows.token(I.row0 + (valid ? rl : 0));
      // ---- Q: every row scaled by a power of two so that its largest element is in [2^7, 2^8).  A warp
      // loads its 32 rows two at a time (16 lanes each), 16 rows in flight.
      float rf = 0.0f;
      {
        const int c = lane & 15, half = lane >> 4, w32 = rl - lane;   // first row of the warp in the block
#pragma unroll 1
        for (int y0 = 0; y0 < 16; y0 += 8) {
          uint4 w[8];
#pragma unroll
          for (int y = 0; y < 8; ++y)
            w[y] = load8(A.q + rows.at(A, u, I.row0 + min(w32 + 2 * (y0 + y) + half, T.rows - 1)) + 8 * c, qal);
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const uint32_t wd[4] = {w[y].x, w[y].y, w[y].z, w[y].w};
            float f[8], mx = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              f[2 * k] = bf_f(wd[k] & 0xFFFFu);
              f[2 * k + 1] = __uint_as_float(wd[k] & 0xFFFF0000u);
              mx = fmaxf(fmaxf(mx, fabsf(f[2 * k])), fabsf(f[2 * k + 1]));
            }
#pragma unroll
            for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            const int e = q_exponent(mx);
            const float mul = q_factor(mx, e, A.scale_log2);
            // (a factor below 1e-30 makes every logit 0, as 1e-30 does; kNever times it must stay far below 0)
            const float rr = fmaxf(fabsf(A.scale_log2) * pow2f(-e), 1e-30f);
            const float mine = __shfl_sync(0xFFFFFFFFu, rr, (lane & 1) << 4);
            if ((lane >> 1) == y0 + y) rf = mine;   // the thread's own row
            *reinterpret_cast<uint4*>(S.q[x] + tile_off(128, (rt & ~31) + 2 * (y0 + y) + half, c)) =
                make_uint4(f16x2(f[0] * mul, f[4] * mul), f16x2(f[1] * mul, f[5] * mul), f16x2(f[2] * mul, f[6] * mul),
                           f16x2(f[3] * mul, f[7] * mul));
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tm_fence_before();   // the previous item's O has been read
      __syncwarp();
      if (lane == 0 && I.tile1 > I.tile0) mb_arrive(&S.q_full);   // an item without tiles has no MMAs
      const uint64_t tm = A.tree ? A.tree[u.tok0 + t] : 0ull;

      float m = -INFINITY, l = 0.0f;
      bool any = false;                                    // O_x has been written in this item
      for (int tile = I.tile0; tile < I.tile1; ++tile) {
        const bool page = tile < T.pages;
        // ---- keys this row sees, 128 bits in the tiles' order
        uint32_t mk[4];
        if (page) {
          const uint4 lv = __ldg(reinterpret_cast<const uint4*>(live) + u.tile_base + tile);   // before the wait below
          mk[0] = lv.x; mk[1] = lv.y; mk[2] = lv.z; mk[3] = lv.w;
        }
        ok = __all_sync(0xFFFFFFFFu, mb_wait(&S.s_full[x], s_phase, gave_up));
        if (!ok) break;
        s_phase ^= 1u;
        tm_fence_after();
        if (!page) {
          const bool list = tile < T.lists;
          const int base = 128 * (tile - (list ? T.pages : T.lists));
          // keys [base, base + n) are seen (with a tree, those of its bits)
          const int n = (list ? u.n_fp : (A.tree ? u.T : t + 1)) - base;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int nw = n - 32 * w;
            uint32_t b = nw >= 32 ? 0xFFFFFFFFu : (nw <= 0 ? 0u : (1u << nw) - 1u);
            if (!list && A.tree) b &= w == 0 ? (uint32_t)tm : (w == 1 ? (uint32_t)(tm >> 32) : 0u);
            mk[w] = order_bits(b);
          }
        }
        // ---- maximum
        uint32_t sv[128];
        tm_ld32_at<0>(sv, ts);
        tm_ld32_at<32>(sv, ts + 32u);
        tm_ld32_at<64>(sv, ts + 64u);
        tm_ld32_at<96>(sv, ts + 96u);
        tm_wait_ld();
        // keys that are not seen (2064 us for 2048 tokens over 32K with 5 % of the slots evicted when this
        // was written back to S before the loads, 1827 so)
        if (!__all_sync(0xFFFFFFFFu, (mk[0] & mk[1] & mk[2] & mk[3]) == 0xFFFFFFFFu)) {
#pragma unroll
          for (int j = 0; j < 128; ++j) sv[j] = (mk[j >> 5] >> (j & 31)) & 1u ? sv[j] : __float_as_uint(kNever);
        }
        float mq[4] = {kNever, kNever, kNever, kNever};
#pragma unroll
        for (int j = 0; j < 128; j += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            mq[y] = fmaxf(fmaxf(mq[y], __uint_as_float(sv[j + 2 * y])), __uint_as_float(sv[j + 2 * y + 1]));
        float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
        mx = mx > kLowest ? fmaxf(mx * rf, kLowest) : -INFINITY;
        const bool grow = mx > m + kGrow || (m == -INFINITY && mx > -INFINITY);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float corr = grow ? ex2f(m - mx) : 1.0f;   // m = -inf: 0
          if (grow) m = mx;
          l *= corr;
          if (any) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tm_ld<16>(o, to + 16u * c);
              tm_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * corr);
              tm_st<16>(to + 16u * c, o);
            }
          }
        }
        any = true;
        // ---- weights (a row that has seen nothing: every weight is 2^(kNever rf) = 0)
        const float nm = m == -INFINITY ? 0.0f : kHead - m;
        float l0 = 0.0f, l1 = 0.0f, l2 = 0.0f, l3 = 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            float a[4];
#pragma unroll
            for (int y = 0; y < 4; y += 2) {
              fma2(a[y], a[y + 1], __uint_as_float(sv[32 * c + j + y]), __uint_as_float(sv[32 * c + j + y + 1]), rf, rf, nm, nm);
              a[y] = ex2f(a[y]);
              a[y + 1] = ex2f(a[y + 1]);
              p[(j + y) >> 1] = f16x2(a[y], a[y + 1]);
            }
            add2f(l0, l1, a[0], a[1]);
            add2f(l2, l3, a[2], a[3]);
          }
          tm_st<16>(ts + 16u * c, p);   // over columns that have been read
        }
        l += (l0 + l1) + (l2 + l3);
        tm_wait_st();
        tm_fence_before();
        __syncwarp();
        if (lane == 0) mb_arrive(&S.p_full[x]);
      }
      if (!ok) break;
      // ---- result of the item
      if (I.tile1 > I.tile0) {
        ok = __all_sync(0xFFFFFFFFu, mb_wait(&S.o_full, o_phase, gave_up));
        if (!ok) break;
        o_phase ^= 1u;
        tm_fence_after();
      }
      const bool whole = I.part < 0;
      const float inv = row_inverse(m, l);
      // an infinite sum or a NaN: a value of the cache past binary16 (or of q)
      if (whole && valid && !(l < INFINITY)) bad = 1u;
      float4* const pp = reinterpret_cast<float4*>(part + (size_t)(whole ? 0 : I.part + x) * 128 * kAttPart) + rt;
      float check = 0.0f;   // becomes a NaN if any element is not finite
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        uint32_t o[16];
        if (any) {
          tm_ld<16>(o, to + 16u * c);
          tm_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = 0u;
        }
        if (whole) {
          // rows go through the warp's own rows of Q, which every MMA has read, to be written whole
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float a = __uint_as_float(o[2 * k]) * inv, b = __uint_as_float(o[2 * k + 1]) * inv;
            check = fmaf(a, 0.0f, fmaf(b, 0.0f, check));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(b), "f"(a));
          }
          *reinterpret_cast<uint4*>(S.q[x] + tile_off(128, rt, 2 * c)) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(S.q[x] + tile_off(128, rt, 2 * c + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
        } else if (valid) {
          // partial: four channels of 128 rows at a time
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            pp[(4 * c + (j >> 2)) * 128] = make_float4(__uint_as_float(o[j]), __uint_as_float(o[j + 1]),
                                                       __uint_as_float(o[j + 2]), __uint_as_float(o[j + 3]));
        }
        __syncwarp();
      }
      if (whole) {
        if (valid && check != 0.0f) bad = 1u;
        const int c = lane & 15, half = lane >> 4, w32 = rl - lane;
#pragma unroll 4
        for (int y = 0; y < 16; ++y) {
          const int r = 2 * y + half;
          if (w32 + r < T.rows) {
            const uint4 w = *reinterpret_cast<const uint4*>(S.q[x] + tile_off(128, (rt & ~31) + r, c));
            uint16_t* op = A.out + rows.at(A, u, I.row0 + w32 + r) + 8 * c;
            if (oal) {
              *reinterpret_cast<uint4*>(op) = w;
            } else {
              const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                op[2 * k] = (uint16_t)wd[k];
                op[2 * k + 1] = (uint16_t)(wd[k] >> 16);
              }
            }
          }
        }
        __syncwarp();   // the rows are Q again in the next item
      } else if (valid) {
        reinterpret_cast<float2*>(part + (size_t)(I.part + x) * 128 * kAttPart + 128 * kHeadDim)[rt] = make_float2(m, l);
      }
    }
    if (bad) atomicOr(A.status, kStatusRange);
  } else if (warp < 10) {
    // ------------------------------------------------- MMA: warp 8 + x issues those of S_x, P_x and O_x
    if (lane == 0) {
      const int x = warp & 1;
      constexpr uint32_t idesc = mma_idesc(128, 128);
      // descriptors of the tiles; a K step of 16 is 32 bytes, a 64-element block 16384 (in units of 16 bytes)
      constexpr uint32_t kTile16 = kTileBytes >> 4;
      const uint64_t qd0 = sw128_desc(sm32(S.q[0])), td0 = sw128_desc(sm32(S.kv[0]));
      const uint32_t ds = tmem + 128u * x, dout = tmem + 256u + 128u * x;
      uint32_t tc0 = 0, q_phase = 0, p_phase = 0, turns = 0;   // tc0: tiles before this item
      bool ok = true;
      // tile t of the CTA's stream: K is ring entry 2 t, V entry 2 t + 1
      auto ready = [&](uint32_t e) {
        return mb_wait(&S.full[e % kRing], (e / kRing) & 1u, gave_up, e ? kAttSpin : first_spins);
      };
      for (int it = i0; it < i1 && ok; ++it) {
        const int n = items[it].tile1 - items[it].tile0;
        if (n == 0) continue;
        ok = mb_wait(&S.q_full, q_phase, gave_up);
        if (!ok) break;
        q_phase ^= 1u;
        const uint64_t qd = qd0 + (uint32_t)x * kTile16;
        // A step: P V of tile t - 1, then Q K^T of tile t into the same S, issued together so that the
        // tensor cores see one run of 16; the other warp's run fills the time that the softmax of this
        // one takes.
#pragma unroll 1
        for (int t = 0; t <= n; ++t) {
          const uint32_t ke = 2u * (tc0 + (uint32_t)t), pv = ke - 1u;
          if (t < n) ok = ready(ke);
          // Runs of the two halves take turns: issued at will they would fall into step, both halves'
          // MMAs at one time and both softmaxes at the next (4100 cycles per tile instead of 3700).
          if (ok && (x || turns)) ok = mb_wait(&S.turn[x], (x ? turns : turns - 1u) & 1u, gave_up);
          ++turns;
          if (ok && t) {
            ok = mb_spin(&S.p_full[x], p_phase, gave_up);
            p_phase ^= 1u;
          }
          if (!ok) break;
          tm_fence_after();
          if (t) {
            const uint64_t b = td0 + (pv % kRing) * kTile16;
#pragma unroll
            for (int s = 0; s < 8; ++s)
              mma_ts(dout, ds + 8u * s, b + ((s >> 2) * 1024 + (s & 3) * 2), idesc, t > 1 || s > 0);
          }
          if (t < n) {
            const uint64_t b = td0 + (ke % kRing) * kTile16;
#pragma unroll
            for (int s = 0; s < 8; ++s)
              mma_ss(ds, qd + ((s >> 2) * 1024 + (s & 3) * 2), b + ((s >> 2) * 1024 + (s & 3) * 2), idesc, s > 0);
            tm_commit(&S.s_full[x]);
            tm_commit(&S.empty[ke % kRing]);
          }
          mb_arrive(&S.turn[x ^ 1]);
          if (t) tm_commit(&S.empty[pv % kRing]);
          if (t == n) break;
          ok = ready(ke + 1u);   // this tile's V
          if (!ok) break;
        }
        if (ok) tm_commit(&S.o_full);
        tc0 += (uint32_t)n;
      }
      if (!ok) {   // let the MMAs that were issued finish before TMEM is given back
        volatile uint32_t never = 0u;
        tm_commit(&S.drain[x]);
        mb_wait(&S.drain[x], 0u, &never);
      }
    }
    __syncwarp();
  } else if (warp == 10) {
    // --------------------------------------------------------------- loader
    if (lane == 0) {
      uint32_t e = 0;   // ring entries issued
      bool ok = true;
      for (int it = i0; it < i1 && ok; ++it) {
        const AttItem I = items[it];
        const uint8_t* src = tiles + (size_t)(units[I.unit].tile_base + I.tile0) * 2 * kTileBytes;
        for (int y = 0; y < 2 * (I.tile1 - I.tile0); ++y, ++e, src += kTileBytes) {
          ok = mb_wait(&S.empty[e % kRing], ((e / kRing) & 1u) ^ 1u, gave_up);
          if (!ok) break;
          bulk_to_smem(S.kv[e % kRing], src, kTileBytes, &S.full[e % kRing]);
        }
      }
      // every copy has landed before the CTA leaves
      volatile uint32_t never = 0u;
      for (uint32_t y = e > kRing ? e - kRing : 0u; y < e; ++y) mb_wait(&S.full[y % kRing], (y / kRing) & 1u, &never);
    }
    __syncwarp();
  }
  tm_fence_before();
  __syncthreads();
  if (tid == 0 && *gave_up) atomicOr(A.status, kStatusTimeout);
  if (warp == 8) {
    tm_fence_after();
    tm_free(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_attend_tiles(kv_pool* P, const AttArgs& A, const AttUnit* d_units, int n_units, int max_tiles,
                                void* d_tiles, uint32_t* d_live, cudaStream_t s) {
  if (n_units <= 0 || max_tiles <= 0) return cudaSuccess;
  ++P->launches;
  attend_tiles_kernel<<<dim3((unsigned)max_tiles, (unsigned)n_units), 256, 0, s>>>(A, d_units, (uint8_t*)d_tiles, d_live);
  return cudaGetLastError();
}

cudaError_t launch_attend_wide(kv_pool* P, const AttArgs& A, const AttUnit* d_units, const AttItem* d_items,
                               const int32_t* d_cta_item, int n_ctas, const void* d_tiles, const uint32_t* d_live,
                               float* d_part, cudaStream_t s) {
  if (n_ctas <= 0) return cudaSuccess;
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(attr_set.load() >> dev & 1u)) {
    const cudaError_t e = cudaFuncSetAttribute(attend_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(WideSmem));
    if (e != cudaSuccess) return e;
    attr_set.fetch_or(uint64_t(1) << dev);
  }
  ++P->launches;
  attend_wide_kernel<<<(unsigned)n_ctas, kThreads, sizeof(WideSmem), s>>>(
      A, d_units, d_items, d_cta_item, (const uint8_t*)d_tiles, d_live, d_part,
      P->first_wait_spins < 0 ? kAttSpin : (uint32_t)P->first_wait_spins);
  return cudaGetLastError();
}

}  // namespace kvq
