// kv_attend for few rows per unit (drafts to be verified, single tokens): tcgen05
// attention bound by the cache's bytes.
//
// With R <= 64 rows the products are taken transposed, so that the 128 rows of an
// MMA are always full:
//     S^T = K Q^T   (128 keys x R),      O^T += V^T P^T   (128 channels x R).
// The A operands, K (a key per TMEM lane) and V^T (a channel per lane), are
// dequantized from the page blocks straight into TMEM: the code words of the
// pages are laid out by mma fragments, and tcgen05.st's 16x256b shape has the same
// ownership (lane 4 r + i: rows r and r + 8, columns 2 i and 2 i + 1 of every 8), so a
// word goes from shared memory through registers to its place with no exchange.
// Through shared memory instead, each tile would cost 64 KB written and 64 KB read
// again, 1000 cycles of its 128 bytes a cycle; TMEM has its own ports.
//
// A CTA takes an item: a block of R rows of one (request, kv head) unit and a run
// of its tiles of 128 keys (four pages, or bf16 rows).  Roles: eight warps for the
// softmax (a key per thread, the rows in two halves), eight (R = 64: four) each for K
// and V (a page, or 32 channels, each or in pairs), one to issue the MMAs of S^T and
// one those of O^T, one that streams pages with bulk copies, six tiles deep.  The
// running maximum of a row is kept while no key exceeds it by more than 2^8 (P is
// binary16 with 2^7 of headroom); otherwise the warps take the maxima of all columns
// and rescale O^T.  The sums of P come from the tensor cores (ones times P).
//
// What bounds it: the instructions of unpacking and softmax and their waits.  A tile
// takes 2750 (R = 32) to 3300 cycles (R = 64): about 7000 warp instructions, in 67 and
// 52 % of the issue slots, against 520 (INT2) to 870 cycles (INT4) that its bytes take
// from HBM and 600 of MMAs at R = 64; two stages of K and V are all that TMEM holds
// beside S and O.  24 requests with 1 to 7 new tokens over 1K to 32K, 32 q on 8 kv
// heads: 285 us, 1.4 TB/s; a tree of 31 for 8 requests over 32K: 381 us.  Slower: K
// and V by the same sixteen warps in turn, one code path at a time (drafts + 10 %);
// softmax warps that skip a half without rows (+ 4 %).
#include <algorithm>
#include <atomic>

#include "kvq_attend_mma.cuh"

namespace kvq {
namespace {

constexpr int kStages = 6;                      // raw tiles in flight
// Warps each for K and for V: with R = 64 the softmax code needs the registers (72 per thread with 27
// warps): 420 us for 31-token trees x 8 over 32K with 4, 478 with 8; ragged drafts (R = 32) 440 and 358.
template <int R>
constexpr int kSide = R == 64 ? 4 : 8;
template <int R>
constexpr int kMma = 8 + 2 * kSide<R>;          // first MMA warp
template <int R>
constexpr int kThreads = 32 * (kMma<R> + 3);
constexpr int kMaskRing = 16;                   // tiles whose live words are kept
constexpr float kHead = 7.0f;                   // P = 2^(x - m + 7)
constexpr float kGrow = 8.0f;                   // a maximum may be stale by this much (base 2)
constexpr float kNever = -3.0e38f;              // S of a key that is not seen
constexpr float kLowest = 0.9f * kNever;        // logits below it count as it
constexpr float kUnseen = -1.0e30f;             // kHead - m of a row that has seen nothing: its weights are 0
// TMEM columns (two stages of K, V and S; kColOne: the ones of the sums, for R <= 32)
constexpr uint32_t kColK = 0, kColV = 128, kColS = 256, kColO = 384, kColL = 448, kColOne = 480;

template <int R>
struct alignas(1024) FewSmem {
  uint8_t q[R * 256], p[2][R * 256];            // operand rows of 128 elements, 128-byte swizzled
  uint8_t one[R == 64 ? 16384 : 16];            // ones (R = 64: TMEM has no columns left for them)
  alignas(128) uint8_t raw[kStages][4][kInt4Block];
  float rf[R], nm[R];                           // per row: factor of S, kHead - m
  float m[R], fac[R], wmax[4][R];
  unsigned long long tree[R];
  uint32_t live[kMaskRing][4];
  int32_t cls[kStages][4];
  uint32_t grow[2][8];
  uint64_t raw_full[kStages], raw_empty[kStages];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], pv_done[2], q_full, drain[2];
  uint32_t tmem, gave_up, unseen;
};
static_assert(sizeof(FewSmem<64>) <= 232448, "one CTA's shared memory");

struct Tiles {   // an item's tiles: [0, pages), [pages, lists), [lists, ..) by kind
  int pages, lists, rows;
};
template <int R>
__device__ __forceinline__ Tiles tiles_of(const AttArgs& A, const AttUnit& u, int row0) {
  Tiles t;
  t.rows = min(R, u.T * (A.hq / A.hkv) - row0);
  t.pages = (u.n_pages + 3) >> 2;
  t.lists = t.pages + ((u.n_fp + 127) >> 7);
  return t;
}

// tcgen05.st of fragments: 16 lanes x (8 N) columns, lane 4 r + i holds rows r and
// r + 8, columns 8 x + 2 i and + 1 (registers 4 x .. 4 x + 3)
__device__ __forceinline__ void tm_st_frag32(uint32_t addr, const uint32_t (&a)[2][4], const uint32_t (&b)[2][4]) {
  // word w = 2 x + c of row r is a[w >> 2][w & 3], of row r + 8 b[w >> 2][w & 3]
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(a[0][0]), "r"(a[0][1]), "r"(b[0][0]), "r"(b[0][1]), "r"(a[0][2]), "r"(a[0][3]), "r"(b[0][2]), "r"(b[0][3]),
      "r"(a[1][0]), "r"(a[1][1]), "r"(b[1][0]), "r"(b[1][1]), "r"(a[1][2]), "r"(a[1][3]), "r"(b[1][2]), "r"(b[1][3])
      : "memory");
}
__device__ __forceinline__ void tm_st_frag16(uint32_t addr, const uint32_t (&a)[4], const uint32_t (&b)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(a[0]), "r"(a[1]),
               "r"(b[0]), "r"(b[1]), "r"(a[2]), "r"(a[3]), "r"(b[2]), "r"(b[3]) : "memory");
}
// Place of element n (0..7) of run (gr, i) in a row of the K contraction, and of
// slot 8 i + n of page gr in one of the V contraction (see tm_st_frag*).
__device__ __forceinline__ int frag_pos(int gr, int i, int n) {
  return 32 * gr + 16 * ((n & 3) >> 1) + 4 * i + 2 * (n & 1) + (n >> 2);
}
__device__ __forceinline__ float warp_max_f(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(y) : "f"(x));
  return y;
}
// Barrier of the softmax warps; true if any thread gives `stop` (every thread
// gets the same answer, so all leave together).
__device__ __forceinline__ bool group_stop(bool stop) {
  uint32_t r;
  asm volatile("{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n barrier.cta.red.or.pred b, 1, 256, a;\n selp.u32 %0, 1, 0, b;\n}"
               : "=r"(r) : "r"((uint32_t)stop) : "memory");
  return r != 0;
}

// P of this thread's key, rows kN ..: row n is 128 n bytes on, its chunks exchanged
// by n & 7 (an exclusive or on the address).
template <int kN, int kC>
__device__ __forceinline__ void store_weights(uint32_t addr, const float (&x)[kC]) {
  if constexpr (kN < kC) {
    const uint32_t h = f16x2(ex2f(x[kN]), ex2f(x[kN + 1]));
    asm volatile("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %4;\n st.shared.b16 [%0 + %2], l;\n st.shared.b16 [%1 + %3], h;\n}"
                 ::"r"(addr ^ ((kN & 7) << 4)), "r"(addr ^ (((kN + 1) & 7) << 4)), "n"(kN * 128), "n"((kN + 1) * 128), "r"(h)
                 : "memory");
    store_weights<kN + 2>(addr, x);
  }
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

template <int R>
__global__ void __launch_bounds__(kThreads<R>, 1) attend_few_kernel(
    AttArgs A, const AttUnit* __restrict__ units, const AttItem* __restrict__ items, const int32_t* __restrict__ cta_item,
    float* __restrict__ part, uint32_t first_spins) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  FewSmem<R>& S = *reinterpret_cast<FewSmem<R>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i0 = cta_item[blockIdx.x], i1 = cta_item[blockIdx.x + 1];
  volatile uint32_t* gave_up = &S.gave_up;
  if (tid == 0) {
    for (int x = 0; x < kStages; ++x) {
      mb_init(&S.raw_full[x], 4);
      mb_init(&S.raw_empty[x], 2 * kSide<R>);
    }
    for (int x = 0; x < 2; ++x) {
      mb_init(&S.k_full[x], kSide<R>);
      mb_init(&S.k_empty[x], 1);
      mb_init(&S.v_full[x], kSide<R>);
      mb_init(&S.v_empty[x], 1);
      mb_init(&S.s_full[x], 1);
      mb_init(&S.p_full[x], 8);
      mb_init(&S.pv_done[x], 1);
    }
    mb_init(&S.q_full, 8);
    mb_init(&S.drain[0], 1);
    mb_init(&S.drain[1], 1);
    S.gave_up = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMma<R>) tm_alloc(&S.tmem, 512);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tmem = S.tmem;
  const int g = A.hq / A.hkv;

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    // hf: the half of the columns (rows of the block) of this warp; its 32 keys are those of page warp & 3
    constexpr int kC = R / 2;
    const int hf = warp >> 2, c0 = hf * kC, wq = warp & 3, key = tid & 127;
    const uint32_t tl = tmem + ((uint32_t)wq << 21);
    // this thread's key in a row of P: its chunk and byte
    const int kp = frag_pos(wq, lane >> 3, lane & 7);
    const uint32_t p_addr = sm32(S.p[0]) + (uint32_t)(kp >> 6) * R * 128 + (uint32_t)c0 * 128 + 2u * (kp & 63);
    uint32_t page_tiles = 0, tc = 0, bad = 0u;   // tc: tiles of this CTA so far
    bool ok = true;
    const bool qal = ((uintptr_t)A.q & 15) == 0;
    const RowMap rows(g);
    if constexpr (R == 64) {
      for (int x = tid; x < 1024; x += 256) reinterpret_cast<uint4*>(S.one)[x] = make_uint4(0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u);
    } else if (hf == 0) {
      uint32_t w[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) w[x] = 0x3C003C00u;
      tm_st<16>(tl + kColOne, w);
      tm_wait_st();
    }
    for (int it = i0; it < i1; ++it) {
      const AttItem I = items[it];
      const AttUnit u = units[I.unit];
      const Tiles T = tiles_of<R>(A, u, I.row0);
      // ---- Q: 256 / R threads per row; scaled by a power of two so that its largest element is in [2^7, 2^8)
      {
        constexpr int kPer = R == 16 ? 16 : 256 / R, kRuns = 16 / kPer;
        const int n = tid / kPer, sub = tid % kPer;
        const bool valid = n < T.rows;
        const uint16_t* qr = A.q + rows.at(A, u, I.row0 + (valid ? n : 0));
        uint4 w[kRuns];
#pragma unroll
        for (int y = 0; y < kRuns; ++y) w[y] = load8(qr + 8 * (sub + kPer * y), qal);
        float mx = 0.0f;
#pragma unroll
        for (int y = 0; y < kRuns; ++y) {
          if (!valid) w[y] = make_uint4(0u, 0u, 0u, 0u);
          const uint32_t wd[4] = {w[y].x, w[y].y, w[y].z, w[y].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx = fmaxf(mx, fmaxf(fabsf(bf_f(wd[k] & 0xFFFFu)), fabsf(__uint_as_float(wd[k] & 0xFFFF0000u))));
        }
#pragma unroll
        for (int o = kPer / 2; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        const int e = q_exponent(mx);
        const float mul = q_factor(mx, e, A.scale_log2);
#pragma unroll
        for (int y = 0; y < kRuns; ++y) {
          const int run = sub + kPer * y, gr = run >> 2, i = run & 3;
          const uint32_t wd[4] = {w[y].x, w[y].y, w[y].z, w[y].w};
          float f[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[2 * k] = bf_f(wd[k] & 0xFFFFu) * mul;
            f[2 * k + 1] = __uint_as_float(wd[k] & 0xFFFF0000u) * mul;
          }
          // elements 0, 4, 1, 5 at frag_pos(gr, i, 0), elements 2, 6, 3, 7 sixteen places on
          const int e0 = 32 * gr + 4 * i;
          uint8_t* base = S.q + (e0 >> 6) * R * 128 + n * 128 + 8 * (i & 1);
          const int c = (e0 & 63) >> 3;
          *reinterpret_cast<uint2*>(base + ((c ^ (n & 7)) << 4)) = make_uint2(f16x2(f[0], f[4]), f16x2(f[1], f[5]));
          *reinterpret_cast<uint2*>(base + (((c + 2) ^ (n & 7)) << 4)) = make_uint2(f16x2(f[2], f[6]), f16x2(f[3], f[7]));
        }
        if (sub == 0) {
          // (a factor below 1e-30 makes every logit 0, as 1e-30 does; kNever times it must stay far below 0)
          S.rf[n] = fmaxf(fabsf(A.scale_log2) * pow2f(-e), 1e-30f);
          S.nm[n] = kUnseen;
          S.m[n] = -INFINITY;
          S.tree[n] = A.tree && valid ? A.tree[u.tok0 + rows.token(I.row0 + n)] : 0ull;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tm_fence_before();   // the previous item's O has been read
      if (group_stop(false)) break;   // rows' factors are in place
      if (lane == 0 && I.tile1 > I.tile0) mb_arrive(&S.q_full);

      bool unseen = true;   // some row has seen no key yet
      bool stop = false;
#pragma unroll 1
      for (int tile = I.tile0; tile < I.tile1; ++tile, ++tc) {
        const uint32_t b = tc & 1u, ts = tl + kColS + 64u * b + (uint32_t)c0;
        // ---- rows of this half that see this thread's key, as bits
        uint32_t vis = 0u;
        bool live_ring = false;
        if (tile < T.pages) {
          live_ring = true;
        } else if (tile < T.lists) {
          if (128 * (tile - T.pages) + key < u.n_fp) vis = 0xFFFFFFFFu;
        } else {
          const int j = 128 * (tile - T.lists) + key;
          if (j < u.T) {
            if (A.tree) {   // u.T <= 64
#pragma unroll 1
              for (int n = 0; n < kC; ++n) vis |= ((S.tree[c0 + n] >> j) & 1ull) ? 1u << n : 0u;
            } else {
              const int64_t f = (int64_t)j * g - I.row0 - c0;   // rows from f on
              vis = f >= 32 ? 0u : (f <= 0 ? 0xFFFFFFFFu : 0xFFFFFFFFu << f);
            }
          }
        }
        ok = __all_sync(0xFFFFFFFFu, mb_wait(&S.s_full[b], (tc >> 1) & 1u, gave_up));
        tm_fence_after();
        if (live_ring) {
          const uint32_t lv = *(volatile uint32_t*)&S.live[page_tiles & (kMaskRing - 1)][wq];
          vis = ((lv >> lane) & 1u) ? 0xFFFFFFFFu : 0u;
          ++page_tiles;
        }
        const bool all_seen = __all_sync(0xFFFFFFFFu, vis == 0xFFFFFFFFu);
        uint32_t s[kC];
        auto load = [&]() {
          if constexpr (kC == 8) tm_ld<8>(s, ts);
          else if constexpr (kC == 16) tm_ld<16>(s, ts);
          else tm_ld<32>(s, ts);
          tm_wait_ld();
          if (!all_seen) {
#pragma unroll
            for (int n = 0; n < kC; ++n) s[n] = ((vis >> n) & 1u) ? s[n] : __float_as_uint(kNever);
          }
        };
        load();
        // ---- x = S rf + 7 - m; does a key exceed its row's maximum by too much?
        float x[kC];
        auto weights_of = [&]() {
#pragma unroll
          for (int n = 0; n < kC; n += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&S.rf[c0 + n]), d = *reinterpret_cast<const float4*>(&S.nm[c0 + n]);
            fma2(x[n], x[n + 1], __uint_as_float(s[n]), __uint_as_float(s[n + 1]), f.x, f.y, d.x, d.y);
            fma2(x[n + 2], x[n + 3], __uint_as_float(s[n + 2]), __uint_as_float(s[n + 3]), f.z, f.w, d.z, d.w);
          }
        };
        weights_of();
        float top = 0.0f, top1 = 0.0f;
#pragma unroll
        for (int n = 0; n < kC; n += 4) {
          top = fmaxf(fmaxf(top, x[n]), x[n + 1]);
          top1 = fmaxf(fmaxf(top1, x[n + 2]), x[n + 3]);
        }
        const bool mine = __any_sync(0xFFFFFFFFu, unseen || fmaxf(top, top1) > kHead + kGrow);
        if (lane == 0) *(volatile uint32_t*)&S.grow[b][warp] = mine;
        // the P buffer of two tiles ago has been used
        if (ok && tile >= I.tile0 + 2)
          ok = __all_sync(0xFFFFFFFFu, mb_wait(&S.pv_done[b], ((tc >> 1) & 1u) ^ 1u, gave_up));
        if (group_stop(!ok)) {
          stop = true;
          break;
        }
        const uint4 g0 = *reinterpret_cast<const uint4*>(&S.grow[b][0]), g1 = *reinterpret_cast<const uint4*>(&S.grow[b][4]);
        if (g0.x | g0.y | g0.z | g0.w | g1.x | g1.y | g1.z | g1.w) {
          // ---- new maxima of all rows
          load();
          float keep = kNever;
#pragma unroll
          for (int n = 0; n < kC; ++n) {
            const float v = __uint_as_float(s[n]);
            const float w = warp_max_f(v == kNever ? kNever : fmaxf(v * S.rf[c0 + n], kLowest));
            if (lane == n) keep = w;
          }
          if (lane < kC) S.wmax[wq][c0 + lane] = keep;
          if (tid == 0) S.unseen = 0u;
          if (tile > I.tile0) ok = mb_wait(&S.pv_done[b ^ 1u], ((tc - 1u) >> 1) & 1u, gave_up);   // O is at rest
          if (group_stop(!ok)) {
            stop = true;
            break;
          }
          if (tid < R) {
            const float w = fmaxf(fmaxf(S.wmax[0][tid], S.wmax[1][tid]), fmaxf(S.wmax[2][tid], S.wmax[3][tid]));
            const float mo = S.m[tid], mn = w > 0.95f * kNever ? fmaxf(mo, w) : mo;
            S.m[tid] = mn;
            S.fac[tid] = mo == -INFINITY ? 1.0f : ex2f(mo - mn);
            S.nm[tid] = mn == -INFINITY ? kUnseen : kHead - mn;
            if (mn == -INFINITY && tid < T.rows) S.unseen = 1u;
          }
          group_stop(false);
          unseen = *(volatile uint32_t*)&S.unseen != 0u;
          weights_of();
          if (tile > I.tile0) {   // O and the sums
            tm_fence_after();
#pragma unroll 1
            for (int y = 0; y < 2; ++y) {
              const uint32_t at = tl + (y ? kColL : kColO) + (uint32_t)c0;
#pragma unroll 1
              for (int c = 0; c < kC; c += 8) {
                uint32_t o[8];
                tm_ld<8>(o, at + (uint32_t)c);
                tm_wait_ld();
#pragma unroll
                for (int n = 0; n < 8; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * S.fac[c0 + c + n]);
                tm_st<8>(at + (uint32_t)c, o);
              }
            }
            tm_wait_st();
          }
        }
        // ---- weights
        store_weights<0>(p_addr + b * (R * 256), x);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the MMAs read P
        tm_fence_before();
        __syncwarp();
        if (lane == 0) mb_arrive(&S.p_full[b]);
      }
      if (stop) break;
      // ---- result of the item: O and the sums (every lane holds them)
      const bool some = I.tile1 > I.tile0;
      if (some) ok = mb_wait(&S.pv_done[(tc - 1u) & 1u], ((tc - 1u) >> 1) & 1u, gave_up);
      if (group_stop(!ok)) break;
      tm_fence_after();
      const bool whole = I.part < 0;
      float* pp = part + (size_t)(whole ? 0 : I.part) * R * kAttPart;
#pragma unroll 1
      for (int c = c0; c < c0 + kC; c += 8) {
        uint32_t o[8], ls[8];
        if (some) {
          tm_ld<8>(o, tl + kColO + (uint32_t)c);
          tm_ld<8>(ls, tl + kColL + (uint32_t)c);
          tm_wait_ld();
        } else {
#pragma unroll
          for (int n = 0; n < 8; ++n) o[n] = ls[n] = 0u;
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          if (c + n >= T.rows) break;
          const float m = S.m[c + n], L = __uint_as_float(ls[n]);
          if (whole && !(L < INFINITY)) bad = 1u;
          if (whole) {
            const float inv = row_inverse(m, L);
            const float v = __uint_as_float(o[n]) * inv;
            if (!(fabsf(v) < INFINITY)) bad = 1u;
            A.out[rows.at(A, u, I.row0 + c + n) + key] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
          } else {
            pp[(size_t)(c + n) * kAttPart + key] = __uint_as_float(o[n]);
            if (key == 0) *reinterpret_cast<float2*>(pp + (size_t)(c + n) * kAttPart + kHeadDim) = make_float2(m, L);
          }
        }
        __syncwarp();
      }
      if (group_stop(false)) break;   // the maxima have been read
    }
    if (bad) atomicOr(A.status, kStatusRange);
  } else if (warp < kMma<R>) {
    // ----------------------------------------------------------- dequantize
    const bool is_k = warp < 8 + kSide<R>;
    // K: a page, channel groups 2 half and 2 half + 1; V: a group, pages 2 half and 2 half + 1 (4 warps a side: both halves)
    const int w4 = warp & 3, h0 = kSide<R> == 8 ? (warp >> 2) & 1 : 0, h1 = kSide<R> == 8 ? h0 + 1 : 2;
    const int r = lane >> 2, i = lane & 3;
    const uint32_t tl = tmem + ((uint32_t)w4 << 21);
    uint32_t page_tiles = 0, tc = 0, bad = 0u;
    const bool kal = (((uintptr_t)A.k | (uintptr_t)A.v) & 15) == 0;
    bool ok = true;
    uint64_t* full = is_k ? S.k_full : S.v_full;
    uint64_t* empty = is_k ? S.k_empty : S.v_empty;
    for (int it = i0; it < i1 && ok; ++it) {
      const AttItem I = items[it];
      const AttUnit u = units[I.unit];
      const Tiles T = tiles_of<R>(A, u, I.row0);
      for (int tile = I.tile0; tile < I.tile1; ++tile, ++tc) {
        const uint32_t st = tc & 1u;
        const uint32_t dst = tl + (is_k ? kColK : kColV) + 64u * st;
        ok = mb_wait(&empty[st], ((tc >> 1) & 1u) ^ 1u, gave_up);
        if (tile < T.pages) {
          const uint32_t sg = page_tiles % kStages;
          if (ok) ok = mb_wait(&S.raw_full[sg], (page_tiles / kStages) & 1u, gave_up, page_tiles ? kAttSpin : first_spins);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          ++page_tiles;
          tm_fence_after();
          if (is_k) {
            const uint8_t* blk = S.raw[sg][w4];
            const int cls = *(volatile int32_t*)&S.cls[sg][w4];
            if (cls == kClsInt2) {
              // a run of 8 channels at a time: its scales serve the lane's four slots
#pragma unroll 1
              for (int gr = 2 * h0; gr < 2 * h1; ++gr) {
                uint32_t sc[4], z[4], a[4][4];
                k_scales2(blk, gr, i, sc, z);
#pragma unroll
                for (int x = 0; x < 4; ++x) k_run2(blk, 8 * x + r, gr, i, sc, z, a[x]);
                tm_st_frag16(dst + 16u * gr, a[0], a[1]);
                tm_st_frag16(dst + 16u * gr + (16u << 16), a[2], a[3]);
              }
            } else {
#pragma unroll 1
              for (int y = 2 * h0; y < 2 * h1; ++y) {      // slots 16 m + r and 16 m + r + 8
                const int m = y & 1, half = y >> 1, t0 = 16 * m + r;
                uint32_t a[2][4], b[2][4];
                if (cls == kClsInt4) {
                  k_slot4(blk, t0, i, half, a);
                  k_slot4(blk, t0 + 8, i, half, b);
                } else if (cls == kClsInt3) {
                  k_slot3(blk, t0, i, half, a);
                  k_slot3(blk, t0 + 8, i, half, b);
                } else if (cls == kClsFp4) {
                  k_slotf(blk, t0, i, half, a);
                  k_slotf(blk, t0 + 8, i, half, b);
                } else {
#pragma unroll
                  for (int x = 0; x < 8; ++x) a[x >> 2][x & 3] = b[x >> 2][x & 3] = 0u;
                }
                tm_st_frag32(dst + 32u * half + ((uint32_t)(16 * m) << 16), a, b);
              }
            }
          } else {
#pragma unroll 1
            for (int p = 2 * h0; p < 2 * h1; ++p) {
              const uint8_t* blk = S.raw[sg][p];
              const int cls = *(volatile int32_t*)&S.cls[sg][p];
              uint32_t v[4][4];
              if (cls == kClsInt2) {
                v_group2(blk, w4, r, i, v);
              } else if (cls == kClsInt4) {
                v_group4(blk, w4, r, i, v);
              } else if (cls == kClsInt3) {
                v_group3(blk, w4, r, i, v);
              } else if (cls == kClsFp4) {
                v_groupf(blk, w4, r, i, v);
              } else {
#pragma unroll
                for (int x = 0; x < 16; ++x) v[x >> 2][x & 3] = 0u;
              }
              tm_st_frag16(dst + 16u * p, v[0], v[1]);
              tm_st_frag16(dst + 16u * p + (16u << 16), v[2], v[3]);
            }
          }
          __syncwarp();
          if (lane == 0) mb_arrive(&S.raw_empty[sg]);
        } else {
          // ---- bf16 rows: list tokens or new tokens (rows past the end: the last one is loaded and used as 0)
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tm_fence_after();
          const bool list = tile < T.lists;
          const int j0 = 128 * (tile - (list ? T.pages : T.lists));
          const int n = list ? u.n_fp : u.T;
          const size_t stride = list ? kHeadDim : (size_t)A.hkv * kHeadDim;
          const uint16_t* src =
              list ? (is_k ? A.fpk : A.fpv) + ((size_t)u.req * A.hkv + u.kvh) * (size_t)A.fp_cap * kHeadDim
                   : (is_k ? A.k : A.v) + ((size_t)u.tok0 * A.hkv + u.kvh) * kHeadDim;
          if (is_k) {
#pragma unroll 1
            for (int yy = 2 * h0; yy < 2 * h1; ++yy) {
              const int m = yy & 1, half = yy >> 1;
              uint32_t a[2][4], b[2][4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int j = j0 + 32 * w4 + 16 * m + 8 * e + r, jc = min(j, n - 1);
                uint4 y[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const int ch = 4 * (2 * half + x) + i;
                  y[x] = load8(src + (size_t)jc * stride + 8 * (list ? ch ^ (jc & 7) : ch), list || kal);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  if (j >= n) y[x] = make_uint4(0u, 0u, 0u, 0u);
                  order8_f16(y[x], 1.0f, e ? b[x] : a[x], bad);
                }
              }
              tm_st_frag32(dst + 32u * half + ((uint32_t)(16 * m) << 16), a, b);
            }
          } else {
#pragma unroll 1
            for (int p = 2 * h0; p < 2 * h1; ++p) {
              uint32_t v[4][4];
              uint16_t y[4][8];
#pragma unroll
              for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int jc = min(j0 + 32 * p + 8 * i + e, n - 1), c = 32 * w4 + 8 * x + r;
                  y[x][e] = __ldg(src + (size_t)jc * stride + (list ? att_list_at(jc, c) : c));
                }
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  f[e] = j0 + 32 * p + 8 * i + e < n ? in_range(bf_f(y[x][e]), bad) : 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[x][k] = f16x2(f[k], f[k + 4]);
              }
              tm_st_frag16(dst + 16u * p, v[0], v[1]);
              tm_st_frag16(dst + 16u * p + (16u << 16), v[2], v[3]);
            }
          }
        }
        tm_wait_st();
        tm_fence_before();
        __syncwarp();
        if (lane == 0) mb_arrive(&full[st]);
      }
    }
    if (bad) atomicOr(A.status, kStatusRange);
  } else if (warp < kMma<R> + 2) {
    // ---------------------------------------------- MMA: one warp Q K^T, one P V and the sums of P
    // The whole warp runs the loop and one elected lane issues: with operands that the compiler knows to
    // be the same in all lanes an MMA of N = 32 issues every 21 cycles, from a branch on the lane every 47.
    constexpr uint32_t idesc = mma_idesc(128, R);
    const bool is_qk = warp == kMma<R>;
    const uint64_t qd = sw128_desc(sm32(S.q)), pd0 = sw128_desc(sm32(S.p[0])), od = sw128_desc(sm32(S.one));
    constexpr uint32_t kP16 = R * 16;   // one P buffer, in units of 16 bytes
    uint32_t tc = 0, q_phase = 0;
    bool ok = true;
    for (int it = i0; it < i1 && ok; ++it) {
      const AttItem I = items[it];
      const int n = I.tile1 - I.tile0;
      if (n == 0) continue;
      ok = mb_wait(&S.q_full, q_phase, gave_up);
      q_phase ^= 1u;
#pragma unroll 1
      for (int t = 0; t < n; ++t, ++tc) {
        const uint32_t b = tc & 1u, ph = (tc >> 1) & 1u;
        if (is_qk) {
          ok = ok && mb_wait(&S.k_full[b], ph, gave_up);
          if (ok && tc >= 2u) ok = mb_wait(&S.p_full[b], ph ^ 1u, gave_up);   // S of two tiles ago has been read
        } else {
          ok = ok && mb_wait(&S.v_full[b], ph, gave_up) && mb_wait(&S.p_full[b], ph, gave_up);
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tm_fence_after();
        if (is_qk) {
          if (elect_one()) {
#pragma unroll
            for (int s = 0; s < 8; ++s)
              mma_ts(tmem + kColS + 64u * b, tmem + kColK + 64u * b + 8u * s, qd + ((s >> 2) * (R * 8) + (s & 3) * 2), idesc, s > 0);
            tm_commit(&S.s_full[b]);
            tm_commit(&S.k_empty[b]);
          }
        } else {
          const uint64_t pd = pd0 + b * kP16;
          if (elect_one()) {
#pragma unroll
            for (int s = 0; s < 8; ++s) {
              const uint64_t at = pd + ((s >> 2) * (R * 8) + (s & 3) * 2);
              mma_ts(tmem + kColO, tmem + kColV + 64u * b + 8u * s, at, idesc, t > 0 || s > 0);
              if constexpr (R == 64) mma_ss(tmem + kColL, od, at, idesc, t > 0 || s > 0);
              else mma_ts(tmem + kColL, tmem + kColOne, at, idesc, t > 0 || s > 0);
            }
            tm_commit(&S.v_empty[b]);
            tm_commit(&S.pv_done[b]);
          }
        }
        __syncwarp();
      }
    }
    if (!ok) {   // let the MMAs that were issued finish before TMEM is given back
      volatile uint32_t never = 0u;
      if (elect_one()) tm_commit(&S.drain[is_qk ? 0 : 1]);
      __syncwarp();
      mb_wait(&S.drain[is_qk ? 0 : 1], 0u, &never);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- loader
    uint32_t page_tiles = 0, issued = 0;   // issued: tiles whose page this lane has issued
    bool ok = true;
    for (int it = i0; it < i1 && ok; ++it) {
      const AttItem I = items[it];
      const AttUnit u = units[I.unit];
      const Tiles T = tiles_of<R>(A, u, I.row0);
      const Entry* tab = A.table + (size_t)u.req * A.max_pages;
      const int end = min(I.tile1, T.pages);
      for (int tile = I.tile0; tile < end; ++tile, ++page_tiles) {
        if (lane < 4) {
          const uint32_t sg = page_tiles % kStages;
          const int pi = 4 * tile + lane;
          Entry e{-1, 0u};
          int cls = -1;
          const uint8_t* blk = nullptr;
          if (pi < u.n_pages) {
            e = tab[pi];
            if (A.hdead) e.live &= ~A.hdead[(size_t)e.id * A.hkv + u.kvh];
            if (e.live) cls = att_page(A, e.id, u.kvh, blk);
          }
          ok = mb_wait(&S.raw_empty[sg], ((page_tiles / kStages) & 1u) ^ 1u, gave_up);
          if (ok) {
            *(volatile int32_t*)&S.cls[sg][lane] = cls;
            *(volatile uint32_t*)&S.live[page_tiles & (kMaskRing - 1)][lane] = e.live;
            ++issued;
            if (cls < 0)
              mb_arrive(&S.raw_full[sg]);
            else
              bulk_to_smem(S.raw[sg][lane], blk,
                           cls == kClsInt2 ? kInt2Block : (cls == kClsInt4 ? kInt4Block : (cls == kClsInt3 ? kInt3Block : kFp4Block)),
                           &S.raw_full[sg]);
          }
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
      }
    }
    // Every copy has landed before the CTA leaves.  A tile of which only some lanes got to issue never
    // completes its barrier; those lanes' copies are waited for by time (the bound of the wait).
    const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, issued);
    if (lane == 0) {
      volatile uint32_t never = 0u;
      for (uint32_t y = most > kStages ? most - kStages : 0u; y < most; ++y)
        mb_wait(&S.raw_full[y % kStages], (y / kStages) & 1u, &never);
    }
    __syncwarp();
  }
  tm_fence_before();
  __syncthreads();
  if (tid == 0 && *gave_up) atomicOr(A.status, kStatusTimeout);
  if (warp == kMma<R>) {
    tm_fence_after();
    tm_free(tmem, 512);
  }
}

template <int R>
cudaError_t launch_r(kv_pool* P, const AttArgs& A, const AttUnit* d_units, const AttItem* d_items,
                     const int32_t* d_cta_item, int n_ctas, float* d_part, cudaStream_t s) {
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(attr_set.load() >> dev & 1u)) {
    const cudaError_t e = cudaFuncSetAttribute(attend_few_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(FewSmem<R>));
    if (e != cudaSuccess) return e;
    attr_set.fetch_or(uint64_t(1) << dev);
  }
  ++P->launches;
  attend_few_kernel<R><<<(unsigned)n_ctas, kThreads<R>, sizeof(FewSmem<R>), s>>>(
      A, d_units, d_items, d_cta_item, d_part, P->first_wait_spins < 0 ? kAttSpin : (uint32_t)P->first_wait_spins);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_few(kv_pool* P, int rows, const AttArgs& A, const AttUnit* d_units, const AttItem* d_items,
                              const int32_t* d_cta_item, int n_ctas, float* d_part, cudaStream_t s) {
  if (n_ctas <= 0) return cudaSuccess;
  switch (rows) {
    case 16: return launch_r<16>(P, A, d_units, d_items, d_cta_item, n_ctas, d_part, s);
    case 32: return launch_r<32>(P, A, d_units, d_items, d_cta_item, n_ctas, d_part, s);
    case 64: return launch_r<64>(P, A, d_units, d_items, d_cta_item, n_ctas, d_part, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
