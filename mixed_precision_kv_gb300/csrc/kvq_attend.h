// Attention of new tokens over the cache (kv_attend): what its host side hands
// to its kernels.
#pragma once
#include "kvq_internal.h"

namespace kvq {

constexpr int kMaxNewTokens = 1 << 20;   // new tokens of one request in a call
constexpr int64_t kMaxRows = int64_t(1) << 31;   // rows of q of a call (512 GB)

// One (request of the call, kv head): T new tokens of g q heads each.  Row i
// of a unit is (new token i / g, q head kvh * g + i % g).  A shared prefix is a
// unit too: its rows are the new tokens of every request that has it.
struct AttUnit {
  int32_t req, kvh;
  int32_t T;          // new tokens
  int32_t n_pages;    // table entries
  int32_t n_fp;       // full-precision list tokens
  int32_t tile_base;  // wide kernel: the unit's first operand tile pair
  int64_t tok0;       // the request's first row in q, k, v and out
  int32_t map;        // -1: new token t is row tok0 + t of q; else row tok_map[map + t]
  int32_t n_own;      // new tokens that are keys too: T, or 0 (none: no k and v, or a prefix)
  int32_t joined;     // the rows' results are joined with another unit's: partials, whatever the plan
  int32_t pad;
};

// A block of a unit's rows over a run of its key tiles, done by one CTA.
struct AttItem {
  int32_t unit, row0;
  int32_t tile0, tile1;   // tiles of 128 keys: pages by fours, then the list's rows, then the new tokens
  int32_t part;           // first partial (see each kernel), or -1: the block is done here
  int32_t pad[3];
};

// Rows whose partials are to be merged: parts part0, part0 + stride, ...
struct AttMerge {
  int32_t unit, row0, rows;
  int32_t part0, n_parts, stride;
};
constexpr int kAttPart = kHeadDim + 4;   // floats per row of a partial: O, then m and l
constexpr float kAttHead = 7.0f;         // weights (and O and l of the partials) are 2^(x - m + kAttHead): headroom of binary16

// The partials of a block of rows of a joined unit.
struct AttSrc {
  int64_t off;       // first part (floats)
  int32_t n_parts;
  int32_t step;      // floats from a part to the next
};
// The rows of a request (and kv head) with a prefix, or of a decode step: the parts of its own unit and those
// of the prefix unit that the rows are also in.
enum : int {
  kJoinOwnTall = 1, kJoinPreTall = 2,   // parts laid out as 128 rows by channel
  kJoinScan = 4                         // own parts are the decode scan's: own0 is a unit of its plan
};
struct AttJoin {
  int64_t tok0;              // the request's first row in q and out
  int32_t kvh, rows;
  int32_t own0, own_shift;   // the own unit's first block in the AttSrc array, log2 of a block's rows
  int32_t pre0, pre_shift;   // the prefix unit's (no prefix: pre0 < 0)
  int32_t pre_row;           // row 0 of the request among the prefix unit's rows
  int32_t flags;
  int32_t req, n_pages;      // the request's own cache
};

// Everything a kernel needs besides its plan.
struct AttArgs {
  const uint8_t* pool;
  size_t int4_off, int3_off, fp4_off;
  int64_t n2, n3b, nfb;          // first INT4, INT3 and FP4 page id
  const Entry* table;
  const uint32_t* hdead;         // null: no slot is excluded for a kv head
  const uint16_t *fpk, *fpv;     // full-precision lists [request][kv head][fp_cap][128], see att_list_at
  const uint16_t *q, *k, *v;     // new tokens, bf16; k and v null: the rows see the cache only
  const uint64_t* tree;          // null: causal
  const int32_t* tok_map;        // rows of q of units whose tokens do not lie together (AttUnit::map)
  uint16_t* out;                 // bf16
  uint32_t* status;
  float scale_log2;
  int32_t max_pages, hkv, hq, fp_cap;
};

// A page's width class and block address.
enum : int { kClsInt2 = 0, kClsInt4 = 1, kClsInt3 = 2, kClsFp4 = 3 };
#ifdef __CUDACC__
__device__ __forceinline__ int att_page(const AttArgs& A, int32_t id, int32_t kvh, const uint8_t*& blk) {
  if (id < A.n2) {
    blk = A.pool + ((size_t)id * A.hkv + kvh) * kInt2Block;
    return kClsInt2;
  }
  if (id < A.n3b) {
    blk = A.pool + A.int4_off + ((size_t)(id - A.n2) * A.hkv + kvh) * kInt4Block;
    return kClsInt4;
  }
  if (id < A.nfb) {
    blk = A.pool + A.int3_off + ((size_t)(id - A.n3b) * A.hkv + kvh) * kInt3Block;
    return kClsInt3;
  }
  blk = A.pool + A.fp4_off + ((size_t)(id - A.nfb) * A.hkv + kvh) * kFp4Block;
  return kClsFp4;
}
// 1 / l of a row with maximum m and sum l.  A row that saw nothing (m = -inf, l = 0)
// is 0, a NaN stays one.  A maximum without a sum: the greatest logit is past
// fp32's range (above: every weight is 2^(x - inf) = 0; below, where it is held at a
// lowest value: every weight is 0 too), and the row is not a number.
__device__ __forceinline__ float row_inverse(float m, float l) {
  return l > 0.0f ? 1.0f / l : (l == 0.0f && m == -INFINITY ? 0.0f : __int_as_float(0x7FFFFFFF));
}
// Offset of channel c in list row t: the 8-channel pieces of a row are stored
// in the order piece ^ (t & 7).
__device__ __forceinline__ int att_list_at(int t, int c) { return (((c >> 3) ^ (t & 7)) << 3) | (c & 7); }
#endif

// CUDA-core kernel (kvq_attend_simt.cu): every unit's rows in blocks of 32.
cudaError_t launch_attend_simt(kv_pool* P, const AttArgs& A, const AttUnit* d_units, int n_units, int max_rows,
                               cudaStream_t s);

// Tensor-core kernel for few rows per unit (kvq_attend_few.cu): blocks of `rows`
// (16, 32 or 64) rows, one partial of that many rows per item.  chain: launched so that the stream's next
// kernel may start as this one's CTAs leave (kChainNext), or as the one before it does so (kChainPrev: this
// launch must not read what that kernel writes); a kernel that follows either with griddepcontrol.wait, or
// plainly, starts when both are done.
enum : int { kChainNext = 1, kChainPrev = 2 };
cudaError_t launch_attend_few(kv_pool* P, int rows, const AttArgs& A, const AttUnit* d_units, const AttItem* d_items,
                              const int32_t* d_cta_item, int n_ctas, float* d_part, cudaStream_t s, int chain = 0);

// Tensor-core kernels for many rows per unit (kvq_attend_wide.cu): the units' keys
// as operand tiles (64 KB and four live words per 128 keys), then blocks of 256
// rows over them.  Partials of 128 rows, two per item (rows 0..127 and 128..255):
// [channels / 4][row][4], then (m, l) [row].
constexpr size_t kAttTileBytes = 65536;
cudaError_t launch_attend_tiles(kv_pool* P, const AttArgs& A, const AttUnit* d_units, int n_units, int max_tiles,
                                void* d_tiles, uint32_t* d_live, cudaStream_t s);
cudaError_t launch_attend_wide(kv_pool* P, const AttArgs& A, const AttUnit* d_units, const AttItem* d_items,
                               const int32_t* d_cta_item, int n_ctas, const void* d_tiles, const uint32_t* d_live,
                               float* d_part, cudaStream_t s);

}  // namespace kvq
