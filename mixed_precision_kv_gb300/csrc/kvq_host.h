// Host helpers shared by the translation units that implement the C ABI:
// errors, the device guard, growing device buffers, pinned uploads, stream
// order and the cached decode plan.
#pragma once
#include <cuda_runtime.h>

#include "kvq_internal.h"

namespace kvq {

// Record a message for kv_last_error() on this thread and return `st`.
kv_status_t fail(kv_status_t st, const char* fmt, ...);

#define KV_CUDA(call)                                                                       \
  do {                                                                                      \
    cudaError_t e_ = (call);                                                                \
    if (e_ != cudaSuccess) return fail(KV_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_)); \
  } while (0)

// Makes the pool's device current for the duration of a call.
struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) ok = cudaSetDevice(dev) == cudaSuccess;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

inline bool req_ok(const kv_pool* P, int32_t r) { return r >= 0 && r < P->cfg.max_requests && P->reqs[r].open; }

// Grow a device buffer to at least `bytes` (contents are not kept), as grow() in
// kvq_grow.h says.  KV_ERR_OOM if there is no memory for it; the buffer is then empty.
kv_status_t ensure(DevBuf& b, size_t bytes, size_t most = SIZE_MAX);

// Several host arrays laid out for one upload (one H2D copy per call); the
// arrays are copied straight into the pinned staging buffer by h2d (they must
// stay alive until then).
struct Upload {
  struct Piece {
    const void* p;
    size_t n, off;
  };
  static constexpr int kMaxPieces = 8;
  Piece pieces[kMaxPieces];
  int n_pieces = 0;
  size_t size = 0;
  size_t add(const void* p, size_t n) {   // byte offset of the array in the upload
    const size_t off = (size + 255) & ~size_t(255);
    pieces[n_pieces++] = Piece{p, n, off};
    size = off + n;
    return off;
  }
};

// Host-to-device copy through a pinned staging slot.
kv_status_t h2d(kv_pool* P, void* dst, const Upload& u, cudaStream_t s);
// ... into the pool's upload buffer.
kv_status_t upload(kv_pool* P, const Upload& u, cudaStream_t s);

// Order this call after the pool's previous work when the stream changes.
kv_status_t order_after_previous(kv_pool* P, cudaStream_t s);

// KV_ERR_STATE if `s` is being captured into a graph: calls that plan on the
// host cannot be replayed (kvq_select.cu).
kv_status_t refuse_capture(const char* what, cudaStream_t s);

// Bring the slots' token positions on the device (P->d_pos) up to date.
kv_status_t sync_positions(kv_pool* P, cudaStream_t s);

// The split plan of a decode over a batch, on the device (kept while it fits).
kv_status_t build_plan(kv_pool* P, const int32_t* req_ids, int32_t batch, int32_t hq, int32_t impl, cudaStream_t s);

}  // namespace kvq
