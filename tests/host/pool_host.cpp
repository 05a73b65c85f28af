// The pool's host side (csrc/kvq_pool.cu, which holds no kernels) on a CUDA runtime of this
// file's own: "device" memory is host memory with a limit, launches check the pointers they
// get.  argv[1]: the scenario; exit 0 if it holds.
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>
#include <vector>

#include "kvq_internal.h"

namespace {
std::map<uint8_t*, size_t> live;   // allocations
size_t most = SIZE_MAX;            // bytes of one allocation at most
int waits = 0, launches = 0, stale = 0;
cudaStream_t capturing = nullptr;

bool inside(const void* p, size_t n) {
  const uint8_t* q = (const uint8_t*)p;
  auto it = live.upper_bound((uint8_t*)q);
  if (it == live.begin()) return false;
  --it;
  return q + n <= it->first + it->second;
}
#define CHECK(x)                                              \
  do {                                                        \
    if (!(x)) {                                               \
      std::printf("line %d: %s (%s)\n", __LINE__, #x, kv_last_error()); \
      std::exit(1);                                           \
    }                                                         \
  } while (0)
}  // namespace

extern "C" {
cudaError_t cudaMalloc(void** p, size_t n) {
  if (n > most) return cudaErrorMemoryAllocation;
  *p = std::calloc(n ? n : 1, 1);
  live[(uint8_t*)*p] = n;
  return cudaSuccess;
}
cudaError_t cudaFree(void* p) {
  if (p) {
    CHECK(live.erase((uint8_t*)p) == 1);
    std::free(p);
  }
  return cudaSuccess;
}
cudaError_t cudaMallocHost(void** p, size_t n) { return (*p = std::malloc(n)) ? cudaSuccess : cudaErrorMemoryAllocation; }
cudaError_t cudaFreeHost(void* p) { return std::free(p), cudaSuccess; }
cudaError_t cudaMemcpy(void* d, const void* s, size_t n, cudaMemcpyKind) { return std::memcpy(d, s, n), cudaSuccess; }
cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, cudaMemcpyKind, cudaStream_t) {
  CHECK(inside(d, n));
  return std::memcpy(d, s, n), cudaSuccess;
}
cudaError_t cudaMemset(void* d, int v, size_t n) { return std::memset(d, v, n), cudaSuccess; }
cudaError_t cudaMemsetAsync(void* d, int v, size_t n, cudaStream_t) { return std::memset(d, v, n), cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { return *v = 152, cudaSuccess; }
cudaError_t cudaGetDeviceCount(int* n) { return *n = 1, cudaSuccess; }
cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "an error"; }
cudaError_t cudaEventCreate(cudaEvent_t* e) { return *e = (cudaEvent_t)1, cudaSuccess; }
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) { return *e = (cudaEvent_t)1, cudaSuccess; }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventElapsedTime(float* t, cudaEvent_t, cudaEvent_t) { return *t = 0.0f, cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t s, cudaStreamCaptureStatus* c) {
  *c = s && s == capturing ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
  return cudaSuccess;
}
cudaError_t cudaStreamWaitEvent(cudaStream_t s, cudaEvent_t, unsigned) {
  ++waits;
  return s && s == capturing ? cudaErrorStreamCaptureIsolation : cudaSuccess;
}
}  // extern "C"

namespace kvq {
cudaError_t launch_append(kv_pool*, const void*, const void*, const AppendJob*, int, const int32_t*, const SmallAppend*,
                          cudaStream_t) { return cudaSuccess; }
cudaError_t launch_bulk_int4(kv_pool*, const void*, const void*, const AppendJob*, int, const int32_t*, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_bulk_int2(kv_pool*, const void*, const void*, const DirectJob*, int, const int32_t*, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_append_int3(kv_pool*, const void*, const void*, const AppendJob*, int, const int32_t*, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_append_fp4(kv_pool*, const void*, const void*, const AppendJob*, int, const int32_t*, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_direct_int2(kv_pool*, const void*, const void*, const DirectJob*, int, const int32_t*, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_repack(kv_pool*, const RepackJob*, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_scatter(kv_pool*, const TableUpd*, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_fp_store(kv_pool*, const void*, const void*, int64_t, const int32_t*, const int32_t*, const int32_t*,
                            const int32_t*, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_fp_move(kv_pool*, int32_t, int32_t, int32_t, int32_t, int32_t, cudaStream_t) { return cudaSuccess; }
int fp_workers(const kv_pool*) { return 152; }
int decode_mma_workers_per_sm(int) { return 16; }
int decode_simt_ctas_per_sm(int) { return 2; }
size_t decode_mma_frag_bytes() { return 4096; }
cudaError_t launch_decode_mma(kv_pool*, const void*, int32_t, float, const Unit* units, int n_units, const Split* splits,
                              const int32_t*, int, void*, float*, float*, cudaStream_t, const GroupPool*, int32_t, bool) {
  ++launches;
  // the plan it is given is there
  if (!inside(units, n_units * sizeof(Unit)) || !inside(splits, sizeof(Split))) ++stale;
  return cudaSuccess;
}
cudaError_t launch_decode_simt(kv_pool* P, const void* q, int32_t hq, float s, const Unit* units, int n_units,
                               const Split* splits, const int32_t* c, int n, float* p, float* out, cudaStream_t st) {
  return launch_decode_mma(P, q, hq, s, units, n_units, splits, c, n, nullptr, p, out, st, nullptr, 0, false);
}
}  // namespace kvq

namespace {
std::vector<uint16_t> rows(1 << 20);
float out[1 << 16];

kv_pool_t* pool_of(int n_req, int tokens) {
  kv_pool_config_t c = {};
  c.num_kv_heads = 2;
  c.head_dim = 128;
  c.page_tokens = c.group = 32;
  c.n_int2_pages = 64;
  c.n_int4_pages = 4096;
  c.max_requests = n_req;
  c.max_pages_per_request = 64;
  kv_pool_t* P = nullptr;
  CHECK(kv_pool_create(&c, &P) == KV_OK);
  std::vector<int32_t> ids((size_t)tokens);
  std::vector<uint8_t> bits((size_t)tokens, 4);
  for (int r = 0; r < n_req; ++r) {
    int32_t id;
    CHECK(kv_request_open(P, &id) == KV_OK && id == r);
    std::fill(ids.begin(), ids.end(), id);
    CHECK(kv_append_quant(P, rows.data(), rows.data(), ids.data(), bits.data(), tokens, nullptr) == KV_OK);
  }
  return P;
}

// A larger plan that gets no memory: the smaller one before it is built again.
void plan_without_memory(bool groups) {
  kv_pool_t* P = pool_of(64, 640);
  std::vector<int32_t> ids;
  for (int r = 0; r < 64; ++r) ids.push_back(r);
  auto decode = [&](int batch) {
    return groups ? kv_decode_attn_groups(&P, 1, rows.data(), ids.data(), batch, 4, 1.0f, out, nullptr)
                  : kv_decode_attn(P, rows.data(), ids.data(), batch, 4, 1.0f, out, nullptr);
  };
  CHECK(decode(1) == KV_OK && launches == 1);
  most = 1 << 14;
  CHECK(decode(64) == KV_ERR_OOM && launches == 1);
  most = SIZE_MAX;
  CHECK(decode(1) == KV_OK && launches == 2 && stale == 0);
  CHECK(decode(64) == KV_OK && launches == 3 && stale == 0);
  CHECK(kv_pool_destroy(P) == KV_OK && live.empty());
}

// A stream waits for the pool's work on another, the default one too; a capture does not.
void streams() {
  kv_pool_t* P = pool_of(1, 64);
  const int32_t id = 0;
  cudaStream_t a = (cudaStream_t)8, b = (cudaStream_t)16;
  auto decode = [&](cudaStream_t s) { return kv_decode_attn(P, rows.data(), &id, 1, 4, 1.0f, out, s); };
  CHECK(decode(nullptr) == KV_OK && waits == 0);
  CHECK(decode(a) == KV_OK && waits == 1);
  CHECK(decode(a) == KV_OK && waits == 1);
  CHECK(decode(nullptr) == KV_OK && waits == 2);
  capturing = b;
  CHECK(decode(b) == KV_OK && waits == 2);
  capturing = nullptr;
  CHECK(decode(nullptr) == KV_OK && waits == 2);   // the capture put nothing on b
  CHECK(decode(b) == KV_OK && waits == 3);
  CHECK(kv_pool_destroy(P) == KV_OK && live.empty());
}
}  // namespace

int main(int, char** v) {
  const std::string what = v[1];
  if (what == "plan") plan_without_memory(false);
  else if (what == "groups") plan_without_memory(true);
  else if (what == "streams") streams();
  else return 2;
  return 0;
}
