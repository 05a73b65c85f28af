// Launchers of the tensor-core split decode (the kernels are in
// kvq_scan_mma.cuh).
#include "kvq_scan_mma.cuh"

namespace kvq {
namespace {

template <int G>
cudaError_t launch_mma_g(kv_pool* P, const void* q, int32_t hq, float scale_log2, const Unit* d_units, int n_units,
                         const Split* d_splits, const int32_t* d_wsplit, int n_workers, void* d_frags, float* d_part,
                         cudaStream_t s, const GroupPool* d_gpools, bool groups_extra, bool in_place) {
  // function attributes are set once per device (bit = device ordinal)
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(attr_set.load() >> dev & 1u)) {
    cudaError_t e = set_scan_attributes<G, false, false, false>();
    if (e == cudaSuccess) e = set_scan_attributes<G, true, false, false>();
    if (e == cudaSuccess) e = set_scan_attributes<G, false, true, false>();
    if (e == cudaSuccess) e = set_scan_attributes<G, false, false, true>();
    if (e == cudaSuccess) e = set_scan_attributes<G, true, false, true>();
    if (e == cudaSuccess) e = set_scan_attributes<G, false, true, true>();
    if (e != cudaSuccess) return e;
    attr_set.fetch_or(uint64_t(1) << dev);
  }
  if (n_workers <= 0 || n_units <= 0) return cudaSuccess;
  const uint32_t* smax = P->d_status + 1;
  P->launches += 2;
  cudaError_t e = launch_pdl(in_place ? frag_kernel<G, true> : frag_kernel<G, false>, dim3((unsigned)n_units), dim3(256), 0, s, (const __nv_bfloat16*)q,
                             (int)hq, scale_log2, d_units, smax, (UnitFrag*)d_frags, d_gpools);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((n_workers + kWarps - 1) / kWarps);
  // pools with INT3 or FP4 pages take the variant that reads them (grouped
  // decodes take no such pool)
  const bool i3 = P->cfg.n_int3_pages > 0 || P->cfg.n_fp4_pages > 0;
  auto* kernel = d_gpools ? (groups_extra ? decode_mma_kernel<G, false, true, true>
                                          : decode_mma_kernel<G, false, true, false>)
                 : i3     ? (P->hdead.empty() ? decode_mma_kernel<G, false, false, true>
                                              : decode_mma_kernel<G, true, false, true>)
                          : (P->hdead.empty() ? decode_mma_kernel<G, false, false, false>
                                              : decode_mma_kernel<G, true, false, false>);
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), (size_t)kScanSmem, s, (const uint8_t*)P->d_pool,
                    P->int4_offset, (int64_t)P->cfg.n_int2_pages, P->cfg.num_kv_heads, P->cfg.max_pages_per_request,
                    (const Entry*)P->d_table, (const UnitFrag*)d_frags, d_splits, d_wsplit, n_workers,
                    (const int32_t*)P->d_ntab, (const uint32_t*)P->d_hdead, d_part, smax, P->d_status,
                    P->first_wait_spins < 0 ? kSpinLimit : (uint32_t)P->first_wait_spins, d_gpools, P->int3_offset,
                    (int64_t)(P->cfg.n_int2_pages + P->cfg.n_int4_pages), P->fp4_offset,
                    (int64_t)(P->cfg.n_int2_pages + P->cfg.n_int4_pages + P->cfg.n_int3_pages), (float*)nullptr);
}

template <int G>
int mma_occupancy() {
  int n = 0;
  if (set_scan_attributes<G, false, false, false>() != cudaSuccess) return 1;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, decode_mma_kernel<G, false, false, false>, kThreads,
                                                    kScanSmem) != cudaSuccess)
    return 1;
  return n > 0 ? n : 1;
}

}  // namespace

size_t decode_mma_frag_bytes() { return sizeof(UnitFrag); }

static cudaError_t launch_scan(kv_pool* P, int g, const void* q, int32_t hq, float scale_log2, const Unit* d_units, int n_units,
                               const Split* d_splits, const int32_t* d_wsplit, int n_workers, void* d_frags, float* d_part,
                               cudaStream_t s, const GroupPool* d_gpools, bool groups_extra, bool in_place) {
#define KVQ_MMA_CASE(gg)                                                                                              \
  case gg:                                                                                                            \
    return launch_mma_g<gg>(P, q, hq, scale_log2, d_units, n_units, d_splits, d_wsplit, n_workers, d_frags, d_part, s, \
                            d_gpools, groups_extra, in_place);
  switch (g) {
    KVQ_MMA_CASE(1)
    KVQ_MMA_CASE(2)
    KVQ_MMA_CASE(3)
    KVQ_MMA_CASE(4)
    KVQ_MMA_CASE(5)
    KVQ_MMA_CASE(6)
    KVQ_MMA_CASE(7)
    KVQ_MMA_CASE(8)
    default: return cudaErrorInvalidValue;
  }
#undef KVQ_MMA_CASE
}

cudaError_t launch_scan_mma(kv_pool* P, const void* q, int32_t hq, float scale_log2, const Unit* d_units, int n_units,
                            const Split* d_splits, const int32_t* d_wsplit, int n_workers, void* d_frags, float* d_part,
                            cudaStream_t s) {
  return launch_scan(P, hq / P->cfg.num_kv_heads, q, hq, scale_log2, d_units, n_units, d_splits, d_wsplit, n_workers, d_frags,
                     d_part, s, nullptr, false, true);
}

cudaError_t launch_decode_mma(kv_pool* P, const void* q, int32_t hq, float scale_log2, const Unit* d_units, int n_units,
                              const Split* d_splits, const int32_t* d_wsplit, int n_workers, void* d_frags,
                              float* d_part, float* out, cudaStream_t s, const GroupPool* d_gpools,
                              int32_t total_kv_heads, bool groups_extra) {
  const int g = hq / (total_kv_heads > 0 ? total_kv_heads : P->cfg.num_kv_heads);
  cudaError_t e = launch_scan(P, g, q, hq, scale_log2, d_units, n_units, d_splits, d_wsplit, n_workers, d_frags, d_part, s,
                              d_gpools, groups_extra, false);
  if (e != cudaSuccess) return e;
  if ((e = launch_fp_pending(P, q, hq, scale_log2, d_units, d_part, s)) != cudaSuccess) return e;
  if (P->merge_event && (e = cudaEventRecord(P->merge_event, s)) != cudaSuccess) return e;
  return launch_merge(P, g, d_units, n_units, d_part, hq, out, s);
}

int decode_mma_workers_per_sm(int g) {
  switch (g) {
    case 1: return kWarps * mma_occupancy<1>();
    case 2: return kWarps * mma_occupancy<2>();
    case 3: return kWarps * mma_occupancy<3>();
    case 4: return kWarps * mma_occupancy<4>();
    case 5: return kWarps * mma_occupancy<5>();
    case 6: return kWarps * mma_occupancy<6>();
    case 7: return kWarps * mma_occupancy<7>();
    default: return kWarps * mma_occupancy<8>();
  }
}

}  // namespace kvq

