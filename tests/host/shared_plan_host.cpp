// The plan of a decode step over shared prefixes beside that of the decode, on the CUDA runtime of pool_host.cpp:
// neither moves or frees the other's.  Exit 0 if it holds.
#define main pool_host_main
#include "pool_host.cpp"
#undef main
#include "kvq_host.h"

int main() {
  kv_pool_t* P = pool_of(64, 640);
  std::vector<int32_t> ids;
  for (int r = 0; r < 64; ++r) ids.push_back(r);
  CHECK(kv_decode_attn(P, rows.data(), ids.data(), 2, 4, 1.0f, out, nullptr) == KV_OK);
  const void *plan = P->plan.buf.ptr, *partials = P->partials.ptr, *frags = P->frags.ptr;
  const size_t bytes = P->plan.n_units * sizeof(kvq::Unit);
  std::vector<uint8_t> units((const uint8_t*)plan, (const uint8_t*)plan + bytes);
  int64_t b0, p0, b1, p1;
  int32_t s0, s1;
  CHECK(kv_last_decode_stats(P, &b0, &s0, &p0) == KV_OK);
  for (int batch : {64, 3, 17}) {
    CHECK(kvq::build_plan(P, P->shared_plan, ids.data(), batch, 4, KV_DECODE_MMA, nullptr) == KV_OK);
    CHECK(P->shared_plan.n_units == 2 * batch && P->shared_plan.buf.ptr != plan);
    CHECK(P->plan.buf.ptr == plan && P->partials.ptr == partials && P->frags.ptr == frags);
    CHECK(std::memcmp(plan, units.data(), bytes) == 0);
    CHECK(kv_last_decode_stats(P, &b1, &s1, &p1) == KV_OK && b0 == b1 && s0 == s1 && p0 == p1);
    const int before = (int)P->shared_plan.n_splits;
    CHECK(kv_decode_attn(P, rows.data(), ids.data(), 2, 4, 1.0f, out, nullptr) == KV_OK && stale == 0);
    CHECK(P->shared_plan.n_splits == before);
  }
  CHECK(kv_pool_destroy(P) == KV_OK && live.empty());
  return 0;
}
