// Appends whose host allocations fail, one after the other, on the CUDA runtime of pool_host.cpp: a call that says
// KV_ERR_OOM leaves the pool as it was, and the same call made again gives what it gives on a pool that never failed.
// argv[1]: the scenario; argv[2]: once (one allocation fails) or on (it and all that follow); exit 0 if it holds.
#include <new>

namespace {
long countdown = -1;   // allocations until one fails (-1: none fails)
bool stays = false;    // those after it fail too
long failed = 0;
}  // namespace

#include <cstdlib>

void* operator new(std::size_t n) {
  if (countdown >= 0 && (countdown == 0 || --countdown == 0)) {
    if (!stays) countdown = -1;
    ++failed;
    throw std::bad_alloc();
  }
  if (void* p = std::malloc(n ? n : 1)) return p;
  throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

#define main pool_host_main
#include "pool_host.cpp"
#undef main
#include "kvq_host.h"

namespace {

// Everything of the pool's host side that a later call goes by.
struct State {
  std::vector<std::vector<int32_t>> table, tails;
  std::vector<std::vector<uint32_t>> loc;
  std::vector<uint64_t> version;
  std::vector<uint8_t> fill;
  std::vector<uint32_t> live, hdead;
  std::vector<std::vector<int32_t>> free, pos;
  std::vector<int32_t> call_slot, page_job;
  bool operator==(const State& o) const {
    return table == o.table && tails == o.tails && loc == o.loc && version == o.version && fill == o.fill && live == o.live &&
           hdead == o.hdead && free == o.free && pos == o.pos && call_slot == o.call_slot && page_job == o.page_job;
  }
};
State state_of(const kv_pool* P) {
  State s;
  for (const auto& R : P->reqs) {
    s.table.push_back(R.table);
    s.tails.push_back({R.tail4, R.tail3, R.tailf, R.staging, R.open, R.dropped});
    s.loc.emplace_back(R.loc.begin(), R.loc.end());
    s.version.push_back(R.version);
  }
  s.fill = P->fill;
  s.live = P->live;
  s.hdead = P->hdead;
  for (const kvq::FreeIds* f : {&P->free2, &P->free4, &P->free3, &P->freef}) {
    kvq::FreeIds x = *f;
    s.free.emplace_back();
    while (!x.empty()) s.free.back().push_back(x.take_lowest());
  }
  for (size_t id = 0; id < P->fill.size(); ++id)   // of slots that hold a token
    s.pos.emplace_back(P->pos.begin() + 32 * id, P->pos.begin() + 32 * id + P->fill[id]);
  for (const auto& v : {P->call_slot, P->page_job})
    for (int32_t x : v) CHECK(x == -1);
  return s;
}

struct Call {
  std::vector<int32_t> ids;
  std::vector<uint8_t> bits;
};
kv_status_t append(kv_pool_t* P, const Call& c, int off = 0) {
  return kv_append_quant(P, rows.data() + off, rows.data() + off, c.ids.data(), c.bits.data(), (int64_t)c.ids.size(), nullptr);
}

// A pool of two to four requests with open tails and staging pages, slots excluded for a head, positions kept on the
// device.
kv_pool_t* begin(int n_req, bool heads, bool positions) {
  kv_pool_config_t c = {};
  c.num_kv_heads = 2;
  c.head_dim = 128;
  c.page_tokens = c.group = 32;
  c.n_int2_pages = c.n_int4_pages = c.n_int3_pages = c.n_fp4_pages = 100;
  c.max_requests = n_req;
  c.max_pages_per_request = 64;
  kv_pool_t* P = nullptr;
  CHECK(kv_pool_create(&c, &P) == KV_OK);
  const uint8_t w[4] = {2, 4, 3, KV_WIDTH_FP4};
  for (int r = 0; r < n_req; ++r) {
    int32_t id;
    CHECK(kv_request_open(P, &id) == KV_OK);
    Call a;
    for (int t = 0; t < 90 + 7 * r; ++t) {
      a.ids.push_back(id);
      a.bits.push_back(w[(t * 7 + t / 5) % (r % 2 ? 4 : 2)]);
    }
    CHECK(append(P, a) == KV_OK);
    if (heads) {
      const int32_t ids[3] = {id, id, id}, h[3] = {0, 1, 1};
      const int64_t n = (int64_t)P->reqs[(size_t)id].loc.size(), pos[3] = {n - 1, n - 2, 3};
      CHECK(kv_evict_slots_head(P, ids, pos, h, 3, nullptr) == KV_OK);
    }
  }
  CHECK(kvq::ensure(P->upload, 1 << 20) == KV_OK);   // the runtime here allocates for itself too
  if (positions) CHECK(cudaMalloc((void**)&P->d_pos, P->fill.size() * 32 * sizeof(int32_t)) == cudaSuccess);
  return P;
}

void failing(int n_req, bool heads, bool positions, const std::vector<Call>& calls, int off) {
  kv_pool_t *P = begin(n_req, heads, positions), *Q = begin(n_req, heads, positions);
  CHECK(state_of(P) == state_of(Q));
  for (const Call& c : calls) {
    long points = 0;
    for (long n = 1;; ++n) {
      const State before = state_of(P);
      const long f0 = failed;
      countdown = n;
      const kv_status_t st = append(P, c, off);
      countdown = -1;
      if (st == KV_OK) {
        if (failed == f0) break;   // every allocation of the call has had its turn
        // one that the call can do without failed: the call is done, and so is the pool's part in this
        CHECK(append(Q, c, off) == KV_OK && state_of(P) == state_of(Q));
        continue;
      }
      ++points;
      CHECK(st == KV_ERR_OOM);
      CHECK(std::strstr(kv_last_error(), "host allocation failed") != nullptr);
      CHECK(state_of(P) == before);
    }
    CHECK(points > 3);
    CHECK(append(Q, c, off) == KV_OK);
    CHECK(state_of(P) == state_of(Q));
  }
  CHECK(kv_pool_destroy(P) == KV_OK && kv_pool_destroy(Q) == KV_OK && live.empty());
}
}  // namespace

int main(int, char** v) {
  const std::string what = v[1];
  stays = std::string(v[2]) == "on";
  std::vector<Call> calls;
  auto call = [&](int n, auto id, auto width) {
    Call c;
    for (int t = 0; t < n; ++t) {
      c.ids.push_back(id(t));
      c.bits.push_back((uint8_t)width(t));
    }
    calls.push_back(c);
  };
  auto two = [](int t) { return (t * 5 + t / 3) % 3 ? 2 : 4; };
  auto four = [](int t) { const int w[4] = {2, 4, 3, KV_WIDTH_FP4}; return w[(t * 5 + t / 3) % 4]; };
  if (what == "runs") {            // prompts: a run of tokens per request
    call(400, [](int t) { return t / 200; }, two);
    call(64, [](int t) { return 1 - t / 32; }, [](int) { return 2; });
    call(200, [](int) { return 0; }, [](int t) { return t < 90 ? 2 : 4; });
  } else if (what == "small") {    // a decode step, and a few tokens of every width
    call(4, [](int t) { return t; }, [](int) { return 4; });
    call(12, [](int t) { return t % 4; }, four);
    call(40, [](int t) { return t % 4; }, two);
  } else if (what == "mixed") {    // token by token, whole INT2 groups among them
    call(500, [](int t) { return t % 3; }, two);
    call(300, [](int t) { return (t / 2) % 4; }, four);
  } else {
    return 2;
  }
  const int n_req = what == "runs" ? 2 : 4;
  for (int y = 0; y < 8; ++y) failing(n_req, y & 1, (y & 2) != 0, calls, y & 4 ? 1 : 0);
  return 0;
}
