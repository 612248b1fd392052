// The launches of more requests than one has threads for (test_attention_launches.py):
// together every request once, each with its own arguments, up to the most requests that
// a call may have.  Addresses are numbers here; nothing is read.
#include <cstdio>
#include <cstdlib>

#include "attention_plan.hpp"

using namespace fp4attn;

#define REQUIRE(ok)                                                                                      \
  do {                                                                                                   \
    if (!(ok)) {                                                                                         \
      std::printf("%s: %d requests, heads %d on %d, from %lld\n", #ok, requests, heads * group, heads,   \
                  (long long)next);                                                                      \
      std::exit(1);                                                                                      \
    }                                                                                                    \
  } while (0)

namespace {

int64_t launches = 0;

void check(int requests, int heads, int group, int forced, int width) {
  int64_t next = 0;
  fp4lib::AttnArgs a{};
  a.cache.heads = heads;
  a.cache.head_dim = 64;
  a.cache.fmt = fp4lib::kKvMx4;
  a.cache.page_shift = 4;
  a.q = {reinterpret_cast<uint16_t*>(int64_t(1) << 40), 64 * heads * group, 64, heads * group};
  a.requests = requests;
  a.table_width = width;
  a.table_stride = width;
  a.table = reinterpret_cast<const int32_t*>(int64_t(1) << 41);
  a.lens = reinterpret_cast<const int32_t*>(int64_t(1) << 42);
  a.out = reinterpret_cast<void*>(int64_t(1) << 43);
  a.lse = reinterpret_cast<float*>(int64_t(1) << 44);
  plan(a, 256, forced);
  const int splits = a.splits;
  const hipError_t e = by_launches(a, [&](const fp4lib::AttnArgs& some) {
    REQUIRE(some.requests >= 1 && next + some.requests <= requests && some.splits == splits);
    REQUIRE(some.planned || some.items == int64_t(some.requests) * splits);
    REQUIRE(some.items * heads * some.tiles < (int64_t(1) << 22) + 8 * some.tiles || some.requests == 1);
    REQUIRE(some.q.x - a.q.x == next * 64 * heads * group && some.table - a.table == next * width);
    REQUIRE(some.lens - a.lens == next && some.lse - a.lse == next * heads * group);
    REQUIRE(static_cast<uint8_t*>(some.out) - static_cast<uint8_t*>(a.out) == next * 128 * heads * group);
    next += some.requests;
    ++launches;
    return hipSuccess;
  });
  REQUIRE(e == hipSuccess && next == requests);
}

}  // namespace

int main() {
  check(1, 8, 4, 0, 100);
  check(200, 8, 4, 0, 1000);
  check((1 << 22) + 5, 1, 1, 0, 4);
  check((1 << 21) + 3, 1, 20, 1, 2);
  check(1030, 8, 1, 512, 8192);
  check(5000, 1024, 1, 0, 50);
  check(5000, 1, 1024, 0, 50);
  check((1 << 30) - 1, 1, 2, 0, 1);
  check(2147483647, 1, 1, 0, 1);           // as many rows of output as there may be
  std::printf("%lld\n", (long long)launches);
  return 0;
}
