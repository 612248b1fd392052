// Whatever the lengths, attention's parts are those that the launch and the workspace
// have room for (test_attention_plan.py).  Runs attention_plan.hpp on the CPU: the host's
// plan, and a workgroup's arithmetic on the lengths, over sizes and lengths drawn from the
// whole range (contexts below 2^30 tokens).  Prints what was checked, or stops at a fault.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "attention_plan.hpp"

using namespace fp4attn;

namespace {

std::mt19937_64 rng(1);
int64_t draw(int64_t lo, int64_t hi) { return lo + static_cast<int64_t>(rng() % static_cast<uint64_t>(hi - lo + 1)); }
// spread over the logarithm
int64_t draw_log(int64_t lo, int64_t hi) {
  const double u = std::uniform_real_distribution<double>(std::log(double(lo)), std::log(double(hi) + 1))(rng);
  return std::min(hi, std::max(lo, static_cast<int64_t>(std::exp(u))));
}

#define REQUIRE(ok)                                                                                          \
  do {                                                                                                       \
    if (!(ok)) {                                                                                             \
      std::printf("%s: requests %d, heads %d on %d of %d, width %d of %d, %d CUs, items %lld, splits %d\n", #ok, \
                  a.requests, a.q.heads, a.cache.heads, a.cache.head_dim, a.table_width, 1 << a.cache.page_shift, \
                  int(cu), (long long)a.items, a.splits);                                                    \
      for (size_t i = 0; i < lens.size() && i < 50; ++i) std::printf("%d ", lens[i]);                        \
      std::printf("\n");                                                                                     \
      std::exit(1);                                                                                          \
    }                                                                                                        \
  } while (0)

int64_t planned = 0, even = 0, rejoined = 0, longest_part = 0;

template <int D>
void by_lengths(const fp4lib::AttnArgs& a, const std::vector<int>& lens, int64_t cu) {
  std::vector<int> size;
  uint32_t all = 0;
  for (int n : lens) {
    size.push_back((n + kStep - 1) / kStep);
    all += size.back();
  }
  Shares s = first_shares<D>(all, a);
  auto count_of = [&](int step) {
    int64_t count = 0;
    for (int n : size) count += parts_of(n, step);
    return count;
  };
  if (a.requests > 1) {
    const int64_t count = count_of(s.step);
    REQUIRE(count <= a.items);
    if (count > s.want && a.requests < s.want) {
      const int before = s.step;
      s.step = longer_step(s.step, static_cast<int>(count), s.want);
      REQUIRE(s.step >= before);
      ++rejoined;
    }
  }
  REQUIRE(s.step >= 1);
  int64_t count = 0;
  for (size_t i = 0; i < size.size(); ++i) {
    const int parts = parts_of(size[i], s.step), per = steps_of(size[i], parts);
    REQUIRE(parts == std::max<int64_t>(1, (int64_t(size[i]) + s.step - 1) / s.step));
    REQUIRE(per == (int64_t(size[i]) + parts - 1) / parts);
    REQUIRE(parts <= a.splits && parts <= kMaxParts);
    REQUIRE(int64_t(parts) * per * kStep >= lens[i]);                     // together the whole request
    REQUIRE(int64_t(parts) * per * kStep < (int64_t(1) << 31));           // in 32 bits
    longest_part = std::max<int64_t>(longest_part, int64_t(per) * kStep);
    count += parts;
  }
  REQUIRE(count <= a.items);
  ++planned;
}

void check(fp4lib::AttnArgs a, const std::vector<int>& lens, int64_t cu) {
  plan(a, cu, 0);
  REQUIRE(a.splits >= 1 && a.splits <= kMaxParts && a.items >= a.requests && a.target[0] >= 1 &&
          a.target[1] >= 1 && a.target[1] <= a.target[0]);
  if (a.planned && a.splits > 1) {
    if (a.cache.head_dim == 64) by_lengths<64>(a, lens, cu);
    else if (a.cache.head_dim == 128) by_lengths<128>(a, lens, cu);
    else by_lengths<256>(a, lens, cu);
  } else if (!a.planned) {
    REQUIRE(a.items == int64_t(a.requests) * a.splits);
    for (int n : lens) {
      const int per = part_tokens(n, a);
      REQUIRE(per >= 1 && (int64_t(n) + per - 1) / per <= a.splits);
    }
    ++even;
  } else {
    REQUIRE(a.items == a.requests);
  }
}

fp4lib::AttnArgs sizes(int requests, int heads, int group, int d, int page, int64_t width) {
  fp4lib::AttnArgs a{};
  a.cache.heads = heads;
  a.cache.head_dim = d;
  a.cache.fmt = fp4lib::kKvMx4;
  a.cache.pages = 4;
  while ((1 << a.cache.page_shift) < page) ++a.cache.page_shift;
  a.q.heads = heads * group;
  a.requests = requests;
  a.table_width = static_cast<int>(width);
  return a;
}

// the table as wide as the longest needs, or wider
void alike(int requests, int heads, int group, int d, int64_t n) {
  check(sizes(requests, heads, group, d, 1024, (n + 1023) / 1024), std::vector<int>(requests, static_cast<int>(n)), 256);
}

}  // namespace

int main(int argc, char** argv) {
  const int draws = argc > 1 ? std::atoi(argv[1]) : 1000;
  const int64_t most = (int64_t(1) << 30) - 1024;           // tokens of 2^20 - 1 pages of 1024
  // quotients, with the reciprocal as far off as an instruction may give it
  int64_t quotients = 0;
  for (int i = 0; i < 200 * draws; ++i) {
    const int x = static_cast<int>(i % 2 ? draw_log(1, (1 << 24) - 1) : draw(0, (1 << 24) - 1));
    const int d = static_cast<int>(i % 3 ? draw_log(1, 1 << 23) : draw(1, 1 << 10));
    const float r = 1.0f / static_cast<float>(d);
    const bool exact = !(d & (d - 1));
    for (float by : {r, exact ? r : std::nextafterf(r, 0.0f), exact ? r : std::nextafterf(r, 1.0f)}) {
      if (quotient(x, d, by) != x / d) return std::printf("%d / %d: %d\n", x, d, quotient(x, d, by)), 1;
      ++quotients;
    }
  }
  // long contexts: parts of more than 2^12 steps
  alike(33, 8, 4, 128, 1572864);
  alike(33, 8, 4, 128, 1200000);
  alike(40, 8, 4, 128, 3145728);
  alike(40, 8, 4, 128, 2560000);
  alike(17, 16, 4, 128, 1572864);
  alike(9, 32, 4, 128, 1572864);
  alike(3, 8, 4, 128, 12582912);
  alike(2, 1, 1, 64, most);
  alike(256, 1, 1, 64, most);
  alike(255, 2, 8, 128, most);
  for (int i = 0; i < draws; ++i) {
    const int heads = static_cast<int>(draw_log(1, 1024)), d = 64 << draw(0, 2), page = 16 << draw(0, 6);
    const int group = static_cast<int>(draw_log(1, std::min(1024 / heads, 128)));
    const int requests = static_cast<int>(draw_log(1, i % 4 ? 256 : 2000));
    const int64_t width = draw_log(1, ((int64_t(1) << 30) - 1) / page);
    const int64_t room = width * page, longest = i % 3 ? room : draw_log(1, room);
    const int64_t cu = i % 5 ? 256 : draw_log(1, 304);
    std::vector<int> lens;
    for (int r = 0; r < requests; ++r)
      switch (i % 6) {
        case 0: lens.push_back(static_cast<int>(longest)); break;
        case 1: lens.push_back(static_cast<int>(draw(0, longest))); break;
        case 2: lens.push_back(static_cast<int>(draw_log(1, longest))); break;
        case 3: lens.push_back(r ? 1 : static_cast<int>(longest)); break;
        case 4: lens.push_back(static_cast<int>(r % 2 ? longest : longest / 2 + 1)); break;
        default: lens.push_back(static_cast<int>(std::min(longest, draw_log(1, longest) / kStep * kStep + draw(0, 1))));
      }
    check(sizes(requests, heads, group, d, page, width), lens, cu);
  }
  std::printf("%lld %lld %lld %lld %lld\n", (long long)quotients, (long long)planned, (long long)rejoined,
              (long long)even, (long long)longest_part);
  return 0;
}
