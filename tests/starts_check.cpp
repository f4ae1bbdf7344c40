// CPU check of the search that finds the documents around one token of cu_seqlens by
// one thread (varlen_depthwise_causal_amd/csrc/vdc_search.h): against a scan of all
// documents for sorted contents, and inside [0, n) with documents that exist for
// contents in no order.  cu is a function of the index, so that 2^31 - 4095 entries need
// no memory.  Prints "starts_check: ok" and exits 0, or names the failing case.
#include <stdint.h>
#include <stdio.h>

#include <functional>
#include <vector>

#include "vdc_search.h"

namespace {

int failures = 0;
typedef std::function<int32_t(int64_t)> At;

struct Probed {
  const At& at;
  int64_t n;
  bool* inside;
  int* count;
  int32_t operator()(int64_t i) const {
    ++*count;
    if (i < 0 || i >= n) {
      *inside = false;
      return 0;
    }
    return at(i);
  }
};

vdc::TokenDocs find(const char* what, const At& at, int64_t n, int64_t v) {
  bool inside = true;
  int count = 0;
  const vdc::TokenDocs d = vdc::token_docs(Probed{at, n, &inside, &count}, n, v);
  const bool ok = inside && count <= 64 && d.ends >= -1 && d.ends < n - 1 && d.starts >= -1 && d.starts < n - 1;
  if (!ok) {
    ++failures;
    printf("FAIL %s: n=%lld v=%lld ends=%lld starts=%lld probes=%d inside=%d\n", what, (long long)n, (long long)v,
           (long long)d.ends, (long long)d.starts, count, (int)inside);
  }
  return d;
}

void scan(const char* what, const std::vector<int32_t>& cu) {
  const int64_t n = (int64_t)cu.size();
  for (int64_t v = 0; v <= (int64_t)cu.back() + 1; ++v) {
    int64_t ends = -1, starts = -1;
    bool any = false;
    for (int64_t d = 0; d < n; ++d) {
      any |= cu[d] == v;
      if (d + 1 == n || cu[d] == cu[d + 1]) continue;  // an empty document
      if (cu[d + 1] == v) ends = d;
      if (cu[d] == v) starts = d;
    }
    const vdc::TokenDocs got = find(what, [&](int64_t i) { return cu[i]; }, n, v);
    // the token of the first documents: none ends there
    if (got.any != any || got.starts != starts || got.ends != ends) {
      ++failures;
      printf("FAIL %s: v=%lld any=%d/%d starts=%lld/%lld ends=%lld/%lld\n", what, (long long)v, got.any, any,
             (long long)got.starts, (long long)starts, (long long)got.ends, (long long)ends);
    }
  }
}

}  // namespace

int main() {
  scan("one", {0, 5});
  scan("none", {0});
  scan("empty ones", {0, 0, 0, 3, 3, 3, 3, 9, 10, 10});
  uint64_t seed = 7;
  for (int rep = 0; rep < 200; ++rep) {
    std::vector<int32_t> cu = {0};
    for (int k = 0; k < 60; ++k) {
      seed = seed * 6364136223846793005ull + 1442695040888963407ull;
      const int draw = (int)(seed >> 60);
      cu.push_back(cu.back() + (draw < 9 ? 0 : draw - 8));
    }
    scan("random", cu);
  }
  const int64_t most = (int64_t(1) << 31) - 4095;
  for (int64_t n : {int64_t(20001), int64_t(1) << 28, most}) {
    // a document of 150 tokens, empty ones, and one of 150 tokens more
    const At at = [n](int64_t i) { return i == 0 ? 0 : i == n - 1 ? 300 : 150; };
    const vdc::TokenDocs d = find("many", at, n, 150);
    if (d.ends != 0 || d.starts != n - 2 || !d.any) ++failures, printf("FAIL many: n=%lld\n", (long long)n);
    const vdc::TokenDocs last = find("many", at, n, 300);
    if (last.ends != n - 2 || last.starts != -1) ++failures, printf("FAIL the last: n=%lld\n", (long long)n);
    const vdc::TokenDocs none = find("many", at, n, 151);
    if (none.any) ++failures, printf("FAIL no entry: n=%lld\n", (long long)n);
    for (uint64_t k = 0; k < 8; ++k) {
      const At junk = [k](int64_t i) { return (int32_t)(((uint64_t)i + k) * 0x9e3779b97f4a7c15ull >> 33) - (1 << 30); };
      for (int64_t v : {int64_t(0), int64_t(150), int64_t(1) << 30, (int64_t(1) << 31) - 1}) {
        find("malformed", junk, n, v);
        find("malformed", [&](int64_t i) { return i % 3 ? (int32_t)v : -5; }, n, v);
      }
    }
  }
  if (failures) {
    printf("starts_check: %d failures\n", failures);
    return 1;
  }
  printf("starts_check: ok\n");
  return 0;
}
