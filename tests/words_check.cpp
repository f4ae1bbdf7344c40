// CPU check of the words that a recurrence's tiles hand on
// (varlen_depthwise_causal_amd/csrc/vdc_words.h): no (P, H) looks like a mark, a fold
// from any known word has the same bits, and a word that a reader waited for in vain
// makes everything that comes from it a NaN, whatever it holds.
// Prints "words_check: ok" and exits 0, or names the failing case.
#include <stdint.h>
#include <stdio.h>

#include <cmath>
#include <limits>
#include <vector>

#include "vdc_words.h"

namespace {

int failures = 0;

void expect(bool ok, const char* what, int at = 0) {
  if (ok) return;
  ++failures;
  printf("FAIL %s (%d)\n", what, at);
}

// The state that reaches a tile, from the words before it, the nearest first.
float fold(const std::vector<uint64_t>& words) {
  float carry = 0.0f;
  for (size_t d = words.size(); d-- > 0;) carry = vdc::folded(words[d], carry);
  return carry;
}

}  // namespace

int main() {
  const float inf = std::numeric_limits<float>::infinity(), nan = std::nanf("");
  const float Ps[] = {0.0f, 1e-45f, 1e-38f, 0.5f, 1.0f, inf, nan, vdc::word_float(0xffffffffu),
                      vdc::word_float(0xfffffffeu), vdc::word_float(0x7fc12345u)};
  const float Hs[] = {0.0f, -0.0f, 1.5f, -3e38f, inf, -inf, nan, vdc::word_float(0xffffffffu)};
  for (float P : Ps)
    for (float H : Hs) {
      const uint64_t w = vdc::word_of(P, H), k = vdc::known(H);
      expect(vdc::there<false>(w) && !vdc::there<true>(w), "a word is there and is no known state");
      expect(vdc::there<false>(k) && vdc::there<true>(k), "a known state is both");
      expect((uint32_t)w == vdc::word_bits(H) && (uint32_t)k == vdc::word_bits(H), "H as it is");
      expect(P != P || vdc::mark(w) == vdc::word_bits(P), "P as it is");
      expect(vdc::taken<false>(w) == w && vdc::taken<false>(k) == k && vdc::taken<true>(k) == k, "what is there is taken");
      expect(vdc::folded(k, nan) == H || H != H, "a known state asks for nothing before it");
    }

  // A chain of tiles: the state behind each, and folds that begin at any of them.
  uint64_t seed = 1;
  auto uniform = [&] {
    seed = seed * 6364136223846793005ull + 1442695040888963407ull;
    return (float)(seed >> 40) / (float)(1 << 24);
  };
  std::vector<uint64_t> words, states;
  float h = 0.0f;
  for (int t = 0; t < 24; ++t) {
    words.push_back(t ? vdc::word_of(uniform(), 2.0f * uniform() - 1.0f) : vdc::known(uniform()));
    h = vdc::folded(words.back(), h);
    states.push_back(vdc::known(h));
  }
  for (int from = 0; from < 24; ++from) {
    std::vector<uint64_t> seen;
    for (int t = 23; t > from; --t) seen.push_back(words[t]);
    seen.push_back(states[from]);
    expect(vdc::word_bits(fold(seen)) == vdc::word_bits(h), "the same bits wherever the fold begins", from);
  }

  // A reader that gave up: on any word at all, or on a known state.
  const uint64_t empty = (uint64_t)vdc::kEmpty << 32 | vdc::kEmpty;
  for (int from = 0; from < 23; ++from)
    for (int kind = 0; kind < 3; ++kind) {
      const uint64_t w = kind == 0   ? vdc::taken<false>(empty)
                         : kind == 1 ? vdc::taken<true>(empty)
                                     : vdc::taken<true>(vdc::word_of(0.25f, 2.0f));
      expect(vdc::there<true>(w), "a wait in vain ends with a state", kind);
      std::vector<uint64_t> seen;
      for (int t = 23; t > from; --t) seen.push_back(t == 20 ? vdc::word_of(0.0f, 1.0f) : words[t]);
      seen.push_back(w);
      expect(std::isnan(fold(seen)), "a wait in vain is a NaN in all that follows", from);
      expect(std::isnan(vdc::word_value(w)), "and in a sum", kind);
    }
  if (failures) {
    printf("words_check: %d failures\n", failures);
    return 1;
  }
  printf("words_check: ok\n");
  return 0;
}
