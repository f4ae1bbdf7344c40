// The words that a recurrence's tiles hand on: 64 bits a channel, of which the lower
// half is H and the upper one P, or a mark in its place.  Kept apart, so that a CPU
// program can fold them as the kernels do.
#pragma once

#include <stdint.h>

#include "vdc_search.h"

namespace vdc {

// The two marks, which no P is: a product of decays is at least 0, and a NaN is written
// as the usual one.
constexpr uint32_t kEmpty = 0xffffffffu, kKnown = 0xfffffffeu;

VDC_HD inline uint32_t word_bits(float v) { return __builtin_bit_cast(uint32_t, v); }
VDC_HD inline float word_float(uint32_t b) { return __builtin_bit_cast(float, b); }

// What a tile makes of any state, h -> P h + H.
VDC_HD inline uint64_t word_of(float P, float H) {
  return (uint64_t)(P != P ? 0x7fc00000u : word_bits(P)) << 32 | word_bits(H);
}
// The state behind a tile.
VDC_HD inline uint64_t known(float H) { return (uint64_t)kKnown << 32 | word_bits(H); }
VDC_HD inline uint32_t mark(uint64_t w) { return (uint32_t)(w >> 32); }
VDC_HD inline float word_value(uint64_t w) { return word_float((uint32_t)w); }

// Whether a word is what its reader waits for: any word, or (kAll) a known state.
template <bool kAll>
VDC_HD inline bool there(uint64_t w) {
  return kAll ? mark(w) == kKnown : mark(w) != kEmpty;
}
// What a reader has that waits no longer: the word, or a state of NaN where it is not
// there, which all that comes from it shows.
template <bool kAll>
VDC_HD inline uint64_t taken(uint64_t w) {
  return there<kAll>(w) ? w : known(__builtin_nanf(""));
}

// The state behind a tile from its word and the state before it.
VDC_HD inline float folded(uint64_t w, float before) {
  return mark(w) == kKnown ? word_value(w) : __builtin_fmaf(word_float(mark(w)), before, word_value(w));
}

}  // namespace vdc
