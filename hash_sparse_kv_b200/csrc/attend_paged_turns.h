// Which tiles the two slots of an attention CTA work on, and for which of them
// their softmax warps take turns (attend_paged_tc.cu).  Plain C++, so that the
// order of the kernel's waits can be walked through on the CPU by these rules.
#pragma once

#ifdef __CUDACC__
#define HKV_BOTH_SIDES __host__ __device__ __forceinline__
#else
#define HKV_BOTH_SIDES inline
#endif

namespace hkv {
namespace pa {

// K and V tiles that shared memory holds.  A tile leaves when both slots have
// used it or passed it by, so a slot can be this many tiles ahead of the other.
constexpr int kKStages = 3, kVStages = 2;

// A slot's tiles: every step-th from first up to last.
struct Run {
  int first, last, step;
  HKV_BOTH_SIDES int count() const { return last > first ? (last - first + step - 1) / step : 0; }
};

// The slots take turns with the exponentials of n tiles, the first of which is
// the slot's own tile number `from`.
struct Turns {
  int from, n;
};

// Slots that share every tile take turns on the tiles that both work on.  Their
// runs may start and end any number of tiles apart (the documents of packed
// prompts): turns counted from each slot's own first tile would make the slot
// that is early wait for one whose tiles cannot be loaded before it goes on.
// Slots that take every other tile of one run pair them in order.
HKV_BOTH_SIDES Turns turns_of(const Run& mine, const Run& other, bool both) {
  if (!both) {
    const int a = mine.count(), b = other.count();
    return Turns{0, a < b ? a : b};
  }
  const int first = mine.first > other.first ? mine.first : other.first;
  const int last = mine.last < other.last ? mine.last : other.last;
  return Turns{first - mine.first, last > first ? last - first : 0};
}

}  // namespace pa
}  // namespace hkv
