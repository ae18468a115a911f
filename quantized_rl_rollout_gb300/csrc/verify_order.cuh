// The order in which the verification of drafts looks at the places of its sequences.  Plain arithmetic, for the device and
// (in tests) the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define QRR_HD __host__ __device__ __forceinline__
#else
#define QRR_HD inline
#endif

namespace qrr {

// First places first: what lies behind a refusal is then mostly known to when its turn comes. Place by place, B sequences each,
// that looks at `most` B places, `most` being those of the longest sequence, where only `rows` exist: a sequence of a million
// drafts among a million short ones would keep the device for minutes. So the places below `level` go that way, kWaste times
// as many as there are rows at most, and the rest by row: what is looked at is kWaste + 1 times the rows at most.
struct PlaceOrder {
  static constexpr int kWaste = 4;
  int64_t level, by_place, total;  // places that go place by place; what that makes, and all, to look at

  PlaceOrder() = default;
  QRR_HD PlaceOrder(int64_t most, int64_t B, int64_t rows) {
    level = most * B <= kWaste * rows ? most : kWaste * rows / B;
    by_place = level * B;
    total = by_place + (level < most ? rows : 0);
  }
};

}  // namespace qrr
