// How attention over the paged NVFP4 cache counts its work: a sequence's rows and
// visible tokens, and the items that the many-rows kernel cuts them into.  Plain
// arithmetic, for the device and (in tests) the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define QRR_HD __host__ __device__ __forceinline__
#else
#define QRR_HD inline
#endif

namespace qrr {

constexpr int kMaxTokens = 1 << 30;  // rows of a call, and positions of a sequence

// x / d for 0 <= x < 2^31 by a multiplication (T. Granlund, P. Montgomery,
// "Division by invariant integers using multiplication", PLDI 1994).
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t d_) : d(d_), mul(0), shift(0) {
    while ((1ull << shift) < d) ++shift;
    mul = static_cast<uint32_t>((((1ull << shift) - d) << 32) / d + 1);
  }
  QRR_HD int div(int x) const {
#ifdef __CUDA_ARCH__
    const uint32_t hi = __umulhi(mul, static_cast<uint32_t>(x));
#else
    const uint32_t hi = static_cast<uint32_t>((static_cast<uint64_t>(mul) * static_cast<uint32_t>(x)) >> 32);
#endif
    return static_cast<int>((hi + static_cast<uint32_t>(x)) >> shift);
  }
  QRR_HD int mod(int x) const { return x - div(x) * static_cast<int>(d); }
};

namespace attn4 {

// A sequence with at most this many rows a KV head takes the first kernel: four
// groups of 8 rows are what a lane's registers hold.  16 sequences over 2250
// tokens, 17..32 rows: 42 us with it, 50 with the other.
constexpr int kFewRows = 32;

// A sequence as the kernels see it: its rows, the position of the first, the
// last visible position of the last (-1: none).
struct Seq {
  int first, n, pos, last;
};

// Of n <= kMaxTokens rows from position pos on, in a table for `cap` <= kMaxTokens
// tokens.  Positions beyond kMaxTokens either way come nearer, which leaves them
// outside; sums with rows and tokens of a tile then stay in 32 bits.
QRR_HD Seq seq_at(int first, int n, int pos, int cap) {
  pos = pos < -kMaxTokens ? -kMaxTokens : pos > kMaxTokens ? kMaxTokens : pos;
  const int last = pos + (n - 1);
  return Seq{first, n, pos, last < 0 ? -1 : last < cap ? last : cap - 1};
}

namespace many {

constexpr int kRows = 256;  // rows of an item
constexpr int kTok = 128;   // tokens of a key tile
// Key tiles that an item's start and end cost (about 10000 cycles beside 3800 a
// tile).  A prompt of 4096 tokens with 2, 3, 4: 158, 156, 161 us; of 64 tokens,
// whose items then fit a range of kMinTiles: 23, 17, 17.
constexpr int kItemCost = 3;

// Items of a sequence with G rows a token (2^30 rows at most): row tiles of 256
// (none if it has few rows), and the key tiles of one (at least 1).
QRR_HD int row_tiles(const FastDiv& byG, const Seq& s) {
  const int rows = s.n * static_cast<int>(byG.d);
  return rows <= kFewRows ? 0 : (rows + kRows - 1) / kRows;
}
QRR_HD int last_seen(const FastDiv& byG, const Seq& s, int qt) {
  const int rows = s.n * static_cast<int>(byG.d), end = (qt + 1) * kRows;
  const int last = s.pos + byG.div((end < rows ? end : rows) - 1);
  return last < s.last ? last : s.last;
}
QRR_HD int key_tiles(const FastDiv& byG, const Seq& s, int qt) {
  const int tiles = (last_seen(byG, s, qt) + kTok) / kTok;
  return tiles > 1 ? tiles : 1;
}

// What an item counts for.
QRR_HD int width(const FastDiv& byG, const Seq& s, int qt) { return key_tiles(byG, s, qt) + kItemCost; }

// What every 32nd row tile of one KV head counts for, from `lane` on.  About
// n^2 G / 65536 in all: a million tokens with 128 rows each pass 32 bits.
QRR_HD int64_t lane_width(const FastDiv& byG, const Seq& s, int lane) {
  const int qts = row_tiles(byG, s);
  int64_t sum = 0;
  for (int qt = lane; qt < qts; qt += 32) sum += width(byG, s, qt);
  return sum;
}

// Of key tile j's tokens, how many a row sees whose last visible position is
// `lim` (any value outside 0 .. kTok: none or all).  A row that needs no mask has
// kAllSeen in its place: behind every position, and seen_of stays in 32 bits.
constexpr int kAllSeen = kMaxTokens;
QRR_HD int seen_of(int lim, int j) { return lim - kTok * j + 1; }

}  // namespace many

}  // namespace attn4

}  // namespace qrr
