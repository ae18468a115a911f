"""How the many-rows attention kernel counts a sequence's work, on the host: the kernel's own arithmetic, compiled with
the host compiler and with signed overflow trapped, against Python's whole numbers."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_rl_rollout_gb300", "csrc")

# row tiles, what they count for, the most of a lane, the last row tile's key tiles
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "attention_nvfp4_items.cuh"
using namespace qrr;
using namespace qrr::attn4;
int main(int argc, char** argv) {
  long v[4];
  while (std::scanf("%ld %ld %ld %ld", v, v + 1, v + 2, v + 3) == 4) {
    const FastDiv byG(static_cast<uint32_t>(v[1]));
    const Seq s{0, static_cast<int>(v[0]), static_cast<int>(v[2]), static_cast<int>(v[3])};
    const int qts = many::row_tiles(byG, s);
    int64_t sum = 0, most = 0;
    for (int lane = 0; lane < 32; ++lane) {
      const int64_t x = many::lane_width(byG, s, lane);
      sum += x;
      if (x > most) most = x;
    }
    std::printf("%d %lld %lld %d\n", qts, static_cast<long long>(sum), static_cast<long long>(most),
                qts ? many::key_tiles(byG, s, qts - 1) : 0);
  }
}
"""


def _compiled(tmp_path_factory, program):
    """A function from cases (four whole numbers each) to the program's lines of whole numbers."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("items")
    src, exe = d / "items.cpp", d / "items"
    src.write_text(program)
    subprocess.run([gxx, "-std=c++17", "-O2", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error",
                    "-I" + CSRC, str(src), "-o", str(exe)], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return run


@pytest.fixture(scope="module")
def counts(tmp_path_factory):
    return _compiled(tmp_path_factory, PROGRAM)


def _want(n, g, pos, last):
    """(row tiles, what they count for, the last tile's key tiles) of a sequence."""
    rows = n * g
    if rows <= 32:
        return 0, 0, 0
    qts = -(-rows // 256)
    tiles = [max(1, (min(pos + (min((qt + 1) * 256, rows) - 1) // g, last) + 128) // 128) for qt in range(qts)]
    return qts, sum(tiles) + 3 * qts, tiles[-1]


def _seq(n, pos, cap):
    return n, pos, max(min(pos + n - 1, cap - 1), -1)


def test_small_and_odd(counts):
    cases = []
    for n in (1, 2, 5, 33, 64, 300, 1000):
        for g in (1, 3, 5, 8, 40, 128):
            for pos in (-400, -1, 0, 7, 5000):
                n_, pos_, last = _seq(n, pos, 5300)
                cases.append((n_, g, pos_, last))
    for case, got in zip(cases, counts(cases)):
        want = _want(*case)
        assert (got[0], got[1], got[3]) == want, case


@pytest.mark.parametrize("n,g,pos", [(1_060_000, 128, 0), (3_000_000, 16, 0), (4_200_000, 8, 0), (1 << 20, 64, 1_600_000), (1 << 23, 128, 0),
                                     (1 << 30, 1, 0)])
def test_prompts_whose_count_passes_32_bits(counts, n, g, pos):
    """Chunks that the interface admits (n g <= 2^30, positions to 2^30): the count is whole, positive and above 2^31."""
    (got,) = counts([(n, g, pos, pos + n - 1)])
    qts = -(-n * g // 256)
    # tiles of row tile qt: (pos + (min(256 (qt + 1), n g) - 1) // g + 128) // 128
    total = sum((pos + (min(256 * (qt + 1), n * g) - 1) // g + 128) // 128 for qt in range(qts)) + 3 * qts
    assert got[0] == qts and got[1] == total > 2 ** 31
    assert got[2] < 2 ** 41  # what the warp's two-part sum rests on


# of rows, rows a token, first position and the table's tokens: the last visible position, the first row tile's key tiles,
# and how many of the first tile's tokens its last row, the loads and the last 32 columns' mask see
POSITIONS = r"""
#include <cstdio>
#include "attention_nvfp4_items.cuh"
using namespace qrr;
using namespace qrr::attn4;
int main() {
  long v[4];
  while (std::scanf("%ld %ld %ld %ld", v, v + 1, v + 2, v + 3) == 4) {
    const FastDiv byG(static_cast<uint32_t>(v[1]));
    const Seq s = seq_at(0, static_cast<int>(v[0]), static_cast<int>(v[2]), static_cast<int>(v[3]));
    const int last = many::last_seen(byG, s, 0), seen = many::seen_of(last, 0);
    std::printf("%d %d %d %d %d\n", s.last, many::key_tiles(byG, s, 0), seen, seen - 112, seen - 96);
  }
}
"""


def test_positions_at_the_ends_of_32_bits(tmp_path_factory):
    """A first position of any value: no sum overflows, and rows before the first token see nothing."""
    lowest, most = -2 ** 31, 2 ** 31 - 1
    cases = [(n, g, pos, cap) for n in (1, 40, 300, 1 << 20, 1 << 30) for g in (1, 5, 64) if n * g <= 1 << 30
             for pos in (lowest, lowest + 5, -2 ** 30 - 1, -2 ** 30, -n, -n + 1, -1, 0, 2 ** 30, most) for cap in (16, 1 << 30)]
    for (n, g, pos, cap), got in zip(cases, _compiled(tmp_path_factory, POSITIONS)(cases)):
        last = max(min(pos + n - 1, cap - 1), -1)
        assert got[0] == last
        tile = min(pos + (min(256, n * g) - 1) // g, last)  # of the first row tile
        if pos + n - 1 < 0 or tile < 0:
            assert got[1] == 1 and all(x <= 0 for x in got[2:]), (n, g, pos, cap)
        elif pos <= 2 ** 30:
            assert got[1] == (tile + 128) // 128 and got[2] == tile + 1


# of rows that need no mask, from key tile v[0] on in steps of v[1] to v[2]: the fewest tokens seen, less the last column's place
UNMASKED = r"""
#include <cstdio>
#include "attention_nvfp4_items.cuh"
using namespace qrr::attn4;
int main() {
  long v[4];
  while (std::scanf("%ld %ld %ld %ld", v, v + 1, v + 2, v + 3) == 4) {
    int least = 2147483647;
    for (int j = static_cast<int>(v[0]); j <= v[2]; j += static_cast<int>(v[1])) {
      const int x = many::seen_of(many::kAllSeen, j) - 96;
      if (x < least) least = x;
    }
    std::printf("%d\n", least);
  }
}
"""


def test_rows_without_a_mask(tmp_path_factory):
    """A row behind the last one sees every column (32 at a time) of every key tile of a table for 2^30 tokens."""
    tiles = 2 ** 30 // 128
    for (least,) in _compiled(tmp_path_factory, UNMASKED)([(0, 1, 1000, 0), (0, 997, tiles - 1, 0), (tiles - 3, 1, tiles - 1, 0)]):
        assert least >= 32
