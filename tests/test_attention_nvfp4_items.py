"""How the many-rows attention kernel counts a sequence's work, on the host: the kernel's own arithmetic, compiled with
the host compiler and with signed overflow trapped, against Python's whole numbers."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_rl_rollout_gb300", "csrc")

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


@pytest.fixture(scope="module")
def counts(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("items")
    src, exe = d / "items.cpp", d / "items"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O2", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error",
                    "-I" + CSRC, str(src), "-o", str(exe)], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return run


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
