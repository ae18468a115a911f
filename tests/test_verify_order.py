"""In which order the verification of drafts looks at places, on the host: the kernel's own arithmetic, compiled with the
host compiler and with signed overflow trapped."""

import random

import pytest

from .test_attention_nvfp4_items import _compiled

PROGRAM = r"""
#include <cstdio>
#include "verify_order.cuh"
int main() {
  long long most, b, rows;
  while (std::scanf("%lld %lld %lld", &most, &b, &rows) == 3) {
    const qrr::PlaceOrder o(most, b, rows);
    std::printf("%lld %lld %lld\n", static_cast<long long>(o.level), static_cast<long long>(o.by_place), static_cast<long long>(o.total));
  }
}
"""


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    return _compiled(tmp_path_factory, PROGRAM)


def test_every_place_once(order):
    """Of sequences of any lengths, the longest far above the others or not: place by place below the level, by row from it on."""
    g = random.Random(1)
    cases = []
    for _ in range(200):
        counts = [int(g.choice([0, 1, 2, 5, g.expovariate(0.05), g.expovariate(0.002)])) for _ in range(g.randint(1, 60))]
        cases.append(counts)
    out = order([(max(c) + 1, len(c), sum(c) + len(c)) for c in cases])
    skewed = 0
    for counts, (level, by_place, total) in zip(cases, out):
        rows = [(b, i) for b, n in enumerate(counts) for i in range(n + 1)]
        seen = [(i % len(counts), i // len(counts)) for i in range(by_place)]
        seen = [(b, i) for b, i in seen if i <= counts[b]]
        if total > by_place:
            assert total - by_place == len(rows)
            seen += [(b, i) for b, i in rows if i >= level]
            skewed += 1
        assert sorted(seen) == rows
    assert 20 < skewed < 200  # both ways


def test_what_is_looked_at_goes_by_the_rows(order):
    """As many as five times the rows at the limits of a call, and one place after another where lengths are alike."""
    big = 1 << 24
    cases = [(big + 1, big, 2 * big), (big + 1, 1, big + 1), (1, big, big), (1000001, 1000000, 2000000), (4097, 4096, 8192), (2, big, big + 1)]
    for (most, b, rows), (level, by_place, total) in zip(cases, order(cases)):
        assert 1 <= level <= most and by_place == level * b and total <= 5 * rows
    assert order([(9, 64, 9 * 64), (10, 200, 1000)]) == [(9, 576, 576), (10, 2000, 2000)]
