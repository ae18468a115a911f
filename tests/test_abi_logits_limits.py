"""Sizes of the calls on rows of logits that are refused, on the host (see test_abi_logits.py)."""

import pytest

from .test_abi_logits import FAKE, _verify, qrr  # noqa: F401

BIG = 1 << 24


@pytest.mark.parametrize("change", [dict(T=BIG + 1, cu=FAKE), dict(B=BIG + 1, cu=FAKE), dict(T=0, B=BIG + 1)])
def test_verification_of_more_drafts_than_it_takes(qrr, change):  # noqa: F811
    assert _verify(qrr, **change) == 2
    assert qrr.lib().qrr_verify_drafts_workspace_bytes(change.get("T", 6), change.get("B", 3), 100, 0) == 0


def test_verification_of_the_most_it_takes(qrr, monkeypatch):  # noqa: F811
    """(An injected fault stops it before a launch.)"""
    monkeypatch.setenv("QRR_INJECT_FAULT", "cuda")
    assert _verify(qrr, T=BIG, B=BIG, cu=FAKE) == 5
    # a part of a row (16 bytes) of each of its rows, a state (8) a sequence, two numbers (4) a place
    assert qrr.lib().qrr_verify_drafts_workspace_bytes(BIG, BIG, 100, 0) == BIG * (3 * 16 + 8 + 2 * 8)
