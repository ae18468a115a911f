"""Sizes of the calls on rows of logits that are refused, on the host (see test_abi_logits.py)."""

import types

import pytest
import torch

from .test_abi_logits import FAKE, _i, _losses, _policy, _t, _verify, binding, qrr  # noqa: F401

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


@pytest.mark.parametrize("T,ld", [(1 << 27, 1 << 40), (1 << 24, 1 << 39), (3, 1 << 62), (1 << 27, (1 << 37) + 1), (1, 1 << 45)])
def test_strides_that_leave_the_address_space(qrr, T, ld):  # noqa: F811
    """Offsets that pass 64 bits, or come near, are refused before they are counted with."""
    assert _losses(qrr, T=T, ld=ld) == (1, 1, 1) and _losses(qrr, T=T, ldd=ld)[1:] == (1, 1)
    assert _policy(qrr, T=T, ld=ld) == 1 and _policy(qrr, T=T, ldd=ld) == 1
    if T <= BIG:
        assert _verify(qrr, T=T, cu=FAKE, ld=ld) == 1 and _verify(qrr, T=T, cu=FAKE, ld_draft=ld) == 1
        assert _verify(qrr, T=T, B=T, cu=FAKE, ld_noise=ld) == 1


@pytest.mark.parametrize("T,ld", [(1 << 24, 1 << 19), (3, 1 << 40), (1, 0)])
def test_strides_of_large_buffers(qrr, monkeypatch, T, ld):  # noqa: F811
    monkeypatch.setenv("QRR_INJECT_FAULT", "cuda")
    far = 1 << 50
    assert _losses(qrr, T=T, ld=ld, ldd=ld, dlogits=far) == (5, 5, 5) and _policy(qrr, T=T, ld=ld, ldd=ld, dlogits=far) == 5
    assert _verify(qrr, T=T, B=T, cu=FAKE, ld=ld or 100, ld_draft=ld, ld_noise=ld) == 5


def test_status_words_off_their_alignment(qrr):  # noqa: F811
    """An atomic there would be a fault of the GPU."""
    lib, s = qrr.lib(), FAKE + 2
    head = (FAKE, 0, 3, 100, 100, FAKE, FAKE, 4, None, 1.0)
    assert lib.qrr_distill_topk(*head, FAKE, FAKE, s, None) == 3
    assert lib.qrr_distill_topk_backward(*head, FAKE, FAKE, 2 * FAKE, 100, s, None) == 3
    assert lib.qrr_distill_topk_grad(*head, FAKE, FAKE, 2 * FAKE, 100, s, None) == 3
    assert lib.qrr_token_logprobs_is_grad(FAKE, 0, 3, 100, 100, FAKE, FAKE, FAKE, 0.0, FAKE, FAKE, 2 * FAKE, 100, s, None) == 3
    assert lib.qrr_verify_drafts(FAKE, 100, FAKE, 100, 0, 6, 3, 100, FAKE, None, FAKE, FAKE, 100, 1.0, FAKE, FAKE, FAKE, FAKE, 1 << 50,
                                 s, None) == 3


def test_binding_refuses_status_words_and_workspaces(binding):  # noqa: F811
    qrr, calls = binding
    x, ids, top, grad = _t(4, 10), _i(4, 3), _t(4, 3), _t(4)
    other = types.SimpleNamespace(index=1)
    verify = lambda **more: qrr.verify_drafts(x, _i(3), _t(3), _t(1, 10), **more)  # noqa: E731
    for status in (_t(1), _t(1, dtype=torch.uint8), _i(0), _t(1, dtype=torch.int32, device=other)):
        for call in (lambda: qrr.distill_topk(x, ids, top, dev_status=status), lambda: qrr.distill_topk_grad(x, ids, top, grad, dev_status=status),
                     lambda: qrr.distill_topk_backward(x, ids, top, _t(4, 2), grad, dev_status=status),
                     lambda: qrr.token_logprobs_is_grad(x, _i(4), grad, dev_status=status), lambda: verify(dev_status=status)):
            with pytest.raises(ValueError):
                call()
    for workspace in (_t(1 << 20, dtype=torch.uint8, device=other), _t(1 << 10, 1 << 10, dtype=torch.uint8, stride=(1 << 11, 1))):
        with pytest.raises(ValueError):
            verify(workspace=workspace)
    assert not calls
    verify(workspace=_t(1 << 20, dtype=torch.uint8), dev_status=_i(1))
    assert len(calls) == 1
