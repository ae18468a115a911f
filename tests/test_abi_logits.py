"""Host-only checks of the calls on rows of logits: bad arguments are refused before anything is launched, by the library
and by the binding.  No call here reaches a GPU."""

import types

import pytest
import torch

FAKE = 0x10000  # a 16-byte-aligned non-null address that is never dereferenced


@pytest.fixture(scope="module")
def qrr():
    from quantized_rl_rollout_gb300 import build, qrr

    build.build()
    qrr.lib()
    return qrr


def _losses(qrr, logits=FAKE, dtype=0, T=3, V=100, ld=100, ids=FAKE, top=FAKE, k=4, lse=None, temp=1.0, grad=FAKE, loss=FAKE,
            stats=FAKE, dlogits=2 * FAKE, ldd=100):
    lib, head = qrr.lib(), (logits, dtype, T, V, ld, ids, top, k, lse, temp)
    return (lib.qrr_distill_topk(*head, loss, stats, None, None),
            lib.qrr_distill_topk_backward(*head, stats, grad, dlogits, ldd, None, None),
            lib.qrr_distill_topk_grad(*head, grad, loss, dlogits, ldd, None, None))


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), 1), (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(T=-1), 1), (dict(V=0), 1), (dict(ld=99), 1),
    (dict(ld=-100, T=1), 1), (dict(k=-1), 1), (dict(k=1025), 2), (dict(ids=None), 1), (dict(top=None), 1), (dict(temp=0.0), 1),
    (dict(temp=-1.0), 1), (dict(temp=float("nan")), 1), (dict(temp=float("inf")), 1), (dict(temp=1e-7), 1),
    (dict(V=786433, ld=786433), 2), (dict(V=393217, ld=393217, dtype=1), 2), (dict(T=(1 << 27) + 1), 2),
    (dict(logits=FAKE + 1), 3), (dict(logits=FAKE + 2, dtype=1), 3), (dict(ids=FAKE + 2), 3), (dict(top=FAKE + 1), 3),
    (dict(lse=FAKE + 2), 3)])
def test_rows_and_teacher(qrr, change, status):
    assert _losses(qrr, **change) == (status,) * 3


def test_loss_outputs(qrr):
    assert _losses(qrr, loss=None)[0::2] == (1, 1) and _losses(qrr, loss=FAKE + 2)[0::2] == (3, 3)
    assert _losses(qrr, stats=None)[:2] == (1, 1) and _losses(qrr, stats=FAKE + 1)[:2] == (3, 3)
    for change, status in [(dict(grad=None), 1), (dict(grad=FAKE + 2), 3), (dict(dlogits=None), 1), (dict(dlogits=FAKE + 1), 3),
                           (dict(ldd=99), 1), (dict(dlogits=FAKE, ldd=104), 1), (dict(dlogits=2 * FAKE + 2, dtype=1), 3)]:
        assert _losses(qrr, **change)[1:] == (status, status), change


def _policy(qrr, logits=FAKE, dtype=0, T=3, V=100, ld=100, tokens=FAKE, adv=FAKE, rollout=FAKE, cap=0.0, logp=FAKE, w=FAKE,
            dlogits=2 * FAKE, ldd=100):
    return qrr.lib().qrr_token_logprobs_is_grad(logits, dtype, T, V, ld, tokens, adv, rollout, cap, logp, w, dlogits, ldd, None, None)


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), 1), (dict(dtype=5), 1), (dict(V=0), 1), (dict(ld=50), 1), (dict(tokens=None), 1), (dict(adv=None), 1),
    (dict(logp=None), 1), (dict(w=None), 1), (dict(dlogits=None), 1), (dict(ldd=1), 1), (dict(V=800000, ld=800000), 2),
    (dict(tokens=FAKE + 2), 3), (dict(adv=FAKE + 1), 3), (dict(rollout=FAKE + 2), 3), (dict(w=FAKE + 2), 3),
    (dict(dlogits=FAKE + 1), 3)])
def test_policy(qrr, change, status):
    assert _policy(qrr, **change) == status


def _verify(qrr, target=FAKE, ld=100, draft=FAKE, ld_draft=100, dtype=0, T=6, B=3, V=100, drafts=FAKE, cu=None, u=FAKE, noise=FAKE,
            ld_noise=100, temp=1.0, tokens=FAKE, accepted=FAKE, logp=FAKE, ws=FAKE, ws_bytes=1 << 50):
    return qrr.lib().qrr_verify_drafts(target, ld, draft, ld_draft, dtype, T, B, V, drafts, cu, u, noise, ld_noise, temp, tokens,
                                       accepted, logp, ws, ws_bytes, None, None)


@pytest.mark.parametrize("change,status", [
    (dict(target=None), 1), (dict(dtype=3), 1), (dict(T=-1), 1), (dict(B=-1), 1), (dict(V=0), 1), (dict(T=7), 1), (dict(B=0), 1),
    (dict(ld=99), 1), (dict(ld_draft=99), 1), (dict(ld_noise=99), 1), (dict(ld_noise=-1, B=1, cu=FAKE), 1), (dict(drafts=None), 1),
    (dict(u=None), 1), (dict(noise=None), 1), (dict(temp=-0.5), 1), (dict(temp=1e-8), 1), (dict(temp=float("nan")), 1),
    (dict(tokens=None), 1), (dict(accepted=None), 1), (dict(logp=None), 1), (dict(B=(1 << 26) + 1, cu=FAKE), 2),
    (dict(V=(1 << 30) + 1), 2), (dict(T=3 << 29, cu=FAKE), 2), (dict(target=FAKE + 1), 3), (dict(draft=FAKE + 2, dtype=1), 3),
    (dict(cu=FAKE + 2), 3), (dict(u=FAKE + 2), 3), (dict(noise=FAKE + 2), 3), (dict(tokens=FAKE + 2), 3), (dict(logp=FAKE + 1), 3),
    (dict(ws=None), 4), (dict(ws_bytes=64), 4), (dict(ws=FAKE + 8), 3)])
def test_verify(qrr, change, status):
    assert _verify(qrr, **change) == status


def test_nothing_to_do(qrr):
    """No rows: nothing is needed and nothing is launched."""
    assert _losses(qrr, T=0, logits=None, ids=None, top=None, grad=None, loss=None, stats=None, dlogits=None) == (0, 0, 0)
    assert _policy(qrr, T=0, logits=None, tokens=None, adv=None, rollout=None, logp=None, w=None, dlogits=None) == 0
    assert _verify(qrr, T=0, B=0, target=None, draft=None, drafts=None, u=None, noise=None, tokens=None, accepted=None, logp=None,
                   ws=None, ws_bytes=0) == 0
    assert qrr.lib().qrr_verify_drafts_workspace_bytes(6, 3, 100, 2) == 0 and qrr.lib().qrr_verify_drafts_workspace_bytes(-1, 3, 100, 0) == 0


def test_injected_fault(qrr, monkeypatch):
    monkeypatch.setenv("QRR_INJECT_FAULT", "cuda")
    assert _losses(qrr) == (5,) * 3 and _policy(qrr) == 5 and _verify(qrr) == 5


class Tensor:
    """What the binding looks at, of a CUDA tensor."""

    is_cuda = True

    def __init__(self, shape, dtype=torch.float32, stride=None, index=0):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, types.SimpleNamespace(index=index)
        self.s = stride or tuple(int(torch.Size(shape[i + 1:]).numel()) for i in range(len(shape)))

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return self.s

    def is_contiguous(self):
        return self.s == Tensor(self.shape).s

    def data_ptr(self):
        return FAKE


DEVICE = types.SimpleNamespace(index=0)


def _t(*shape, dtype=torch.float32, stride=None, device=DEVICE):
    t = Tensor(shape, dtype, stride)
    t.device = device
    return t


def _i(*shape):
    return _t(*shape, dtype=torch.int32)


@pytest.fixture
def binding(monkeypatch):
    from quantized_rl_rollout_gb300 import qrr

    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 4096 if name.endswith("_bytes") else calls.append((name, a)) or 0

    monkeypatch.setattr(qrr, "lib", lambda: Lib())
    monkeypatch.setattr(qrr, "_stream", lambda s: 0)
    monkeypatch.setattr(qrr, "_on_stream", lambda shape, dtype, device, stream, returned=True: _t(*shape, dtype=dtype))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return qrr, calls


def test_binding_passes_strides(binding):
    qrr, calls = binding
    x = _t(4, 10, dtype=torch.bfloat16, stride=(16, 1))
    loss, stats = qrr.distill_topk(x, _i(4, 3), _t(4, 3))
    assert tuple(loss.shape) == (4,) and tuple(stats.shape) == (4, 2)
    assert calls[-1][1][1:5] == (0, 4, 10, 16)
    d = qrr.distill_topk_backward(x, _i(4, 3), _t(4, 3), stats, _t(4), dlogits=_t(4, 10, dtype=torch.bfloat16, stride=(12, 1)))
    assert calls[-1][1][13] == 12 and d.stride() == (12, 1)
    _, _, d = qrr.token_logprobs_is_grad(_t(4, 10), _i(4), _t(4))
    assert d.dtype == torch.float32 and calls[-1][1][9:11] == (FAKE, None)
    tokens, accepted, logp = qrr.verify_drafts(_t(9, 10), _i(6), _t(6), _t(3, 10, stride=(20, 1)), cu=_i(4))
    assert tuple(tokens.shape) == (9,) and tuple(accepted.shape) == (3,) and calls[-1][1][12] == 20
    qrr.verify_drafts(_t(9, 10), _i(6), temperature=0)
    assert calls[-1][1][2] is None and calls[-1][1][10:12] == (None, None)


def test_binding_refuses(binding):
    qrr, calls = binding
    x, ids, top = _t(4, 10), _i(4, 3), _t(4, 3)
    other = types.SimpleNamespace(index=1)
    bad = [
        lambda: qrr.distill_topk(_t(4, 10, dtype=torch.float16), ids, top),
        lambda: qrr.distill_topk(_t(4, 10, stride=(1, 4)), ids, top),
        lambda: qrr.distill_topk(_t(4, 10, stride=(0, 1)), ids, top),
        lambda: qrr.distill_topk(_t(40), ids, top),
        lambda: qrr.distill_topk(_t(4, 10, device=other), ids, top),
        lambda: qrr.distill_topk(x, _t(4, 3, dtype=torch.int64), top),
        lambda: qrr.distill_topk(x, _i(3, 3), top),
        lambda: qrr.distill_topk(x, ids, _t(4, 2)),
        lambda: qrr.distill_topk(x, ids, _t(4, 3, device=other)),
        lambda: qrr.distill_topk(x, ids, top, top_lse=_t(3)),
        lambda: qrr.distill_topk(x, ids, top, loss=_t(5)),
        lambda: qrr.distill_topk(x, ids, top, stats=_t(4)),
        lambda: qrr.distill_topk_backward(x, ids, top, _t(4, 2), _t(4), dlogits=_t(4, 10, dtype=torch.bfloat16)),
        lambda: qrr.distill_topk_backward(x, ids, top, _t(4, 2), _t(4), dlogits=_t(4, 9)),
        lambda: qrr.distill_topk_backward(x, ids, top, _t(4, 2), _t(1)),
        lambda: qrr.distill_topk_grad(x, ids, top, _t(4), dlogits=_t(4, 10, device=other)),
        lambda: qrr.token_logprobs_is_grad(x, _i(5), _t(4)),
        lambda: qrr.token_logprobs_is_grad(x, _i(4), _t(4), _t(4), w=_t(4, dtype=torch.bfloat16)),
        lambda: qrr.verify_drafts(x, _i(5), _t(5), _t(1, 10)),
        lambda: qrr.verify_drafts(x, _i(3)),
        lambda: qrr.verify_drafts(x, _i(3), _t(3)),
        lambda: qrr.verify_drafts(x, _i(3), _t(2), _t(1, 10)),
        lambda: qrr.verify_drafts(x, _i(3), _t(3), _t(1, 9)),
        lambda: qrr.verify_drafts(x, _i(3), _t(3), _t(1, 10), draft_logits=_t(4, 10)),
        lambda: qrr.verify_drafts(x, _i(3), _t(3), _t(1, 10), draft_logits=_t(3, 10, dtype=torch.bfloat16)),
        lambda: qrr.verify_drafts(x, _i(3), _t(3), _t(1, 10), cu=_i(3)),
        lambda: qrr.verify_drafts(x, _i(3), _t(3), _t(1, 10), tokens=_t(4)),
        lambda: qrr.verify_drafts(x, _i(3), _t(3), _t(1, 10, device=other)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            raise AssertionError(f"call {i} was not refused")
    assert not calls


@pytest.mark.parametrize("change,status", [
    (dict(dlogits=FAKE + 2), 1), (dict(dlogits=FAKE + 2 * 50), 1), (dict(logits=FAKE + 2 * 250, dlogits=FAKE), 1),  # rows in others
    (dict(dlogits=FAKE + 2 * 100), 1), (dict(T=1, dlogits=FAKE + 2), 1), (dict(dlogits=FAKE + 2 * 104, ld=104, ldd=108), 1),
    (dict(dlogits=FAKE + 2 * 100, ld=199, ldd=199), 1), (dict(dlogits=FAKE + 2 * 300, ld=250, ldd=250), 1)])
def test_gradients_that_overlap_the_logits(qrr, change, status):
    assert _losses(qrr, **change)[1:] == (status, status)
    assert _policy(qrr, **change) == status


def test_gradients_beside_the_logits(qrr, monkeypatch):
    """Columns of one buffer, and the logits themselves, pass the checks (an injected fault stops them before a launch)."""
    monkeypatch.setenv("QRR_INJECT_FAULT", "cuda")
    ok = _losses(qrr)[2]
    assert ok not in (0, 1, 2, 3)
    for change in (dict(dlogits=FAKE + 2 * 100, ld=200, ldd=200), dict(logits=FAKE + 2 * 100, dlogits=FAKE, ld=208, ldd=208),
                   dict(dlogits=FAKE), dict(dlogits=FAKE + 2 * 300), dict(T=1, dlogits=FAKE, ldd=300)):
        assert _losses(qrr, **change)[1:] == (ok, ok) and _policy(qrr, **change) == ok, change
