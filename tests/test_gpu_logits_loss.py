"""GPU parity of the losses over rows of logits and their gradients against the float64 oracle.

Tolerances, from the arithmetic.  A term of a row's sum is off by the hardware exponential (2^-22), the rounding of its
argument (2^-23 of at most 40, where a term still counts, times ln 2: 4e-6) and the sum's (at most 100 additions in sequence:
2^-24 each, 6e-6): the log-sum-exp is within LSE = 1.2e-5, and its own rounding 2^-24.  Teacher probabilities come of expf
(2^-22), an argument's rounding (2 2^-24 of at most 40: 5e-6) and a sum of k terms by lanes (k / 32 + 5 additions; 40
2^-24 = 2.4e-6): P = 8e-6 relative.  A loss adds p (ln p - ln q): LSE + P (1 + |ln p - ln q|) of the mass, for the tail
too, where p_r = 1 - sum p is off by P of the sum, not of itself (and so its logarithm by P / p_r).  A gradient element is off
by (LSE + P) of the terms that it is the difference of, and the rounding to its type."""

import numpy as np
import pytest
import torch

from oracle import distill

pytestmark = pytest.mark.gpu
DEV = "cuda"
LSE, P, EPS = 1.2e-5, 8e-6, 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    from quantized_rl_rollout_gb300 import build, qrr

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    qrr.lib()
    return qrr


def _rows(t, v, dtype, seed, pad=0, start=0):
    """Logits [t, v], rows v + pad apart, from element `start` of their buffer on."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((start + t * (v + pad),), float("nan"), dtype=dtype)
    x = buf[start:].view(t, v + pad)[:, :v]
    x[:] = (2.5 * torch.randn(t, v, generator=g)).to(dtype)
    whole = buf.to(DEV)
    return whole[start:].view(t, v + pad)[:, :v], whole


def _teacher(x, k, seed, temperature, tail, idle=0):
    """Ids in any order, the teacher's logits there, its log-sum-exp; some slots unused, every idle-th row without any."""
    g = torch.Generator().manual_seed(seed)
    t, v = x.shape
    y = x.float().cpu() + 0.8 * torch.randn(t, v, generator=g)
    ids = torch.stack([torch.randperm(v, generator=g)[:k] for _ in range(t)]).to(torch.int32)
    if k > v:
        ids = torch.nn.functional.pad(ids, (0, k - v), value=-1)
    top = y.gather(1, ids.clamp(min=0).long())
    if t > 1 and k > 2:
        ids[1, ::2] = -1
    if idle:
        ids[::idle] = -1
    lse = torch.logsumexp(y.double() / temperature, -1).float()
    return ids.to(DEV), top.to(DEV), lse.to(DEV) if tail else None


def _oracle(x, ids, top, lse, temperature):
    x, ids, top = x.float().cpu().numpy().astype(np.float64), ids.cpu().numpy(), top.cpu().numpy().astype(np.float64)
    with np.errstate(all="ignore"):
        return distill.distill(x, ids, top, None if lse is None else lse.cpu().numpy().astype(np.float64), temperature)


def _loss_bound(x, ids, top, lse, temperature, stats):
    """See above, a row."""
    out = []
    for t in range(x.shape[0]):
        z = x[t].double().cpu().numpy() / temperature
        i, p, lnp, rest = distill.teacher(ids[t].cpu().numpy(), top[t].cpu().numpy(), None if lse is None else float(lse[t]), temperature)
        if i.size == 0:
            out.append(0.0)
            continue
        some = p > 0
        d = np.abs(lnp[some] - (z[i[some]] - stats[t, 0]))
        b = (LSE + P) * p.sum() + P * (p[some] * d).sum() + 4 * EPS * (p[some] * d).sum()
        if lse is not None and rest > (0 if stats[t, 1] > -np.inf else 2.0 ** -16):
            b += 2 * LSE * rest + P * (1 + abs(np.log(rest) - (stats[t, 1] - stats[t, 0])))
        out.append(b)
    return np.array(out)


def _gradient_bound(x, ids, top, lse, temperature, stats, grad, ref, dtype):
    b = np.zeros_like(ref)
    for t in range(ref.shape[0]):
        z = x[t].double().cpu().numpy() / temperature
        i, p, _, rest = distill.teacher(ids[t].cpu().numpy(), top[t].cpu().numpy(), None if lse is None else float(lse[t]), temperature)
        if i.size == 0:
            continue
        terms = (LSE + P + 3 * EPS * (1 + abs(stats[t, 0]))) * np.exp(z - stats[t, 0]) if stats[t, 0] > -np.inf else np.zeros_like(z)
        np.add.at(terms, i, P * p)
        if lse is not None and stats[t, 1] > -np.inf:
            u = np.exp(z - stats[t, 1])
            u[i] = 0
            # q_r off by 2 LSE of itself, p_r by P of 1, and the shared factor by LSE and the logarithm's rounding
            q_r = np.exp(stats[t, 1] - stats[t, 0])
            terms += u * (2 * LSE * q_r + P + (LSE + 3 * EPS * (1 + abs(stats[t, 1]))) * abs(q_r - rest))
        b[t] = abs(float(grad[t])) / temperature * terms
    return b + np.abs(ref) * (torch.finfo(dtype).eps / 2 + 4 * EPS) + 1e-37


def _close(got, ref, bound, what):
    got = got.double().cpu().numpy().reshape(ref.shape)
    same = got == ref  # infinities
    # A loss of ids at fp32's lowest value is p 3.4028235e38 over a mass of 1 +- P: what passes the largest fp32 number,
    # 3.4028235e38, by less than its bound rounds to infinity.
    same |= np.isinf(got) & (np.sign(got) == np.sign(ref)) & (np.abs(ref) + bound > np.finfo(np.float32).max)
    with np.errstate(all="ignore"):
        worst = np.where(same, 0.0, np.abs(got - ref) / np.maximum(bound, 1e-300))
    assert np.all(worst <= 1.0), f"{what}: {np.max(worst):.3g} of the bound at {np.unravel_index(np.argmax(worst), worst.shape)}"


def _check(q, x, ids, top, lse, temperature, dlogits=None, flags=0):
    t = x.shape[0]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    grad = torch.linspace(-1.5, 2.0, t, device=DEV) if t > 1 else torch.ones(1, device=DEV)
    loss, stats, ref = _oracle(x, ids, top, lse, temperature)
    with np.errstate(all="ignore"):
        l_bound = _loss_bound(x, ids, top, lse, temperature, stats)
        ref = ref * grad.double().cpu().numpy()[:, None]
        g_bound = _gradient_bound(x, ids, top, lse, temperature, stats, grad, ref, x.dtype)
    s_bound = LSE + EPS * np.abs(stats)
    more = dict(top_lse=lse, temperature=temperature, dev_status=st)
    got, got_stats = q.distill_topk(x, ids, top, **more)
    _close(got, loss, l_bound + EPS * np.abs(loss), "loss")
    _close(got_stats, stats, s_bound, "stats")
    _close(q.distill_topk_backward(x, ids, top, got_stats, grad, dlogits=dlogits, **more), ref, g_bound, "backward")
    again, d = q.distill_topk_grad(x, ids, top, grad, dlogits=dlogits, **more)
    _close(again, loss, l_bound + EPS * np.abs(loss), "loss with its gradient")  # summed in another order
    _close(d, ref, g_bound, "gradient")
    assert q.get_last_device_status(st) == flags
    return got, d


SHAPES = [(1, 1, 1, 0, 0), (3, 7, 3, 1, 1), (2, 8, 8, 0, 0), (5, 100, 100, 4, 3), (4, 500, 1, 0, 0), (6, 1003, 20, 0, 0),
          (3, 4096, 64, 8, 0), (4, 8195, 256, 5, 7), (2, 32000, 1024, 0, 8), (3, 50001, 33, 63, 1), (2, 128256, 64, 0, 0)]


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("t,v,k,pad,start", SHAPES)
def test_shapes(q, t, v, k, pad, start, dtype, tail):
    x, _ = _rows(t, v, dtype, v, pad, start)
    ids, top, lse = _teacher(x, k, v + 1, 1.0, tail)
    _check(q, x, ids, top, lse, 1.0)


@pytest.mark.parametrize("temperature", [0.5, 2.0, 7.0])
@pytest.mark.parametrize("tail", [False, True])
def test_temperature_and_idle_rows(q, temperature, tail):
    x, _ = _rows(9, 3000, BF16, 1)
    ids, top, lse = _teacher(x, 17, 2, temperature, tail, idle=3)
    loss, d = _check(q, x, ids, top, lse, temperature)
    assert not loss[::3].any() and not d[::3].any() and d[1].any()


@pytest.mark.parametrize("v,dtype", [(393216, FP32), (786432, BF16), (262145, FP32)])
def test_longest_rows(q, v, dtype):
    x, _ = _rows(1, v, dtype, 3, start=1)
    ids, top, lse = _teacher(x, 40, 4, 1.0, True)
    _check(q, x, ids, top, lse, 1.0)


@pytest.mark.parametrize("t", [1, 37, 151, 700])
def test_many_rows(q, t):
    """Rows by one CTA, and by clusters of several."""
    for v in (64, 5000):
        x, _ = _rows(t, v, BF16, t)
        ids, top, lse = _teacher(x, 5, t + 1, 1.0, True)
        _check(q, x, ids, top, lse, 1.0)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_slots_that_name_one_id(q, dtype, tail):
    x, _ = _rows(4, 900, dtype, 5)
    ids, top, lse = _teacher(x, 90, 6, 1.0, False)
    ids[:, 1::2] = ids[:, ::2]
    ids[3] = 17
    lse = torch.logsumexp(torch.where(ids >= 0, top.double(), -torch.inf), -1).float() + 0.2 if tail else None
    _check(q, x, ids, top, lse, 1.0)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_masked_logits(q, dtype, tail):
    """-inf and the type's lowest value: in most places, beside the ids, at them, everywhere."""
    low = torch.finfo(dtype).min
    x, _ = _rows(6, 3001, dtype, 7)
    ids, top, lse = _teacher(x, 12, 8, 1.0, tail)
    ids[1] = ids[2]
    x[0, 5:] = low
    x[0, ids[0].long()] = 1.0
    keep = x[1].clone()
    x[1] = -torch.inf
    x[1, ids[1].long()] = keep[ids[1].long()]  # nothing is left outside the ids
    x[2, ids[2, 3].long()] = -torch.inf  # an id that the student rules out
    x[3] = -torch.inf
    x[4, ids[4].long()] = low  # the ids' probability is 0, the logarithms are large
    x[5, : 3000] = -torch.inf
    if tail:
        lse[1] = torch.logsumexp(top[1].double(), -1).float() - 0.01  # no rest
    loss, d = _check(q, x, ids, top, lse, 1.0)
    assert torch.isinf(loss[2]) and torch.isfinite(d).all()


def test_rows_at_the_lowest_value(q):
    """All logits equal, at the lowest value: probabilities are 1 / V (of the loss and gradient at once, which hold the row;
    its log-sum-exp in 32 bits, which the other call starts from, has no digits for ln V)."""
    for dtype in (BF16, FP32):
        x = torch.full((2, 1000), torch.finfo(dtype).min, dtype=dtype, device=DEV)
        ids = torch.tensor([[3], [999]], dtype=torch.int32, device=DEV)
        loss, d = q.distill_topk_grad(x, ids, torch.zeros(2, 1, device=DEV), torch.ones(2, device=DEV))
        assert torch.allclose(loss.double().cpu(), torch.full((2,), 1000.0).double().log(), rtol=0, atol=2 * LSE)
        want = torch.full((2, 1000), 1e-3, device=DEV)
        want[0, 3] = want[1, 999] = 1e-3 - 1
        assert torch.allclose(d.float(), want, rtol=torch.finfo(dtype).eps / 2 + LSE, atol=0)


@pytest.mark.parametrize("v,pad", [(1003, 0), (4096, 8)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_in_place_and_strided_gradients(q, dtype, v, pad):
    t = 5
    x, _ = _rows(t, v, dtype, 9, pad)
    ids, top, lse = _teacher(x, 21, 10, 1.0, True)
    grad = torch.rand(t, device=DEV)
    loss, want = q.distill_topk_grad(x, ids, top, grad, top_lse=lse)
    _, stats = q.distill_topk(x, ids, top, top_lse=lse)
    back = q.distill_topk_backward(x, ids, top, stats, grad, top_lse=lse)
    tokens = torch.arange(t, dtype=torch.int32, device=DEV) * 7
    _, _, pol = q.token_logprobs_is_grad(x, tokens, grad)
    for call, ref in [(lambda z, o: q.distill_topk_grad(z, ids, top, grad, top_lse=lse, dlogits=o), want),
                      (lambda z, o: q.distill_topk_backward(z, ids, top, stats, grad, top_lse=lse, dlogits=o), back),
                      (lambda z, o: q.token_logprobs_is_grad(z, tokens, grad, dlogits=o), pol)]:
        for gap in (0, 1, 3, 16):  # rows of the gradient that start elsewhere than the logits'
            buf = torch.full((t, v + gap), 7.0, dtype=dtype, device=DEV)
            call(x, buf[:, :v])
            assert torch.equal(buf[:, :v], ref) and (buf[:, v:] == 7.0).all()
        own = torch.empty_strided(x.shape, x.stride(), dtype=dtype, device=DEV).copy_(x)
        call(own, own)
        assert torch.equal(own, ref)


def test_flags(q):
    x, _ = _rows(4, 600, BF16, 11)
    ids, top, lse = _teacher(x, 6, 12, 1.0, False)
    grad, st = torch.ones(4, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    loss, want = q.distill_topk_grad(x, ids, top, grad, dev_status=st)
    assert q.get_last_device_status(st) == 0
    more, tops = torch.nn.functional.pad(ids, (0, 2)), torch.nn.functional.pad(top, (0, 2), value=3.0)
    more[:, 6], more[:, 7] = 600, 2 ** 31 - 1  # no ids of this vocabulary: unused
    got, d = q.distill_topk_grad(x, more, tops, grad, dev_status=st)
    assert q.get_last_device_status(st) == q.DEV_BAD_INDEX
    assert torch.equal(got, loss) and torch.equal(d, want)
    for bad in (float("nan"), float("inf")):
        for at in (0, 300, 599):
            y = x.clone()
            y[2, at] = bad
            for call in (lambda: q.distill_topk(y, ids, top, dev_status=st), lambda: q.distill_topk_grad(y, ids, top, grad, dev_status=st),
                         lambda: q.token_logprobs_is_grad(y, ids[:, 0].contiguous(), grad, dev_status=st)):
                st.zero_()
                call()
                assert q.get_last_device_status(st) == q.DEV_NONFINITE, (bad, at)
        y = top.clone()
        y[1, 1] = bad
        st.zero_()
        q.distill_topk(x, ids, y, dev_status=st)
        assert q.get_last_device_status(st) == q.DEV_NONFINITE


def test_no_slots(q):
    x, _ = _rows(3, 40, BF16, 13)
    none = torch.empty(3, 0, dtype=torch.int32, device=DEV)
    loss, d = q.distill_topk_grad(x, none, none.float(), torch.ones(3, device=DEV))
    assert not loss.any() and not d.any()
    empty = x[:0]
    loss, stats = q.distill_topk(empty, none[:0], none[:0].float())
    assert loss.shape == (0,) and stats.shape == (0, 2)


def _policy(q, x, tokens, adv, rollout, cap):
    xs = x.double().cpu().numpy()
    with np.errstate(all="ignore"):
        logp, w, ref = distill.policy_gradient(xs, tokens.cpu().numpy(), adv.double().cpu().numpy(),
                                               None if rollout is None else rollout.double().cpu().numpy(), cap)
    got = q.token_logprobs_is_grad(x, tokens, adv, rollout, cap)
    lp_bound = LSE + 3 * EPS * np.abs(logp)
    _close(got[0], logp, lp_bound, "logp")
    if rollout is None:
        assert got[1] is None
    else:
        _close(got[1], w, w * (lp_bound + 2 ** -21 + EPS * np.abs(logp)), "w")
    a = np.abs(adv.double().cpu().numpy() * w)[:, None]
    lse = np.where(np.isfinite(xs), xs, -1e300).max(-1) + np.log(np.exp(xs - xs.max(-1, keepdims=True)).sum(-1))
    terms = np.exp(xs - lse[:, None])
    live = np.nonzero(tokens.cpu().numpy() >= 0)[0]
    terms[live, tokens.cpu().numpy()[live]] += 2 ** -20
    w_err = (lp_bound + 2 ** -21 + EPS * np.abs(logp))[:, None] * np.abs(ref)
    bound = a * (LSE + P) * terms + w_err + np.abs(ref) * (torch.finfo(x.dtype).eps / 2 + 4 * EPS) + 1e-37
    _close(got[2], ref, bound, "policy gradient")
    return got


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("t,v,pad", [(1, 1, 0), (3, 7, 2), (40, 1000, 0), (5, 8195, 1), (3, 32003, 0), (2, 128256, 0)])
def test_policy_gradient(q, t, v, pad, dtype):
    x, _ = _rows(t, v, dtype, v, pad)
    g = torch.Generator().manual_seed(v)
    tokens = torch.randint(0, v, (t,), generator=g).to(torch.int32)
    if t > 2:
        tokens[1] = -1
        tokens[2] = v - 1
    lp = torch.log_softmax(x.double(), -1).cpu().gather(1, tokens.clamp(min=0).long()[:, None])[:, 0]
    rollout = (lp + 0.4 * torch.randn(t, generator=g)).float().to(DEV)
    adv, tokens = torch.randn(t, generator=g).to(DEV), tokens.to(DEV)
    for r, cap in ((None, 0.0), (rollout, 0.0), (rollout, 1.1)):
        logp, w, d = _policy(q, x, tokens, adv, r, cap)
    if t > 2:
        assert logp[1] == 0 and w[1] == 0 and not d[1].any()
    # the forward call's numbers (which has its own kernel)
    if dtype == BF16 and pad == 0:
        lp2, w2 = q.token_logprobs_is(x, tokens, rollout, 1.1)
        assert torch.allclose(logp, lp2, rtol=1e-6, atol=1e-4) and torch.allclose(w, w2, rtol=2e-4, atol=0)


def test_policy_masked_and_bad_tokens(q):
    x, _ = _rows(4, 500, BF16, 14)
    x[0, 9] = -torch.inf
    x[1, 10:] = torch.finfo(BF16).min
    tokens = torch.tensor([9, 3, 500, 7], dtype=torch.int32, device=DEV)
    adv, st = torch.ones(4, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    logp, w, d = q.token_logprobs_is_grad(x, tokens, adv, torch.zeros(4, device=DEV), dev_status=st)
    assert q.get_last_device_status(st) == q.DEV_BAD_INDEX
    assert torch.isneginf(logp[0]) and w[0] == 0 and not d[0].any()  # never taken under this policy
    assert logp[2] == 0 and w[2] == 0 and not d[2].any()
    assert torch.isfinite(logp[1]) and not d[1, 10:].any()
    logp, w, d = q.token_logprobs_is_grad(x, tokens, adv)
    assert w is None and d[0, 9] == -1 and abs(float(d[0].float().sum())) < 0.02


def test_offsets_behind_2_31(q):
    """Rows whose elements lie behind 2^31, in place: the last ones as the same rows alone."""
    t, v = 17000, 128256
    x = torch.zeros(t, v, dtype=BF16, device=DEV)
    tail, _ = _rows(4, v, BF16, 15)
    x[-4:] = tail
    ids = torch.full((t, 3), -1, dtype=torch.int32, device=DEV)
    ids[-4:] = torch.tensor([5, 128255, 77], dtype=torch.int32, device=DEV)
    top, grad = torch.rand(t, 3, device=DEV), torch.rand(t, device=DEV)
    want = q.distill_topk_grad(tail, ids[-4:].contiguous(), top[-4:].contiguous(), grad[-4:].contiguous())
    loss, d = q.distill_topk_grad(x, ids, top, grad, dlogits=x)
    assert d.data_ptr() == x.data_ptr()
    assert torch.allclose(loss[-4:], want[0], rtol=1e-6, atol=2 * LSE) and not loss[:-4].any()
    assert torch.allclose(d[-4:].float(), want[1].float(), rtol=2 ** -7, atol=1e-9)
    assert not d[:4].any() and not d[-5].any()


def test_streams_and_graphs(q):
    """On a side stream beside other work, and captured: a graph that is replayed on new inputs."""
    x, _ = _rows(64, 9000, BF16, 16)
    other, _ = _rows(64, 9000, BF16, 17)
    ids, top, lse = _teacher(x, 30, 18, 1.0, True)
    grad, tokens = torch.rand(64, device=DEV), torch.arange(64, dtype=torch.int32, device=DEV)

    def calls(z, stream=None):
        loss, stats = q.distill_topk(z, ids, top, top_lse=lse, stream=stream)
        return (loss, stats, q.distill_topk_backward(z, ids, top, stats, grad, top_lse=lse, stream=stream),
                *q.distill_topk_grad(z, ids, top, grad, top_lse=lse, stream=stream),
                *q.token_logprobs_is_grad(z, tokens, grad, grad, stream=stream))

    want = [calls(x), calls(other)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        got = [(calls(x), 0), (calls(other, side), 1), (calls(x), 0)]
        torch.cuda.synchronize()
        for g, i in got:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
        del got, g
    z = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls(z)
    for i, y in ((1, other), (0, x), (1, other)):
        z.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


@pytest.mark.parametrize("y", [1e-9, 1e-7, 0.3, 0.69, 0.7, 3.0, 20.0])
@pytest.mark.parametrize("spread", [0.0, 4.0, 9.0])
def test_rests_of_any_size(q, y, spread):
    """The teacher's rest from 1e-9 to nearly all, beside students with little and with most at the id."""
    v = 1000
    x = torch.zeros(3, v)
    x[:, 17] = torch.tensor([0.0, 1.0, 2.0]) * spread
    x = x.to(DEV)
    ids = torch.full((3, 1), 17, dtype=torch.int32, device=DEV)
    top = torch.zeros(3, 1, device=DEV)
    lse = torch.full((3,), y, device=DEV)
    _check(q, x, ids, top, lse, 1.0)
    _check(q, x.to(BF16), ids, top, lse, 0.7)


def test_slots_in_one_granule(q):
    """Ids side by side, more of them than threads that have a granule, and some of them twice."""
    for dtype in (BF16, FP32):
        x, _ = _rows(3, 2053, dtype, 41, start=3)
        ids = torch.arange(1000, dtype=torch.int32).repeat(3, 1)
        ids[1] += 1053
        ids[2, 500:] = ids[2, :500]
        top = x.float().cpu().gather(1, ids.long()) + 0.3
        lse = torch.logsumexp(x.double(), -1).float() + 1.0
        _check(q, x, ids.to(DEV), top.to(DEV), lse.to(DEV), 1.0)
        _check(q, x, ids.to(DEV), top.to(DEV), None, 1.0)


@pytest.mark.parametrize("temperature", [1e-6, 1e-3, 1e3, 1e6])
def test_extreme_temperatures(q, temperature):
    """Logits over 1e-6 reach 1e7, where a row is its largest logit alone: differences are taken first, and rounded three times
    (the difference, 1 / t, their product) beside what holds at ordinary temperatures."""
    x, _ = _rows(5, 3001, BF16, 51)
    x[3] = torch.where(torch.arange(3001, device=DEV) % 2 == 0, x[3], -torch.inf)
    ids, top, _ = _teacher(x.nan_to_num(neginf=-9.0), 12, 52, 1.0, False)
    ids[3] = ids[3] // 2 * 2
    grad = torch.ones(5, device=DEV)
    loss, stats, ref = _oracle(x, ids, top, None, temperature)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, got_stats = q.distill_topk(x, ids, top, temperature=temperature, dev_status=st)
    again, d = q.distill_topk_grad(x, ids, top, grad, temperature=temperature, dev_status=st)
    d2 = q.distill_topk_backward(x, ids, top, got_stats, grad, temperature=temperature, dev_status=st)
    # of a loss sum p (ln p - ln q) every logarithm is rounded by itself: 3 EPS of (y - y_max) / t and (x - x_max) / t each
    _close(got, loss, 2 * (LSE + P) + 8 * EPS * np.abs(loss), "loss")
    _close(again, loss, 2 * (LSE + P) + 8 * EPS * np.abs(loss), "loss with its gradient")
    _close(got_stats, stats, LSE + 3 * EPS * np.abs(stats), "stats")
    # q and p each within LSE + P and what 3 EPS of an exponent that still counts (below 100) make of them
    scale = (LSE + P + 3 * EPS * 100) * 2 / temperature
    _close(d, ref, scale + np.abs(ref) * 2 ** -8, "gradient")
    if temperature >= 1e-3:  # (below, a known log-sum-exp of 1e7 is rounded to whole numbers)
        known = EPS * np.abs(stats[:, :1]) * 2 / temperature
        _close(d2, ref, scale + 2 * known + np.abs(ref) * 2 ** -8, "backward")
    assert q.get_last_device_status(st) == 0
