"""The drafted rollout and the training step behind it, as the example puts them together: what is verified, learned and
handed on to the adapters, against the float64 oracle, and all of it captured and replayed.

Bounds: log-probabilities and losses as the operators' own tests derive them (LSE = 1.2e-5 for a log-sum-exp, P = 8e-6 for a
teacher's probability); gradients by (LSE + P) of the terms that they are the difference of, here at most the row's weight
each, and the rounding to bf16; the adapters' gradients by the acceptance tolerance of the linear (5e-3 of the norm)."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import distill, verify

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV, LSE, P, EPS = "cuda", 1.2e-5, 8e-6, 2.0 ** -24


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("drafted_policy_update", os.path.join(ROOT, "examples", "drafted_policy_update.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _np(x):
    return x.double().cpu().numpy()


@pytest.mark.parametrize("sequences,n", [(1, 1), (6, 4), (33, 7)])
def test_step(example, sequences, n):
    model, r, out, flags = example.main(sequences, n)
    assert flags == 0
    given = example.numbers(sequences, n, 7, DEV)
    want = verify.batch(_np(r["target"]), r["drafts"].cpu().numpy(), [n] * sequences, _np(given["uniforms"]), _np(given["noise"]),
                        _np(r["draft_logits"]), example.TEMPERATURE)
    tokens, accepted = r["tokens"].cpu().numpy().reshape(sequences, n + 1), r["accepted"].cpu().numpy()
    clear = want[3] > 1e-4
    assert clear.mean() >= 0.9
    assert np.array_equal(tokens[clear], want[0].reshape(sequences, n + 1)[clear]) and np.array_equal(accepted[clear], want[1][clear])
    for b in range(sequences):
        assert np.all(tokens[b, :accepted[b] + 1] >= 0) and np.all(tokens[b, accepted[b] + 1:] == -1)

    # the policy: the same logits as in the rollout, so weights of 1 but for the two calls' roundings
    flat = tokens.reshape(-1)
    logp, w, grad = distill.policy_gradient(_np(out["policy_logits"]), flat, _np(out["weight"]), _np(r["logp"]), 2.0)
    assert np.all(np.abs(_np(out["logp"]) - logp) <= LSE + 3 * EPS * np.abs(logp))
    assert np.all(np.abs(_np(out["w"]) - (flat >= 0)) <= 2 * (LSE + 3 * EPS * np.abs(logp)) + 4 * EPS)
    size = np.abs(_np(out["weight"]))[:, None]
    q = np.exp(_np(out["policy_logits"]) - np.logaddexp.reduce(_np(out["policy_logits"]), -1)[:, None])
    hit = np.zeros_like(q)
    hit[np.arange(len(flat)), np.maximum(flat, 0)] = 1
    bound = size * (3 * LSE + P) * (q + hit) + np.abs(grad) * (2 ** -8 + 4 * EPS) + 1e-37
    assert np.all(np.abs(_np(out["dpolicy"]) - grad) <= bound)
    assert not out["dpolicy"][torch.from_numpy(flat < 0).to(DEV)].any()

    # the draft model
    loss, _, grad = distill.distill(_np(r["draft_logits"]), out["ids"].cpu().numpy(), _np(out["top"]), _np(out["lse"]), example.TEMPERATURE)
    weight = _np(out["grad"])
    assert np.all(np.abs(_np(out["loss"]) - loss) <= 4 * (LSE + P) * (1 + np.abs(loss)))
    grad *= weight[:, None]
    z = _np(r["draft_logits"])
    q = np.exp(z - np.logaddexp.reduce(z, -1)[:, None])
    live = (out["ids"].cpu().numpy() >= 0).any(-1)
    # of the teacher's share of an element: its own probability, or the tail's times the student's share of the tail, where
    # the tail is off by P of the whole mass
    teacher = np.abs(grad / np.maximum(weight, 1e-30)[:, None] - q) + P
    bound = weight[:, None] * ((3 * LSE + P) * (q + teacher) + P * q) + np.abs(grad) * (2 ** -8 + 4 * EPS) + 1e-37
    assert np.all(np.abs(_np(out["ddraft"]) - grad)[live] <= bound[live]) and not _np(out["ddraft"])[~live].any()
    assert live.sum() == np.minimum(accepted + 1, n).sum()

    for got, d, x, lora in ((out["policy"], out["dpolicy"], r["x"], model.policy), (out["draft"], out["ddraft"], r["draft_x"], model.draft)):
        s = lora["alpha"] / lora["lora_A"].shape[0]
        d, x, a, b = d.double(), x.double(), lora["lora_A"].double(), lora["lora_B"].double()
        for g, ref in zip(got, (s * (d @ b).T @ x, s * d.T @ (x @ a.T))):
            assert (g.double() - ref).norm() <= 5e-3 * ref.norm()


def test_captured(example):
    """Rollout and step in one graph, replayed on other numbers: the same bits as eagerly."""
    b, n = 5, 3
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    model = example.Model(n + 1, torch.device(DEV, 0))
    advantages = torch.linspace(-1.0, 1.0, b, device=DEV)

    def run(given):
        r = example.rollout(model, n=n, status=status, **given)
        out = example.step(model, r, n, advantages, status)
        return [r["tokens"], r["accepted"], r["logp"], out["dpolicy"], out["loss"], out["ddraft"], *out["policy"], *out["draft"]]

    sets = [example.numbers(b, n, seed, DEV) for seed in (11, 12, 13)]
    want = [run(s) for s in sets]
    held = {k: v.clone() for k, v in sets[0].items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(held)
    for i in (2, 0, 1):
        for k, v in held.items():
            v.copy_(sets[i][k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want[i])), i
    assert int(status.item()) == 0


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("temperature", [0.7, 1.0])
def test_gradient_is_the_difference(example, tail, temperature):
    """The losses' own gradient along a direction d, |d| <= 1, against their central difference at h = 0.05.

    A loss is off by (LSE + P) (2 + loss) at most, which the difference divides by h; and the difference by h^2 / 6 of the
    third derivative, which for each of two log-sum-exps is a third cumulant of d / t, below (1 / t)^3."""
    from quantized_rl_rollout_gb300 import qrr

    g = torch.Generator().manual_seed(3)
    t, v, k, h = 7, 1500, 40, 0.05
    x = (2 * torch.randn(t, v, generator=g)).to(DEV)
    y = x.cpu() + torch.randn(t, v, generator=g)
    top, ids = torch.topk(y, k, -1)
    more = dict(top_lse=torch.logsumexp(y / temperature, -1).to(DEV) if tail else None, temperature=temperature)
    top, ids = top.to(DEV), ids.to(torch.int32).to(DEV)
    d = torch.where(y > y.median(), 1.0, -1.0).to(DEV) * torch.rand(t, v, generator=g).to(DEV)
    loss, grad = qrr.distill_topk_grad(x, ids, top, torch.ones(t, device=DEV), **more)
    sides = [qrr.distill_topk(x + s * h * d, ids, top, **more)[0].double() for s in (1, -1)]
    along = (grad.double() * d.double()).sum(-1)
    size = (grad.abs().double() * d.abs().double()).sum(-1)
    bound = (LSE + P) * (2 + loss.double()) / h + h * h / 3 / temperature ** 3 + (LSE + P) * (2 + size)
    assert torch.all(((sides[0] - sides[1]) / (2 * h) - along).abs() <= bound)
    # (what is compared is mostly large beside the bound: its sign, and so its being small in some row, is the rows' chance)
    assert (along.abs() > 3 * bound).double().mean() >= 0.5


def test_two_streams(example):
    """Rollouts on two streams at once, each with its own adapters' gradients: the same bits as one after the other."""
    b, n = 9, 4
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    model = example.Model(n + 1, torch.device(DEV, 0))
    advantages = torch.linspace(-1.0, 1.0, b, device=DEV)
    sets = [example.numbers(b, n, seed, DEV) for seed in (21, 22)]

    def run(given):
        r = example.rollout(model, n=n, status=status, **given)
        out = example.step(model, r, n, advantages, status)
        return [r["tokens"], r["accepted"], r["logp"], out["dpolicy"], out["loss"], out["ddraft"], *out["policy"], *out["draft"]]

    want = [run(s) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for stream, given in zip(streams, sets):
            with torch.cuda.stream(stream):
                got.append(run(given))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(g, w))
