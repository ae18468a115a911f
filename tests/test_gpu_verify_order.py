"""Verification of sequences of very different lengths, whose places are not all looked at place by place (test_verify_order.py
says which): against the oracle, as test_gpu_verify_drafts.py does."""

import pytest
import torch

from .test_gpu_verify_drafts import BF16, DEV, FORMS, FP32, _case, _check, _run, q  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("counts,v", [([700] + [0, 1] * 300, 40), ([0, 1, 2] * 200 + [900], 17), ([1] * 100 + [300] + [0] * 400 + [250], 9000)])
def test_one_long_sequence(q, counts, v, dtype, form):  # noqa: F811
    s = _case(counts, v, dtype, form, len(counts), spread=0.01, temperature=0.5)
    if form != "greedy":
        s["uniforms"] *= 0.05
    else:
        n, at = counts.index(max(counts)), 0
        first = sum(counts[:n])
        rows = s["target"][first + n:first + n + counts[n]]
        s["drafts"][first:first + counts[n]] = rows.float().argmax(-1).to(torch.int32)
    long = counts.index(max(counts))
    for last in (None, v - 1, -1):  # its drafts are taken nearly all; to a place far behind the others' ends; padded from there on
        if last is not None:
            s["drafts"][sum(counts[:long]) + counts[long] * 3 // 4] = last
        _, accepted, _ = _check(q, s, enough=0.8)
        if form != "lookup":
            assert accepted.max() > 100


def test_among_bad_offsets_and_padding(q):  # noqa: F811
    """One long sequence, offsets that descend elsewhere, places of no sequence: the others' outputs are as without them."""
    counts = [2] * 300 + [600] + [1] * 300
    s = _case(counts, 50, BF16, "model", 3, spread=0.01, temperature=0.5)
    s["uniforms"] *= 0.05
    want = _run(q, s)
    cu = torch.zeros(len(counts) + 1, dtype=torch.int64)
    cu[1:] = torch.tensor(counts).cumsum(0)
    b = len(counts)
    ws = torch.randint(-2 ** 31, 2 ** 31 - 1, (1 << 20,), dtype=torch.int32, device=DEV).view(torch.uint8)  # what stood there does not count
    for bad, at in ((b - 1, -5), (b, 2 ** 31 - 1), (b, -2 ** 31)):
        given = cu.clone()
        given[bad] = at if bad == b else given[bad - 1] - 3
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        n = s["target"].shape[0]
        tokens, logp = torch.full((n,), 12345, dtype=torch.int32, device=DEV), torch.full((n,), 0.5, device=DEV)
        accepted = torch.full((b,), 777, dtype=torch.int32, device=DEV)
        q.verify_drafts(s["target"], s["drafts"], uniforms=s["uniforms"], noise=s["noise"], draft_logits=s["draft_logits"],
                        cu=given.to(torch.int32).to(DEV), temperature=s["temperature"], tokens=tokens, accepted=accepted, logp=logp,
                        workspace=ws.clone(), dev_status=st)
        assert q.get_last_device_status(st) == q.DEV_BAD_INDEX
        live = min(bad, b) - 4  # (those behind share places with the bad one)
        rows = int(cu[live]) + live
        assert torch.equal(accepted[:live], want[1][:live]) and accepted[300] > 100
        assert torch.equal(tokens[:rows], want[0][:rows]) and torch.equal(logp[:rows], want[2][:rows])


@pytest.mark.parametrize("form", FORMS)
def test_a_sequence_alone(q, form):  # noqa: F811
    """A sequence's outputs are bit for bit those that it has without the others (of rows that start alike)."""
    counts, v = [3, 0, 5, 1, 2] * 40, 20000
    s = _case(counts, v, BF16, form, 4)
    tokens, accepted, logp = _run(q, s)
    at = 0
    for b, n in enumerate(counts[:15]):
        rows, drafts = slice(at + b, at + b + n + 1), slice(at, at + n)
        of = lambda x, i: None if x is None else x[i]  # noqa: E731
        one = q.verify_drafts(s["target"][rows], s["drafts"][drafts], uniforms=of(s["uniforms"], drafts), noise=of(s["noise"], slice(b, b + 1)),
                              draft_logits=of(s["draft_logits"], drafts), temperature=s["temperature"])
        assert torch.equal(one[0], tokens[rows]) and int(one[1]) == int(accepted[b]) and torch.equal(one[2], logp[rows])
        at += n
