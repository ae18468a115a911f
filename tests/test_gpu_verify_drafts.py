"""GPU parity of the verification of drafted tokens against the float64 oracle.

Tokens and counts have to be the oracle's wherever its decisions are not nearer than NEAR (relative) to going the other way:
probabilities are off by the exponentials (2^-22), their arguments' rounding (2^-23 of at most 40: 5e-6) and a row's sum
(1.2e-5, as test_gpu_logits_loss.py derives).  Log-probabilities are within 1.2e-5 + 3 2^-24 of themselves."""

import numpy as np
import pytest
import torch

from oracle import verify

pytestmark = pytest.mark.gpu
DEV = "cuda"
NEAR, LSE, EPS = 6e-5, 1.2e-5, 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    from quantized_rl_rollout_gb300 import build, qrr

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    qrr.lib()
    return qrr


def _case(counts, v, dtype, form, seed, temperature=1.0, pad=0, spread=0.7):
    """Target rows (some tokens stand out), drafts that mostly pass, random numbers."""
    g = torch.Generator().manual_seed(seed)
    t, b = sum(counts), len(counts)

    def padded(x, dt=dtype, gap=pad):
        out = torch.full((x.shape[0], v + gap), float("nan"), dtype=dt)
        out[:, :v] = x.to(dt)
        return out.to(DEV)[:, :v]

    x = 1.5 * torch.randn(t + b, v, generator=g)
    peaks = torch.randint(0, v, (t + b, 6), generator=g)
    x.scatter_add_(1, peaks, 8 * torch.rand(t + b, 6, generator=g))
    x = x.to(dtype).float()
    rows = torch.tensor([sum(counts[:i]) + i + j for i in range(b) for j in range(counts[i])], dtype=torch.long)
    s = dict(target=padded(x), counts=counts, temperature=temperature, draft_logits=None, uniforms=None, noise=None)
    y = x[rows]
    if form == "model":
        y = (y + spread * torch.randn(t, v, generator=g)).to(dtype).float()
        s["draft_logits"] = padded(y)
        y = y / temperature - torch.log(-torch.log(torch.rand(t, v, generator=g).clamp(1e-9, 1 - 1e-7)))
    if form != "greedy":
        s["uniforms"] = torch.rand(t, generator=g).to(DEV)
        s["noise"] = padded(torch.empty(b, v).exponential_(generator=g).clamp(min=1e-20), FP32, pad)
    drafts = y.argmax(-1) if t else torch.empty(0, dtype=torch.long)
    if form == "greedy":
        drafts = torch.where(torch.rand(t, generator=g) < 0.25, torch.randint(0, v, (t,), generator=g), drafts)
        s["temperature"] = 0.0
    s["drafts"] = drafts.to(torch.int32).to(DEV)
    return s


def _cu(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)


def _run(q, s, **more):
    args = dict(uniforms=s["uniforms"], noise=s["noise"], draft_logits=s["draft_logits"], temperature=s["temperature"])
    if "cu" not in more:
        args["cu"] = _cu(s["counts"])
    args.update(more)
    return q.verify_drafts(s["target"], s["drafts"], **args)


def _check(q, s, enough=0.9, flags=0, **more):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    tokens, accepted, logp = _run(q, s, dev_status=st, **more)
    assert q.get_last_device_status(st) == flags
    host = lambda x: None if x is None else x.double().cpu().numpy()  # noqa: E731
    want = verify.batch(host(s["target"]), s["drafts"].cpu().numpy(), s["counts"], host(s["uniforms"]), host(s["noise"]),
                        host(s["draft_logits"]), s["temperature"])
    clear = want[3] > NEAR
    assert clear.mean() >= enough
    at = 0
    for b, n in enumerate(s["counts"]):
        if clear[b]:
            rows = slice(at, at + n + 1)
            assert int(accepted[b]) == want[1][b], b
            assert tokens[rows].tolist() == want[0][rows].tolist(), b
            lp = want[2][rows]
            assert np.all(np.abs(logp[rows].double().cpu().numpy() - lp) <= LSE + 3 * EPS * np.abs(lp)), b
        at += n + 1
    return tokens, accepted, logp


FORMS = ["model", "lookup", "greedy"]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("counts,v,pad", [([0], 1, 0), ([1], 2, 0), ([3, 0, 2], 7, 1), ([4] * 5, 1000, 0), ([2, 9, 0, 1], 8195, 3),
                                          ([5, 3], 32000, 8), ([1, 4], 50001, 0), ([4], 128256, 0), ([0, 0, 0], 300, 0)])
def test_shapes(q, counts, v, pad, dtype, form):
    _check(q, _case(counts, v, dtype, form, v + len(counts), pad=pad), enough=0.5 if len(counts) < 10 else 0.9)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("batch", [1, 40, 160, 400])
def test_batches(q, batch, form):
    """Clusters of many CTAs, rows in one group; of few, row by row."""
    s = _case([(3 * b) % 7 for b in range(batch)] if batch > 1 else [6], 3000, BF16, form, batch, temperature=0.8)
    tokens, accepted, _ = _check(q, s)
    if batch >= 40:
        assert accepted.max() >= 3 and (accepted.cpu() < torch.tensor(s["counts"])).any()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("batch", [2, 320])
def test_more_drafts_than_a_group(q, batch, form):
    """Dozens of drafts that nearly all pass: groups after groups, with a refusal in the second or third."""
    s = _case([40] * batch, 600, FP32, form, 3, spread=0.02, temperature=0.25)
    if form != "greedy":
        s["uniforms"] *= 0.05
        s["uniforms"][33::80] = 0.999
    else:
        s["drafts"] = torch.tensor([int(x) for b in range(batch) for x in s["target"][41 * b:41 * b + 40].argmax(-1)],
                                   dtype=torch.int32, device=DEV)
        s["drafts"][33::80] = 0
    _, accepted, _ = _check(q, s)
    assert accepted.max() > 32


@pytest.mark.parametrize("temperature", [0.3, 1.0, 3.0])
def test_temperature(q, temperature):
    _check(q, _case([4] * 30, 2001, BF16, "model", 5, temperature=temperature))


def test_even_counts_need_no_offsets(q):
    s = _case([3] * 20, 1001, BF16, "model", 6)
    for a, b in zip(_run(q, s), _run(q, s, cu=None)):
        assert torch.equal(a, b)


def test_same_logits_pass_and_masked_ones_do_not(q):
    s = _case([5] * 12, 700, BF16, "model", 7)
    rows = [i for i in range(72) if i % 6 != 5]
    s["draft_logits"] = s["target"][rows].contiguous()
    s["uniforms"].fill_(1 - 2.0 ** -24)  # the largest below 1
    # Rows of 700 start at either half of a 16-byte granule, so the two sums of one row are taken in different orders and
    # differ by up to 2 LSE of themselves; u is 2^-24 from 1: nearer than that, and a draft may be refused.  (Once u is
    # farther than NEAR from 1, none is; and where rows start alike, the sums are the same and none is whatever u is.)
    _check(q, s, enough=0.0)
    s["uniforms"].fill_(1 - 2 * NEAR)
    _, accepted, _ = _run(q, s)
    assert (accepted == 5).all()
    even = _case([5] * 12, 704, BF16, "model", 7)
    even["draft_logits"] = even["target"][rows].contiguous()
    even["uniforms"].fill_(1 - 2.0 ** -24)
    _, accepted, _ = _run(q, even)
    assert (accepted == 5).all()
    s["uniforms"].zero_()
    for b in range(12):  # the target rules the third draft out
        s["target"][6 * b + 2, s["drafts"][5 * b + 2].long()] = -torch.inf
    # what is left is q p_d / (1 - p_d): for two sequences, whose p_d is small, less than NEAR lies between the first scores
    tokens, accepted, _ = _check(q, s, enough=10 / 12)
    assert (accepted == 2).all()
    # Refused though nothing is left of p behind q: a token of p.  (Of the rows that start alike, see above.)
    even["uniforms"].fill_(1.0)
    tokens, accepted, logp = _run(q, even)
    first = tokens.view(12, 6)[:, 0]
    p = torch.softmax(even["target"][::6].double(), -1)
    assert (accepted == 0).all() and torch.equal(first.long(), (p / even["noise"].double()).argmax(-1)) and (logp.view(12, 6)[:, 0] < 0).all()


def test_padded_drafts(q):
    """A negative draft ends its sequence's drafts, and the token there is one of p; an id behind the vocabulary as well,
    with a flag."""
    s = _case([4] * 9, 900, BF16, "model", 8)
    s["uniforms"].zero_()
    s["drafts"][2::4] = -1
    tokens, accepted, _ = _check(q, s)
    assert (accepted == 2).all() and (tokens.view(9, 5)[:, 3:] == -1).all()
    s["drafts"][1::4] = 900
    tokens, accepted, _ = _check(q, s, flags=q.DEV_BAD_INDEX)
    assert (accepted == 1).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_likeliest_of_equals_is_the_lowest(q, dtype):
    for v in (9, 5000, 70001):
        x = torch.zeros(6, v, dtype=dtype, device=DEV)
        x[1, v // 2:] = 1.0
        x[2, v - 1] = 1.0
        x[3] = torch.finfo(dtype).min
        x[4, 1] = -torch.inf
        x[5, 0] = -torch.inf
        tokens, accepted, logp = q.verify_drafts(x, torch.empty(0, dtype=torch.int32, device=DEV), temperature=0.0)
        assert tokens.tolist() == [0, v // 2, v - 1, 0, 0, 1] and not accepted.any()
        assert torch.allclose(logp[3].double(), -torch.tensor(float(v)).double().log().to(DEV), rtol=0, atol=2 * LSE)


@pytest.mark.parametrize("form", FORMS)
def test_rows_without_probabilities(q, form):
    """A row of -inf gives -1, a NaN or +inf a token of the vocabulary or -1; each is flagged, and other sequences keep theirs."""
    for bad in (float("nan"), float("inf"), -float("inf")):
        s = _case([2] * 6, 800, BF16, form, 9)
        want = _run(q, s)
        if bad < 0:
            s["target"][3] = bad
        else:
            s["target"][3, 77] = bad
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = _run(q, s, dev_status=st)
        assert q.get_last_device_status(st) == q.DEV_NONFINITE
        assert got[0][3] == -1 if bad < 0 else -1 <= int(got[0][3]) < 800
        keep = [i for i in range(18) if i // 3 != 1]
        assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[2][keep], want[2][keep])


def test_offsets(q):
    """Places that belong to no sequence are left as they were; offsets that descend or leave the drafts write nothing."""
    s = _case([2, 3, 1], 500, BF16, "model", 10)
    t, b = 6, 3
    want = _run(q, s)

    def call(cu, flags, target=s["target"], drafts=s["drafts"], draft=s["draft_logits"], u=s["uniforms"]):
        n = drafts.numel() + b
        tokens, logp = torch.full((n,), 12345, dtype=torch.int32, device=DEV), torch.full((n,), 0.5, device=DEV)
        accepted, st = torch.full((b,), 777, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        q.verify_drafts(target, drafts, uniforms=u, noise=s["noise"], draft_logits=draft, cu=torch.tensor(cu, dtype=torch.int32, device=DEV),
                        tokens=tokens, accepted=accepted, logp=logp, dev_status=st)
        assert q.get_last_device_status(st) == flags
        return tokens, accepted, logp

    pad = lambda x, rows, at: torch.cat([x[:at], x.new_zeros((rows,) + tuple(x.shape[1:])), x[at:]])  # noqa: E731
    # two drafts before the first sequence and two behind the last
    big = dict(target=pad(pad(s["target"], 2, 0), 2, t + b + 2), drafts=pad(pad(s["drafts"], 2, 0), 2, t + 2),
               draft=pad(pad(s["draft_logits"], 2, 0), 2, t + 2), u=pad(pad(s["uniforms"], 2, 0), 2, t + 2))
    tokens, accepted, logp = call([2, 4, 7, 8], 0, **big)
    assert torch.equal(tokens[2:-2], want[0]) and torch.equal(accepted, want[1]) and torch.equal(logp[2:-2], want[2])
    assert (tokens[:2] == 12345).all() and (tokens[-2:] == 12345).all() and (logp[:2] == 0.5).all() and (logp[-2:] == 0.5).all()
    for cu, live in [([0, 2, 5, 7], [0, 1]), ([-1, 2, 5, 6], [1, 2]), ([0, 2, 1, 6], [0]), ([0, 2, 5, -2 ** 31], [0, 1]),
                     ([0, 2, 5, 2 ** 31 - 1], [0, 1])]:
        tokens, accepted, _ = call(cu, q.DEV_BAD_INDEX)
        assert accepted[live].tolist() == want[1][live].tolist()
        bad = [i for i in range(b) if cu[i] < 0 or cu[i + 1] < cu[i] or cu[i + 1] > t]
        assert bad and (accepted[bad] == 777).all()


def test_noise_rows_and_alignment(q):
    """Rows of the target, the draft and the noise that start at different places of a 16-byte granule."""
    for v, gaps in ((1000, (0, 1, 3)), (1003, (2, 5, 1)), (2048, (8, 4, 2))):
        s = _case([3] * 8, v, BF16, "model", 11)
        want = _check(q, s)
        for name, gap in zip(("target", "draft_logits", "noise"), gaps):
            wide = torch.full((s[name].shape[0], v + gap), float("nan"), dtype=s[name].dtype, device=DEV)
            wide[:, :v] = s[name]
            s[name] = wide[:, :v]
        got = _run(q, s)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.allclose(got[2], want[2], rtol=1e-6, atol=LSE)


def test_distribution(q):
    """First tokens of many sequences with one target row: as often as its probabilities say (5 sigma)."""
    n, v = 20000, 6
    g = torch.Generator(device=DEV).manual_seed(12)
    p, y = torch.tensor([0.3, 1.0, -1.0, 0.7, 0.0, -2.0], device=DEV), torch.tensor([1.2, -0.5, 0.4, 0.1, 0.0, 1.0], device=DEV)
    drafts = torch.multinomial(torch.softmax(y, -1), n, replacement=True, generator=g).to(torch.int32)
    for draft_logits in (y.expand(n, v).contiguous(), None):
        tokens, _, _ = q.verify_drafts(p.expand(2 * n, v).contiguous(), drafts, uniforms=torch.rand(n, generator=g, device=DEV),
                                       noise=torch.empty(n, v, device=DEV).exponential_(generator=g), draft_logits=draft_logits)
        want = torch.softmax(p.double(), -1)
        got = torch.bincount(tokens[::2].long(), minlength=v).double() / n
        if draft_logits is None:  # lookups follow p whatever the drafts are
            assert got.shape == want.shape
        assert torch.all((got - want).abs() <= 5 * torch.sqrt(want * (1 - want) / n))


def test_nothing(q):
    x = torch.empty(0, 50, dtype=BF16, device=DEV)
    tokens, accepted, logp = q.verify_drafts(x, torch.empty(0, dtype=torch.int32, device=DEV), temperature=0.0)
    assert tokens.numel() == accepted.numel() == logp.numel() == 0


def test_streams_and_graphs(q):
    cases = [_case([4] * 24, 6001, BF16, "model", 13 + i) for i in range(2)]
    want = [_run(q, s, cu=None) for s in cases]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        got = [(_run(q, cases[0], cu=None), 0), (_run(q, cases[1], cu=None, stream=side), 1), (_run(q, cases[0], cu=None), 0)]
        torch.cuda.synchronize()
        for g, i in got:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
        del got, g
    z = {k: x.clone() if torch.is_tensor(x) else x for k, x in cases[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _run(q, z, cu=None)
    for i in (1, 0, 1):
        for k in ("target", "draft_logits", "uniforms", "noise", "drafts"):
            z[k].copy_(cases[i][k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


@pytest.mark.parametrize("form", FORMS)
def test_counts_far_apart(q, form):
    """One long sequence among short and empty ones, and many sequences: more parts of rows than there are CTAs to sum them."""
    _check(q, _case([0] * 20 + [120] + [1, 0, 2] * 20, 5000, BF16, form, 31, spread=0.05), enough=0.5)
    _check(q, _case([3, 1, 0, 2] * 400, 300, FP32, form, 32), enough=0.8)


def test_refusals_are_seen_in_time(q):
    """Sequences that are refused at each place in turn, with rows behind the refusal that would raise a flag if they counted."""
    n, v = 12, 40000
    s = _case([n] * (n + 1), v, BF16, "greedy", 33)
    target = s["target"].clone()
    s["drafts"] = s["drafts"].view(n + 1, n).clone()
    best = target.float().argmax(-1).view(n + 1, n + 1)
    for b in range(n + 1):
        s["drafts"][b] = best[b, :n].to(torch.int32)
        if b < n:
            s["drafts"][b, b] = (best[b, b] + 1) % v
        target.view(n + 1, n + 1, v)[b, b + 1:] = float("nan")
    s["drafts"], s["target"] = s["drafts"].view(-1), target
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(20):
        tokens, accepted, logp = _run(q, s, dev_status=st)
        assert accepted.tolist() == list(range(n + 1))
        tokens = tokens.view(n + 1, n + 1)
        for b in range(n + 1):
            assert torch.equal(tokens[b, :b + 1].long(), best[b, :b + 1]) and torch.all(tokens[b, b + 1:] == -1)
    assert q.get_last_device_status(st) == 0


@pytest.mark.parametrize("form", ["model", "lookup"])
@pytest.mark.parametrize("temperature", [1e-6, 1e-3, 1e3, 1e6])
def test_extreme_temperatures(q, form, temperature):
    """Near 0 the likeliest token, as if greedy; far above nearly uniform. A log-probability is (x - x_max) / t - ln s: 3 EPS of
    the first more than at ordinary temperatures, which `_check` grants of the whole."""
    s = _case([3, 0, 5, 2] * 3, 3001, BF16, form, 61, temperature=1.0, spread=0.2)
    s["temperature"] = temperature
    _check(q, s, enough=0.7)
    if temperature == 1e-6 and form == "lookup":  # (a model's draft is taken by p / q, however unlikely both are)
        tokens, _, _ = _run(q, s)
        used, rows = tokens >= 0, s["target"].float()
        # (an exponential noise of 1e-20 at another token cannot make up for e^-7000)
        assert torch.equal(rows[used].gather(1, tokens[used].long()[:, None])[:, 0], rows[used].amax(-1))
