"""GPU parity of the paged NVFP4 cache against the oracle: written codes and
scales and values read back bit for bit, attention within a derived tolerance,
and refusals.

Tolerances of attention.  A weight p_j carries a relative error of 2^-11 (its
rounding to f16) plus that of its score: products are exact and summed in fp32
by the tensor core, an absolute error of at most 2^-20 M with M the largest
scale sum_d |q_d k_d| of the row; exponentials add 2^-21.  So lse is within
2^-19 (M + 1), and out within 2^-9 |out| (its own rounding to bf16) plus
(2^-11 + 2^-19 (M + 1)) times sum_j p_j |v_j| / sum_j p_j.  f16 has an absolute
spacing of 2^-24 below 2^-14, and the row's largest weight is carried as at
least 2^7: a weight below 2^-21 of it is off by up to 2^-32 of it, which adds
2^-32 sum_j |v_j|.  All doubled."""

import numpy as np
import pytest
import torch

from oracle import kv_nvfp4 as kv
from oracle.formats import bf16_rne
from quantized_rl_rollout_gb300 import inputs

from .conftest import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def q():
    from quantized_rl_rollout_gb300 import build, qrr

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    qrr.lib()
    return qrr


class Bed:
    """A cache of ``lens`` tokens a sequence, every byte that no token wrote 0xFF (scales that decode to NaN), pages in
    a shuffled order, and its oracle copy.  The global scales differ by head."""

    def __init__(self, q, lens, hkv, dim, page, seed, gs=True, spread=1.0):
        self.q, self.lens, self.hkv, self.dim, self.page = q, lens, hkv, dim, page
        b = len(lens)
        per = max(1, max(-(-max(n, 0) // page) for n in lens))
        g = torch.Generator().manual_seed(seed)
        pages = b * per + 2
        table = torch.randperm(pages, generator=g)[:b * per].view(b, per).to(torch.int32)
        self.table = table.numpy()
        self.gs = [torch.linspace(0.01, 0.05, hkv), torch.linspace(0.02, 0.004, hkv)] if gs else [torch.ones(hkv)] * 2
        full = [torch.full((pages, hkv, page, dim // d), 0xFF, dtype=torch.uint8, device=DEV) for d in (2, 16, 2, 16)]
        self.cache = q.KvCacheNvfp4(*full, table.to(DEV), *([x.to(DEV) for x in self.gs] if gs else (None, None)))
        cu = np.concatenate([[0], np.cumsum([max(n, 0) for n in lens])]).astype(np.int32)
        t = int(cu[-1])
        self.k = (spread * inputs.activations(max(t, 1) * hkv, dim, inputs.derive_seed(seed, "k"), device=DEV).float()).to(
            torch.bfloat16).view(-1, hkv, dim)[:t]
        self.v = inputs.activations(max(t, 1) * hkv, dim, inputs.derive_seed(seed, "v"), device=DEV).view(-1, hkv, dim)[:t]
        self.cu = cu
        if t:
            q.kv_append_nvfp4(self.k, self.v, self.cache, torch.zeros(b, dtype=torch.int32, device=DEV),
                              cu=torch.from_numpy(cu).to(DEV))

    def values(self, b):
        """The oracle's values of sequence b, from its own quantization of the rows."""
        s = slice(self.cu[b], self.cu[b + 1])
        return [kv.kv_values(*kv.kv_quantize(to_np(x[s]), to_np(g)), to_np(g)) for x, g in ((self.k, self.gs[0]), (self.v, self.gs[1]))]


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _attend(bed, hq, news, strided=False, stream=None, q_scale=1.0, scale=None):
    """Attention of the last ``news[b]`` tokens of every sequence, checked against the oracle; returns (out, lse)."""
    q = bed.q
    t = sum(news)
    wide = torch.randn(t, hq + 3, bed.dim, generator=torch.Generator(device=DEV).manual_seed(t + hq), device=DEV) * q_scale
    wide = wide.to(torch.bfloat16)
    x = wide[:, 1:hq + 1] if strided else wide[:, :hq].contiguous()
    pos = [n - m for n, m in zip(bed.lens, news)]
    one = all(m == 1 for m in news)
    cu = None if one else _dev(np.concatenate([[0], np.cumsum(news)]))
    st = _dev([0])
    if stream is not None:
        torch.cuda.synchronize()
    out, lse = q.attention_nvfp4(x, bed.cache, _dev(pos), cu=cu, max_new=max(news), return_lse=True, dev_status=st,
                                 stream=stream, scale=scale)
    assert q.get_last_device_status(st, stream) == 0
    sc = bed.dim ** -0.5 if scale is None else scale
    xs, o, e = to_np(x), to_np(out), to_np(lse)
    at = 0
    for b, m in enumerate(news):
        k, v = bed.values(b)
        rows = xs[at:at + m]
        want, want_lse, spread = kv.attention(rows, k, v, pos[b], sc)
        g = hq // bed.hkv
        big = np.zeros((m, hq))
        for h in range(hq):
            if len(k):
                big[:, h] = (np.abs(rows[:, h].astype(np.float64)) @ np.abs(k[:, h // g]).T).max(-1) * sc
        tol = 2 ** -18 * (big + 1)
        got, got_lse = o[at:at + m], e[at:at + m]
        none = np.isneginf(want_lse)
        assert np.array_equal(none, np.isneginf(got_lse))
        assert not got[none].any()
        off = np.abs(got_lse[~none] - want_lse[~none])
        assert (off <= tol[~none]).all(), (b, off.max())
        bound = 2 ** -8 * np.abs(want) + (2 ** -10 + tol)[..., None] * spread + 2 ** -31 * np.repeat(np.abs(v).sum(0), g, 0) + 1e-30
        worst = (np.abs(got - want) / bound).max() if m else 0
        assert worst <= 1, (b, worst)
        at += m
    return out, lse


@pytest.mark.parametrize("dim,hkv,page,gs", [(128, 8, 16, True), (64, 3, 32, True), (128, 1, 64, False), (64, 4, 256, False)])
def test_write_and_read_back(q, dim, hkv, page, gs):
    lens = [1, 37, 0, 130, 16]
    bed = Bed(q, lens, hkv, dim, page, 3, gs=gs)
    kc, ks, vc, vs = (x.cpu().numpy() for x in bed.cache.tensors[:4])
    touched = np.zeros(kc.shape[:3], bool)
    for b, n in enumerate(lens):
        s = slice(bed.cu[b], bed.cu[b + 1])
        for pool, scales, rows, g in ((kc, ks, bed.k, bed.gs[0]), (vc, vs, bed.v, bed.gs[1])):
            c, e = kv.kv_quantize(to_np(rows[s]), to_np(g))
            assert np.array_equal(kv.gather(pool, bed.table[b], n), c) and np.array_equal(kv.gather(scales, bed.table[b], n), e)
        p = np.arange(n)
        touched[bed.table[b][p // page], :, p % page] = True
    assert (kc[~touched] == 0xFF).all() and (vs[~touched] == 0xFF).all()  # nothing else is written
    # back: from the start, and a range inside
    for pos, news in (([0] * 5, lens), ([0, 20, 0, 100, 15], [1, 9, 0, 30, 1])):
        cu = np.concatenate([[0], np.cumsum(news)])
        got = q.kv_read_nvfp4(bed.cache, _dev(pos), cu=_dev(cu), rows=int(cu[-1]))
        for b in range(5):
            for x, want, g in zip(got, bed.values(b), bed.gs):
                unit = (want / to_np(g).astype(np.float64)[:, None]).astype(np.float32)  # code x block scale: exact
                r = bf16_rne(unit * to_np(g)[:, None])[pos[b]:pos[b] + news[b]]
                assert np.array_equal(to_np(x[cu[b]:cu[b + 1]]), r)


def test_write_extremes(q):
    """Zero blocks, subnormals, saturation, the largest finite values, and both signs of zero."""
    dim = 64
    x = torch.zeros(6, 1, dim, dtype=torch.bfloat16, device=DEV)
    x[1] = 1e-39
    x[2] = torch.linspace(-3, 3, dim).to(torch.bfloat16)
    x[3, 0, ::2] = 3.3e38
    x[4] = -0.0
    x[5, 0, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 2)  # the grid's midpoints
    x[5, 0, 16:32] = -x[5, 0, :16]
    cache = q.KvCacheNvfp4.empty(1, 1, 16, dim, _dev([[0]]))
    st = _dev([0])
    q.kv_append_nvfp4(x, x, cache, _dev([0]), cu=_dev([0, 6]), dev_status=st)
    assert q.get_last_device_status(st) == 0
    c, e = kv.kv_quantize(to_np(x), [1.0])
    assert np.array_equal(cache.tensors[0][0, :, :6].cpu().numpy().transpose(1, 0, 2), c)
    assert np.array_equal(cache.tensors[1][0, :, :6].cpu().numpy().transpose(1, 0, 2), e)


def test_write_places_and_flags(q):
    cache = q.KvCacheNvfp4.empty(3, 2, 16, 64, _dev([[0, 1], [2, 7]]))
    x = torch.randn(6, 2, 64, device=DEV).to(torch.bfloat16)
    st = _dev([0])
    q.kv_append_nvfp4(x, x, cache, _dev([-2, 15]), cu=_dev([0, 3, 4]), dev_status=st)  # rows 4 and 5 belong to nobody
    assert q.get_last_device_status(st) == 0
    k = cache.tensors[1]
    assert k[0, :, 0].any() and not k[0, :, 1:].any() and not k[1].any() and k[2, :, 15].any() and not k[2, :, :15].any()
    a, _ = q.kv_read_nvfp4(cache, _dev([-2, 15]), cu=_dev([0, 3, 4]), k=torch.full_like(x, 7), v=torch.full_like(x, 7))
    assert not a[:2].any() and a[2].any() and a[3].any()
    for pos in ([0, 16], [0, 32], [40, 0]):  # a page that is not there, positions behind the table
        st.zero_()
        before = [t.clone() for t in cache.tensors[:4]]
        q.kv_append_nvfp4(x[:2], x[:2], cache, _dev(pos), dev_status=st)
        assert q.get_last_device_status(st) == q.DEV_BAD_INDEX
        bad = 1 if pos[0] == 0 else 0
        seq = [0, 1] if bad else [2]
        rest = [i for i in range(3) if i not in seq]
        assert all(torch.equal(t[rest], o[rest]) for t, o in zip(cache.tensors[:4], before))
        st.zero_()
        got = q.kv_read_nvfp4(cache, _dev(pos), dev_status=st)
        assert q.get_last_device_status(st) == q.DEV_BAD_INDEX and not got[0][bad].any()
        q.attention_nvfp4(torch.randn(2, 4, 64, device=DEV).to(torch.bfloat16), cache, _dev(pos), dev_status=st)
        assert q.get_last_device_status(st) == q.DEV_BAD_INDEX
    x[1, 1, 5] = float("inf")
    st.zero_()
    q.kv_append_nvfp4(x[:2], x[:2], cache, _dev([0, 0]), dev_status=st)
    assert q.get_last_device_status(st) == q.DEV_NONFINITE


HEADS = [(8, 8), (8, 4), (32, 8), (10, 2), (7, 1), (16, 2), (48, 3)]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_decode_heads(q, dim, hq, hkv):
    _attend(Bed(q, [1, 300, 17], hkv, dim, 32, 5), hq, [1, 1, 1], strided=True)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("lens", [[1, 15, 16, 17, 31, 32, 33], [127, 128, 129, 0, 255, 257], [2000], [5, 3000, 64, 1]])
def test_decode_lengths(q, page, lens):
    """A sequence without tokens (length 0: its row stands at -1) sees nothing."""
    _attend(Bed(q, lens, 2, 128, page, 6), 8, [1] * len(lens))


@pytest.mark.parametrize("dim,hq,hkv", [(128, 8, 2), (64, 4, 4), (128, 5, 1), (64, 16, 2), (128, 32, 2)])
@pytest.mark.parametrize("lens,news", [
    ([40, 300, 9], [3, 2, 5]), ([64, 1], [64, 1]), ([129, 200], [129, 33]), ([20, 0, 400], [20, 0, 257]), ([3], [7]),
    ([130, 0, 260], [131, 4, 1])])
def test_several_rows(q, dim, hq, hkv, lens, news):
    """Rows before the first token (more rows than tokens) see nothing; a sequence may bring no row."""
    _attend(Bed(q, lens, hkv, dim, 16, 7), hq, news, strided=True)


@pytest.mark.parametrize("dim,page", [(128, 64), (64, 16)])
def test_many_items_a_range(q, dim, page):
    """Several whole items in every CTA's range, of one key tile to four."""
    lens = [17 + 97 * i % 487 for i in range(40)]
    _attend(Bed(q, lens, 8, dim, page, 37 + dim), 32, lens)


@pytest.mark.parametrize("dim", [64, 128])
def test_long_prompt_has_the_same_bits_every_time(q, dim):
    """A prompt whose items fill the GPU several times over: 60 runs agree bit for bit, and sampled rows with the oracle."""
    n, hq, hkv = 4096, 32, 8
    bed = Bed(q, [n], hkv, dim, 64, 39)
    x = inputs.activations(n * hq, dim, 40, device=DEV).view(n, hq, dim)
    pos, cu = _dev([0]), _dev([0, n])
    first = None
    for i in range(60):
        out, lse = q.attention_nvfp4(x, bed.cache, pos, cu=cu, max_new=n, return_lse=True)
        if first is None:
            first = out, lse
        else:
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), i
    k, v = bed.values(0)
    xs, o, e = to_np(x), to_np(first[0]), to_np(first[1])
    for t in (0, 63, 64, 368, 1000, 2047, 3071, 4095):
        want, want_lse, spread = kv.attention(xs[t:t + 1], k[:t + 1], v[:t + 1], t, dim ** -0.5)
        big = np.stack([(np.abs(xs[t, h].astype(np.float64)) @ np.abs(k[:t + 1, h // 4]).T).max() for h in range(hq)]) * dim ** -0.5
        tol = 2 ** -18 * (big + 1)
        assert (np.abs(e[t] - want_lse[0]) <= tol).all()
        bound = 2 ** -8 * np.abs(want[0]) + (2 ** -10 + tol)[:, None] * spread[0] + 2 ** -31 * np.repeat(np.abs(v[:t + 1]).sum(0), 4, 0) + 1e-30
        assert (np.abs(o[t] - want[0]) <= bound).all()


def test_peaked_scores(q):
    """Scores of some hundreds: the running reference moves, weights underflow."""
    _attend(Bed(q, [700, 90], 2, 128, 32, 8, spread=4.0), 8, [1, 1], q_scale=8.0)
    _attend(Bed(q, [700, 90], 2, 64, 32, 8, spread=4.0), 8, [40, 3], q_scale=8.0, scale=0.3)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,news", [(4, [5, 8, 1, 4]), (8, [3, 4, 2, 1]), (16, [2, 1, 2, 1]), (32, [1, 1, 1, 1]), (17, [1, 1, 1, 1])])
def test_rows_17_to_32(q, dim, hq, news):
    """More than 16 rows a KV head beside fewer, in one piece and in many, with plain and with peaked scores."""
    _attend(Bed(q, [900, 33, 16, 2000], 1, dim, 16, 11), hq, news, strided=True)
    _attend(Bed(q, [300, 70, 5, 31], 1, dim, 32, 12, spread=4.0), hq, news, q_scale=8.0)


@pytest.mark.parametrize("dim", [64, 128])
def test_rows_17_to_32_of_many_items(q, dim):
    """Items of a few pieces each: 40 sequences, 8 KV heads, two to eight new tokens over ragged lengths."""
    lens = [200 + 53 * i % 700 for i in range(40)]
    _attend(Bed(q, lens, 8, dim, 64, 13), 32, [2 + i % 7 for i in range(40)])


def test_query_magnitudes(q):
    """Queries far from one, zero rows among them."""
    for s in (1e-30, 1e20, 0.0):
        _attend(Bed(q, [50, 20], 1, 128, 16, 9), 4, [1, 1], q_scale=s, scale=min(1.0, 0.1 / s) if s > 1 else None)


def test_rescored_rows_agree(q):
    """A prompt in one call gives what its tokens give one at a time, within the tolerance of both."""
    bed = Bed(q, [150], 2, 128, 16, 10)
    x = torch.randn(150, 8, 128, device=DEV).to(torch.bfloat16)
    whole = q.attention_nvfp4(x, bed.cache, _dev([0]), cu=_dev([0, 150]), max_new=150)
    for t in (0, 1, 77, 149):
        one = q.attention_nvfp4(x[t:t + 1], bed.cache, _dev([t]))
        d = (one - whole[t:t + 1]).float().abs().max().item()
        assert d <= 2 ** -6 * whole[t].float().abs().max().item()


def test_same_bits_again_and_on_another_stream(q):
    bed = Bed(q, [3000, 5, 1700, 900], 2, 128, 64, 11)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for news in ([1] * 4, [70, 5, 1, 300]):
        a = _attend(bed, 8, news)
        b = _attend(bed, 8, news)
        c = _attend(bed, 8, news, stream=side)
        side.synchronize()
        for x, y in zip(a, b):
            assert torch.equal(x, y)
        for x, y in zip(a, c):
            assert torch.equal(x, y)


def test_captured(q):
    bed = Bed(q, [600, 33], 2, 128, 32, 12)
    x = torch.randn(2, 8, 128, device=DEV).to(torch.bfloat16)
    kn = torch.randn(2, 2, 128, device=DEV).to(torch.bfloat16)
    pos = _dev([599, 32])
    ws = torch.empty(q.attention_nvfp4_workspace_bytes(bed.cache, 2, 8), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(x)

    def step():
        q.kv_append_nvfp4(kn, kn, bed.cache, pos)
        q.attention_nvfp4(x, bed.cache, pos, out=out, workspace=ws)

    step()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_captured_rows_of_every_kind(q):
    """A call whose sequences take every kernel, replayed with other queries."""
    bed = Bed(q, [600, 33, 300], 2, 128, 32, 20)
    news = [1, 30, 200]
    x = torch.randn(sum(news), 8, 128, device=DEV).to(torch.bfloat16)
    pos, cu = _dev([n - m for n, m in zip(bed.lens, news)]), _dev(np.concatenate([[0], np.cumsum(news)]))
    ws = torch.empty(q.attention_nvfp4_workspace_bytes(bed.cache, sum(news), 8, 200), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(x)

    def step():
        q.attention_nvfp4(x, bed.cache, pos, cu=cu, max_new=200, out=out, workspace=ws)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        x.copy_(torch.randn(sum(news), 8, 128, device=DEV))
        step()
        want = out.clone()
        out.zero_()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("hq,rows", [(4, 1), (4, 2), (20, 1), (40, 1)])
def test_many_sequences(q, hq, rows):
    """More sequences than a CTA has threads, and than the many-rows kernel keeps in shared memory; some without tokens."""
    g = np.random.default_rng(3)
    lens = [int(x) for x in g.integers(0, 40, 1100)]
    lens[7], lens[1050] = 300, 260
    bed = Bed(q, lens, 1, 64, 16, 21)
    x = torch.randn(1100 * rows, hq, 64, device=DEV).to(torch.bfloat16)
    pos, st = _dev([n - rows for n in lens]), _dev([0])
    cu = None if rows == 1 else _dev(np.arange(0, 1101) * rows)
    out, lse = q.attention_nvfp4(x, bed.cache, pos, cu=cu, max_new=rows, return_lse=True, dev_status=st)
    assert q.get_last_device_status(st) == 0
    o, e, xs = to_np(out), to_np(lse), to_np(x)
    for b in list(range(0, 1100, 37)) + [7, 1050, 1099]:
        k, v = bed.values(b)
        want, want_lse, spread = kv.attention(xs[b * rows:(b + 1) * rows], k, v, lens[b] - rows, 0.125)
        got, got_lse = o[b * rows:(b + 1) * rows], e[b * rows:(b + 1) * rows]
        none = np.isneginf(want_lse)
        assert np.array_equal(none, np.isneginf(got_lse)) and not got[none].any()
        assert (np.abs(got_lse[~none] - want_lse[~none]) <= 2 ** -18 * 64).all()  # |scale q.k| terms sum to well under 63
        assert (np.abs(got - want) <= 2 ** -8 * np.abs(want) + (2 ** -10 + 2 ** -18 * 64) * spread + 2 ** -31 * np.abs(v).sum(0) + 1e-30).all()


def test_rows_of_nobody_stay(q):
    """Rows in front of cu[0] and behind cu[B] are left alone by every call."""
    bed = Bed(q, [40, 200], 2, 128, 16, 22)
    for news in ([1, 2], [9, 150]):
        cu = _dev([3, 3 + news[0], 3 + sum(news)])
        t = 3 + sum(news) + 5
        x = torch.randn(t, 8, 128, device=DEV).to(torch.bfloat16)
        out, lse = torch.full_like(x, 7), torch.full((t, 8), 7.0, device=DEV)
        pos = _dev([40 - news[0], 200 - news[1]])
        q.attention_nvfp4(x, bed.cache, pos, cu=cu, max_new=max(news), out=out, lse=lse)
        whole = q.attention_nvfp4(x[3:-5], bed.cache, pos, cu=cu - 3, max_new=max(news))
        assert torch.equal(out[3:-5], whole)
        for z in (out, lse):
            assert (z[:3] == 7).all() and (z[-5:] == 7).all()
        k, v = torch.full((t, 2, 128), 7, dtype=torch.bfloat16, device=DEV), torch.full((t, 2, 128), 7, dtype=torch.bfloat16, device=DEV)
        q.kv_read_nvfp4(bed.cache, pos, cu=cu, k=k, v=v)
        assert (k[:3] == 0).all() and (v[-5:] == 0).all()  # no token: reads zeros


def test_non_finite_queries_are_told(q):
    bed = Bed(q, [40, 200], 2, 128, 16, 23)
    for news in ([1, 1], [40, 60]):
        x = torch.randn(sum(news), 8, 128, device=DEV).to(torch.bfloat16)
        x[-1, 3, 17] = float("nan")
        st = _dev([0])
        q.attention_nvfp4(x, bed.cache, _dev([40 - news[0], 200 - news[1]]), cu=_dev([0, news[0], sum(news)]), max_new=max(news), dev_status=st)
        assert q.get_last_device_status(st) == q.DEV_NONFINITE


def test_offsets_that_leave_the_rows(q):
    """Offsets outside [0, T] and descending ones are flagged; what they name stays inside the call's rows."""
    bed = Bed(q, [40, 200], 2, 128, 16, 24)
    x = torch.randn(12, 8, 128, device=DEV).to(torch.bfloat16)
    for cu in ([0, 6, 50], [-3, 6, 12], [0, 9, 4]):
        st = _dev([0])
        q.attention_nvfp4(x, bed.cache, _dev([30, 180]), cu=_dev(cu), max_new=12, dev_status=st)
        assert q.get_last_device_status(st) & q.DEV_BAD_INDEX


def test_pages_behind_32_bits(q):
    """Code offsets above 2^32: the last pages of a pool of 4.6 GB."""
    pages, hkv, page, dim = 70000, 8, 128, 128
    pool = [torch.empty(pages, hkv, page, dim // d, dtype=torch.uint8, device=DEV) for d in (2, 16, 2, 16)]
    table = _dev([[pages - 1, pages - 2]])
    far = q.KvCacheNvfp4(*pool, table)
    near = q.KvCacheNvfp4.empty(2, hkv, page, dim, _dev([[0, 1]]))
    x = torch.randn(200, hkv, dim, device=DEV).to(torch.bfloat16)
    qq = torch.randn(200, 16, dim, device=DEV).to(torch.bfloat16)
    got = []
    for c in (far, near):
        q.kv_append_nvfp4(x, x, c, _dev([0]), cu=_dev([0, 200]))
        got.append(q.kv_read_nvfp4(c, _dev([0]), cu=_dev([0, 200]), rows=200) + (
            q.attention_nvfp4(qq[:1], c, _dev([199])), q.attention_nvfp4(qq, c, _dev([0]), cu=_dev([0, 200]), max_new=200)))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    del pool, far


def test_refusals(q):
    bed = Bed(q, [40, 3], 2, 128, 16, 13)
    c, pos = bed.cache, _dev([39, 2])
    x = torch.randn(2, 8, 128, device=DEV).to(torch.bfloat16)
    with pytest.raises(ValueError, match="one row a sequence"):
        q.attention_nvfp4(x[:1], c, pos)
    with pytest.raises(ValueError, match="max_new"):
        q.attention_nvfp4(x, c, pos, cu=_dev([0, 1, 2]))
    with pytest.raises(ValueError, match="pos"):
        q.attention_nvfp4(x, c, pos[:1])
    with pytest.raises(TypeError):
        q.attention_nvfp4(x.float(), c, pos)
    with pytest.raises(ValueError, match="q must be"):
        q.attention_nvfp4(x[..., :64], c, pos)
    with pytest.raises(q.QrrError, match="UNSUPPORTED"):
        q.attention_nvfp4(x[:, :7].contiguous(), c, pos)  # 7 query heads on 2 KV heads
    with pytest.raises(q.QrrError, match="WORKSPACE"):
        q.attention_nvfp4(x, c, pos, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(q.QrrError, match="INVALID"):
        q.attention_nvfp4(x, c, pos, scale=-1.0)
    with pytest.raises(ValueError, match="rows"):
        q.kv_read_nvfp4(c, pos, cu=_dev([0, 1, 2]))
    with pytest.raises(ValueError, match="k_new must be"):
        q.kv_append_nvfp4(x, x, c, pos)
    with pytest.raises(ValueError, match="k_scales"):
        q.KvCacheNvfp4(c.tensors[0], c.tensors[0], *c.tensors[2:5])
    with pytest.raises(q.QrrError, match="UNSUPPORTED"):  # pages of 24 tokens
        q.kv_read_nvfp4(q.KvCacheNvfp4.empty(2, 2, 24, 128, _dev([[0], [1]])), pos)
    y = torch.randn(2, 2 * 128 + 4, device=DEV).to(torch.bfloat16)
    with pytest.raises(q.QrrError, match="MISALIGNED"):
        q.kv_append_nvfp4(y.as_strided((2, 2, 128), (260, 128, 1)), x[:, :2].contiguous(), c, pos)


def test_a_sequence_longer_than_promised(q):
    bed = Bed(q, [40, 30], 2, 128, 16, 14)
    x = torch.randn(35, 8, 128, device=DEV).to(torch.bfloat16)
    st = _dev([0])
    q.attention_nvfp4(x, bed.cache, _dev([10, 25]), cu=_dev([0, 30, 35]), max_new=5, dev_status=st)
    assert q.get_last_device_status(st) == q.DEV_BAD_INDEX


def test_no_rows(q):
    bed = Bed(q, [4], 2, 64, 16, 15)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    q.kv_append_nvfp4(e, e, bed.cache, _dev([0]), cu=_dev([0, 0]))
    k, v = q.kv_read_nvfp4(bed.cache, _dev([0]), cu=_dev([0, 0]), rows=0)
    out = q.attention_nvfp4(torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV), bed.cache, _dev([0]), cu=_dev([0, 0]), max_new=0)
    assert k.shape[0] == v.shape[0] == out.shape[0] == 0
