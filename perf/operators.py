"""The paged NVFP4 key/value cache: writing it, reading it back, and attention over it.

A cache page holds `page` tokens of every key/value head as E2M1 codes (two a byte, the even index in the low nibble) with
one E4M3 scale per 16 values; a table of page numbers a sequence maps token positions to pages, and a global scale a head
multiplies everything. A call covers a batch of sequences: sequence b brings the rows cu[b] .. cu[b + 1] - 1 of the call's
tensors (one row each without cu), at the positions pos[b], pos[b] + 1, ...; a negative position is no token at all.

  write      rows of k and v are quantized into the cache, and read back as the bf16 values that attention will see
  read       the values of a range of positions of every sequence
  attention  softmax(q k^T / sqrt(dim)) v of every query row over the positions up to its own, and its log-sum-exp
"""
import math
import random

import torch

own = False

MID = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # midpoints between neighbouring E2M1 magnitudes
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decode step of a rollout batch: 64 sequences of an 8B-class layer write a token each
        dict(name="write step", kind="write", batch=64, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=4000, hq=32, hkv=8, dim=128, page=64, idle=0),
        # prompts of a batch of ragged lengths, behind a shared beginning that is in the cache
        dict(name="write prompts", kind="write", batch=32, new_lo=100, new_hi=1001, ctx_lo=0, ctx_hi=500, hq=32, hkv=8, dim=128, page=16, idle=0),
        # long documents
        dict(name="write long", kind="write", batch=4, new_lo=30000, new_hi=32768, ctx_lo=0, ctx_hi=0, hq=32, hkv=8, dim=128, page=128, idle=0),
        # a turn of a few sequences with heads of 64, to be scored again elsewhere
        dict(name="read turn", kind="read", batch=3, new_lo=77, new_hi=333, ctx_lo=0, ctx_hi=1000, hq=8, hkv=4, dim=64, page=32, idle=0),
        # a whole rollout batch
        dict(name="read batch", kind="read", batch=32, new_lo=2048, new_hi=4096, ctx_lo=0, ctx_hi=0, hq=32, hkv=8, dim=128, page=64, idle=0),
        # the first tokens of a single sequence: latency
        dict(name="decode first", kind="attention", batch=1, new_lo=1, new_hi=1, ctx_lo=36, ctx_hi=36, hq=32, hkv=8, dim=128, page=16, idle=0),
        # a rollout batch of an 8B-class layer; every eighth sequence has ended and sees nothing
        dict(name="decode batch", kind="attention", batch=64, new_lo=1, new_hi=1, ctx_lo=2047, ctx_hi=4095, hq=32, hkv=8, dim=128, page=64, idle=8),
        # long contexts of a 32B-class layer, five query heads to a key head
        dict(name="decode long", kind="attention", batch=8, new_lo=1, new_hi=1, ctx_lo=20000, ctx_hi=33000, hq=40, hkv=8, dim=128, page=128, idle=0),
        # many short sequences of a small model without shared heads
        dict(name="decode small heads", kind="attention", batch=128, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=1500, hq=16, hkv=16, dim=64, page=32, idle=0),
        # a few drafted tokens a sequence, scored in one call
        dict(name="drafts", kind="attention", batch=32, new_lo=1, new_hi=9, ctx_lo=500, ctx_hi=4000, hq=32, hkv=8, dim=128, page=64, idle=0),
        # a new turn of several hundred tokens over a long conversation
        dict(name="turn", kind="attention", batch=4, new_lo=300, new_hi=700, ctx_lo=6000, ctx_hi=10000, hq=40, hkv=8, dim=128, page=64, idle=0),
        # a whole prompt
        dict(name="prompt", kind="attention", batch=1, new_lo=4096, new_hi=4096, ctx_lo=0, ctx_hi=0, hq=32, hkv=8, dim=128, page=64, idle=0),
    ]


def draw(rng):
    most = [max(work(c)[w] for c in listed()) for w in ("bytes", "flops")]
    while True:
        case = _draw(rng)
        if work(case)["bytes"] <= most[0] and work(case)["flops"] <= most[1]:
            return case


def _draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["write", "read", "attention", "attention", "attention"])
    dim = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    case = dict(kind=kind, hq=hq, hkv=hkv, dim=dim, page=page, idle=0)
    if kind != "attention":
        batch = log(1, 128)
        new = log(1, max(1, 100000 // batch))
        return dict(case, batch=batch, new_lo=max(1, new // 2), new_hi=new, ctx_lo=0, ctx_hi=log(1, 2000))
    form = rng.choice(["decode", "decode", "drafts", "turn", "prompt"])
    if form == "decode":
        batch = log(1, 128)
        ctx = log(1, 200000 // batch)
        return dict(case, batch=batch, new_lo=1, new_hi=1, ctx_lo=ctx // 2, ctx_hi=ctx, idle=rng.choice([0, 0, 3]))
    if form == "drafts":
        return dict(case, batch=log(1, 32), new_lo=1, new_hi=rng.randint(2, 12), ctx_lo=rng.randint(0, 300), ctx_hi=log(301, 4000))
    if form == "turn":
        new = log(20, 700)
        ctx = log(100, 9000)
        return dict(case, batch=rng.randint(1, 4), new_lo=new // 2, new_hi=new, ctx_lo=ctx // 2, ctx_hi=ctx)
    new = log(30, 2000)
    return dict(case, batch=rng.randint(1, 2), new_lo=new, new_hi=new, ctx_lo=0, ctx_hi=0)


def _lengths(case, seed):
    """Rows and first positions of the sequences; the rows' lengths spread evenly over their range, in an order of the seed's."""
    r, b = random.Random(seed), case["batch"]
    n = [case["new_lo"] + (case["new_hi"] - case["new_lo"]) * (2 * i + 1) // (2 * b) for i in range(b)]
    r.shuffle(n)
    pos = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(b)]
    if case["idle"]:
        pos = [-1 if b % case["idle"] == case["idle"] - 1 else p for b, p in enumerate(pos)]
    return n, pos


def work(case):
    b, d, hq, hkv = case["batch"], case["dim"], case["hq"], case["hkv"]
    n, ctx = (case["new_lo"] + case["new_hi"]) / 2, (case["ctx_lo"] + case["ctx_hi"]) / 2
    row, packed = 2 * hkv * d * 2, 2 * hkv * d * 0.5625
    if case["kind"] == "write":  # k and v in, codes and scales out and in again, values out
        return {"bytes": b * n * (2 * row + 2 * packed), "flops": 0}
    if case["kind"] == "read":
        return {"bytes": b * n * (row + packed), "flops": 0}
    if case["idle"]:
        b -= b // case["idle"]
    seen = n * ctx + n * (n + 1) / 2
    return {"bytes": b * ((ctx + n) * packed + n * hq * (4 * d + 4)), "flops": 4.0 * b * hq * d * seen}


def _quantize(x, gs):
    """Codes [.., dim] (0 .. 15) and E4M3 scales [.., dim / 16] of fp32 rows x [.., hkv, dim]."""
    blocks = x.unflatten(-1, (-1, 16))
    g = gs[:, None]
    s = (blocks.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = (s.float() * g)[..., None]
    a = torch.where(d > 0, blocks.abs() / d, torch.zeros_like(blocks))
    up = (a > MID[0]).to(torch.uint8) + (a >= MID[1]) + (a > MID[2]) + (a >= MID[3]) + (a > MID[4]) + (a >= MID[5]) + (a > MID[6])
    codes = up + 8 * ((blocks < 0) & (d > 0)).to(torch.uint8)
    return codes.to(torch.uint8).flatten(-2), s


def _values(packed, scales, gs, grid):
    """The fp32 values [.., hkv, .., dim] of packed codes [.., dim / 2] and E4M3 scales; gs has the values' rank."""
    codes = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).to(torch.int64)
    return (grid[codes].unflatten(-1, (-1, 16)) * scales.float()[..., None]).flatten(-2) * gs


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    n, pos = _lengths(case, seed)
    b, d, hq, hkv, page = case["batch"], case["dim"], case["hq"], case["hkv"], case["page"]
    per = max(1, max(-(-(p + m) // page) for m, p in zip(n, pos)))
    pages = b * per + 3
    table = torch.randperm(pages, generator=g, device=dev)[: b * per].to(torch.int32).view(b, per)
    gs = [torch.full((hkv,), v, device=dev) * (1 + torch.rand(hkv, generator=g, device=dev)) for v in (0.03, 0.01)]
    cu = [sum(n[:i]) for i in range(b + 1)]
    s = dict(kind=case["kind"], page=page, hq=hq, hkv=hkv, dim=d, max_new=case["new_hi"], k_gs=gs[0], v_gs=gs[1], table=table,
             one=case["new_hi"] == 1, scale=1.0 / math.sqrt(d),
             grid=torch.tensor(GRID + tuple(-v for v in GRID), device=dev), cu=torch.tensor(cu, dtype=torch.int32, device=dev),
             pos=torch.tensor(pos, dtype=torch.int32, device=dev))
    channel = 0.5 + 2.0 * torch.rand(hkv, d, generator=g, device=dev)  # keys differ by channel, values do not
    channel[:, ::37] *= 4.0

    def rows(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    for name, factor, scale in (("k", channel, gs[0]), ("v", None, gs[1])):
        codes = torch.zeros(pages, hkv, page, d // 2, dtype=torch.uint8, device=dev)
        scales = torch.zeros(pages, hkv, page, d // 16, dtype=torch.uint8, device=dev)
        if case["kind"] != "write":
            for at in range(0, pages, 512):  # a bounded number of pages at a time
                x = rows(min(512, pages - at), page, hkv, d) * 0.5
                c, e = _quantize(x * factor if factor is not None else x, scale)
                codes[at:at + 512] = (c[..., 0::2] | c[..., 1::2] << 4).transpose(1, 2)
                scales[at:at + 512] = e.view(torch.uint8).transpose(1, 2)
        s[name + "_codes"], s[name + "_scales"] = codes, scales
    t = cu[-1]
    # a projection's output: the rows of q, k and v side by side
    qkv = rows(t, hq + 2 * hkv, d).to(torch.bfloat16)
    qkv[:, hq:hq + hkv] *= channel.to(torch.bfloat16)
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    return s


def run(s):
    if own:
        return _run_own(s)
    if s["kind"] == "attention":
        return _attention(s)
    seq, at, ok, page, slot = _places(s)
    if s["kind"] == "write":
        for_k, for_v = _written(s, "k", page, slot, ok), _written(s, "v", page, slot, ok)
        return {"k": for_k, "v": for_v}
    return {"k": _read(s, "k", page, slot, ok), "v": _read(s, "v", page, slot, ok)}


def _run_own(s):
    from quantized_rl_rollout_gb300 import qrr

    if "cache" not in s:  # the handle on the cache's buffers that a program keeps with them
        s["cache"] = qrr.KvCacheNvfp4(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["table"], s["k_gs"], s["v_gs"])
    cu = None if s["one"] else s["cu"]
    if s["kind"] == "attention":
        out, lse = qrr.attention_nvfp4(s["q"], s["cache"], s["pos"], cu=cu, max_new=s["max_new"], scale=s["scale"], return_lse=True)
        return {"out": out, "lse": lse}
    if s["kind"] == "write":
        qrr.kv_append_nvfp4(s["k"], s["v"], s["cache"], s["pos"], cu=cu)
    k, v = qrr.kv_read_nvfp4(s["cache"], s["pos"], cu=cu, rows=s["q"].shape[0])
    return {"k": k, "v": v}


def _places(s):
    """Of every row: its sequence, its position, whether it has one, its page and the slot in it."""
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.bucketize(t, s["cu"][1:], right=True)
    at = s["pos"][seq] + (t - s["cu"][seq])
    ok = at >= 0
    safe = at.clamp(min=0)
    page = s["table"][seq, safe // s["page"]].to(torch.int64)
    return seq, at, ok, page, safe % s["page"]


def _written(s, name, page, slot, ok):
    codes, scales = _quantize(s[name].float(), s[name + "_gs"])
    s[name + "_codes"][page, :, slot] = codes[..., 0::2] | codes[..., 1::2] << 4
    s[name + "_scales"][page, :, slot] = scales.view(torch.uint8)
    return _read(s, name, page, slot, ok)


def _read(s, name, page, slot, ok):
    x = _values(s[name + "_codes"][page, :, slot], s[name + "_scales"][page, :, slot].view(torch.float8_e4m3fn), s[name + "_gs"][:, None], s["grid"])
    return torch.where(ok[:, None, None], x, torch.zeros_like(x)).to(torch.bfloat16)


def _attention(s):
    b, hkv, hq, d = s["table"].shape[0], s["hkv"], s["hq"], s["dim"]
    table = s["table"].to(torch.int64)
    seq, at, _, _, _ = _places(s)
    i = torch.arange(seq.shape[0], device="cuda") - s["cu"][seq]

    def cached(name):
        x = _values(s[name + "_codes"][table], s[name + "_scales"][table].view(torch.float8_e4m3fn), s[name + "_gs"][:, None, None], s["grid"])
        return x.transpose(1, 2).flatten(2, 3)  # [b, hkv, tokens, dim]

    k, v = cached("k"), cached("v")
    q = torch.zeros(b, s["max_new"], hq, d, device="cuda")
    q[seq, i] = s["q"].float()
    q = q.unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [b, hkv, new x group, dim]
    scores = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    last = s["pos"][:, None] + torch.arange(s["max_new"], device="cuda")  # [b, new]
    last = last.repeat_interleave(hq // hkv, dim=1)[:, None, :, None]
    scores.masked_fill_(torch.arange(k.shape[2], device="cuda") > last, -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = top + total.log()

    def back(x):
        return x.unflatten(2, (s["max_new"], -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, i]

    return {"out": back(out).to(torch.bfloat16), "lse": back(lse)[..., 0]}


def _decoded(codes, scales, gs):
    """float64 values of packed bytes: sign, two exponent bits and a mantissa bit of E2M1; E4M3 by its fields."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    e, m = ((c >> 1) & 3).double(), (c & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1))
    nib = torch.where(c >= 8, -mag, mag)
    e, m = ((scales >> 3) & 15).double(), (scales & 7).double()
    sc = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2(e - 7))
    return nib * sc.repeat_interleave(16, dim=-1) * gs


def _rounded(x, gs):
    """float64 rows [rows, hkv, dim] on their NVFP4 grids, from the definition."""
    b = x.reshape(*x.shape[:-1], -1, 16)
    want = (b.abs().amax(-1) / (6 * gs[:, None])).clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3)
    s = torch.round(want / step) * step  # torch.round takes ties to even
    d = (s * gs[:, None])[..., None]
    a = torch.where(d > 0, b.abs() / d.clamp(min=1e-300), torch.zeros_like(b)).clamp(max=6.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=1.0))) - 1)
    return (torch.sign(b) * torch.round(a / step) * step * d).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    n, pos = _lengths(case, seed)
    gk, gv = s["k_gs"].double(), s["v_gs"].double()
    if case["kind"] == "write":
        return {"k": _rounded(s["k"].double(), gk), "v": _rounded(s["v"].double(), gv)}
    hkv, d, page, group = case["hkv"], case["dim"], case["page"], case["hq"] // case["hkv"]
    first, outs = 0, ([], [])
    for b in range(case["batch"]):
        end = pos[b] + n[b]
        used = s["table"][b, : max(0, -(-end // page))].long()
        k, v = (_decoded(s[m + "_codes"][used], s[m + "_scales"][used], g[:, None, None]).permute(1, 0, 2, 3).reshape(hkv, -1, d) for m, g in (("k", gk), ("v", gv)))
        q = s["q"][first:first + n[b]].double()
        first += n[b]
        if case["kind"] == "read":
            for o, x in zip(outs, (k, v)):
                o.append(x[:, pos[b]:end].transpose(0, 1))
            continue
        for at in range(0, n[b], 512):  # rows of queries at a time
            m = min(512, n[b] - at)
            last = pos[b] + at + torch.arange(m, device="cuda")
            seen = torch.arange(k.shape[1], device="cuda")[None, :] <= last[:, None]
            x = torch.einsum("ihgd,hjd->hgij", q[at:at + m].reshape(m, hkv, group, d), k) * s["scale"]
            x = x.masked_fill(~seen, -math.inf)
            lse = torch.logsumexp(x, -1) if k.shape[1] else x.new_full(x.shape[:-1], -math.inf)
            p = torch.nan_to_num(torch.exp(x - lse[..., None]), nan=0.0)
            outs[0].append(torch.einsum("hgij,hjd->ihgd", p, v).reshape(m, hkv * group, d))
            outs[1].append(lse.permute(2, 0, 1).reshape(m, hkv * group))
    names = ("k", "v") if case["kind"] == "read" else ("out", "lse")
    return {name: torch.cat(o) for name, o in zip(names, outs)}
