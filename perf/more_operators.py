"""Logits at both ends of a rollout: drafted tokens verified while it runs, and the losses of the training step after it.

  verify    drafted tokens are tested one after another against the target's probabilities; where one is refused, and behind
            the last one, a token is drawn from what is left of the target's distribution. Random numbers are inputs.
  loss      distillation: sum_j p_j (ln p_j - ln q_j) of every row, p from a teacher's top logits, q = softmax of the row
  backward  its gradient in the logits, for a gradient that arrives a row
  step      loss and gradient at once, for row weights that are known beforehand
  policy    token log-probabilities, capped importance weights and the policy gradient in the logits at once

With a tail, the teacher's probability outside its top logits is one more outcome, beside the student's probability outside them;
without it the teacher's probabilities are taken among the top logits alone.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SPREAD = {0.9: 0.3, 0.85: 0.5, 0.7: 1.0}  # how far a draft model's logits are off, by the drafts that are accepted


def listed():
    return [
        # one sequence, four tokens from a draft model: latency
        dict(name="verify one", kind="verify", form="model", batch=1, n_lo=4, n_hi=4, vocab=128256, pad=0, dtype="bf16", temp=1.0, accept=0.9),
        # a rollout batch, tokens from a draft model, sampled below temperature 1
        dict(name="verify batch", kind="verify", form="model", batch=64, n_lo=8, n_hi=8, vocab=128256, pad=0, dtype="bf16", temp=0.7, accept=0.7),
        # tokens looked up in the prompt, 0 to 8 a sequence; an odd vocabulary in padded rows
        dict(name="verify lookup", kind="verify", form="lookup", batch=200, n_lo=0, n_hi=8, vocab=50001, pad=63, dtype="fp32", temp=1.0, accept=0.45),
        # an evaluation that takes the likeliest token
        dict(name="verify greedy", kind="verify", form="greedy", batch=32, n_lo=1, n_hi=5, vocab=32000, pad=0, dtype="bf16", temp=0.0, accept=0.85),
        # the divergence of a few positions, to watch it
        dict(name="loss few", kind="loss", rows=5, vocab=32000, pad=0, dtype="bf16", k=20, tail=True, temp=1.0, idle=0),
        # an evaluation batch; every fifth row is a prompt's and has no teacher
        dict(name="loss batch", kind="loss", rows=2048, vocab=128256, pad=0, dtype="bf16", k=64, tail=True, temp=1.0, idle=5),
        # a small model's step in 32 bits, odd vocabulary, softened
        dict(name="backward odd", kind="backward", rows=777, vocab=50001, pad=0, dtype="fp32", k=33, tail=False, temp=2.0, idle=0),
        # an 8B-class model's batch
        dict(name="backward batch", kind="backward", rows=2048, vocab=128256, pad=0, dtype="bf16", k=64, tail=True, temp=1.0, idle=5),
        # one rollout's few tokens
        dict(name="step few", kind="step", rows=24, vocab=128256, pad=0, dtype="bf16", k=8, tail=False, temp=1.0, idle=0),
        # a training batch of an 8B-class model
        dict(name="step batch", kind="step", rows=4096, vocab=128256, pad=0, dtype="bf16", k=64, tail=True, temp=1.0, idle=7),
        # the policy gradient of a micro-batch of a small vocabulary with rows of an odd length
        dict(name="policy odd", kind="policy", rows=300, vocab=32003, pad=0, dtype="bf16", cap=2.0, idle=4),
        # and of a whole batch
        dict(name="policy batch", kind="policy", rows=4096, vocab=128256, pad=0, dtype="bf16", cap=5.0, idle=7),
    ]


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        case = _draw(rng)
        if work(case)["bytes"] <= most:
            return case


def _draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    vocab = rng.choice([log(500, 160000), log(500, 160000), 8 * log(100, 20000), 32000, 128256])
    case = dict(vocab=vocab, pad=rng.choice([0, 0, rng.randint(1, 64)]), dtype=rng.choice(["bf16", "bf16", "fp32"]))
    kind = rng.choice(["verify", "verify", "loss", "backward", "step", "policy"])
    if kind == "verify":
        form = rng.choice(["model", "model", "lookup", "greedy"])
        hi = rng.randint(1, 9)
        return dict(case, kind=kind, form=form, batch=log(1, 256), n_lo=rng.choice([hi, rng.randint(0, hi)]), n_hi=hi,
                    temp=0.0 if form == "greedy" else rng.choice([0.7, 1.0, 1.0, 1.3]),
                    accept=0.45 if form == "lookup" else rng.choice(list(SPREAD)))
    case.update(kind=kind, rows=log(1, 6000), idle=rng.choice([0, 0, 3, 6]))
    if kind == "policy":
        return dict(case, cap=rng.choice([0.0, 1.5, 4.0]))
    return dict(case, k=log(1, 256), tail=rng.choice([True, False]), temp=rng.choice([0.8, 1.0, 1.0, 2.0]))


def _drafts(case):
    """Drafted tokens of the sequences, spread evenly over their range."""
    b, lo, hi = case["batch"], case["n_lo"], case["n_hi"]
    n = [lo + (hi - lo + 1) * (2 * i + 1) // (2 * b) for i in range(b)]
    random.Random(b).shuffle(n)
    return n


def _idle(case):
    """Rows that have nothing to learn."""
    t = range(case["rows"])
    return [i for i in t if case["idle"] and i % case["idle"] == case["idle"] - 1]


def work(case):
    v, e = case["vocab"], 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "verify":  # rows up to the first refusal, as many as that is on average
        a, n = case["accept"], _drafts(case)
        drafted = sum(a ** i for m in n for i in range(m))
        rows = drafted + sum(a ** m for m in n)
        if case["form"] == "model":
            rows += drafted
        noise = 0 if case["form"] == "greedy" else case["batch"] * v * 4
        return {"bytes": rows * v * e + noise, "flops": 4.0 * rows * v}
    rows = case["rows"]
    live = rows - len(_idle(case))
    if case["kind"] == "policy":
        return {"bytes": (live + rows) * v * e + rows * 20, "flops": 6.0 * live * v}
    small = rows * (case["k"] * 8 + 12)
    if case["kind"] == "loss":
        return {"bytes": live * v * e + small, "flops": 4.0 * live * v}
    return {"bytes": (live + rows) * v * e + small, "flops": 6.0 * live * v}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype, v = TYPES[case["dtype"]], case["vocab"]

    def logits(rows):
        """A model's rows: a broad mass and some tokens that stand out; the rows may be longer than the vocabulary."""
        out = torch.empty(rows, v + case["pad"], dtype=dtype, device="cuda")
        for at in range(0, rows, 512):
            x = 2.0 * torch.randn(min(512, rows - at), v, generator=g, device="cuda")
            up = torch.randint(v, (x.shape[0], 32), generator=g, device="cuda")
            x.scatter_add_(1, up, 4.0 + 8.0 * torch.rand(up.shape, generator=g, device="cuda"))
            out[at:at + 512, :v] = x.to(dtype)
        return out[:, :v]

    if case["kind"] == "verify":
        return _prepare_verify(case, g, logits)
    rows = case["rows"]
    s = dict(kind=case["kind"], logits=logits(rows), dlogits=torch.empty(rows, v, dtype=dtype, device="cuda"))
    idle = torch.tensor(_idle(case), dtype=torch.int64, device="cuda")
    if case["kind"] == "policy":
        s["tokens"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        s["rollout"] = torch.empty(rows, device="cuda")
        for at in range(0, rows, 512):
            x = s["logits"][at:at + 512].float()
            e = torch.empty_like(x).exponential_(generator=g)
            token = (torch.softmax(x, -1) / e).argmax(-1)
            s["tokens"][at:at + 512] = token.to(torch.int32)
            s["rollout"][at:at + 512] = torch.log_softmax(x, -1).gather(1, token[:, None])[:, 0]
        s["rollout"] += 0.3 * torch.randn(rows, generator=g, device="cuda")  # another engine's, and a policy some steps older
        s["tokens"][idle] = -1
        s["advantages"] = torch.randn(rows, generator=g, device="cuda") / rows
        s["cap"] = case["cap"]
        return s
    s["temp"], k = case["temp"], case["k"]
    s["ids"] = torch.empty(rows, k, dtype=torch.int32, device="cuda")
    s["top"] = torch.empty(rows, k, device="cuda")
    lse = torch.empty(rows, device="cuda")
    for at in range(0, rows, 512):  # the teacher's logits, of which its top ones are kept
        x = s["logits"][at:at + 512].float()
        x = x + 0.7 * torch.randn(x.shape, generator=g, device="cuda")
        s["top"][at:at + 512], ids = x.topk(k, dim=-1)
        s["ids"][at:at + 512] = ids.to(torch.int32)
        lse[at:at + 512] = torch.logsumexp(x.double() / case["temp"], -1).float()
    s["ids"][idle] = -1
    s["ids"][1::11, k // 2 + 1:] = -1  # a teacher that gave fewer
    s["lse"] = lse if case["tail"] else None
    s["grad"] = torch.rand(rows, generator=g, device="cuda") / rows
    if case["kind"] == "backward":
        s["stats"] = _distill(s)[1]
    return s


def _prepare_verify(case, g, logits):
    b, v, n = case["batch"], case["vocab"], _drafts(case)
    cu = [sum(n[:i]) for i in range(b + 1)]
    t = cu[-1]
    s = dict(kind="verify", temp=case["temp"], form=case["form"], target=logits(t + b), draft=None, uniforms=None, noise=None,
             cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), even=case["n_lo"] == case["n_hi"])
    of = torch.tensor([cu[i] + i + j for i in range(b) for j in range(n[i])], dtype=torch.int64, device="cuda")
    x = s["target"][of].float()
    if case["form"] == "model":  # the draft model's logits, from which the drafts were drawn
        x = x + SPREAD[case["accept"]] * torch.randn(x.shape, generator=g, device="cuda")
        wide = torch.empty(t, v + case["pad"], dtype=TYPES[case["dtype"]], device="cuda")
        wide[:, :v] = x.to(wide.dtype)
        s["draft"] = wide[:, :v]
        x = s["draft"].float() / case["temp"]
    elif case["form"] == "lookup":
        x = x * 3.0
    if case["form"] != "greedy":
        x = x - torch.empty_like(x).exponential_(generator=g).log()
        s["uniforms"] = torch.rand(t, generator=g, device="cuda")
        s["noise"] = torch.empty(b, v, device="cuda").exponential_(generator=g).clamp_(min=1e-30)
    s["drafts"] = x.argmax(-1).to(torch.int32)
    if case["form"] == "greedy":
        other = torch.randint(v, (t,), generator=g, device="cuda").to(torch.int32)
        s["drafts"] = torch.where(torch.rand(t, generator=g, device="cuda") < case["accept"], s["drafts"], other)
    return s


def run(s):
    if own:
        return _run_own(s)
    if s["kind"] == "verify":
        return _verify(s)
    if s["kind"] == "policy":
        return _policy(s)
    if s["kind"] == "backward":
        return {"dlogits": _distill_gradient(s, s["stats"])}
    loss, stats = _distill(s)
    if s["kind"] == "loss":
        return {"loss": loss, "stats": stats}
    return {"loss": loss, "dlogits": _distill_gradient(s, stats)}


def _run_own(s):
    from quantized_rl_rollout_gb300 import qrr

    if s["kind"] == "verify":
        tokens, accepted, logp = qrr.verify_drafts(s["target"], s["drafts"], uniforms=s["uniforms"], noise=s["noise"], draft_logits=s["draft"],
                                                   cu=None if s["even"] else s["cu"], temperature=s["temp"])
        return {"tokens": tokens, "accepted": accepted, "logp": logp}
    if s["kind"] == "policy":
        logp, w, dlogits = qrr.token_logprobs_is_grad(s["logits"], s["tokens"], s["advantages"], s["rollout"], s["cap"], dlogits=s["dlogits"])
        return {"logp": logp, "w": w, "dlogits": dlogits}
    teacher = dict(top_lse=s["lse"], temperature=s["temp"])
    if s["kind"] == "loss":
        loss, stats = qrr.distill_topk(s["logits"], s["ids"], s["top"], **teacher)
        return {"loss": loss, "stats": stats}
    if s["kind"] == "backward":
        return {"dlogits": qrr.distill_topk_backward(s["logits"], s["ids"], s["top"], s["stats"], s["grad"], dlogits=s["dlogits"], **teacher)}
    loss, dlogits = qrr.distill_topk_grad(s["logits"], s["ids"], s["top"], s["grad"], dlogits=s["dlogits"], **teacher)
    return {"loss": loss, "dlogits": dlogits}


def _normaliser(x):
    """Log of the sum of exp over each row of fp32 x, in 64 bits: decisions that are near their border hang on it."""
    top = x.amax(-1, keepdim=True)
    return top[:, 0].double() + torch.exp(x - top).sum(-1, dtype=torch.float64).log()


def _verify(s):
    target, drafts, cu = s["target"], s["drafts"].to(torch.int64), s["cu"].to(torch.int64)
    rows, v = target.shape
    t, dev = drafts.shape[0], target.device
    b = rows - t
    n = cu[1:] - cu[:-1]
    first = cu[:-1] + torch.arange(b, device=dev)  # of each sequence, its first row of the target's
    at = torch.arange(t, device=dev)
    seq = torch.bucketize(at, cu[1:], right=True)
    row = at + seq
    temp = s["temp"] if s["temp"] > 0 else 1.0
    x = target.float() / temp
    z = _normaliser(x)
    if s["form"] == "greedy":
        best = torch.where(x == x.amax(-1, keepdim=True), torch.arange(v, device=dev), v).amin(-1)
        ok = best[row] == drafts
    else:
        p = x[row, drafts].double() - z[row]
        q = 0.0
        if s["form"] == "model":
            y = s["draft"].float() / temp
            zy = _normaliser(y)
            q = y[at, drafts].double() - zy
        ok = s["uniforms"].double().log() + q < p
    place = at - cu[seq]
    accepted = n.scatter_reduce(0, seq, torch.where(ok, n[seq], place), "amin")
    last = first + accepted  # the row that the next token is drawn from
    if s["form"] == "greedy":
        token = best[last]
    else:
        p = torch.exp(x[last].double() - z[last, None])
        refused = (accepted < n).nonzero()[:, 0]
        which = cu[:-1][refused] + accepted[refused]
        left = p.clone()
        if s["form"] == "model":
            left[refused] = (p[refused] - torch.exp(y[which].double() - zy[which, None])).clamp(min=0)
        else:
            left[refused, drafts[which]] = 0
        left = torch.where(left.sum(-1, keepdim=True) > 0, left, p)
        token = (left / s["noise"]).argmax(-1)
    tokens = torch.full((rows,), -1, dtype=torch.int64, device=dev)
    tokens[row] = torch.where(place < accepted[seq], drafts, -1)
    tokens[last] = token
    logp = x.gather(1, tokens.clamp(min=0)[:, None])[:, 0].double() - z
    logp = torch.where(tokens >= 0, logp, torch.zeros_like(logp))
    return {"tokens": tokens.to(torch.int32), "accepted": accepted.to(torch.int32), "logp": logp.float()}


def _teacher(s):
    """Which slots count, and of those the teacher's probabilities and their logarithms (in 64 bits: a divergence is a small
    difference of large logarithms)."""
    used = s["ids"] >= 0
    y = s["top"].double() / s["temp"]
    y = torch.where(used, y, torch.full_like(y, -math.inf))
    if s["lse"] is None:
        top = y.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        lse = top + torch.exp(y - top).sum(-1, keepdim=True).log()
    else:
        lse = s["lse"].double()[:, None]
    logp = torch.where(used, y - lse, torch.full_like(y, -math.inf))
    p = torch.exp(logp)
    return used, p, logp, (1 - p.sum(-1)).clamp(min=0)


def _outside(s, x):
    """Rows of x with -inf at the teacher's ids."""
    row, slot = (s["ids"] >= 0).nonzero(as_tuple=True)
    x = x.clone()
    x[row, s["ids"][row, slot].to(torch.int64)] = -math.inf
    return x


def _distill(s):
    used, p, logp, rest = _teacher(s)
    x = s["logits"].float() / s["temp"]
    lse = _normaliser(x)
    outside = lse if s["lse"] is None else _normaliser(_outside(s, x))
    logq = s["logits"].gather(1, s["ids"].clamp(min=0).to(torch.int64)).double() / s["temp"] - lse[:, None]
    loss = torch.where(p > 0, p * (logp - logq), torch.zeros_like(p)).sum(-1)
    if s["lse"] is not None:
        loss = loss + torch.where(rest > 0, rest * (rest.log() - (outside - lse)), torch.zeros_like(rest))
    live = used.any(-1)
    stats = torch.stack((lse, outside), -1)
    return torch.where(live, loss, torch.zeros_like(loss)).float(), torch.where(live[:, None], stats, torch.zeros_like(stats)).float()


def _distill_gradient(s, stats):
    used, p, _, rest = _teacher(s)
    p = p.float()
    x = s["logits"].float() / s["temp"]
    factor = torch.where(used.any(-1), s["grad"] / s["temp"], torch.zeros_like(s["grad"]))[:, None]
    lse, outside = stats[:, :1], stats[:, 1:]
    ids = s["ids"].clamp(min=0).to(torch.int64)
    if s["lse"] is None:
        d = torch.exp(x - lse)
    else:
        d = torch.exp(x - outside) * (torch.exp(outside.double() - lse.double()) - rest[:, None]).float()
        row, slot = used.nonzero(as_tuple=True)
        at = ids[row, slot]
        d[row, at] = torch.exp(x[row, at] - lse[row, 0])
    d.scatter_add_(1, ids, torch.where(used, -p, torch.zeros_like(p)))
    return (d * factor).to(s["logits"].dtype)


def _policy(s):
    x = s["logits"].float()
    lse = _normaliser(x)
    live = s["tokens"] >= 0
    token = s["tokens"].clamp(min=0).to(torch.int64)[:, None]
    logp = x.gather(1, token)[:, 0] - lse
    w = torch.exp(logp - s["rollout"])
    if s["cap"] > 0:
        w = w.clamp(max=s["cap"])
    logp, w = (torch.where(live, a, torch.zeros_like(a)).float() for a in (logp, w))
    d = torch.exp(x - lse.float()[:, None])
    d.scatter_add_(1, token, -torch.ones_like(logp)[:, None])
    return {"logp": logp, "w": w, "dlogits": (d * (w * s["advantages"])[:, None]).to(s["logits"].dtype)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "verify":
        return _exact_verify(case, s)
    out = {}
    for at in range(0, case["rows"], 512):  # rows at a time
        x = s["logits"][at:at + 512].double()
        if case["kind"] == "policy":
            one = _exact_policy(case, s, x, at)
        else:
            one = _exact_distill(case, s, x, at)
        for name, value in one.items():
            out.setdefault(name, []).append(value)
    return {name: torch.cat(parts) for name, parts in out.items()}


def _exact_policy(case, s, x, at):
    token = s["tokens"][at:at + 512].long()
    live = (token >= 0).double()
    z = torch.logsumexp(x, -1)
    here = torch.arange(x.shape[0], device="cuda")
    logp = (x[here, token.clamp(min=0)] - z) * live
    w = torch.exp(logp - s["rollout"][at:at + 512].double())
    w = (torch.clamp(w, max=case["cap"]) if case["cap"] > 0 else w) * live
    d = torch.exp(x - z[:, None])
    d[here, token.clamp(min=0)] -= 1.0
    return {"logp": logp, "w": w, "dlogits": d * (w * s["advantages"][at:at + 512].double())[:, None]}


def _exact_distill(case, s, x, at):
    ids = s["ids"][at:at + 512].long()
    y = s["top"][at:at + 512].double() / case["temp"]
    x = x / case["temp"]
    used = ids >= 0
    live = used.any(-1)
    y = y.masked_fill(~used, -math.inf)
    logp = y - (s["lse"][at:at + 512].double() if case["tail"] else torch.logsumexp(y, -1))[:, None]
    p = torch.exp(logp).masked_fill(~used, 0.0)
    z = torch.logsumexp(x, -1)
    mark = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), used.double()) > 0
    logq = x.gather(1, ids.clamp(min=0)) - z[:, None]
    loss = torch.where(p > 0, p * (logp - logq), 0.0).sum(-1)
    q = torch.exp(x - z[:, None])
    teacher = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), p)
    outside = z
    if case["tail"]:
        rest = (1.0 - p.sum(-1)).clamp(min=0.0)
        outside = torch.logsumexp(x.masked_fill(mark, -math.inf), -1)
        loss = loss + torch.where(rest > 0, rest * (torch.log(rest) - (outside - z)), 0.0)
        teacher = torch.where(mark, teacher, rest[:, None] * torch.exp(x - outside[:, None]))
    stats = torch.stack((z, outside), -1)
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    factor = torch.where(live, s["grad"][at:at + 512].double() / case["temp"], zero)
    full = {"loss": torch.where(live, loss, zero), "stats": torch.where(live[:, None], stats, zero)}
    if case["kind"] == "loss":
        return full
    d = {"dlogits": torch.where(live[:, None], (q - teacher) * factor[:, None], zero)}
    return d if case["kind"] == "backward" else {"loss": full["loss"], **d}


def _exact_verify(case, s):
    n, temp = _drafts(case), case["temp"] or 1.0
    tokens, logps, accepted, row, at = [], [], [], 0, 0
    drafts = s["drafts"].tolist()
    for b, m in enumerate(n):
        logp = torch.log_softmax(s["target"][row:row + m + 1].double() / temp, -1)
        mine = drafts[at:at + m]
        q = torch.exp(torch.log_softmax(s["draft"][at:at + m].double() / temp, -1)) if case["form"] == "model" else None
        taken = 0
        while taken < m:
            x = mine[taken]
            if case["form"] == "greedy":
                top = s["target"][row + taken]
                if int((top == top.max()).nonzero()[0]) != x:
                    break
            else:
                chance = float(torch.exp(logp[taken, x])) / (float(q[taken, x]) if q is not None else 1.0)
                if not float(s["uniforms"][at + taken]) < chance:
                    break
            taken += 1
        if case["form"] == "greedy":
            top = s["target"][row + taken]
            token = int((top == top.max()).nonzero()[0])
        else:
            p = torch.exp(logp[taken])
            if taken < m:
                other = q[taken] if q is not None else torch.nn.functional.one_hot(torch.tensor(mine[taken], device="cuda"), p.shape[0]).double() * 2
                p = torch.clamp(p - other, min=0.0)
            token = int((p / s["noise"][b].double()).argmax())
        new = mine[:taken] + [token]
        tokens += new + [-1] * (m - taken)
        logps += [float(logp[i, x]) for i, x in enumerate(new)] + [0.0] * (m - taken)
        accepted.append(taken)
        row, at = row + m + 1, at + m
    whole = dict(dtype=torch.int32, device="cuda")
    return {"tokens": torch.tensor(tokens, **whole), "accepted": torch.tensor(accepted, **whole),
            "logp": torch.tensor(logps, dtype=torch.float64, device="cuda")}
