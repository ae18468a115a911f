"""A drafted rollout and the training step that follows it, on the logits of one 4-bit output layer.

The draft model is the frozen NVFP4 output layer with one LoRA adapter, the policy the same layer with another.  The draft
model proposes tokens one at a time; the policy scores all places of a sequence in one call; the verification takes
drafts as far as it agrees and draws the token behind, so that the tokens are the policy's own.  Then both adapters learn: the
policy by the advantages of its tokens, with importance weights against the log-probabilities of the rollout, and the draft
model from the policy's likeliest tokens at the places that were reached.  Rows behind a refusal take no part: their token
is -1.  Nothing is copied to the host in between.

    python examples/drafted_policy_update.py [--sequences 6] [--drafts 4]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_rl_rollout_gb300 import build, inputs, qrr  # noqa: E402

HIDDEN, VOCAB, RANK, TOP = 512, 4096, 16, 32
TEMPERATURE = 1.0


def adapter(seed, dev):
    a, b, alpha = inputs.lora(RANK, HIDDEN, VOCAB, seed, device=dev)
    return dict(lora_A=a, lora_B=b, alpha=8 * alpha)  # (far enough apart for some drafts to be refused)


class Model:
    """States are the embedding of the token before and of the place; logits are the output layer's."""

    def __init__(self, places, dev):
        g = torch.Generator(device=dev).manual_seed(0)
        codes, scales, ts = qrr.quantize_nvfp4(inputs.weight(VOCAB, HIDDEN, 1, device=dev))
        self.head = dict(codes=codes, scales=scales, tensor_scale=ts)
        self.tokens = torch.randn(VOCAB, HIDDEN, generator=g, device=dev)
        self.places = torch.randn(places, HIDDEN, generator=g, device=dev)
        self.draft, self.policy = adapter(3, dev), adapter(5, dev)

    def states(self, before, place):
        return (self.tokens[before.clamp(min=0).long()] + self.places[place]).to(torch.bfloat16)

    def logits(self, x, lora, status):
        return qrr.linear_nvfp4_lora(x, dev_status=status, **self.head, **lora)

    def gradients(self, dlogits, x, lora, status):
        return qrr.lora_backward_nvfp4(dlogits, x, **self.head, **lora, dev_status=status)[1:]


def rollout(model, last, n, uniforms, noise, draft_noise, status):
    """n drafts behind the tokens `last` [B], and what the policy makes of them.

    Returns the policy's states [B (n + 1), HIDDEN] and logits, the draft model's [B n, ...], and the verification's outputs."""
    b, dev = last.numel(), last.device
    states, logits, drafts = [], [], [last]
    for i in range(n):
        states.append(model.states(drafts[-1], i))
        logits.append(model.logits(states[-1], model.draft, status))
        p = torch.softmax(logits[-1].float() / TEMPERATURE, -1)
        drafts.append(torch.argmax(p / draft_noise[i], -1).to(torch.int32))
    before = torch.stack(drafts, 1)  # [B, n + 1]
    x = model.states(before.reshape(-1), torch.arange(n + 1, device=dev).repeat(b))
    target = model.logits(x, model.policy, status)
    draft_x, draft_logits = torch.stack(states, 1).view(b * n, -1), torch.stack(logits, 1).view(b * n, -1)
    drafted = before[:, 1:].reshape(-1).contiguous()
    tokens, accepted, logp = qrr.verify_drafts(target, drafted, uniforms=uniforms, noise=noise, draft_logits=draft_logits,
                                               temperature=TEMPERATURE, dev_status=status)
    return dict(x=x, target=target, draft_x=draft_x, draft_logits=draft_logits, drafts=drafted, tokens=tokens, accepted=accepted,
                logp=logp)


def step(model, r, n, advantages, status):
    """The gradients of both adapters from a rollout. `advantages` [B]; the policy's logits are taken again, as after an update."""
    b, dev = advantages.numel(), advantages.device
    out = {}
    logits = model.logits(r["x"], model.policy, status)
    weight = advantages.repeat_interleave(n + 1) / b
    out["logp"], out["w"], out["dpolicy"] = qrr.token_logprobs_is_grad(logits, r["tokens"], weight, r["logp"], cap=2.0, dev_status=status)
    out["policy_logits"], out["weight"] = logits, weight
    out["policy"] = model.gradients(out["dpolicy"], r["x"], model.policy, status)

    # the policy's likeliest tokens teach the draft model at the places that were reached
    place = torch.arange(n, device=dev)
    reached = (place[None] <= r["accepted"][:, None]).view(-1, 1)
    rows = r["target"].view(b, n + 1, VOCAB)[:, :n].reshape(b * n, VOCAB).float()
    top, ids = torch.topk(rows, TOP, -1)
    out["ids"], out["top"] = torch.where(reached, ids, -1).to(torch.int32), top
    out["lse"] = torch.logsumexp(rows / TEMPERATURE, -1)
    out["grad"] = reached.view(-1).float() / reached.sum()
    out["loss"], out["ddraft"] = qrr.distill_topk_grad(r["draft_logits"], out["ids"], top, out["grad"], top_lse=out["lse"],
                                                       temperature=TEMPERATURE, dev_status=status)
    out["draft"] = model.gradients(out["ddraft"], r["draft_x"], model.draft, status)
    return out


def numbers(b, n, seed, dev):
    """The random numbers of a rollout."""
    g = torch.Generator(device=dev).manual_seed(seed)
    return dict(last=torch.randint(VOCAB, (b,), generator=g, device=dev, dtype=torch.int32),
                uniforms=torch.rand(b * n, generator=g, device=dev),
                noise=torch.empty(b, VOCAB, device=dev).exponential_(generator=g).clamp_(min=1e-30),
                draft_noise=torch.empty(n, b, VOCAB, device=dev).exponential_(generator=g).clamp_(min=1e-30))


def main(sequences, drafts):
    build.build()
    dev = torch.device("cuda:0")
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    model = Model(drafts + 1, dev)
    r = rollout(model, n=drafts, status=status, **numbers(sequences, drafts, 7, dev))
    advantages = torch.linspace(-1.0, 1.0, sequences, device=dev)
    out = step(model, r, drafts, advantages, status)
    flags = qrr.get_last_device_status(status)
    print(f"{sequences} sequences of {drafts} drafts: {r['accepted'].tolist()} taken, loss of the draft model "
          f"{(out['loss'] * out['grad']).sum().item():.4f}, largest importance weight {out['w'].max().item():.4f}, status {flags}")
    return model, r, out, flags


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--sequences", type=int, default=6)
    a.add_argument("--drafts", type=int, default=4)
    args = a.parse_args()
    main(args.sequences, args.drafts)
