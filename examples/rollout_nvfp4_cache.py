"""A rollout through one attention layer with 4-bit weights and a 4-bit key/value cache.

Two groups of rollouts each share a prompt's pages.  The prompts are scored in
one call (a chunk of rows a sequence), then every rollout takes decode steps of
one token: projection by the NVFP4 + LoRA linear, append to its own pages,
attention over the cache, output projection.  At the end a rollout's keys and
values are read back, and the last step is compared with attention over them in
float32.

    python examples/rollout_nvfp4_cache.py [--steps 8]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_rl_rollout_gb300 import build, inputs, qrr  # noqa: E402

HIDDEN, HQ, HKV, DIM, PAGE = 1024, 8, 2, 128, 32
PROMPTS, GROUP = (70, 45), 3  # tokens of the prompts; rollouts of each


def linear(n, k, seed, dev):
    """An NVFP4 weight with a LoRA adapter, as keyword arguments of the linear call."""
    codes, scales, ts = qrr.quantize_nvfp4(inputs.weight(n, k, seed, device=dev))
    a, b, alpha = inputs.lora(8, k, n, seed + 1, device=dev)
    return dict(codes=codes, scales=scales, tensor_scale=ts, lora_A=a, lora_B=b, alpha=alpha)


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class Layer:
    def __init__(self, dev):
        self.qkv = linear((HQ + 2 * HKV) * DIM, HIDDEN, 1, dev)
        self.out = linear(HIDDEN, HQ * DIM, 3, dev)

    def __call__(self, x, cache, pos, cu=None, max_new=None, dev_status=None):
        """x [T, HIDDEN] -> [T, HIDDEN]: rows cu[b] .. cu[b + 1] - 1 are sequence b's tokens from position pos[b] on."""
        rows = qrr.linear_nvfp4_lora(x, dev_status=dev_status, **self.qkv).view(-1, HQ + 2 * HKV, DIM)
        q, k, v = rows[:, :HQ], rows[:, HQ:HQ + HKV], rows[:, HQ + HKV:]  # slices: no copies
        qrr.kv_append_nvfp4(k, v, cache, pos, cu=cu, dev_status=dev_status)
        o = qrr.attention_nvfp4(q, cache, pos, cu=cu, max_new=max_new, dev_status=dev_status)
        return q, qrr.linear_nvfp4_lora(o.view(-1, HQ * DIM), dev_status=dev_status, **self.out), o


def main(steps):
    build.build()
    dev = torch.device("cuda:0")
    layer, status = Layer(dev), torch.zeros(1, dtype=torch.int32, device=dev)

    # pages: the prompt's whole pages are shared by its group; the page that a
    # prompt ends in is copied to each rollout, which goes on in it
    per = -(-(max(PROMPTS) + steps) // PAGE)
    prompt_table, table, free = [], [], 0
    for n in PROMPTS:
        used = -(-n // PAGE)
        prompt_table.append(list(range(free, free + used)) + [0] * (per - used))
        free += used
    for g, n in enumerate(PROMPTS):
        for _ in range(GROUP):
            shared = n // PAGE
            table.append(prompt_table[g][:shared] + list(range(free, free + per - shared)))
            free += per - shared
    gs = [torch.full((HKV,), 0.05, device=dev) for _ in range(2)]
    prompts = qrr.KvCacheNvfp4.empty(free, HKV, PAGE, DIM, i32(prompt_table, dev), *gs)
    rollouts = qrr.KvCacheNvfp4(*prompts.tensors[:4], i32(table, dev), *gs)  # the same buffers, another table

    cu = [0]
    for n in PROMPTS:
        cu.append(cu[-1] + n)
    x = inputs.activations(cu[-1], HIDDEN, 5, device=dev)
    _, y, _ = layer(x, prompts, i32([0] * len(PROMPTS), dev), cu=i32(cu, dev), max_new=max(PROMPTS), dev_status=status)

    for buffer in prompts.tensors[:4]:
        for g, n in enumerate(PROMPTS):
            if n % PAGE:
                for r in range(GROUP):
                    buffer[table[g * GROUP + r][n // PAGE]] = buffer[prompt_table[g][n // PAGE]]

    # each rollout starts from its prompt's last token, with a little noise of its own
    h = torch.cat([y[c - 1:c].expand(GROUP, -1) for c in cu[1:]]).float()
    h = (h / h.std() + 0.1 * torch.randn_like(h)).to(torch.bfloat16).contiguous()
    length = [n for n in PROMPTS for _ in range(GROUP)]
    for t in range(steps):
        q, y, o = layer(h, rollouts, i32([n + t for n in length], dev), dev_status=status)
        h = (y.float() / y.float().std()).to(torch.bfloat16)

    # the last step of one rollout again, from the values read back
    b, n = 1, length[1] + steps
    counts = [n if i == b else 0 for i in range(len(length))]
    ends = [sum(counts[:i]) for i in range(len(counts) + 1)]
    k, v = qrr.kv_read_nvfp4(rollouts, i32([0] * len(length), dev), cu=i32(ends, dev), rows=n, dev_status=status)
    kf, vf = (z.float().repeat_interleave(HQ // HKV, dim=1) for z in (k, v))
    p = torch.softmax(torch.einsum("hd,jhd->hj", q[b].float(), kf) * DIM ** -0.5, dim=-1)
    want = torch.einsum("hj,jhd->hd", p, vf)
    err = ((o[b].float() - want).norm() / want.norm()).item()
    flags = qrr.get_last_device_status(status)
    cached = sum(length) + steps * len(length)
    print(f"{len(length)} rollouts, {steps} steps, {cached} cached tokens, {free} pages of {PAGE}: "
          f"attention against its read-back values {err:.2e}, status {flags}")
    return err, flags


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--steps", type=int, default=8)
    main(a.parse_args().steps)
