"""Scores that are equal, or nearly so, in many places: the exact score decides, and of equals the lowest index."""

import numpy as np
import pytest
import torch

from .test_gpu_verify_drafts import BF16, DEV, FP32, NEAR, q  # noqa: F401

pytestmark = pytest.mark.gpu
NONE = torch.empty(0, dtype=torch.int32)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("v,gap", [(9, 0), (700, 1), (5000, 0), (70001, 3)])
def test_equal_scores(q, dtype, v, gap):  # noqa: F811
    """Rows of equal logits under equal noise, of all tokens and of those behind some place."""
    first = [0, 1, 7, v // 2, v - 1]
    x = torch.full((len(first), v + gap), float("nan"), dtype=dtype, device=DEV)[:, :v]
    x[:] = 0.5
    for b, f in enumerate(first):
        x[b, :f] = -torch.inf
    tokens, accepted, _ = q.verify_drafts(x, NONE.to(DEV), noise=torch.full((len(first), v), 0.7, device=DEV))
    assert tokens.tolist() == first and not accepted.any()
    # behind a refused draft: of a looked-up one's place nothing is left, of a model's what p has above q
    x = x.repeat_interleave(2, 0)
    n = len(first)
    drafts, noise = torch.tensor(first, dtype=torch.int32, device=DEV), torch.full((n, v), 0.7, device=DEV)
    tokens, accepted, _ = q.verify_drafts(x, drafts, uniforms=torch.full((n,), 1.0, device=DEV), noise=noise)
    assert not accepted.any() and tokens[::2].tolist() == [f + 1 if f + 1 < v else f for f in first]
    y = torch.full((n, v), -torch.inf, dtype=dtype, device=DEV)
    y[torch.arange(n), drafts.long()] = 3.0
    tokens, accepted, _ = q.verify_drafts(x, drafts, uniforms=torch.full((n,), 1.0, device=DEV), noise=noise, draft_logits=y)
    assert not accepted.any() and tokens[::2].tolist() == [f + 1 if f + 1 < v else f for f in first]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("v,gap", [(700, 1), (8200, 0), (70001, 3)])
def test_nearly_equal_scores(q, dtype, v, gap):  # noqa: F811
    """Noise of a few neighbouring numbers: hundreds of scores within the bounds of the best, several in every granule.  The
    chosen one is among those that rounding cannot tell from the best, and the same wherever the noise's rows start."""
    g = torch.Generator().manual_seed(1)
    n = 6
    x = torch.zeros(n, v, dtype=dtype, device=DEV)
    noise = (1 + 2.0 ** -23 * torch.randint(0, 200, (n, v), generator=g)).float()
    wide = torch.full((n, v + gap), float("nan"), device=DEV)
    wide[:, :v] = noise.to(DEV)
    tokens, _, _ = q.verify_drafts(x, NONE.to(DEV), noise=wide[:, :v])
    again, _, _ = q.verify_drafts(x, NONE.to(DEV), noise=noise.to(DEV))
    assert torch.equal(tokens, again)
    score = (1 / noise.double()).numpy()
    for b in range(n):
        assert score[b, int(tokens[b])] >= score[b].max() * (1 - 2.0 ** -22)  # (p / e is rounded twice)
        equal = np.nonzero(noise[b].numpy() == noise[b, int(tokens[b])].item())[0]
        assert int(tokens[b]) == equal[0]
