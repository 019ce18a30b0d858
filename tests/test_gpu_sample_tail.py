"""bm_sample where weights are so small that their integers round: tail tokens, and sums over many of them."""

import math

import numpy as np
import pytest
import torch

from test_gpu_sample import _call, bm  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [2, 1000, 50257])
@pytest.mark.parametrize("T", [1.0, 0.05, 8.0])
def test_logprob_of_a_tail_token(bm, V, T):
    """u = 0 draws the lowest kept index, u above 1 the highest, whatever is left of their weights; the log probability is
    that of the logit, not of the rounded weight."""
    below = [1.0, 7.3, 17.77, 23.1, 25.5, 28.0, 29.5, 30.4]      # log of the weights: 2^-1.4 to 2^-43.9
    for u, at in ((0.0, 0), (2.0, V - 1)):
        x = torch.full((len(below), V), -float("inf"), device="cuda")
        x[:, V // 2] = 1.25
        if at == V // 2:
            continue
        x[:, at] = 1.25 - T * torch.tensor(below, device="cuda")
        ids, lp = _call(bm, x, temp=np.full(len(below), T), u=np.full(len(below), u))
        assert (ids == at).all()
        gap = (x[:, at].double() - 1.25).cpu().numpy() / np.float64(np.float32(T))
        want = gap - np.log1p(np.exp(gap))
        # one rounding to fp32; the sum of the weights is good to 2^-29
        assert (np.abs(lp - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -27).all(), lp - want


def test_weights_below_the_smallest_are_never_drawn(bm):
    """Below 2^-45 of the largest a weight counts as 0: neither end of u reaches it."""
    V = 300
    x = torch.full((2, V), -40.0, device="cuda")                 # e^-40 = 2^-57.7
    x[:, 100] = 0.0
    x[:, 200] = -1.0
    total = 1 + math.exp(-1.0)
    for u, at, w in ((0.0, 100, 1.0), (1.0, 200, math.exp(-1.0)), (7.0, 200, math.exp(-1.0))):
        ids, lp = _call(bm, x, u=np.full(2, u))
        assert (ids == at).all()
        want = math.log(w / total)
        assert (np.abs(lp - want) <= 2.0 ** -24 * abs(want) + 2.0 ** -27).all()


@pytest.mark.parametrize("V", [20000, 40000, 151936])
def test_sums_of_tiny_weights_do_not_depend_on_the_batch(bm, V):
    """Two equal largest logits at top-p 0.5: one of them holds half of the weight, unless anything else has any.  What
    else there is are weights of 0.4 units (2^-44) far apart, which add up the same however many CTAs share the row."""
    x = torch.full((1, V), -float("inf"), device="cuda")
    x[0, :2] = 0.0
    x[0, torch.arange(4, device="cuda") * (V // 4) + 77] = math.log(0.4) - 44 * math.log(2.0)
    ids, lp = _call(bm, x, top_p=[0.5], u=[0.9])
    assert ids[0] == 1 and abs(lp[0] + math.log(2.0)) <= 2.0 ** -24
    for B in (2, 9, 17, 40, 70, 130, 300):
        many, mlp = _call(bm, x.expand(B, V).contiguous(), top_p=np.full(B, 0.5), u=np.full(B, 0.9))
        assert (many == ids[0]).all() and (mlp == lp[0]).all(), B
