"""Calls of the speculative step's operators that lie at the edge of what their documentation allows, on the GPU against
the fp64 oracle (oracle/speculative.py)."""
import numpy as np
import pytest

from oracle import speculative as sp
from test_speculative_gpu import U, dev, f32
from weight_quantized_expert_b200 import api

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- probabilities
# The bar is that of test_probs: |err| <= (8 + 2 max|l - max| / temperature) u p, and a step of the subnormal numbers.

def check_probs(x, temp):
    """Out of place, in place, and with logits and probabilities off 16-byte boundaries, alike and unlike each other."""
    import torch
    T, V = x.shape
    want = sp.token_probs(x, temp)
    span = np.where(np.isfinite(x), x.max(-1, keepdims=True).astype(np.float64) - x, 0.0) / temp
    flat, out = torch.zeros(4 + T * V, device="cuda"), torch.zeros(4 + T * V, device="cuda")
    got = [api.focr_token_probs(dev(x), temp)]
    same = dev(x)
    got.append(api.focr_token_probs(same, temp, out=same))
    logits = flat[1:1 + T * V].view(T, V)
    logits.copy_(dev(x))
    got += [api.focr_token_probs(logits, temp, out=out[s:s + T * V].view(T, V)).clone() for s in (1, 2)]
    for g in got:
        g = g.cpu().numpy().astype(np.float64)
        assert not np.isnan(g).any()
        assert (np.abs(g - want) <= (8 + 2 * span) * U * want + 1e-44).all()
        assert (g[np.isneginf(x)] == 0).all()


@pytest.mark.parametrize("V", [1, 3, 5, 10, 100, 777, 1000, 1920, 1921, 10000, 129280])
def test_probs_of_rows_far_below_zero(V):
    # parts of a row that hold no value, or none that is finite, take part in no sum
    rng = np.random.default_rng(V)
    x = 4 * f32(rng, 3, V)
    check_probs(x - np.float32(200), 1.0)
    logp = np.log(sp.token_probs(x)).astype(np.float32)
    check_probs(logp, 0.05)
    check_probs(logp, 1e-6)


@pytest.mark.parametrize("left", [1, 10, 1000])
@pytest.mark.parametrize("T", [1, 60])
def test_probs_of_rows_that_a_mask_leaves_few_tokens_of(left, T):
    rng = np.random.default_rng(left)
    x = np.full((T, 129280), -np.inf, np.float32)
    for t in range(T):
        x[t, rng.choice(129280, left, replace=False)] = -12
    check_probs(x, 0.1)
    x += f32(rng, *x.shape)
    check_probs(x, 0.01)


def test_probs_stay_nan_where_a_row_has_no_distribution():
    for V in (5, 3000, 129280):
        x = np.full((4, V), -np.inf, np.float32)
        x[1, V // 2], x[2, 0], x[3] = np.nan, np.inf, -200
        x[3, 1] = np.nan
        got = api.focr_token_probs(dev(x), 0.5).cpu().numpy()
        assert np.isnan(got[[0, 1, 3]]).all() and np.isnan(got[2]).any()
