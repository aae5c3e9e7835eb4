"""The bounds that the 4-bit attention and weights are held to see a lost, a
repeated or a wrong entry: mistakes planted in the reference, on the CPU."""
import numpy as np
import pytest
import torch

from tests import fp4_bounds as B


def _bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


def _case(n, c, H, spread, seed):
    g = np.random.default_rng(seed)
    V = _bf16(g.standard_normal((1, n, c)))
    q = _bf16(spread * g.standard_normal((1, H, c)))
    return q, V, np.arange(n)[None]


@pytest.mark.parametrize("n", [1, 64, 512, 1024, 2000, 8999])
def test_equal_logits_show_every_entry(n):
    """Queries of zeros: every entry has the same weight, and lse counts them."""
    q, V, idx = _case(n, 128, 2, 0, n)
    out, lse, lim, lim_l = B.attention(q, V, idx, 128 ** -0.5)
    assert B.outside(_bf16(out), out, lim) <= 1 and B.outside(lse.astype(np.float32), lse, lim_l) <= 1
    for wrong in (idx[:, 1:], idx[:, :-1], np.concatenate((idx, idx[:, -1:]), 1)):
        bad = B.attention(q, V, wrong, 128 ** -0.5)
        assert B.outside(lse, bad[1], bad[3]) > 1


@pytest.mark.parametrize("n", [512, 2000])
def test_equal_logits_show_another_row(n):
    q, V, idx = _case(n, 128, 2, 0, n)
    out, lse, lim, _ = B.attention(q, V, idx, 128 ** -0.5)
    for at in (0, 63, n // 2, n - 1):
        other = idx.copy()
        other[0, at] = (at + 7) % n
        bad = B.attention(q, V, other, 128 ** -0.5)
        assert B.outside(_bf16(out), bad[0], bad[2]) > 1


@pytest.mark.parametrize("n", [512, 2000])
def test_a_query_of_its_own_shows_an_entry(n):
    """A query along an entry: nearly all its weight lies there, and the output is that row."""
    c = 128
    _, V, idx = _case(n, c, 1, 0, n)
    for at in (0, 63, 64, n // 2, n - 1):
        q = _bf16(2 * V[0, at])[None, None]
        out, lse, lim, lim_l = B.attention(q, V, idx, c ** -0.5)
        assert B.outside(_bf16(out), out, lim) <= 1
        bad = B.attention(q, V, np.delete(idx, at, 1), c ** -0.5)
        assert B.outside(_bf16(out), bad[0], bad[2]) > 10 and B.outside(lse, bad[1], bad[3]) > 10


def test_weights_show_half_a_percent():
    q, V, _ = _case(300, 512, 64, 2, 1)
    lse = B.attention(q, V, np.arange(300)[None], 512 ** -0.5)[1]
    w, lim = B.weights(q[0], lse[0], V[0], 512 ** -0.5)
    assert abs(w.sum() - 64) < 1e-9 and (lim < 0.005 * w).all()
