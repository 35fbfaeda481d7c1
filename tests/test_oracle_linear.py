"""Pins of the linear-attention oracle against closed forms and torch operations (CPU)."""

import numpy as np
import pytest
import torch

from oracle import linear as OL


def _case(seed, n, hk, h, d):
    r = np.random.default_rng(seed)
    return r.normal(size=(h, d, d)), r.normal(size=(n, hk, d)), r.normal(size=(n, hk, d)), r.normal(size=(n, h, d)), -r.random((n, h))


@pytest.mark.parametrize("hk,h", [(2, 2), (1, 3)])
def test_rows_against_the_sum_over_all_earlier_rows(hk, h):
    s0, q, k, v, g = _case(0, 7, hk, h, 5)
    out, s, bound, size, chain = OL.linear_attention(s0, q, k, v, g, 0.3)
    share, c = h // hk, np.cumsum(g, 0)
    for t in range(7):
        for a in range(h):
            w = np.array([np.exp(c[t, a] - c[j, a]) * (q[t, a // share] @ k[j, a // share]) for j in range(t + 1)])
            want = 0.3 * (w @ v[:t + 1, a] + np.exp(c[t, a]) * q[t, a // share] @ s0[a])
            assert np.allclose(out[t, a], want, rtol=1e-12)
    want = np.exp(c[-1])[:, None, None] * s0 + np.einsum("th,thi,thj->hij", np.exp(c[-1] - c), np.repeat(k, share, 1), v)
    assert np.allclose(s, want, rtol=1e-12)
    assert np.all(np.abs(out) <= bound * (1 + 1e-12)) and np.all(np.abs(s) <= size * (1 + 1e-12)) and np.all(size <= chain * (1 + 1e-12))


def test_no_decay_is_a_running_sum_and_full_decay_forgets():
    s0, q, k, v, g = _case(1, 4, 1, 1, 3)
    _, s, *_ = OL.linear_attention(s0, q, k, v, 0 * g, 1.0)
    assert np.allclose(s[0], s0[0] + k[:, 0].T @ v[:, 0])
    out, s, *_ = OL.linear_attention(s0, q, k, v, np.full_like(g, -np.inf), 1.0)
    assert np.allclose(s[0], np.outer(k[3, 0], v[3, 0])) and np.allclose(out[:, 0], (q[:, 0] * k[:, 0]).sum(1)[:, None] * v[:, 0])


def test_a_tree_is_its_chains():
    s0, q, k, v, g = _case(2, 4, 2, 2, 3)
    masks = [0b1, 0b11, 0b101, 0b1011]
    out, _ = OL.tree_attention(s0, q, k, v, g, masks, 0.5)
    for path in ([0, 1, 3], [0, 2]):
        want, s, *_ = OL.linear_attention(s0, q[path], k[path], v[path], g[path], 0.5)
        assert np.allclose(out[path], want, rtol=1e-12)
        assert np.allclose(OL.advance(s0, k, v, g, sum(1 << i for i in path))[0], s, rtol=1e-12)
    assert np.array_equal(OL.advance(s0, k, v, g, 0)[0], s0)


def test_norms_and_gates_against_torch():
    r = np.random.default_rng(3)
    y, w, g, res = r.normal(size=(3, 12)), r.normal(size=4), r.normal(size=(3, 12)), r.normal(size=(3, 12))
    t = torch.from_numpy
    want = torch.nn.functional.rms_norm(t(y).view(3, 3, 4), (4,), t(w), 1e-3).view(3, 12)
    for kind, f in (("mul", lambda x: x), ("sigmoid", torch.sigmoid), ("silu", torch.nn.functional.silu)):
        got, size = OL.block_sum(y, w, 4, g, kind, res, 0.5, 2.0, 1e-3)
        assert np.allclose(got, (0.5 * want * f(t(g)) + 2 * t(res)).numpy(), rtol=1e-12) and np.all(np.abs(got) <= size + 1e-12)
    assert np.allclose(OL.rmsnorm(y, r.normal(size=12) * 0 + 1, 0.0).var(-1) + OL.rmsnorm(y, np.ones(12), 0.0).mean(-1) ** 2, 1)
    assert np.array_equal(OL.block_sum(y, branch_scale=2.0)[0], 2 * y)
