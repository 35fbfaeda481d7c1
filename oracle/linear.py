"""Float64 oracle of the linear-attention sub-layer: rows one after the other, trees of drafted tokens, and the
norm, gate and residual between two sub-layers.

Test infrastructure (see ``oracle/__init__.py``). The formulas are the plain recurrences, written out in each docstring;
beside each result stands the sum of its terms' magnitudes, which bounds what rounding can do to it.
"""

from __future__ import annotations

import numpy as np


def _step(state, size, k, v, g, share: int):
    """S <- e^g S + k v^T for every value head, and the same of the magnitudes."""
    with np.errstate(invalid="ignore", over="ignore"):
        kk = np.repeat(np.asarray(k, np.float64), share, 0)
        f = np.exp(np.asarray(g, np.float64))[:, None, None]
        return state * f + kk[:, :, None] * v[:, None, :], size * f + np.abs(kk)[:, :, None] * np.abs(v)[:, None, :]


def _read(state, size, q, share: int, scale: float):
    with np.errstate(invalid="ignore", over="ignore"):
        qq = np.repeat(np.asarray(q, np.float64), share, 0)
        return scale * np.einsum("hi,hij->hj", qq, state), abs(scale) * np.einsum("hi,hij->hj", np.abs(qq), size)


def linear_attention(state, q, k, v, g, scale: float):
    """One request: state [heads, d, d], q, k [n, key heads, d], v [n, heads, d], g [n, heads] log decays.
    S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t; value head h uses key head h // share. Returns out, the state
    after, the magnitudes of both, and the sum over steps of the state's magnitude as it decays (what a rounding in
    every step can come to)."""
    state, v = np.array(state, np.float64), np.asarray(v, np.float64)
    share, size, chain = v.shape[1] // q.shape[1], np.abs(state), np.zeros_like(state)
    out, bound = np.zeros(v.shape), np.zeros(v.shape)
    for t in range(len(v)):
        state, size = _step(state, size, k[t], v[t], g[t], share)
        chain = chain * np.exp(np.asarray(g[t], np.float64))[:, None, None] + size
        out[t], bound[t] = _read(state, size, q[t], share, scale)
    return out, state, bound, size, chain


def tree_attention(state, q, k, v, g, masks, scale: float):
    """The same for the nodes of a tree: node i comes after the nodes j < i whose bit is set in masks[i], in order."""
    v = np.asarray(v, np.float64)
    share = v.shape[1] // q.shape[1]
    out, bound = np.zeros(v.shape), np.zeros(v.shape)
    for i in range(len(v)):
        s, size = np.array(state, np.float64), np.abs(state)
        for j in range(i + 1):
            if j == i or int(masks[i]) >> j & 1:
                s, size = _step(s, size, k[j], v[j], g[j], share)
        out[i], bound[i] = _read(s, size, q[i], share, scale)
    return out, bound


def advance(state, k, v, g, accepted: int):
    """The state after the rows whose bits are set, in order, and its magnitude."""
    v = np.asarray(v, np.float64)
    s, size = np.array(state, np.float64), np.abs(state)
    for j in range(len(v)):
        if int(accepted) >> j & 1:
            s, size = _step(s, size, k[j], v[j], g[j], v.shape[1] // k.shape[1])
    return s, size


def gate(kind: str, x):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return {"mul": lambda: x, "sigmoid": lambda: 1 / (1 + np.exp(-x)), "silu": lambda: x / (1 + np.exp(-x))}[kind]()


def rmsnorm(x, w, eps: float, group=None):
    """x / sqrt(mean(x^2) + eps) * w over groups of the last dimension (all of it by default)."""
    x = np.asarray(x, np.float64)
    parts = x.reshape(*x.shape[:-1], -1, group or x.shape[-1])
    return (parts / np.sqrt((parts ** 2).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)).reshape(x.shape)


def block_sum(y, post_w=None, group=None, gate_values=None, kind="none", residual=None, branch_scale=1.0, residual_scale=1.0, eps=1e-6):
    """residual_scale * residual + branch_scale * gate * norm(y), and the magnitudes of the terms."""
    z = np.asarray(y, np.float64) if post_w is None else rmsnorm(y, post_w, eps, group)
    if kind != "none":
        z = z * gate(kind, gate_values)
    r = 0.0 if residual is None else residual_scale * np.asarray(residual, np.float64)
    return r + branch_scale * z, np.abs(r) + np.abs(branch_scale * z)
