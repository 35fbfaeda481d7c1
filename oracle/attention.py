"""Float64 oracle of a verify window's attention sub-layer: int4 projection, cache plan, cache
writer and tree attention.

Test infrastructure (see ``oracle/__init__.py``). The pages name the window only ("Multi-token
prediction turns each verification into four tokens"); the formulas are the plain ones, written
out in each docstring.
"""

from __future__ import annotations

import numpy as np

from .formats import float_to_e4m3_rne_sat


def w4_weight(q, scale, zero, group: int) -> np.ndarray:
    """w[n, k] = (code - zero) * scale; code k of a row is the low (k even) or high nibble of byte k / 2."""
    q = np.asarray(q)
    n, k = q.shape[0], 2 * q.shape[1]
    code = np.empty((n, k))
    code[:, 0::2], code[:, 1::2] = q & 15, q >> 4
    z = np.full((n, k // group), 8.0) if zero is None else np.asarray(zero, dtype=np.float64)
    return ((code.reshape(n, k // group, group) - z[:, :, None]) * np.asarray(scale, np.float64)[:, :, None]).reshape(n, k)


def w4_linear(q, scale, zero, group: int, x, bias=None, residual=None) -> np.ndarray:
    """y = x . W^T (+ bias) (+ residual)."""
    y = np.asarray(x, np.float64) @ w4_weight(q, scale, zero, group).T
    y = y if bias is None else y + np.asarray(bias, np.float64)
    return y if residual is None else y + np.asarray(residual, np.float64)


def kv_plan(ctx, new, page: int, num_pages: int, table, free, t: int, parents=None, with_mask=True) -> dict:
    """Plan of one step, request after request; ``bad`` says that a status was raised. The whole plan
    fails on bad lengths (start None), single rows fail on bad page ids or parents."""
    table, total, used, bad = np.array(table), 0, 0, False
    slot, pos, mask = np.full(t, -1, np.int64), np.full(t, -1, np.int64), np.zeros(t, np.uint64)
    start = [0]
    trees = parents is not None or with_mask
    for c, n in zip(ctx, new):
        if c < 0 or n < 0 or c + n > table.shape[1] * page or (trees and n > 64):
            return dict(fail=True)
        total += n
        used += -(-(c + n) // page) - -(-c // page)
        if total > t or used > len(free):
            return dict(fail=True)
        start.append(total)
    used = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        for i in range(-(-c // page), -(-(c + n) // page)):
            ok = 0 <= free[used] < num_pages
            table[b, i] = free[used] if ok else -1
            bad |= not ok
            used += 1
        good = []
        for j in range(n):
            row = start[b] + j
            up = j - 1 if parents is None else int(parents[row])
            m, depth, ok = 1 << j, 0, True
            if parents is None:
                m, depth = (2 << j) - 1, j
            elif up < -1 or up >= j:
                ok = False
            elif up >= 0:
                ok = good[up] is not None
                if ok:
                    m, depth = m | good[up][0], good[up][1] + 1
            good.append((m, depth) if ok else None)
            ident = int(table[b, (c + j) // page])
            if not 0 <= ident < num_pages:
                ok = False
            bad |= not ok
            if ok:
                slot[row], pos[row], mask[row] = ident * page + (c + j) % page, c + depth, m & (2 ** 64 - 1)
    return dict(fail=False, bad=bad, table=table, start=np.array(start), slot=slot, pos=pos, mask=mask, taken=used)


def kv_write(cache, rows, slots, page: int, scale=None) -> np.ndarray:
    """The cache [pages, heads, page, dim] (values, or E4M3 codes with scale [heads]) after rows [T, heads, dim]
    went to their slots; slots outside it are skipped."""
    out = np.array(cache)
    for r, s in zip(np.asarray(rows, np.float32), slots):
        if 0 <= s < out.shape[0] * page:
            v = r if scale is None else float_to_e4m3_rne_sat(r / np.asarray(scale, np.float32)[:, None])
            out[s // page, :, s % page] = v
    return out


def tree_attention(q, k, v, seen, scale: float):
    """softmax(scale q k^T over the seen keys) v of one request: q [n, heads, dim], k, v [keys, kv heads, dim],
    seen bool [n, keys]. Returns out [n, heads, dim], lse [n, heads], and for error bounds
    sum_j p_j |v_j| and scale * max_j sum_d |q_d k_jd|. A row that sees nothing gives 0 and -inf."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    n, hq, d = q.shape
    group = hq // k.shape[1]
    out, lse, spread, size = np.zeros((n, hq, d)), np.full((n, hq), -np.inf), np.zeros((n, hq, d)), np.zeros((n, hq))
    for i in range(n):
        ks, vs = k[seen[i]], v[seen[i]]
        if not len(ks):
            continue
        for h in range(hq):
            z = scale * (ks[:, h // group] @ q[i, h])
            top = z.max()
            if top == -np.inf:
                continue
            p = np.exp(z - top)
            lse[i, h] = top + np.log(p.sum())
            p /= p.sum()
            out[i, h] = p @ vs[:, h // group]
            spread[i, h] = p @ np.abs(vs[:, h // group])
            size[i, h] = scale * (np.abs(ks[:, h // group]) @ np.abs(q[i, h])).max()
    return out, lse, spread, size
