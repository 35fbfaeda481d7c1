"""The operators of a window's linear-attention sub-layer, in plain form and as the library's calls.

Beside softmax attention a hybrid decoder has layers whose attention is linear, with a decay for each head: a
request then holds a matrix for each value head instead of a cache that grows. A serving program runs

* ``mdw_linear_attention``      -- the rows of prompts and of decoded tokens, from one state to the next;
* ``mdw_linear_tree_attention`` -- the nodes of a tree of drafted tokens; the state stays as it is;
* ``mdw_linear_state_advance``  -- the state along the path that was accepted;
* ``mdw_block_norm``            -- what stands between two sub-layers: the norm after one, its gate, the scaled
  residual and the norm before the next (or the gated norm of each head, without a residual).

``run`` computes them with elementary torch operations in 32 bits (``own`` false) or by the
library's entry points (``own`` true); ``exact`` gives the definition in 64 bits.
"""

import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one decoded token of one request: the smallest call of a layer
        {"name": "lin_token", "op": "lin", "b": 1, "hqk": 20, "h": 20, "d": 128, "new_lo": 1, "new_hi": 1,
         "steps": False, "fresh": False, "inplace": True},
        # a decode batch in which some requests take up to 4 tokens, decays of each token, two value heads to a key head
        {"name": "lin_tokens_batch", "op": "lin", "b": 61, "hqk": 16, "h": 32, "d": 128, "new_lo": 1, "new_hi": 4,
         "steps": True, "fresh": False, "inplace": True},
        # one long prompt of odd length from an empty state
        {"name": "lin_prompt_long", "op": "lin", "b": 1, "hqk": 32, "h": 32, "d": 128, "new_lo": 16301, "new_hi": 16301,
         "steps": False, "fresh": True, "inplace": False},
        # chunks of prompts beside decoded tokens, decays of each token
        {"name": "lin_prompts_mixed", "op": "lin", "b": 24, "hqk": 20, "h": 20, "d": 128, "new_lo": 1, "new_hi": 2100,
         "steps": True, "fresh": False, "inplace": False},
        # a chain of 4 drafted tokens of one request
        {"name": "tree_window", "op": "tree", "b": 1, "hqk": 20, "h": 20, "d": 128, "new_lo": 4, "new_hi": 4, "steps": False},
        # a batch of trees
        {"name": "tree_batch", "op": "tree", "b": 48, "hqk": 16, "h": 32, "d": 128, "new_lo": 1, "new_hi": 16, "steps": True},
        # the largest trees: 64 nodes, heads of 64
        {"name": "tree_wide", "op": "tree", "b": 12, "hqk": 32, "h": 64, "d": 64, "new_lo": 64, "new_hi": 64, "steps": True},
        # the accepted path of one window
        {"name": "advance_window", "op": "advance", "b": 1, "hqk": 20, "h": 20, "d": 128, "new_lo": 4, "new_hi": 4,
         "steps": False, "inplace": True},
        # the accepted paths of a batch
        {"name": "advance_batch", "op": "advance", "b": 48, "hqk": 16, "h": 32, "d": 128, "new_lo": 1, "new_hi": 16,
         "steps": True, "inplace": True},
        # between two sub-layers, one token: norm after, residual, norm before
        {"name": "norm_token", "op": "norm", "t": 1, "w": 2560, "group": 0, "post": True, "gate": "none", "rows": False,
         "res": "bf16", "pre": True, "x": "bf16", "y": "bf16"},
        # the gated norm of each head of a prompt's linear attention
        {"name": "norm_heads", "op": "norm", "t": 4099, "w": 4096, "group": 128, "post": True, "gate": "sigmoid", "rows": True,
         "res": "none", "pre": False, "x": "bf16", "y": "bf16"},
        # between two sub-layers of a prompt: gate by channel, residual in fp32
        {"name": "norm_prompt", "op": "norm", "t": 16381, "w": 2560, "group": 0, "post": True, "gate": "mul", "rows": False,
         "res": "f32", "pre": True, "x": "bf16", "y": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["lin", "lin", "lin", "tree", "advance", "norm", "norm"])
    if op == "norm":
        x = rng.choice(["bf16", "f16"])
        group = rng.choice([0, 0, 64, 128])
        w = group * _log(rng, 1, 64) if group else _log(rng, 65, 12288)
        pre = rng.random() < 0.7
        return {"op": op, "t": _log(rng, 1, 16381 * 2560 // max(w, 2560)), "w": w, "group": group, "post": bool(group) or rng.random() < 0.7,
                "gate": rng.choice(["none", "mul", "sigmoid", "silu"]), "rows": rng.random() < 0.5,
                "res": rng.choice([x, x, "f32", "none"]), "pre": pre, "x": x, "y": rng.choice([x, x, "f32"])}
    d = rng.choice([64, 128, 128])
    hqk, share = _log(rng, 1, 32), rng.choice([1, 1, 2, 4])
    h = hqk * share
    b = _log(rng, 1, max(1, min(64, 61 * 32 * 128 * 128 // (h * d * d))))
    steps = rng.random() < 0.5
    if op != "lin":
        hi = _log(rng, 1, 64)
        c = {"op": op, "b": b, "hqk": hqk, "h": h, "d": d, "new_lo": rng.randint(1, hi), "new_hi": hi, "steps": steps}
        return {**c, "inplace": rng.random() < 0.5} if op == "advance" else c
    hi = _log(rng, 1, max(1, min(16301, 16301 * 32 * 128 // (b * h * d))))
    return {"op": op, "b": b, "hqk": hqk, "h": h, "d": d, "new_lo": rng.randint(0 if b > 1 else 1, hi), "new_hi": hi, "steps": steps,
            "fresh": rng.random() < 0.3, "inplace": rng.random() < 0.5}


def _lengths(c):
    """Rows of each request, spread over the case's range, the last of them the longest."""
    v = [c["new_lo"] + int((c["new_hi"] + 1 - c["new_lo"]) * ((i + 1) * 0.7548776662 % 1.0)) for i in range(c["b"])]
    v[-1] = c["new_hi"]
    return np.array(v, dtype=np.int64)


def work(c):
    if c["op"] == "norm":
        n, e = c["t"] * c["w"], {"bf16": 2, "f16": 2, "f32": 4, "none": 0}
        byts = n * e[c["y"]] + 2 * (c["group"] or c["w"]) * c["post"] + (0 if c["gate"] == "none" else 2 * (n if c["rows"] else c["w"]))
        byts += n * (2 * e[c["res"]] if c["res"] != "none" else e[c["x"]]) + (2 * n + 2 * c["w"]) * c["pre"]
        return {"bytes": byts, "flops": 0}
    t, state = int(_lengths(c).sum()), c["h"] * c["d"] * c["d"] * 4
    decay = 4 * c["h"] * (t if c["steps"] else 1)
    if c["op"] == "lin":
        return {"bytes": c["b"] * state * (1 if c["fresh"] else 2) + t * (c["hqk"] + c["h"]) * c["d"] * 4 + decay + 12 * c["b"],
                "flops": 4.0 * t * c["h"] * c["d"] ** 2}
    if c["op"] == "tree":
        return {"bytes": c["b"] * state + t * (c["hqk"] + c["h"]) * c["d"] * 4 + decay + 8 * t + 8 * c["b"],
                "flops": 2.0 * t * c["h"] * c["d"] ** 2}
    taken = int(sum((n + 1) // 2 for n in _lengths(c)))   # about half of a tree's nodes lie on the path
    return {"bytes": 2 * c["b"] * state + taken * (c["hqk"] + c["h"]) * c["d"] * 2 + (4 * c["h"] * taken if c["steps"] else 4 * c["h"]) + 20 * c["b"],
            "flops": 2.0 * taken * c["h"] * c["d"] ** 2}


# ------------------------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _int(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _masks(rs, lengths):
    """Trees of drafted tokens: node 0 is the root, each other one hangs on one of the three before it. Bit j of a node's
    mask: node j is the node itself or an ancestor."""
    out = []
    for n in lengths:
        m = []
        for i in range(n):
            p = max(i - 1 - int(rs.randint(0, 3)), 0)
            m.append((m[p] if i else 0) | 1 << i)
        out.append(m)
    return out


def prepare(c, seed):
    g, rs = _gen(seed), np.random.RandomState(int(seed) % (1 << 31))
    s = {"case": c}
    if c["op"] == "norm":
        t, w, x = c["t"], c["w"], DT[c["x"]]
        s["y"] = _normal(g, (t, w), DT[c["y"]])
        s["post"] = _normal(g, (c["group"] or w,), x, 0.2).add_(1) if c["post"] else None
        s["gate"] = None if c["gate"] == "none" else _normal(g, (t, w) if c["rows"] else (w,), x)
        res = None if c["res"] == "none" else DT[c["res"]]
        s["r"] = None if res is None else _normal(g, (t, w), res, 3.0)
        s["pre"] = _normal(g, (w,), x, 0.2).add_(1) if c["pre"] else None
        s["sum"] = torch.empty((t, w), dtype=res or x, device="cuda")
        s["out"] = torch.empty((t, w), dtype=x, device="cuda") if c["pre"] else None
        return s
    b, hqk, h, d, n = c["b"], c["hqk"], c["h"], c["d"], _lengths(c)
    t = int(n.sum())
    # queries, keys (of unit length) and values as slices of one projection's rows
    qkv = _normal(g, (t, (2 * hqk + h) * d + 64), torch.bfloat16)
    s["q"] = qkv[:, 64:64 + hqk * d].unflatten(1, (hqk, d))
    s["k"] = qkv[:, 64 + hqk * d:64 + 2 * hqk * d].unflatten(1, (hqk, d))
    s["v"] = qkv[:, 64 + 2 * hqk * d:].unflatten(1, (h, d))
    s["k"].copy_(torch.nn.functional.normalize(s["k"].float(), dim=-1))
    # decays of the heads from a token's to a thousand tokens' memory; of each token around them, now and then a strong one
    rate = torch.exp(torch.linspace(0, math.log(1e-3), h, device="cuda"))
    if c["steps"]:
        step = torch.nn.functional.softplus(torch.randn((t, h), generator=g, device="cuda"))
        s["decay"] = -rate * step * torch.where(torch.rand((t, h), generator=g, device="cuda") < 0.01, 20.0, 1.0)
    else:
        s["decay"] = -rate * (torch.rand(h, generator=g, device="cuda") + 0.5)
    s["start"] = _int(np.concatenate([[0], np.cumsum(n)]))
    # states of the requests somewhere in a pool, those after the call in place or in other slots
    fresh, inplace = c.get("fresh", False), c.get("inplace", c["op"] == "tree")
    slots = rs.permutation(b + 1 if inplace else 2 * b + 1)
    s["pool"] = _normal(g, (len(slots), h, d, d), torch.float32)
    s["slot_in"] = _int(np.full(b, -1) if fresh else slots[:b])
    s["slot_out"] = _int(slots[:b] if inplace else slots[-b:])
    if c["op"] != "lin":
        masks = _masks(rs, n)
        s["mask"] = _int(np.array([m for r in masks for m in r], dtype=np.uint64).view(np.int64), torch.int64)
        s["accepted"] = _int(np.array([r[rs.randint(len(r) // 2, len(r))] for r in masks], dtype=np.uint64).view(np.int64), torch.int64)
    if c["op"] != "advance":
        s["out"] = torch.empty((t, h, d), dtype=torch.bfloat16, device="cuda")
    if own:  # the handle of the states and the workspace that a program keeps
        from moe_decode_weight_gb300 import api
        s["state"] = api.LinearState(s["pool"])
        if c["op"] == "lin":
            nbytes = api.mdw_linear_attention_workspace_bytes(s["state"], b, t, hqk, c["new_hi"])
            s["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------ plain forms


def _padded(s, x, width):
    """Rows of the requests side by side: [requests, width, ...] in fp32 (zeros behind each one's last row)."""
    start = s["start"].long()
    at = start[:-1, None] + torch.arange(width, device=x.device)
    live = at < start[1:, None]
    rows = x[at.clamp(max=max(x.shape[0] - 1, 0))]
    return torch.where(live.view(*live.shape, *[1] * (x.dim() - 1)), rows, torch.zeros((), dtype=x.dtype, device=x.device))


def _heads_of(s, width):
    """q, k, v [requests, value heads, width, d] in fp32 and log decays [requests, value heads, width] in 64 bits."""
    c = s["case"]
    share = c["h"] // c["hqk"]
    q, k = (_padded(s, s[x], width).float().repeat_interleave(share, 2).transpose(1, 2) for x in "qk")
    v = _padded(s, s["v"], width).float().transpose(1, 2)
    g = s["decay"] if c["steps"] else s["decay"].expand(s["v"].shape[0], c["h"])
    return q, k, v, _padded(s, g, width).double().transpose(1, 2)


def _states(s):
    slots = s["slot_in"].long()
    return torch.where((slots >= 0)[:, None, None, None], s["pool"][slots.clamp(min=0)], 0.0)


def _packed(s, o):
    """[requests, heads, width, d] back to the packed rows."""
    start = s["start"].long()
    r = torch.arange(s["out"].shape[0], device=o.device)
    req = torch.searchsorted(start[1:], r, right=True)
    return o.transpose(1, 2)[req, r - start[req]]


def _plain_lin(s):
    c, size = s["case"], 128
    b, h, d = c["b"], c["h"], c["d"]
    chunks = -(-c["new_hi"] // size)
    q, k, v, g = (x.reshape(b, h, chunks, size, *x.shape[3:]) for x in _heads_of(s, chunks * size))
    cum = torch.cumsum(g, -1)
    total = cum[..., -1]
    # inside a chunk
    lower = torch.ones((size, size), dtype=torch.bool, device=q.device).tril()
    gap = torch.where(lower, cum[..., :, None] - cum[..., None, :], -math.inf)
    o = ((q @ k.transpose(-1, -2)) * torch.exp(gap).float()) @ v
    # what a chunk adds to the state, and the states between the chunks
    add = (k * torch.exp(total[..., None] - cum).float()[..., None]).transpose(-1, -2) @ v
    edge = torch.cat((torch.zeros_like(total[..., :1]), torch.cumsum(total, -1)), -1)
    before = torch.arange(chunks + 1, device=q.device)[:, None] > torch.arange(chunks, device=q.device)
    weight = torch.exp(torch.where(before, edge[..., :, None] - edge[..., None, 1:], -math.inf)).float()
    state = weight @ add.reshape(b, h, chunks, d * d) + torch.exp(edge).float()[..., None] * _states(s).reshape(b, h, 1, d * d)
    o = o + torch.exp(cum).float()[..., None] * (q @ state[:, :, :-1].reshape(b, h, chunks, d, d))
    s["out"].copy_(_packed(s, (o * d ** -0.5).reshape(b, h, chunks * size, d)))
    s["pool"][s["slot_out"].long()] = state[:, :, -1].reshape(b, h, d, d)
    return [s["out"], s["pool"]]


def _bits(mask, width):
    return (mask[..., None] >> torch.arange(width, device=mask.device)) & 1 == 1


def _plain_tree(s):
    c = s["case"]
    width = c["new_hi"]
    q, k, v, g = _heads_of(s, width)
    seen = _bits(_padded(s, s["mask"], width), width)[:, None]
    cum = torch.where(seen, g[:, :, None, :], 0.0).sum(-1)
    gap = torch.where(seen, cum[..., :, None] - cum[..., None, :], -math.inf)
    o = ((q @ k.transpose(-1, -2)) * torch.exp(gap).float()) @ v + torch.exp(cum).float()[..., None] * (q @ _states(s))
    s["out"].copy_(_packed(s, o * c["d"] ** -0.5))
    return s["out"]


def _plain_advance(s):
    width = s["case"]["new_hi"]
    q, k, v, g = _heads_of(s, width)
    taken = _bits(s["accepted"], width)[:, None]
    cum = torch.cumsum(torch.where(taken, g, 0.0), -1)
    total = cum[..., -1:]
    f = torch.where(taken, torch.exp(total - cum), 0.0).float()
    s["pool"][s["slot_out"].long()] = torch.exp(total).float()[..., None] * _states(s) + (k * f[..., None]).transpose(-1, -2) @ v
    return s["pool"]


def _act(kind, gate):
    if kind == "mul":
        return gate
    f = 1 / (1 + torch.exp(-gate))
    return f if kind == "sigmoid" else gate * f


def _plain_norm(s):
    c = s["case"]
    z = s["y"].float()
    if c["post"]:
        z = z.view(c["t"], -1, c["group"] or c["w"])
        z = (z * torch.rsqrt(z.square().mean(-1, keepdim=True) + 1e-6) * s["post"].float()).view(c["t"], c["w"])
    if c["gate"] != "none":
        z = z * _act(c["gate"], s["gate"].float())
    z = 0.5 * z
    if c["res"] != "none":
        z = z + 0.75 * s["r"].float()
    r = z.to(s["sum"].dtype)
    if not c["pre"]:
        return r
    x = r.float()
    return [r, (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["pre"].float()).to(DT[c["x"]])]


# ------------------------------------------------------------------------------------ the calls


def _own(s):
    from moe_decode_weight_gb300 import api
    c = s["case"]
    if c["op"] == "norm":
        api.mdw_block_norm(s["y"], s["sum"], post_weight=s["post"], group=c["group"] or None, gate=s["gate"],
                           gate_kind=c["gate"], residual=s["r"], pre_weight=s["pre"], x=s["out"], branch_scale=0.5, residual_scale=0.75)
        return [s["sum"], s["out"]] if c["pre"] else s["sum"]
    if c["op"] == "lin":
        api.mdw_linear_attention(s["state"], s["q"], s["k"], s["v"], s["decay"], s["out"], s["start"], s["slot_in"], s["slot_out"],
                                 c["new_hi"], s["ws"])
        return [s["out"], s["pool"]]
    if c["op"] == "tree":
        api.mdw_linear_tree_attention(s["state"], s["q"], s["k"], s["v"], s["decay"], s["out"], s["start"], s["slot_in"], c["new_hi"],
                                      tree_mask=s["mask"])
        return s["out"]
    api.mdw_linear_state_advance(s["state"], s["k"], s["v"], s["decay"], s["start"], s["accepted"], s["slot_in"], s["slot_out"], c["new_hi"])
    return s["pool"]


def run(s):
    if own:
        return _own(s)
    return {"lin": _plain_lin, "tree": _plain_tree, "advance": _plain_advance, "norm": _plain_norm}[s["case"]["op"]](s)


# ------------------------------------------------------------------------------------ 64 bits


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm":
        y = s["y"].double()
        if c["post"]:
            parts = y.split(c["group"] or c["w"], dim=1)
            y = torch.cat([p / torch.sqrt((p * p).sum(1, keepdim=True) / p.shape[1] + 1e-6) * s["post"].double() for p in parts], 1)
        if c["gate"] != "none":
            a = s["gate"].double()
            y = y * {"mul": lambda: a, "sigmoid": lambda: torch.sigmoid(a), "silu": lambda: a * torch.sigmoid(a)}[c["gate"]]()
        r = 0.5 * y + (0.75 * s["r"].double() if c["res"] != "none" else 0.0)
        if not c["pre"]:
            return r
        # the norm before the next sub-layer is of the residual as it is stored
        x = r.to(s["sum"].dtype).double()
        return [r, x / torch.sqrt((x * x).sum(1, keepdim=True) / c["w"] + 1e-6) * s["pre"].double()]
    n, start = _lengths(c), np.concatenate([[0], np.cumsum(_lengths(c))])
    share, scale = c["h"] // c["hqk"], c["d"] ** -0.5
    dev = "cuda"

    def step(state, row):
        """The states of some requests after one row of each."""
        k = s["k"][row].double().repeat_interleave(share, 1)
        g = s["decay"][row].double() if c["steps"] else s["decay"].double()
        return state * torch.exp(g)[..., None, None] + k[..., :, None] * s["v"][row].double()[..., None, :]

    def read(state, row):
        q = s["q"][row].double().repeat_interleave(share, 1)
        return torch.einsum("bhi,bhij->bhj", q, state) * scale

    slots = s["slot_in"].cpu().numpy()
    state = torch.stack([s["pool"][i].double() if i >= 0 else torch.zeros_like(s["pool"][0], dtype=torch.float64) for i in slots])
    if c["op"] == "lin":
        out = torch.empty(s["out"].shape, dtype=torch.float64, device=dev)
        order = np.argsort(-n, kind="stable")               # long requests first: those still going are the first ones
        state = state[torch.from_numpy(order).to(dev)]
        begin = torch.from_numpy(start[:-1][order]).to(dev)
        for t in range(int(n.max())):
            live = int((n > t).sum())
            row = begin[:live] + t
            state[:live] = step(state[:live], row)
            out[row] = read(state[:live], row)
        pool = s["pool"].double()
        pool[s["slot_out"].long()[torch.from_numpy(order).to(dev)]] = state
        return [out, pool]
    if c["op"] == "tree":
        out = torch.empty(s["out"].shape, dtype=torch.float64, device=dev)
        mask = s["mask"].cpu().numpy().view(np.uint64)
        for b in range(c["b"]):
            after = []
            for i in range(int(n[b])):
                above = int(mask[start[b] + i]) & ((1 << i) - 1)
                row = torch.tensor([int(start[b]) + i], device=dev)
                after.append(step(after[above.bit_length() - 1] if above else state[b:b + 1], row))
                out[row] = read(after[-1], row)
        return out
    pool = s["pool"].double()
    accepted = s["accepted"].cpu().numpy().view(np.uint64)
    for b in range(c["b"]):
        now = state[b:b + 1]
        for i in range(int(n[b])):
            if int(accepted[b]) >> i & 1:
                now = step(now, torch.tensor([int(start[b]) + i], device=dev))
        pool[int(s["slot_out"][b])] = now[0]
    return pool


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(case, work(case))
