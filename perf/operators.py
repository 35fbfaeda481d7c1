"""The operators of a verify window's attention sub-layer, in plain form and as the library's calls.

Around the decode step's MoE layers and LM head a serving program runs, for every window of
drafted tokens:

* ``w4_linear``          -- the dense projections, int4 weights with group scales (q/k/v, output);
* ``mdw_kv_plan``        -- block tables, slot map, positions and tree masks from request lengths;
* ``mdw_kv_write``       -- the window's keys and values into the paged cache (16-bit or E4M3);
* ``mdw_tree_attention`` -- attention of a tree of drafted tokens over that cache.

``run`` computes them with elementary torch operations in 32 bits (``own`` false) or by the
library's entry points (``own`` true); ``exact`` gives the definition in 64 bits.
"""

import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3_MAX = 448.0


def listed():
    return [
        # the fused q/k/v projection of one decoded token: the smallest call of a layer
        {"name": "w4_qkv_m1", "op": "w4", "m": 1, "n": 3584, "k": 2560, "group": 128, "zero": False,
         "x": "bf16", "y": "bf16", "bias": True, "residual": False},
        # the output projection of a 4-token verify window, zero points, residual added
        {"name": "w4_out_m4", "op": "w4", "m": 4, "n": 2560, "k": 2560, "group": 64, "zero": True,
         "x": "f16", "y": "f16", "bias": False, "residual": True},
        # the widest window, an odd number of rows, the finest groups
        {"name": "w4_odd_m32", "op": "w4", "m": 32, "n": 10007, "k": 5120, "group": 32, "zero": True,
         "x": "bf16", "y": "bf16", "bias": False, "residual": False},
        # a 4-bit vocabulary projection of one token, fp32 logits
        {"name": "w4_vocab_m1", "op": "w4", "m": 1, "n": 157184, "k": 2560, "group": 128, "zero": False,
         "x": "bf16", "y": "f32", "bias": False, "residual": False},
        # trees of up to 16 drafted tokens for a batch of requests, padded to the captured size
        {"name": "plan_trees", "op": "plan", "b": 64, "ctx_lo": 0, "ctx_hi": 8000, "new_lo": 1, "new_hi": 16,
         "page": 16, "tree": True, "pad": 37},
        # admission of a batch of prompts
        {"name": "plan_prompts", "op": "plan", "b": 199, "ctx_lo": 0, "ctx_hi": 1000, "new_lo": 0, "new_hi": 4096,
         "page": 64, "tree": False, "pad": 0},
        # one window's keys and values
        {"name": "write_window", "op": "write", "t": 32, "hkv": 8, "d": 128, "page": 16, "x": "bf16", "cache": "bf16",
         "pages": 300, "pad": 3},
        # a prompt chunk into an E4M3 cache
        {"name": "write_prompt_e4m3", "op": "write", "t": 16381, "hkv": 8, "d": 128, "page": 64, "x": "bf16",
         "cache": "e4m3", "pages": 300, "pad": 0},
        # one request, a chain of 4 drafted tokens, odd group of 5 query heads per kv head
        {"name": "attn_window", "op": "attn", "b": 1, "hq": 20, "hkv": 4, "d": 128, "ctx_lo": 1500, "ctx_hi": 1500,
         "new_lo": 4, "new_hi": 4, "page": 16, "x": "bf16", "cache": "bf16"},
        # a ragged batch with trees
        {"name": "attn_trees", "op": "attn", "b": 16, "hq": 32, "hkv": 8, "d": 128, "ctx_lo": 300, "ctx_hi": 12000,
         "new_lo": 1, "new_hi": 16, "page": 32, "x": "bf16", "cache": "bf16"},
        # one very long request, one token, E4M3 cache
        {"name": "attn_long_e4m3", "op": "attn", "b": 1, "hq": 64, "hkv": 8, "d": 128, "ctx_lo": 131001,
         "ctx_hi": 131001, "new_lo": 1, "new_hi": 1, "page": 64, "x": "bf16", "cache": "e4m3"},
        # the largest trees: 64 nodes, heads of 64
        {"name": "attn_wide_trees", "op": "attn", "b": 6, "hq": 32, "hkv": 4, "d": 64, "ctx_lo": 1000, "ctx_hi": 9000,
         "new_lo": 64, "new_hi": 64, "page": 128, "x": "f16", "cache": "f16"},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["w4", "w4", "plan", "write", "attn", "attn", "attn"])
    x = rng.choice(["bf16", "f16"])
    if op == "w4":
        group = rng.choice([32, 64, 128])
        k = group * _log(rng, 4 * 128 // group, 16384 // group)
        n = _log(rng, 100, min(157184, 300_000_000 // k))
        return {"op": op, "m": _log(rng, 1, 32), "n": n, "k": k, "group": group, "zero": rng.random() < 0.5, "x": x,
                "y": rng.choice([x, "f32"]), "bias": rng.random() < 0.3, "residual": rng.random() < 0.3}
    if op == "plan":
        tree = rng.random() < 0.5
        b = _log(rng, 1, 512)
        new_hi = _log(rng, 1, 64 if tree else min(4096, 400000 // b))
        ctx_hi = _log(rng, 1, 20000)
        return {"op": op, "b": b, "ctx_lo": rng.randint(0, ctx_hi), "ctx_hi": ctx_hi, "new_lo": rng.randint(0 if b > 1 else 1, 1),
                "new_hi": new_hi, "page": rng.choice([16, 32, 64, 128]), "tree": tree, "pad": rng.randint(0, 50)}
    hkv, d = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128])
    cache = rng.choice([x, x, "e4m3"])
    if op == "write":
        t = _log(rng, 1, min(16384, 16384 * 8 * 128 // (hkv * d)))
        page = rng.choice([16, 32, 64, 128])
        return {"op": op, "t": t, "hkv": hkv, "d": d, "page": page, "x": x, "cache": cache,
                "pages": -(-t // page) + rng.randint(1, 200), "pad": rng.randint(0, 9)}
    b = _log(rng, 1, 48)
    new_hi = _log(rng, 1, 64)
    group = min(rng.randint(1, 16), max(1, 512 // new_hi))
    most = min(131072, 131072 * 8 * 128 // (b * hkv * d), 16_000_000_000 // (4 * b * hkv * group * new_hi * d))
    ctx_hi = _log(rng, 16, max(16, most))
    return {"op": op, "b": b, "hq": hkv * group, "hkv": hkv, "d": d, "ctx_lo": rng.randint(0, ctx_hi), "ctx_hi": ctx_hi,
            "new_lo": rng.randint(1, new_hi), "new_hi": new_hi, "page": rng.choice([16, 32, 64, 128]), "x": x, "cache": cache}


def _spread(count, lo, hi, step):
    """`count` whole numbers spread over [lo, hi], the last of them hi: the case's lengths."""
    v = [lo + int((hi - lo) * ((i + 1) * step % 1.0)) for i in range(count)]
    v[-1] = hi
    return np.array(v, dtype=np.int64)


def _lengths(c):
    return _spread(c["b"], c["ctx_lo"], c["ctx_hi"], 0.6180339887), _spread(c["b"], c["new_lo"], c["new_hi"], 0.7548776662)


def _pages(tokens, page):
    return -(-tokens // page)


def work(c):
    if c["op"] == "w4":
        groups = c["n"] * (c["k"] // c["group"])
        xb, yb = 2, 4 if c["y"] == "f32" else 2
        byts = c["n"] * c["k"] // 2 + groups * (3 if c["zero"] else 2) + c["m"] * (c["k"] * xb + c["n"] * yb)
        byts += c["n"] * 2 if c["bias"] else 0
        byts += c["m"] * c["n"] * 2 if c["residual"] else 0
        return {"bytes": byts, "flops": 2.0 * c["m"] * c["n"] * c["k"]}
    if c["op"] == "plan":
        ctx, new = _lengths(c)
        t, taken = int(new.sum()), int((_pages(ctx + new, c["page"]) - _pages(ctx, c["page"])).sum())
        # lengths read, row starts written; slot and position of every row; pages read and written; trees
        return {"bytes": c["b"] * 12 + (t + c["pad"]) * 12 + taken * 8 + ((t + c["pad"]) * 8 + t * 4 if c["tree"] else 0), "flops": 0}
    if c["op"] == "write":
        e = 1 if c["cache"] == "e4m3" else 2
        return {"bytes": c["t"] * c["hkv"] * c["d"] * 2 * (2 + e) + (c["t"] + c["pad"]) * 8, "flops": 0}
    ctx, new = _lengths(c)
    e = 1 if c["cache"] == "e4m3" else 2
    keys, rows = int((ctx + new).sum()), int(new.sum())
    byts = keys * c["hkv"] * c["d"] * 2 * e + rows * c["hq"] * (c["d"] * 4 + 4) + rows * 8 + int(_pages(ctx + new, c["page"]).sum()) * 4
    return {"bytes": byts, "flops": 4.0 * c["hq"] * c["d"] * float((new * (ctx + (new + 1) / 2)).sum())}


# ------------------------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _int(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _trees(rs, new):
    """Parents of every request's drafted tokens: node 0 is the root, later ones hang on one of the four before."""
    out = []
    for n in new:
        i = np.arange(n)
        out.append(np.maximum(i - 1 - rs.randint(0, 4, n), np.where(i > 0, 0, -1)))
    return np.concatenate(out) if out else np.zeros(0, dtype=np.int64)


def _masks(parents, new):
    """Bit j of a node's mask: node j is the node itself or an ancestor."""
    out, at = [], 0
    for n in new:
        m = []
        for i in range(n):
            p = int(parents[at + i])
            m.append((m[p] if p >= 0 else 0) | 1 << i)
        out += m
        at += n
    return np.array(out, dtype=np.uint64).view(np.int64)


def _cache(g, c, pages):
    shape = (pages, c["hkv"], c["page"], c["d"])
    if c["cache"] == "e4m3":
        k, v = (_normal(g, shape, torch.float32, 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = ((torch.rand(c["hkv"], generator=g, device="cuda") + 0.5) / 100.0 for _ in range(2))
        return k, v, ks, vs
    return _normal(g, shape, DT[c["cache"]]), _normal(g, shape, DT[c["cache"]]), None, None


def prepare(c, seed):
    g, rs = _gen(seed), np.random.RandomState(int(seed) % (1 << 31))
    s = {"case": c}
    if c["op"] == "w4":
        m, n, k, ng = c["m"], c["n"], c["k"], c["k"] // c["group"]
        # codes of normally distributed weights, two to a byte, the even one in the low nibble
        q = torch.empty((n, k // 2), dtype=torch.uint8, device="cuda")
        for a in range(0, n, 16384):
            code = (torch.randn((min(16384, n - a), k), generator=g, device="cuda") * 2.7 + 8).round_().clamp_(0, 15).to(torch.uint8)
            q[a:a + 16384] = code[:, 0::2] | code[:, 1::2] << 4
        s["q"] = q
        s["scale"] = ((torch.rand((n, ng), generator=g, device="cuda") + 0.5) * 0.02).to(DT[c["x"]])
        s["zero"] = torch.randint(5, 12, (n, ng), generator=g, device="cuda", dtype=torch.uint8) if c["zero"] else None
        s["x"] = _normal(g, (m, k), DT[c["x"]])
        s["bias"] = _normal(g, (n,), DT[c["x"]]) if c["bias"] else None
        s["residual"] = _normal(g, (m, n), DT[c["x"]]) if c["residual"] else None
        s["y"] = torch.empty((m, n), dtype=DT[c["y"]], device="cuda")
        if own:  # the weight handle a program keeps: the same tensors, no copy
            from moe_decode_weight_gb300 import api
            s["w"] = api.W4Weights(s["q"], s["scale"], s["zero"])
        return s
    if c["op"] == "plan":
        ctx, new = _lengths(c)
        have, need = _pages(ctx, c["page"]), _pages(ctx + new, c["page"])
        t, width = int(new.sum()) + c["pad"], int(need.max()) + 3
        pool = rs.permutation(int(need.sum()) + 5)
        table = np.full((c["b"], width), -1, dtype=np.int64)
        at = 0
        for b in range(c["b"]):
            table[b, :have[b]] = pool[at:at + have[b]]
            at += have[b]
        s.update(ctx=_int(ctx), new=_int(new), table=_int(table), free=_int(pool[at:]), num_pages=len(pool),
                 slot=torch.empty(t, dtype=torch.int64, device="cuda"), pos=torch.empty(t, dtype=torch.int32, device="cuda"),
                 start=torch.empty(c["b"] + 1, dtype=torch.int32, device="cuda"),
                 taken=torch.empty(1, dtype=torch.int32, device="cuda"), parents=None, mask=None)
        if c["tree"]:
            s["parents"] = _int(np.concatenate([_trees(rs, new), np.zeros(c["pad"], dtype=np.int64)]))
            s["mask"] = torch.empty(t, dtype=torch.int64, device="cuda")
        return s
    if c["op"] == "write":
        t = c["t"] + c["pad"]
        s["kc"], s["vc"], s["ks"], s["vs"] = _cache(g, c, c["pages"])
        # keys and values as slices of a fused projection's rows
        qkv = _normal(g, (t, 2 * c["hkv"] * c["d"] + 64), DT[c["x"]])
        s["k"] = qkv[:, 64:64 + c["hkv"] * c["d"]].unflatten(1, (c["hkv"], c["d"]))
        s["v"] = qkv[:, 64 + c["hkv"] * c["d"]:].unflatten(1, (c["hkv"], c["d"]))
        slots = (rs.permutation(c["pages"])[:, None] * c["page"] + np.arange(c["page"])).reshape(-1)[:c["t"]]
        s["slot"] = _int(np.concatenate([slots, np.full(c["pad"], -1)]), torch.int64)
    else:
        ctx, new = _lengths(c)
        need = _pages(ctx + new, c["page"])
        t, pages = int(new.sum()), int(need.sum()) + 3
        s["kc"], s["vc"], s["ks"], s["vs"] = _cache(g, c, pages)
        s["qt"] = _normal(g, (t, c["hq"], c["d"]), DT[c["x"]])
        table = np.full((c["b"], int(need.max())), -1, dtype=np.int64)
        pool, at = rs.permutation(pages), 0
        for b in range(c["b"]):
            table[b, :need[b]] = pool[at:at + need[b]]
            at += need[b]
        parents = _trees(rs, new)
        s.update(table=_int(table), ctx=_int(ctx), start=_int(np.concatenate([[0], np.cumsum(new)])),
                 mask=_int(_masks(parents, new), torch.int64), out=torch.empty_like(s["qt"]),
                 lse=torch.empty((t, c["hq"]), dtype=torch.float32, device="cuda"))
    if own:  # the cache handle and the workspace a program keeps
        from moe_decode_weight_gb300 import api
        s["cache"] = api.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
        if c["op"] == "attn":
            nbytes = api.mdw_tree_attention_workspace_bytes(s["cache"], c["b"], t, c["hq"], c["new_hi"])
            s["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------ plain forms


def _plain_w4(s):
    c = s["case"]
    n, ng = c["n"], c["k"] // c["group"]
    code = torch.stack((s["q"] & 15, s["q"] >> 4), dim=2).view(n, ng, c["group"]).float()
    zero = s["zero"].float().unsqueeze(2) if c["zero"] else 8.0
    w = ((code - zero) * s["scale"].float().unsqueeze(2)).view(n, c["k"])
    y = s["x"].float() @ w.t()
    if c["bias"]:
        y = y + s["bias"].float()
    if c["residual"]:
        y = y + s["residual"].float()
    return y.to(DT[c["y"]])


def _plain_plan(s):
    c, dev = s["case"], s["ctx"].device
    page, b, t, width = c["page"], c["b"], s["slot"].numel(), s["table"].shape[1]
    ctx, new = s["ctx"].long(), s["new"].long()
    have, need = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    take = need - have
    first = torch.cumsum(take, 0) - take
    col = torch.arange(width, device=dev)
    fresh = (col >= have[:, None]) & (col < need[:, None])
    at = (first[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    start = torch.cat((new.new_zeros(1), torch.cumsum(new, 0)))
    row = torch.arange(t, device=dev)
    req = torch.searchsorted(start[1:], row, right=True).clamp(max=b - 1)
    node = row - start[req]
    valid = row < start[b]
    place = torch.where(valid, ctx[req] + node, 0)
    slot = torch.where(valid, table[req, place // page].long() * page + place % page, -1)
    out = [table, start.int(), slot, take.sum().int().view(1)]
    if not c["tree"]:
        return [*out, torch.where(valid, place, -1).int()]
    # ancestors of every node: reach[i, j], squared until it covers the deepest tree
    size = c["new_hi"]
    grid = start[:b, None] + torch.arange(size, device=dev)
    parent = torch.where(torch.arange(size, device=dev) < new[:, None], s["parents"][grid.clamp(max=t - 1)].long(), -1)
    reach = (parent[:, :, None] == torch.arange(size, device=dev)).float() + torch.eye(size, device=dev)
    for _ in range(max(1, (size - 1).bit_length())):
        reach = (reach @ reach > 0).float()
    bits = (reach.long() << torch.arange(size, device=dev)).sum(2)
    depth = reach.sum(2).long() - 1
    node = node.clamp(0, size - 1)
    return [*out, torch.where(valid, ctx[req] + depth[req, node], -1).int(), torch.where(valid, bits[req, node], 0)]


def _plain_write(s):
    c = s["case"]
    at = (s["slot"] >= 0).nonzero().squeeze(1)
    slot = s["slot"][at]
    for rows, cache, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        v = rows[at]
        if scale is not None:
            v = (v.float() / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
            cache = cache.view(torch.uint8)
        cache.permute(0, 2, 1, 3)[slot // c["page"], slot % c["page"]] = v
    return [s["kc"], s["vc"]]


def _plain_attn(s):
    c, dev = s["case"], s["qt"].device
    b, hkv, d, group, size = c["b"], c["hkv"], c["d"], c["hq"] // c["hkv"], c["new_hi"]
    width = s["table"].shape[1] * c["page"]
    table = s["table"].long().clamp(min=0)
    ctx, start = s["ctx"].long(), s["start"].long()
    new = start[1:] - start[:-1]
    k, v = (x[table].float().transpose(1, 2).reshape(b, hkv, width, d) for x in (s["kc"], s["vc"]))
    if s["ks"] is not None:
        k, v = k * s["ks"][:, None, None], v * s["vs"][:, None, None]
    node = torch.arange(size, device=dev)
    row = (start[:b, None] + node).clamp(max=s["qt"].shape[0] - 1)
    q = s["qt"].float()[row].view(b, size, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, size * group, d)
    score = (q @ k.transpose(2, 3)).view(b, hkv, size, group, width) / math.sqrt(d)
    key = torch.arange(width, device=dev) - ctx[:, None]
    bit = (s["mask"][row][:, :, None] >> key.clamp(0, 63)[:, None, :]) & 1
    seen = (key < 0)[:, None, :] | ((bit == 1) & (key < new[:, None])[:, None, :])
    score = torch.where(seen[:, None, :, None, :], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = (p / torch.where(total > 0, total, 1.0)).view(b, hkv, size * group, width) @ v
    o = o.view(b, hkv, size, group, d).permute(0, 2, 1, 3, 4).reshape(b, size, c["hq"], d)
    lse = (top + torch.log(total)).view(b, hkv, size, group).permute(0, 2, 1, 3).reshape(b, size, c["hq"])
    r = torch.arange(s["qt"].shape[0], device=dev)
    req = torch.searchsorted(start[1:], r, right=True)
    return [o[req, r - start[req]].to(s["qt"].dtype), lse[req, r - start[req]]]


# ------------------------------------------------------------------------------------ the calls


def _own(s):
    from moe_decode_weight_gb300 import api
    c = s["case"]
    if c["op"] == "w4":
        api.w4_linear(s["w"], s["x"], s["y"], bias=s["bias"], residual=s["residual"])
        return s["y"]
    if c["op"] == "plan":
        api.mdw_kv_plan(s["ctx"], s["new"], c["page"], s["num_pages"], s["table"], s["free"], s["start"], s["slot"],
                        s["pos"], s["taken"], parents=s["parents"], tree_mask=s["mask"])
        out = [s["table"], s["start"], s["slot"], s["taken"], s["pos"]]
        return out + [s["mask"]] if c["tree"] else out
    if c["op"] == "write":
        api.mdw_kv_write(s["cache"], s["k"], s["v"], s["slot"])
        return [s["kc"], s["vc"]]
    api.mdw_tree_attention(s["cache"], s["qt"], s["out"], s["table"], s["ctx"], s["start"], c["new_hi"], s["ws"],
                           tree_mask=s["mask"], lse=s["lse"])
    return [s["out"], s["lse"]]


def run(s):
    if own:
        return _own(s)
    return {"w4": _plain_w4, "plan": _plain_plan, "write": _plain_write, "attn": _plain_attn}[s["case"]["op"]](s)


# ------------------------------------------------------------------------------------ 64 bits


def exact(c, seed):
    if c["op"] == "plan":
        return None  # whole numbers only
    s = prepare(c, seed)
    if c["op"] == "w4":
        x, ng = s["x"].double(), c["k"] // c["group"]
        out = torch.empty((c["m"], c["n"]), dtype=torch.float64, device="cuda")
        for a in range(0, c["n"], 8192):
            q = s["q"][a:a + 8192]
            w = torch.empty((q.shape[0], c["k"]), dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = q % 16, q // 16
            w = w.view(-1, ng, c["group"])
            w -= s["zero"][a:a + 8192].double()[:, :, None] if c["zero"] else 8.0
            w *= s["scale"][a:a + 8192].double()[:, :, None]
            out[:, a:a + 8192] = (w.view(-1, c["k"]) @ x.t()).t()
        for extra in (s["bias"], s["residual"]):
            if extra is not None:
                out += extra.double()
        return out
    if c["op"] == "write":
        out = []
        live = s["slot"][:c["t"]]
        for rows, cache, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
            v = rows[:c["t"]].double()
            if scale is not None:
                v = torch.clamp(v / scale.double()[:, None], -E4M3_MAX, E4M3_MAX)
            flat = cache.to(torch.float64).transpose(1, 2).reshape(-1, c["hkv"], c["d"])
            flat[live] = v
            out.append(flat.view(c["pages"], c["page"], c["hkv"], c["d"]).transpose(1, 2).contiguous())
        return out
    ctx, new = _lengths(c)
    out = torch.empty(s["qt"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    group, at = c["hq"] // c["hkv"], 0
    mask = s["mask"].cpu().numpy()
    for b in range(c["b"]):
        n, keys = int(new[b]), int(ctx[b] + new[b])
        pages = s["table"][b, :_pages(keys, c["page"])].long()
        bits = np.array([[int(mask[at + i]) >> j & 1 for j in range(n)] for i in range(n)], dtype=bool).reshape(n, n)
        seen = torch.ones((n, keys), dtype=torch.bool, device="cuda")
        seen[:, int(ctx[b]):] = torch.from_numpy(bits).cuda()
        for h in range(c["hkv"]):
            k, v = (x[pages, h].to(torch.float64).reshape(-1, c["d"])[:keys] for x in (s["kc"], s["vc"]))
            if s["ks"] is not None:
                k, v = k * s["ks"][h].double(), v * s["vs"][h].double()
            q = s["qt"][at:at + n, h * group:(h + 1) * group].double()
            z = torch.einsum("ngd,kd->ngk", q, k) * (c["d"] ** -0.5)
            z = z.masked_fill(~seen[:, None, :], -math.inf)
            norm = torch.logsumexp(z, -1)
            out[at:at + n, h * group:(h + 1) * group] = torch.einsum("ngk,kd->ngd", torch.exp(z - norm[:, :, None]), v)
            lse[at:at + n, h * group:(h + 1) * group] = norm
        at += n
    return [out, lse]


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(case, work(case))
