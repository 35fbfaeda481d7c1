"""GPU parity of the attention sub-layer (int4 projection, cache plan, cache writer, tree attention)
against the float64 oracle.

Tolerances, derived from the arithmetic the entry points promise:
* a rounding to type t is off by at most eps(t) / 2 relative to the value;
* fp32 sums of the tensor cores or of warps: each of at most c chained additions is off by 2^-23 of
  the partial sum, which sum |term| bounds, so a dot product is off by c 2^-23 sum |term|;
* a probability off by the relative error r, or rounded to type p, moves an output by at most
  (r + eps(p) / 2) sum_j p_j |v_j|, twice that where the sum of probabilities moves too.
"""

import numpy as np
import pytest
import torch

from moe_decode_weight_gb300 import api
from oracle import attention as OA
from oracle import formats as OF

pytestmark = pytest.mark.gpu
BF, HF, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def host(t):
    return t.detach().to(torch.float64).cpu().numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------------------ w4_linear


def w4_case(seed, n, k, group, zero, dtype):
    g = gen(seed)
    q = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = ((torch.rand((n, k // group), generator=g, device="cuda") + 0.5) * 0.02).to(dtype)
    z = torch.randint(0, 16, (n, k // group), generator=g, device="cuda", dtype=torch.uint8) if zero else None
    return api.W4Weights(q, scale, z)


def w4_want(w, x, bias=None, residual=None):
    """The oracle's y and the bound of an fp32 sum in k / 16 + 64 chained steps (at most 16 products enter the
    tensor core's sum at once; groups, warps and blocks add at most 64 more)."""
    group = w.c.group
    args = (w.q.cpu().numpy(), host(w.scale), None if w.zero is None else w.zero.cpu().numpy(), group)
    extra = dict(bias=None if bias is None else host(bias), residual=None if residual is None else host(residual))
    y = OA.w4_linear(*args, host(x), **extra)
    size = np.abs(host(x)) @ np.abs(OA.w4_weight(*args)).T
    for e in extra.values():
        size = size if e is None else size + np.abs(e)
    steps = w.c.k / 16 + w.c.k / group + 64
    return y, steps * 2.0 ** -23 * size


def assert_close(got, want, tol, what=""):
    got, bad = np.asarray(got, np.float64), None
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], np.asarray(want)[bad][:4])


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 32])
@pytest.mark.parametrize("n,k,group,zero,dtype,ydtype", [
    (257, 2560, 128, False, BF, BF), (64, 2560, 64, True, HF, HF), (33, 1280, 32, True, BF, F32), (1, 128, 128, False, HF, F32)])
def test_w4_linear(m, n, k, group, zero, dtype, ydtype):
    w = w4_case(m * n, n, k, group, zero, dtype)
    x = torch.randn((m, k), generator=gen(m), device="cuda").to(dtype)
    y = torch.full((m, n), float("nan"), dtype=ydtype, device="cuda")
    api.w4_linear(w, x, y)
    want, tol = w4_want(w, x)
    assert_close(host(y), want, tol + half_step(ydtype) * np.abs(want))


@pytest.mark.parametrize("n,k,group", [(17, 32, 32), (1, 32, 32), (15, 96, 32), (16, 64, 64), (100, 192, 64), (48, 384, 128),
                                       (31, 16384, 32), (2049, 640, 128), (10007, 512, 64), (7, 9984, 128),
                                       (300, 2592, 32), (50, 2624, 64), (5000, 1024, 32)])
@pytest.mark.parametrize("m", [1, 6, 32])
def test_w4_linear_shapes(m, n, k, group):
    w = w4_case(n + k, n, k, group, n % 2 == 1, BF if k % 3 else HF)
    x = torch.randn((m, k), generator=gen(m), device="cuda").to(w.scale.dtype)
    y = torch.empty((m, n), dtype=F32, device="cuda")
    api.w4_linear(w, x, y)
    want, tol = w4_want(w, x)
    assert_close(host(y), want, tol + half_step(F32) * np.abs(want))


@pytest.mark.parametrize("m", [1, 4, 19])
def test_w4_linear_strides_bias_and_residual_in_place(m):
    n, k = 203, 768
    w = w4_case(5, n, k, 64, True, BF)
    x = torch.randn((m, k + 40), generator=gen(m), device="cuda").to(BF)[:, 24:24 + k]
    bias = torch.randn(n + 1, generator=gen(2), device="cuda").to(BF)[1:]
    full = torch.randn((m, n + 5), generator=gen(3), device="cuda").to(BF)
    y = full[:, 3:3 + n]
    before = full.clone()
    api.w4_linear(w, x, y, bias=bias, residual=y)
    want, tol = w4_want(w, x, bias, before[:, 3:3 + n])
    assert_close(host(y), want, tol + half_step(BF) * np.abs(want))
    assert torch.equal(full[:, :3], before[:, :3]) and torch.equal(full[:, 3 + n:], before[:, 3 + n:])


def test_w4_linear_stays_in_its_rows_and_repeats_bit_for_bit():
    """Features behind the last and tokens behind the window are not written; two calls give the same bits."""
    for m, n in ((3, 37), (32, 1003)):
        w = w4_case(6, n, 1024, 128, False, BF)
        x = torch.randn((m, 1024), generator=gen(m), device="cuda").to(BF)
        buf = torch.full((m + 2, n + 9), 7.0, dtype=F32, device="cuda")
        api.w4_linear(w, x, buf[:m, :n])
        assert (buf[m:] == 7).all() and (buf[:, n:] == 7).all()
        again = torch.empty((m, n), dtype=F32, device="cuda")
        api.w4_linear(w, x, again)
        assert torch.equal(buf[:m, :n], again)


def test_w4_linear_nonfinite_input_stays_in_its_token():
    w = w4_case(8, 130, 256, 32, True, BF)
    x = torch.randn((9, 256), generator=gen(1), device="cuda").to(BF)
    x[4, 100] = float("inf")
    y = torch.empty((9, 130), dtype=F32, device="cuda")
    api.w4_linear(w, x, y)
    keep = [i for i in range(9) if i != 4]
    want, tol = w4_want(w, x[keep])
    assert_close(host(y[keep]), want, tol + half_step(F32) * np.abs(want))
    assert not torch.isfinite(y[4]).any()


def test_w4_linear_large_window_of_rows():
    """Row offsets of q beyond 2^31 bytes: the last rows of a 2.2 GB weight."""
    n, k = 135_000, 32768
    q = torch.zeros((n, k // 2), dtype=torch.uint8, device="cuda")
    scale = torch.ones((n, k // 128), dtype=BF, device="cuda")
    tail = w4_case(3, 40, k, 128, False, BF)
    q[-40:], scale[-40:] = tail.q, tail.scale
    x = torch.randn((2, k), generator=gen(4), device="cuda").to(BF)
    y = torch.empty((2, n), dtype=F32, device="cuda")
    api.w4_linear(api.W4Weights(q, scale), x, y)
    want, tol = w4_want(tail, x)
    assert_close(host(y[:, -40:]), want, tol + half_step(F32) * np.abs(want))


# ---------------------------------------------------------------------------- mdw_kv_plan


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def plan_call(ctx, new, page, num_pages, table, free, t, parents=None, mask=True):
    out = dict(table=i32(table), start=i32(np.full(len(ctx) + 1, -7)), slot=torch.full((t,), -7, dtype=torch.int64, device="cuda"),
               pos=i32(np.full(t, -7)), mask=torch.full((t,), -7, dtype=torch.int64, device="cuda") if mask else None, taken=i32([-7]),
               status=i32([0]))
    api.mdw_kv_plan(i32(ctx), i32(new), page, num_pages, out["table"], i32(free), out["start"], out["slot"], out["pos"], out["taken"],
                    parents=None if parents is None else i32(parents), tree_mask=out["mask"], status=out["status"])
    return {k: None if v is None else v.cpu().numpy() for k, v in out.items()}


def random_plan(seed, b, page, ctx_hi, new_hi, tree, pad):
    rng = np.random.default_rng(seed)
    ctx, new = rng.integers(0, ctx_hi + 1, b), rng.integers(0, new_hi + 1, b)
    have, need = -(-ctx // page), -(-(ctx + new) // page)
    pool = rng.permutation(int(need.sum()) + 4)
    table = np.full((b, int(need.max()) + 2), -5)
    at = 0
    for i in range(b):
        table[i, :have[i]] = pool[at:at + have[i]]
        at += have[i]
    t = int(new.sum()) + pad
    parents = None
    if tree:
        parents = np.concatenate([rng.integers(-1, np.arange(n)) if n else np.zeros(0, int) for n in new] + [np.full(pad, -9)])
    return ctx, new, page, len(pool), table, pool[at:], max(t, 1), parents


@pytest.mark.parametrize("b,page,ctx_hi,new_hi,tree,pad", [
    (1, 16, 0, 1, False, 0), (1, 16, 1000, 64, True, 3), (3, 32, 40, 4, False, 5), (64, 16, 300, 16, True, 11), (257, 64, 5, 1, False, 1),
    (300, 16, 200, 64, True, 0), (4096, 16, 60, 3, True, 100), (17, 256, 3000, 5000, False, 7), (1500, 128, 0, 300, False, 0)])
def test_plan(b, page, ctx_hi, new_hi, tree, pad):
    args = random_plan(b, b, page, ctx_hi, new_hi, tree, pad)
    mask = new_hi <= 64
    want, got = OA.kv_plan(*args, with_mask=mask), plan_call(*args, mask=mask)
    assert not want["fail"] and not want["bad"] and got["status"][0] == 0
    for key in ("table", "start", "slot", "pos"):
        assert np.array_equal(got[key], want[key]), key
    assert got["taken"][0] == want["taken"]
    if mask:
        assert np.array_equal(got["mask"].view(np.uint64), want["mask"])


@pytest.mark.parametrize("ctx,new,free,t", [
    ([31, 0], [2, 1], [3, 4], 5), ([-1, 0], [1, 1], [3, 4], 5), ([0, 0], [1, -1], [3, 4], 5), ([0, 16], [1, 1], [3], 5),
    ([0, 0], [3, 3], [3, 4], 5), ([0, 2147483647], [1, 2147483647], [3, 4], 5)])
def test_plan_that_fails_whole(ctx, new, free, t):
    table = [[0, 1], [2, 5]]
    assert OA.kv_plan(ctx, new, 16, 9, table, free, t)["fail"]
    got = plan_call(ctx, new, 16, 9, table, free, t)
    assert got["status"][0] == 7 and np.array_equal(got["table"], table) and not got["start"].any() and got["taken"][0] == 0
    assert (got["slot"] == -1).all() and (got["pos"] == -1).all() and not got["mask"].any()


def test_plan_with_trees_too_large():
    got = plan_call([0], [65], 16, 9, [[-1] * 5], [0, 1, 2, 3, 4], 70)
    assert got["status"][0] == 7 and not got["start"].any()
    got = plan_call([0], [65], 16, 9, [[-1] * 5], [0, 1, 2, 3, 4], 70, mask=False)
    assert got["status"][0] == 0 and got["start"].tolist() == [0, 65]


@pytest.mark.parametrize("table,free,parents", [
    ([[9, -1, -1], [2, -1, -1]], [3, 4, 5], None), ([[0, -1, -1], [2, -1, -1]], [3, -4, 5], None),
    ([[0, -1, -1], [2, -1, -1]], [3, 4, 5], [-1, 0, 2, 2, -1, 0, 1, 1]), ([[0, -1, -1], [2, -1, -1]], [3, 4, 5], [-1, 0, -2, 2, -1, 3, 0, 1])])
def test_plan_with_bad_pages_or_parents(table, free, parents):
    args = ([15, 14], [4, 4], 16, 9, table, free, 8, parents)
    want, got = OA.kv_plan(*args), plan_call(*args)
    assert want["bad"] and got["status"][0] == 7
    for key in ("table", "start", "slot", "pos"):
        assert np.array_equal(got[key], want[key]), key
    assert np.array_equal(got["mask"].view(np.uint64), want["mask"])


# --------------------------------------------------------------------------- mdw_kv_write


def make_cache(seed, pages, hkv, page, d, ctype, fill=None):
    g = gen(seed)
    shape = (pages, hkv, page, d)
    if ctype == E4:
        k, v = ((torch.randn(shape, generator=g, device="cuda") * 100).clamp_(-448, 448).to(E4) for _ in range(2))
        ks, vs = ((torch.rand(hkv, generator=g, device="cuda") + 0.5) / 100 for _ in range(2))
        return api.KVCache(k, v, ks, vs)
    return api.KVCache(torch.randn(shape, generator=g, device="cuda").to(ctype), torch.randn(shape, generator=g, device="cuda").to(ctype))


@pytest.mark.parametrize("t,hkv,page,d,dtype,ctype", [
    (1, 1, 16, 64, BF, BF), (4, 4, 16, 128, HF, HF), (33, 3, 32, 128, BF, E4), (200, 8, 64, 64, HF, E4), (7, 5, 256, 128, BF, BF),
    (300, 2, 128, 64, HF, HF), (1000, 1, 16, 128, BF, E4)])
def test_kv_write(t, hkv, page, d, dtype, ctype):
    pages = t // page + 5
    cache = make_cache(t, pages, hkv, page, d, ctype)
    rng = np.random.default_rng(t)
    slots = rng.permutation(pages * page)[:t]
    slots[rng.random(t) < 0.1] = -1
    rows = (torch.randn((t, 2 * hkv * d + 24), generator=gen(t), device="cuda") * 2).to(dtype)
    rows[0, 8] = float("nan")
    rows[0, 9], rows[0, 10] = float("inf"), -6.0
    k, v = (rows[:, 8 + i * hkv * d:8 + (i + 1) * hkv * d].unflatten(1, (hkv, d)) for i in range(2))
    fp8 = ctype == E4
    bits = torch.uint8 if fp8 else torch.int16
    before = [c.view(bits).cpu().numpy() for c in (cache.k, cache.v)]
    status = i32([0])
    api.mdw_kv_write(cache, k, v, torch.tensor(slots, device="cuda"), status=status)
    assert status.item() == 0
    for rows_, c, old, scale in ((k, cache.k, before[0], cache.k_scale), (v, cache.v, before[1], cache.v_scale)):
        got = c.view(bits).cpu().numpy()
        if fp8:
            clean = torch.nan_to_num(rows_.float(), nan=0.0, posinf=3e38, neginf=-3e38).cpu().numpy()
            want = OA.kv_write(old, clean, slots, page, scale.cpu().numpy())
            nan = OA.kv_write(np.zeros(old.shape, bool), torch.isnan(rows_.float()).cpu().numpy(), slots, page)
            assert ((got[nan] & 127) == 127).all()
            got, want = got[~nan], want[~nan]
        else:
            want = old.copy()
            src = rows_.contiguous().view(bits).cpu().numpy()
            for r, s in zip(src, slots):
                if s >= 0:
                    want[s // page, :, s % page] = r
        assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_kv_write_codes_of_every_element_at_many_scales(dtype):
    """Every 16-bit element at scales of all magnitudes: the codes are those of the fp32 quotient, also where
    it lies next to the middle of two codes, below E4M3's normal range or beyond its largest value."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.uint16).view(dtype)
    x = bits[torch.isfinite(bits.float())]
    x = torch.cat([x, x.new_zeros(-len(x) % 64)]).view(-1, 1, 64).cuda()
    t = x.shape[0]
    rng = np.random.default_rng(0)
    scales = list(np.exp2(rng.uniform(-12, 12, 24))) + [1.0, 2.0 ** -9, 1.5, 1e-38, 3e38, 1e-45, 1 / 3, 0.99999994]
    slots = torch.arange(t, device="cuda")
    for s in scales:
        shape = (t // 16 + 1, 1, 16, 64)
        cache = api.KVCache(*(torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)),
                            *(torch.full((1,), float(s), dtype=F32, device="cuda") for _ in range(2)))
        api.mdw_kv_write(cache, x, -x, slots)
        with np.errstate(over="ignore"):
            q = x.float().cpu().numpy().reshape(t, 64) / np.float32(s)
        for c, sign in ((cache.k, 1), (cache.v, -1)):
            got = c.reshape(-1, 64)[:t].cpu().numpy()
            want = OF.float_to_e4m3_rne_sat(np.clip(sign * q, -1e30, 1e30))
            assert np.array_equal(got, want), (s, int((got != want).sum()))


def test_kv_write_skips_slots_outside_the_cache():
    cache = make_cache(1, 3, 2, 16, 64, BF)
    before = cache.k.clone()
    rows = torch.randn((4, 2, 64), generator=gen(1), device="cuda").to(BF)
    status = i32([0])
    api.mdw_kv_write(cache, rows, rows, torch.tensor([48, 5, -2, 1 << 40], device="cuda"), status=status)
    assert status.item() == 7
    before[0, :, 5] = rows[1]
    assert torch.equal(cache.k, before)


def test_kv_write_with_k_and_v_in_one_allocation_beyond_2_31_elements():
    pool = torch.zeros((5, 2, 1024, 256, 128), dtype=BF, device="cuda")        # 5 pages of 2 x 33.5 M elements
    pool = torch.zeros((33, 2, 1024, 256, 128), dtype=torch.uint8, device="cuda") if pool.numel() < 1 << 31 else pool
    one = torch.ones(1024, device="cuda")
    cache = api.KVCache(pool[:, 0], pool[:, 1], one, one)
    rows = torch.full((1, 1024, 128), 1.0, dtype=BF, device="cuda")
    api.mdw_kv_write(cache, rows, 2 * rows, torch.tensor([33 * 256 - 1], device="cuda"))
    assert pool[32, 0, :, 255].view(E4).float().eq(1).all() and pool[32, 1, :, 255].view(E4).float().eq(2).all()
    assert int(pool[32].count_nonzero()) == 2 * 1024 * 128 and int(pool[:32].count_nonzero()) == 0


# --------------------------------------------------------------------- mdw_tree_attention


class Attn:
    """A case: cache, shuffled pages, packed rows and random trees (or random masks)."""

    def __init__(self, seed, ctx, new, hq, hkv, d, page, dtype, ctype, masks="tree", pad=0, spare=3):
        rng = np.random.default_rng(seed)
        self.ctx, self.new = np.array(ctx), np.array(new)
        need = -(-(self.ctx + self.new) // page)
        pages = int(need.sum()) + spare
        self.cache = make_cache(seed, pages, hkv, page, d, ctype)
        self.table = np.full((len(ctx), max(1, int(need.max()))), -1)
        pool, at = rng.permutation(pages), 0
        for b, n in enumerate(need):
            self.table[b, :n] = pool[at:at + n]
            at += n
        self.start = np.concatenate([[0], np.cumsum(new)])
        self.t = int(self.start[-1]) + pad
        self.q = torch.randn((max(self.t, 1), hq, d), generator=gen(seed), device="cuda").to(dtype)
        self.seen = []
        for n in new:
            s = np.zeros((n, n), bool)
            for i in range(n):
                if masks == "tree":
                    p = int(rng.integers(-1, i)) if i else -1
                    s[i] = s[p] if p >= 0 else False
                    s[i, i] = True
                elif masks == "chain":
                    s[i, :i + 1] = True
                else:
                    s[i] = rng.random(n) < 0.3
            self.seen.append(s)
        bits = [sum(1 << int(j) for j in np.nonzero(r)[0]) for s in self.seen for r in s] + [0] * pad
        self.mask = torch.tensor(np.array(bits or [0], np.uint64).view(np.int64), device="cuda")
        self.page, self.d, self.scale = page, d, d ** -0.5

    def call(self, q=None, out=None, mask=True, max_new=None, ws=None, stream=None, status=None, lse=True, table=None, ctx=None):
        q = self.q if q is None else q
        out = torch.full_like(self.q, 5.0) if out is None else out
        lse = torch.full(self.q.shape[:2], 5.0, device="cuda") if lse is True else lse
        max_new = max(1, int(self.new.max())) if max_new is None else max_new
        nbytes = api.mdw_tree_attention_workspace_bytes(self.cache, len(self.ctx), self.q.shape[0], self.q.shape[1], max_new)
        ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
        api.mdw_tree_attention(self.cache, q, out, i32(self.table if table is None else table), i32(self.ctx if ctx is None else ctx),
                               i32(self.start), max_new, ws, tree_mask=self.mask if mask is True else mask, lse=lse, scale=self.scale,
                               status=status, stream=stream)
        return out, lse

    def keys(self, b):
        """Keys and values of request b, in float64."""
        n = int(self.ctx[b] + self.new[b])
        ids = torch.tensor(self.table[b, :-(-n // self.page)], dtype=torch.int64, device="cuda")
        kv = []
        for c, s in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            x = c.view(torch.uint8)[ids].view(c.dtype).to(torch.float64).transpose(1, 2).reshape(-1, c.shape[1], c.shape[3])[:n]
            kv.append((x if s is None else x * s.double()[:, None]).cpu().numpy())
        return kv

    def check(self, out, lse, hide=None, requests=None, k_v=None):
        """`hide`: more keys (bool [keys]) that no row of a request sees."""
        prob = half_step(HF if self.cache.k.dtype == E4 else self.q.dtype)
        for b in range(len(self.ctx)) if requests is None else requests:
            k, v = self.keys(b) if k_v is None else k_v(b)
            rows = slice(int(self.start[b]), int(self.start[b + 1]))
            seen = np.concatenate([np.ones((self.new[b], self.ctx[b]), bool), self.seen[b]], 1)
            if hide is not None:
                seen &= ~hide[b][None]
            qd = host(self.q[rows])
            o, z, spread, size = OA.tree_attention(qd, k, v, seen, self.scale)
            # scores: d products in fp32 (and an f16 query element off by 2^-24 of its row's largest
            # with an E4M3 cache), scaled once: at most d / 16 + 8 chained steps; exponentials and their
            # sums: 2^-20 relative, one chain of keys / 16 + 64 steps per sum
            delta = (self.d / 16 + 8) * 2.0 ** -23 * size + 2.0 ** -23 * np.where(np.isfinite(z), np.abs(z), 0)
            if self.cache.k.dtype == E4 and len(k):
                delta = delta + self.scale * 2.0 ** -24 * np.abs(qd).max(-1) * np.abs(k).sum(-1).max()
            chain = (len(k) / 16 + 64) * 2.0 ** -23
            rel = 2 * np.expm1(delta) + 2.0 ** -20 + chain
            assert_close(host(out[rows]), o, half_step(self.q.dtype) * np.abs(o) + (rel[:, :, None] + 2 * prob) * spread + 1e-30, f"out {b}")
            if lse is not None:
                got, fin = host(lse[rows]), np.isfinite(z)
                assert np.array_equal(got[~fin], z[~fin])
                assert_close(got[fin], z[fin], (delta + 2.0 ** -20 + chain + 2.0 ** -22 * np.where(fin, np.abs(z), 0))[fin], f"lse {b}")


SHAPES = [
    # ctx, new, hq, hkv, d, page
    ([5], [1], 1, 1, 64, 16), ([0], [1], 4, 1, 128, 16), ([0], [64], 8, 2, 64, 32), ([1500], [4], 20, 4, 128, 16),
    ([127, 128, 129, 0, 1], [1, 1, 2, 3, 0], 8, 8, 128, 16), ([200, 0, 0, 700], [0, 0, 5, 16], 16, 2, 128, 64),
    ([1000, 30, 4000], [16, 7, 33], 32, 8, 64, 128), ([63, 64, 65, 190], [64, 63, 62, 1], 12, 3, 128, 256), ([300], [64], 64, 1, 128, 32),
    ([511, 513], [3, 5], 64, 4, 64, 64), ([9001], [1], 8, 8, 128, 16), ([20000, 7], [2, 1], 7, 1, 128, 128),
    ([40] * 37, [2] * 37, 6, 2, 64, 16), ([90, 300], [17, 11], 10, 2, 128, 16)]


@pytest.mark.parametrize("dtype,ctype", [(BF, BF), (HF, HF), (BF, E4), (HF, E4)])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attention(i, dtype, ctype):
    c = Attn(i, *SHAPES[i], dtype, ctype, masks="random" if i % 3 == 2 else "tree")
    status = i32([0])
    out, lse = c.call(status=status)
    assert status.item() == 0
    c.check(out, lse)


@pytest.mark.parametrize("ctype", [BF, E4])
def test_attention_long_context(ctype):
    c = Attn(3, [50001, 3], [2, 5], 8, 2, 128, 64, BF, ctype)
    c.check(*c.call())


def test_attention_many_requests():
    rng = np.random.default_rng(0)
    c = Attn(4, rng.integers(0, 40, 700), rng.integers(0, 3, 700), 4, 2, 64, 16, HF, HF)
    c.check(*c.call())


def test_attention_chain_without_a_mask_and_a_loose_row_limit():
    c = Attn(5, [100, 0, 31], [4, 64, 9], 8, 2, 128, 16, BF, BF, masks="chain")
    out, lse = c.call()
    c.check(out, lse)
    for kw in (dict(mask=None), dict(mask=None, lse=None)):
        got, _ = c.call(**kw)
        assert torch.equal(got, out)
    c = Attn(5, [100, 0, 31], [4, 1, 9], 8, 2, 128, 16, BF, BF)
    c.check(*c.call(max_new=64))


@pytest.mark.parametrize("ctype", [BF, E4])
@pytest.mark.parametrize("hq", [2, 32, 128])
def test_attention_ignores_what_masked_keys_hold(ctype, hq):
    """NaN and infinities in slots behind the sequence, in spare pages and in nodes that a row does not see."""
    c = Attn(6, [70, 0, 129], [9, 20, 40], hq, 2, 128, 32, BF, ctype, masks="random", spare=4)
    poison = {}
    for b in range(3):
        # node 3 holds NaN values and node 5 NaN keys and infinite values; rows that see one are not compared
        c.seen[b][0], c.seen[b][1] = False, False
        for node in (3, 5):
            key = int(c.ctx[b]) + node
            page, off = int(c.table[b, key // 32]), key % 32
            poison[page, off] = node
        n = int(c.ctx[b] + c.new[b])
        for off in range(n % 32, 32 if n % 32 else 0):
            poison[int(c.table[b, n // 32]), off] = 5
    used = set(c.table[c.table >= 0].tolist())
    for page in range(c.cache.k.shape[0]):
        if page not in used:
            for off in range(32):
                poison[page, off] = 5
    bits = [sum(1 << int(j) for j in np.nonzero(r)[0]) for s in c.seen for r in s]
    c.mask = torch.tensor(np.array(bits, np.uint64).view(np.int64), device="cuda")
    clean = [c.keys(b) for b in range(3)]
    raw = torch.uint8 if ctype == E4 else torch.int16
    nan, inf = (127, 127) if ctype == E4 else (0x7FC0, 0x7F80)
    for (page, off), node in poison.items():
        c.cache.v.view(raw)[page, :, off, ::3] = nan if node == 3 else inf
        if node == 5:
            c.cache.k.view(raw)[page, :, off, 1::5] = nan
    out, lse = c.call()
    whole = Attn.keys
    c.keys = lambda b: clean[b]
    keep = [np.nonzero(~(c.seen[b][:, 3] | c.seen[b][:, 5]))[0] for b in range(3)]
    for b in range(3):
        assert len(keep[b]) > 2
        rows = torch.tensor(keep[b] + c.start[b], device="cuda")
        sub = Attn.__new__(Attn)
        sub.__dict__.update(c.__dict__, ctx=c.ctx[b:b + 1], new=np.array([len(keep[b])]), start=np.array([0, len(keep[b])]), q=c.q[rows],
                            seen=[c.seen[b][keep[b]]])
        seen = np.concatenate([np.ones((len(keep[b]), c.ctx[b]), bool), c.seen[b][keep[b]]], 1)
        sub.seen, sub.ctx = [seen], np.array([0])
        sub.check(out[rows], lse[rows], k_v=lambda _: clean[b])
    # rows that see a poisoned node are not finite there
    for b in range(3):
        hit = torch.tensor(np.nonzero(c.seen[b][:, 3])[0] + c.start[b], device="cuda")
        assert not torch.isfinite(out[hit][:, :, ::3]).any()
    assert whole is Attn.keys


def test_attention_rows_that_see_nothing():
    c = Attn(7, [0, 0], [6, 1], 8, 2, 64, 16, HF, HF, masks="random")
    for s in c.seen:
        s[:] = False
    c.mask.zero_()
    out, lse = c.call()
    assert not out[:7].any() and (lse[:7] == -float("inf")).all()


def test_attention_strides_padding_and_untouched_rows():
    c = Attn(8, [50, 7], [5, 3], 6, 2, 128, 16, BF, BF, pad=4)
    wide = torch.full((c.t, 6 * 128 + 48), 3.0, dtype=BF, device="cuda")
    q = wide[:, 16:16 + 768].unflatten(1, (6, 128))
    q.copy_(c.q)
    buf = torch.full((c.t, 6 * 128 + 8), 9.0, dtype=BF, device="cuda")
    out, lse = c.call(q=q, out=buf[:, :768].unflatten(1, (6, 128)))
    c.check(out, lse)
    assert (buf[8:] == 9).all() and (buf[:, 768:] == 9).all() and (lse[8:] == 5).all()


def test_attention_with_keys_and_values_in_one_allocation():
    c = Attn(9, [200, 17], [4, 4], 8, 4, 64, 16, BF, BF)
    both = torch.stack((c.cache.k, c.cache.v), 1).contiguous()
    want, _ = c.call()
    c.cache = api.KVCache(both[:, 0], both[:, 1])
    got, lse = c.call()
    assert torch.equal(got, want)
    c.check(got, lse)


def test_attention_bad_pages_are_not_seen():
    c = Attn(10, [100, 40], [3, 3], 8, 2, 128, 16, BF, BF)
    table = c.table.copy()
    table[0, 2], table[0, 6], table[1, 0] = 1 << 30, -3, c.cache.k.shape[0]
    status = i32([0])
    out, lse = c.call(table=table, status=status)
    assert status.item() == 7
    hide = [np.zeros(103, bool), np.zeros(43, bool)]
    hide[0][32:48], hide[0][96:], hide[1][:16] = True, True, True
    c.check(out, lse, hide=hide)


def test_attention_bad_lengths_skip_the_request():
    c = Attn(11, [30, 40, 50, 20], [2, 2, 2, 2], 4, 2, 64, 16, HF, HF)
    for ctx, bad in (([30, -1, 50, 20], [1]), ([30, 40, 2147483647, 20], [2]), ([30, 64, 50, 2000], [1, 3])):
        status = i32([0])
        out, lse = c.call(ctx=ctx, status=status)
        assert status.item() == 7
        c.check(out, lse, requests=[b for b in range(4) if b not in bad])
        for b in bad:
            assert (out[2 * b:2 * b + 2] == 5).all() and (lse[2 * b:2 * b + 2] == 5).all()
    status = i32([0])
    out, lse = c.call(max_new=1, status=status)
    assert status.item() == 7 and (out == 5).all()
    c.start[4] = 9
    status = i32([0])
    out, lse = c.call(max_new=64, status=status)
    assert status.item() == 7 and (out[6:] == 5).all()
    c.start[4] = 8
    c.check(out, lse, requests=[0, 1, 2])


def test_attention_large_scores_and_values():
    c = Attn(12, [300], [4], 8, 2, 128, 16, BF, BF)
    c.q *= 200                                      # scores of thousands: one key holds the whole row
    c.check(*c.call())
    c = Attn(13, [300], [4], 8, 2, 64, 16, HF, E4)
    c.q *= 100
    c.check(*c.call())
    c = Attn(14, [300], [4], 8, 2, 64, 16, BF, E4)
    c.q *= 2.0 ** 100                               # beyond f16; values of the query rows are scaled, not clipped
    c.scale = 2.0 ** -104
    c.check(*c.call())


def test_attention_beyond_2_31_elements():
    pages, hkv, page, d = 70, 1024, 256, 128        # 2.3 G elements each
    k, v = (torch.zeros((pages, hkv, page, d), dtype=torch.uint8, device="cuda").view(E4) for _ in range(2))
    ks = torch.full((hkv,), 0.01, device="cuda")
    c = Attn(15, [300], [2], 8, 2, 128, 256, BF, E4)
    small = c.cache
    for i, p in enumerate(c.table[0]):
        k.view(torch.uint8)[pages - 1 - i, -2:] = small.k.view(torch.uint8)[int(p)]
        v.view(torch.uint8)[pages - 1 - i, -2:] = small.v.view(torch.uint8)[int(p)]
    ks[-2:] = small.k_scale
    vs = ks.clone()
    vs[-2:] = small.v_scale
    big = api.KVCache(k, v, ks, vs)
    q = torch.zeros((2, hkv * 4, d), dtype=BF, device="cuda")
    q[:, -8:] = c.q
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = torch.empty(api.mdw_tree_attention_workspace_bytes(big, 1, 2, hkv * 4, 2), dtype=torch.uint8, device="cuda")
    api.mdw_tree_attention(big, q, out, i32([[pages - 1 - i for i in range(c.table.shape[1])]]), i32([300]), i32([0, 2]), 2, ws,
                           tree_mask=c.mask, lse=lse, scale=c.scale)
    c.check(out[:, -8:], lse[:, -8:])


def test_attention_repeats_bit_for_bit_on_other_streams_and_in_graphs():
    a = Attn(16, [700, 90], [8, 3], 16, 4, 128, 16, BF, BF)
    b = Attn(17, [40, 1300], [2, 16], 16, 4, 128, 16, BF, BF)
    wa, wb = (x.call() for x in (a, b))
    again, _ = a.call()
    assert torch.equal(again, wa[0])
    side = torch.cuda.Stream()
    ws = torch.empty(max(api.mdw_tree_attention_workspace_bytes(x.cache, 2, x.t, 16, 16) for x in (a, b)), dtype=torch.uint8, device="cuda")
    fixed = [(x, torch.zeros_like(x.q), torch.zeros(x.q.shape[:2], device="cuda"), i32(x.table), i32(x.ctx), i32(x.start)) for x in (a, b)]

    def run(x, out, lse, table, ctx, start, stream=None):
        api.mdw_tree_attention(x.cache, x.q, out, table, ctx, start, 16, ws, tree_mask=x.mask, lse=lse, scale=x.scale, stream=stream)

    side.wait_stream(torch.cuda.current_stream())
    run(*fixed[0], stream=side)
    run(*fixed[1], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for (x, out, lse, *_), w in zip(fixed, (wa, wb)):
        x.check(out, lse)
        out.zero_()
        lse.zero_()
    torch.cuda.synchronize()
    graphs = []
    for f in fixed:                                  # two graphs that share one workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(*f)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for x, out, lse, *_ in fixed:
        x.check(out, lse)


# ------------------------------------------------------------------------------- together


def test_sublayer_of_a_verify_window():
    """Projection, plan, writer, attention and output projection of one window of two trees, then the decode
    step's own MoE layer and head on what comes out: each step against the oracle on the device's input."""
    from _cases import Layer
    hidden, hq, hkv, d, page = 2560, 20, 4, 128, 16
    ctx, new = np.array([37, 130]), np.array([4, 7])
    t = int(new.sum())
    parents = np.array([-1, 0, 0, 1, -1, 0, 1, 1, 0, 4, 4])
    g = gen(0)
    cache = make_cache(1, 24, hkv, page, d, BF)
    wqkv, wo = w4_case(1, (hq + 2 * hkv) * d, hidden, 128, False, BF), w4_case(2, hidden, hq * d, 64, True, BF)
    x = torch.randn((t, hidden), generator=g, device="cuda").to(BF)
    table = np.full((2, 10), -1)
    table[0, :3], table[1, :9] = [5, 1, 9], [2, 3, 4, 6, 7, 8, 10, 11, 12]
    status = torch.zeros(4, dtype=torch.int32, device="cuda")[:1]
    dt, ct, st = i32(table), i32(ctx), torch.empty(3, dtype=torch.int32, device="cuda")
    slot, pos, mask = torch.empty(t, dtype=torch.int64, device="cuda"), i32(np.zeros(t)), torch.empty(t, dtype=torch.int64, device="cuda")
    taken, qkv = i32([0]), torch.empty((t, (hq + 2 * hkv) * d), dtype=BF, device="cuda")
    att, y = torch.empty((t, hq, d), dtype=BF, device="cuda"), torch.empty((t, hidden), dtype=BF, device="cuda")
    lse = torch.empty((t, hq), device="cuda")
    q, k, v = qkv.split([hq * d, hkv * d, hkv * d], 1)
    q, k, v = q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))
    ws = torch.empty(api.mdw_tree_attention_workspace_bytes(cache, 2, t, hq, 7), dtype=torch.uint8, device="cuda")
    old_k = host(cache.k)
    api.mdw_kv_plan(ct, i32(new), page, 24, dt, i32([20, 21]), st, slot, pos, taken, parents=i32(parents), tree_mask=mask, status=status)
    api.w4_linear(wqkv, x, qkv)
    api.mdw_kv_write(cache, k, v, slot, status=status)
    api.mdw_tree_attention(cache, q, att, dt, ct, st, 7, ws, tree_mask=mask, lse=lse, status=status)
    api.w4_linear(wo, att.flatten(1), y, residual=x)
    assert api.mdw_device_status(status) == 0
    want, tol = w4_want(wqkv, x)
    assert_close(host(qkv), want, tol + half_step(BF) * np.abs(want), "qkv")
    plan = OA.kv_plan(ctx, new, page, 24, table, [20, 21], t, parents)
    assert np.array_equal(slot.cpu().numpy(), plan["slot"]) and np.array_equal(dt.cpu().numpy(), plan["table"])
    assert np.array_equal(host(cache.k), OA.kv_write(old_k, host(k), plan["slot"], page))
    c = Attn(0, ctx, new, hq, hkv, d, page, BF, BF)
    c.cache, c.table, c.q = cache, plan["table"], q.contiguous()
    c.seen = [np.array([[int(plan["mask"][plan["start"][b] + i]) >> j & 1 for j in range(n)] for i in range(n)], bool) for b, n in enumerate(new)]
    c.check(att, lse)
    want, tol = w4_want(wo, att.flatten(1), residual=x)
    assert_close(host(y), want, tol + half_step(BF) * np.abs(want), "output projection")
    layer = Layer(seed=3, layer=0, num_experts=64, top_k=8, shared=True)
    mws = torch.zeros(api.mdw_moe_workspace_bytes(layer.weights, t), dtype=torch.uint8, device="cuda")
    z = torch.empty_like(y)
    api.moe_decode_layer(layer.weights, y, z, mws, residual=y)
    assert api.mdw_device_status(mws) == 0 and torch.isfinite(z.float()).all()


def test_binding_refuses():
    c = Attn(18, [20], [2], 4, 2, 64, 16, BF, BF)
    w = w4_case(1, 8, 64, 32, False, BF)
    x, y = torch.zeros((2, 64), dtype=BF, device="cuda"), torch.zeros((2, 8), dtype=BF, device="cuda")
    for args, code in (((x.half(), y), 3), ((x, y.half()), 3), ((x[:, :32], y), 1), ((x.t().contiguous().t(), y), 1), ((x, y[:1]), 1),
                       ((x.cpu(), y), 1), ((x.new_zeros((33, 64)), y.new_zeros((33, 8))), 1)):
        with pytest.raises(api.MdwError) as e:
            api.w4_linear(w, *args)
        assert e.value.code == code
    for kw in (dict(q=c.q.half()), dict(mask=c.mask[:1]), dict(out=c.q.new_zeros((2, 4, 128))[:, :, ::2]), dict(table=c.table[:, :0]),
               dict(ws=torch.empty(8, dtype=torch.uint8, device="cuda")), dict(max_new=65), dict(lse=torch.zeros(2, 4, device="cuda").half())):
        with pytest.raises(api.MdwError):
            c.call(**kw)
    with pytest.raises(api.MdwError):
        api.KVCache(c.cache.k, c.cache.v, torch.ones(2, device="cuda"), torch.ones(2, device="cuda"))
    with pytest.raises(api.MdwError):
        api.KVCache(c.cache.k.view(torch.uint8), c.cache.v.view(torch.uint8))
    with pytest.raises(api.MdwError):
        api.KVCache(c.cache.k.transpose(1, 2), c.cache.v.transpose(1, 2))


def test_attention_wait_that_runs_out_is_reported():
    """A bounded wait of the copy pipeline that gives up ends in MDW_ERR_TIMEOUT, a clean exit and a usable
    device; rows are then not stored."""
    c = Attn(19, [40000, 500], [4, 2], 8, 2, 128, 16, BF, BF)
    ws = torch.empty(api.mdw_tree_attention_workspace_bytes(c.cache, 2, c.t, 8, 4), dtype=torch.uint8, device="cuda")
    api.mdw_debug_set_spin_budget(1)
    try:
        status = i32([0])
        torch.zeros(1 << 28, dtype=torch.int32, device="cuda")  # the cache leaves the L2: its copies are waited for
        c.call(status=status, ws=ws)
        assert status.item() == 6
    finally:
        api.mdw_debug_set_spin_budget(0)
    status = i32([0])
    out, lse = c.call(status=status)
    assert status.item() == 0
    c.check(out, lse)


# ---- the binding ----------------------------------------------------------------------------------
def test_handles_of_another_kind_are_refused():
    kv = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    cache = api.KVCache(kv, kv.clone())
    w = api.W4Weights(torch.zeros(64, 32, dtype=torch.uint8, device="cuda"), torch.zeros(64, 1, dtype=torch.bfloat16, device="cuda"))
    x = torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    cache.q, w.k = x, rows
    with pytest.raises(api.MdwError) as e:
        api.w4_linear(cache, x, x.clone())
    assert e.value.code == 3
    with pytest.raises(api.MdwError) as e:
        api.mdw_kv_write(w, rows, rows, torch.zeros(1, dtype=torch.int64, device="cuda"))
    assert e.value.code == 3


@pytest.mark.parametrize("m,n,k,group,zero,dtype,ydtype", [
    (9, 8192, 256, 32, True, BF, BF), (16, 8200, 320, 32, True, HF, F32), (17, 8193, 384, 128, True, BF, F32), (32, 20000, 2560, 64, False, HF, HF),
    (32, 8321, 2880, 32, True, BF, BF), (31, 8200, 5120, 128, False, BF, F32), (13, 9001, 6400, 64, True, HF, F32), (8, 8192, 12800, 128, True, BF, F32)])
def test_w4_linear_many_features(m, n, k, group, zero, dtype, ydtype):
    """Features for every block and more, with tokens that fit a block's shared memory and ones that do not."""
    w = w4_case(m + n, n, k, group, zero, dtype)
    x = torch.randn((m, k), generator=gen(2), device="cuda").to(dtype)
    bias = torch.randn(n, generator=gen(3), device="cuda").to(dtype)
    res = torch.randn((m, n), generator=gen(4), device="cuda").to(dtype)
    y = torch.full((m + 1, n), 7.0, dtype=ydtype, device="cuda")
    api.w4_linear(w, x, y[:m], bias=bias, residual=res)
    want, tol = w4_want(w, x, bias, res)
    assert_close(host(y[:m]), want, tol + half_step(ydtype) * np.abs(want))
    assert (y[m] == 7.0).all()
    again = torch.empty_like(y[:m])
    api.w4_linear(w, x, again, bias=bias, residual=res)
    assert torch.equal(again, y[:m])


# ---- every kernel of mdw_tree_attention: up to 16 rows a request and kv head, up to 32, more
PATHS = [(8, BF, BF, 128), (8, BF, E4, 128), (8, HF, HF, 64), (8, HF, E4, 64), (16, BF, BF, 128), (16, BF, E4, 128), (16, HF, HF, 64),
         (16, HF, E4, 64), (64, BF, BF, 128), (64, BF, E4, 128), (64, HF, HF, 64), (64, HF, E4, 64)]   # query heads over 2 kv heads


@pytest.mark.parametrize("hq,dtype,ctype,d", PATHS)
def test_attention_bad_pages_on_every_path(hq, dtype, ctype, d):
    c = Attn(30, [400, 40, 16], [4, 3, 1], hq, 2, d, 16, dtype, ctype)
    table = c.table.copy()
    table[0, 2], table[0, 6], table[0, 20], table[1, 0] = 1 << 30, -3, -1, c.cache.k.shape[0]
    status = i32([0])
    out, lse = c.call(table=table, status=status)
    assert status.item() == 7
    hide = [np.zeros(404, bool), np.zeros(43, bool), np.zeros(17, bool)]
    hide[0][32:48], hide[0][96:112], hide[0][320:336], hide[1][:16] = True, True, True, True
    c.check(out, lse, hide=hide)


@pytest.mark.parametrize("hq,dtype,ctype,d", PATHS)
def test_attention_bad_lengths_and_empty_requests_on_every_path(hq, dtype, ctype, d):
    c = Attn(31, [30, 40, 50, 0, 300], [2, 4, 2, 0, 1], hq, 2, d, 32, dtype, ctype, pad=3)
    for ctx, bad in (([30, -1, 50, 0, 300], [1]), ([30, 40, 2147483647, 0, 300], [2]), ([2000, 40, 50, 0, 300], [0])):
        status = i32([0])
        out, lse = c.call(ctx=ctx, status=status)
        assert status.item() == 7
        c.check(out, lse, requests=[b for b in range(5) if b not in bad])
        for b in bad:
            rows = slice(int(c.start[b]), int(c.start[b + 1]))
            assert (out[rows] == 5).all() and (lse[rows] == 5).all()
        assert (out[9:] == 5).all() and (lse[9:] == 5).all()


@pytest.mark.parametrize("hq,dtype,ctype,d", PATHS)
def test_attention_nothing_seen_on_every_path(hq, dtype, ctype, d):
    c = Attn(32, [0, 0, 40], [4, 1, 2], hq, 2, d, 16, dtype, ctype)
    for s in c.seen[:2]:
        s[:] = False
    c.mask[:5] = 0
    out, lse = c.call()
    assert not out[:5].any() and (lse[:5] == -float("inf")).all()
    c.check(out, lse, requests=[2])


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("hq,dtype,ctype,d", [(2, BF, BF, 128), (2, HF, E4, 128), (2, HF, HF, 64), (2, BF, E4, 64), (8, BF, BF, 128), (8, HF, E4, 128),
                                              (8, HF, HF, 64), (8, BF, E4, 64), (32, BF, BF, 128), (32, HF, E4, 64)])
def test_attention_ignores_what_masked_keys_hold_on_every_path(hq, dtype, ctype, d, page):
    """NaN and infinities behind the sequence, in spare pages and in nodes that a row does not see; rows that see
    NaN values are NaN there."""
    ctx, new = [70, 0, 1029], [8, 7, 8]
    c = Attn(33, ctx, new, hq, 2, d, page, dtype, ctype, masks="random", spare=4)
    for s in c.seen:
        s[0], s[1], s[2] = False, False, False
        s[0, 0], s[2, 3] = True, True
    bits = [sum(1 << int(j) for j in np.nonzero(r)[0]) for s in c.seen for r in s]
    c.mask = torch.tensor(np.array(bits, np.uint64).view(np.int64), device="cuda")
    clean = [c.keys(b) for b in range(3)]
    raw = torch.uint8 if ctype == E4 else torch.int16
    nan, inf = (127, 255) if ctype == E4 else (0x7FC0, 0x7F80) if dtype == BF else (0x7E00, 0x7C00)

    def spoil(page_id, off, node):
        c.cache.v.view(raw)[page_id, :, off, ::3] = nan if node == 3 else inf
        if node != 3:
            c.cache.k.view(raw)[page_id, :, off, 1::5] = nan

    used = set(c.table[c.table >= 0].tolist())
    for b in range(3):
        for node in (3, 5):
            key = ctx[b] + node
            spoil(int(c.table[b, key // page]), key % page, node)
        n = ctx[b] + new[b]
        for off in range(n % page, page if n % page else 0):
            spoil(int(c.table[b, n // page]), off, 5)
    for page_id in set(range(c.cache.k.shape[0])) - used:
        for off in range(page):
            spoil(page_id, off, 5)
    out, lse = c.call()
    for b in range(3):
        keep = np.nonzero(~(c.seen[b][:, 3] | c.seen[b][:, 5]))[0]
        assert {0, 1} <= set(keep.tolist())
        rows = torch.tensor(keep + c.start[b], device="cuda")
        sub = Attn.__new__(Attn)
        seen = np.concatenate([np.ones((len(keep), ctx[b]), bool), c.seen[b][keep]], 1)
        sub.__dict__.update(c.__dict__, ctx=np.array([0]), new=np.array([len(keep)]), start=np.array([0, len(keep)]), q=c.q[rows], seen=[seen])
        sub.check(out[rows], lse[rows], k_v=lambda _: clean[b])
        row = out[int(c.start[b]) + 2].float()
        assert torch.isnan(row[:, ::3]).all() and torch.isfinite(row[:, 1::3]).all()


def test_calls_on_two_streams_do_not_disturb_each_other():
    cs = [Attn(34 + i, [900, 40], [4, 2], 16 * (1 + 3 * i), 4, 128, 16, BF, BF) for i in range(2)]
    ws = [w4_case(40 + i, 2000, 2560, 64, True, BF) for i in range(2)]
    xs = [torch.randn((3 + 20 * i, 2560), generator=gen(i), device="cuda").to(BF) for i in range(2)]
    want = [c.call()[0] for c in cs]
    ys = [torch.empty((x.shape[0], 2000), dtype=BF, device="cuda") for x in xs]
    for w, x, y in zip(ws, xs, ys):
        api.w4_linear(w, x, y)
    got = [[torch.empty_like(y) for _ in range(8)] for y in ys]
    outs = [[torch.empty_like(c.q) for _ in range(8)] for c in cs]
    space = [torch.empty(api.mdw_tree_attention_workspace_bytes(c.cache, 2, c.t, c.q.shape[1], 4), dtype=torch.uint8, device="cuda") for c in cs]
    fixed = [(i32(c.table), i32(c.ctx), i32(c.start)) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(8):
        for i, (c, s) in enumerate(zip(cs, streams)):
            api.w4_linear(ws[i], xs[i], got[i][k], stream=s)
            api.mdw_tree_attention(c.cache, c.q, outs[i][k], *fixed[i], 4, space[i], tree_mask=c.mask, scale=c.scale, stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, ys[i]) for g in got[i]) and all(torch.equal(o, want[i]) for o in outs[i])


def test_w4_linear_wait_that_runs_out_is_reported():
    w = w4_case(50, 3000, 5120, 64, False, BF)
    x = torch.randn((20, 5120), generator=gen(0), device="cuda").to(BF)
    y, status = torch.empty((20, 3000), dtype=BF, device="cuda"), i32([0])
    api.mdw_debug_set_spin_budget(1)
    try:
        api.w4_linear(w, x, y, status=status)
        assert status.item() == 6
    finally:
        api.mdw_debug_set_spin_budget(0)
    status = i32([0])
    api.w4_linear(w, x, y, status=status)
    want, tol = w4_want(w, x)
    assert status.item() == 0
    assert_close(host(y), want, tol + half_step(BF) * np.abs(want))


FIRST_CALLS_CAPTURED = """
import sys; sys.path[:0] = [{root!r}, {tests!r}]
import torch
import test_attention_gpu as t
from moe_decode_weight_gb300 import api
c = [t.Attn(60 + i, [300, 20], [4, 2], hq, 2, 64, 16, t.HF, t.HF) for i, hq in enumerate((4, 16, 64))]
w = t.w4_case(61, 900, 640, 64, True, t.HF)
x = [torch.randn((m, 640), device="cuda").half() for m in (2, 12, 25)]
y = [torch.zeros((v.shape[0], 900), dtype=torch.half, device="cuda") for v in x]
out = [torch.zeros_like(v.q) for v in c]
args = [(t.i32(v.table), t.i32(v.ctx), t.i32(v.start)) for v in c]
ws = [torch.empty(api.mdw_tree_attention_workspace_bytes(v.cache, 2, v.t, v.q.shape[1], 4), dtype=torch.uint8, device="cuda") for v in c]
slot = torch.arange(6, device="cuda")
ctx, new, free, table = t.i32([3, 20]), t.i32([2, 4]), t.i32([5, 6, 7]), t.i32([[1, -1, -1], [2, 3, -1]])
start, slots, pos, taken = t.i32([0] * 3), torch.zeros(6, dtype=torch.int64, device="cuda"), t.i32([0] * 6), t.i32([0])
keys = torch.randn((6, 2, 64), device="cuda").half()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    api.mdw_kv_plan(ctx, new, 16, 8, table, free, start, slots, pos, taken)
    api.mdw_kv_write(c[0].cache, keys, keys, slot)
    for a, b in zip(x, y):
        api.w4_linear(w, a, b)
    for v, o, a, s in zip(c, out, args, ws):
        api.mdw_tree_attention(v.cache, v.q, o, *a, 4, s, tree_mask=v.mask, scale=v.scale)
g.replay()
g.replay()
torch.cuda.synchronize()
assert slots.tolist() == [19, 20, 52, 53, 54, 55] and start.tolist() == [0, 2, 6], (slots, start)
for a, b in zip(x, y):
    want, tol = t.w4_want(w, a)
    t.assert_close(t.host(b), want, tol + t.half_step(t.HF) * abs(want))
for v, o in zip(c, out):
    v.check(o, None)
print("ok")
"""


def test_first_calls_of_a_process_can_be_captured():
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALLS_CAPTURED.format(root=os.path.dirname(here), tests=here)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]


@pytest.mark.parametrize("m,n,k,group,zero,dtype,ydtype", [
    (1, 5000, 512, 128, False, BF, F32), (3, 5130, 2560, 64, True, HF, HF), (8, 9001, 640, 32, True, BF, BF), (2, 20011, 1152, 128, False, BF, F32),
    (1, 7001, 16384, 32, True, HF, F32), (4, 4880, 4096, 128, True, BF, BF), (1, 12001, 96, 32, False, BF, F32)])
def test_w4_linear_few_tokens_many_features(m, n, k, group, zero, dtype, ydtype):
    """More tiles of features than blocks, whose units clusters of blocks share out."""
    w = w4_case(m + n, n, k, group, zero, dtype)
    x = torch.randn((m, k), generator=gen(2), device="cuda").to(dtype)
    res = torch.randn((m, n), generator=gen(4), device="cuda").to(dtype)
    y = torch.full((m + 1, n), 7.0, dtype=ydtype, device="cuda")
    api.w4_linear(w, x, y[:m], residual=res)
    want, tol = w4_want(w, x, residual=res)
    assert_close(host(y[:m]), want, tol + half_step(ydtype) * np.abs(want))
    assert (y[m] == 7.0).all()
    again = torch.empty_like(y[:m])
    api.w4_linear(w, x, again, residual=res)
    assert torch.equal(again, y[:m])


# ---- waits that run out: every copy arrives before its block ends, whenever the wait runs out


@pytest.mark.parametrize("hq,dtype,ctype,d", PATHS)
def test_attention_is_right_after_waits_that_ran_out(hq, dtype, ctype, d):
    """Shares of a few tiles, whose copies are all requested at once: those of a block that gave up do not reach
    into the shared memory of the next call's blocks, which follow at once."""
    c = Attn(70, [900, 0, 300, 140], [4, 3, 1, 4], hq, 2, d, 16, dtype, ctype)
    want = c.call()
    args = i32(c.table), i32(c.ctx), i32(c.start)
    ws = [torch.empty(api.mdw_tree_attention_workspace_bytes(c.cache, 4, c.t, hq, 4), dtype=torch.uint8, device="cuda") for _ in range(2)]
    junk, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    outs = [torch.empty_like(c.q) for _ in range(16)]
    lost, good = i32([0]), i32([0])
    try:
        for out in outs:
            api.mdw_debug_set_spin_budget(1)
            api.mdw_tree_attention(c.cache, c.q, junk, *args, 4, ws[0], tree_mask=c.mask, lse=lse, scale=c.scale, status=lost)
            api.mdw_debug_set_spin_budget(0)
            api.mdw_tree_attention(c.cache, c.q, out, *args, 4, ws[1], tree_mask=c.mask, lse=lse, scale=c.scale, status=good)
    finally:
        api.mdw_debug_set_spin_budget(0)
    assert lost.item() == 6 and good.item() == 0
    assert all(torch.equal(out, want[0]) for out in outs) and torch.equal(lse, want[1])


@pytest.mark.parametrize("m,n,k,group,dtype", [(2, 3000, 2560, 64, BF), (12, 3000, 640, 32, HF), (12, 40000, 640, 128, BF), (32, 3000, 5120, 32, BF)])
def test_w4_linear_is_right_after_waits_that_ran_out(m, n, k, group, dtype):
    w = w4_case(71, n, k, group, True, dtype)
    x = torch.randn((m, k), generator=gen(1), device="cuda").to(dtype)
    want, junk = torch.empty((m, n), dtype=F32, device="cuda"), torch.empty((m, n), dtype=F32, device="cuda")
    api.w4_linear(w, x, want)
    outs = [torch.empty_like(want) for _ in range(16)]
    lost, good = i32([0]), i32([0])
    try:
        for out in outs:
            api.mdw_debug_set_spin_budget(1)
            api.w4_linear(w, x, junk, status=lost)
            api.mdw_debug_set_spin_budget(0)
            api.w4_linear(w, x, out, status=good)
    finally:
        api.mdw_debug_set_spin_budget(0)
    assert good.item() == 0 and (m <= 8 or lost.item() == 6)
    assert all(torch.equal(out, want) for out in outs)


@pytest.mark.parametrize("hq,dtype,ctype,d", PATHS)
def test_attention_that_gives_up_reads_no_bad_page(hq, dtype, ctype, d):
    """A block whose wait runs out goes on with what its shared memory holds, here NaN of the same tiles' other
    pages: it reads neither pages outside the cache nor behind the table's end."""
    c = Attn(72, [900, 90], [4, 3], hq, 2, d, 16, dtype, ctype)
    table = c.table.copy()
    table[0, 1::2], table[1, 3:] = 1 << 30, -(1 << 30)
    c.cache.v.view(torch.uint8 if ctype == E4 else torch.int16).fill_(127 if ctype == E4 else -1)
    ws = torch.empty(api.mdw_tree_attention_workspace_bytes(c.cache, 2, c.t, hq, 4), dtype=torch.uint8, device="cuda")
    for budget in (0, 1, 1, 1):                       # the first call leaves its tiles in shared memory
        api.mdw_debug_set_spin_budget(budget)
        try:
            status = i32([0])
            out, _ = c.call(table=table, ws=ws, status=status)
            assert status.item() in ((7,) if budget == 0 else (6, 7))
        finally:
            api.mdw_debug_set_spin_budget(0)
    c = Attn(73, [900, 90], [4, 3], hq, 2, d, 16, dtype, ctype)
    c.check(*c.call())


@pytest.mark.parametrize("hq,dtype,ctype,d", PATHS + [(32, BF, BF, 128), (32, HF, HF, 64), (32, HF, E4, 128)])
def test_attention_stores_nothing_of_items_with_a_lost_part(hq, dtype, ctype, d):
    """Requests cut between blocks of which some give up: rows are right or left as they were, not joined from what
    the workspace holds (finite sums here)."""
    c = Attn(74, [40000, 500], [4, 2], hq, 2, d, 16, dtype, ctype)
    want, want_lse = c.call()
    nbytes = api.mdw_tree_attention_workspace_bytes(c.cache, 2, c.t, hq, 4)
    flush = torch.empty(1 << 28, dtype=torch.int32, device="cuda")
    for _ in range(4):
        ws = torch.full((nbytes // 4,), 1.0, device="cuda").view(torch.uint8)
        out, lse, status = torch.full_like(c.q, 5.0), torch.full(c.q.shape[:2], 5.0, device="cuda"), i32([0])
        flush.zero_()                                # the cache leaves the L2: its first copies are waited for
        api.mdw_debug_set_spin_budget(1)
        try:
            c.call(out=out, lse=lse, ws=ws, status=status)
        finally:
            api.mdw_debug_set_spin_budget(0)
        assert status.item() == 6
        kept = (out == 5).all(2) & (lse == 5)        # (blocks whose copies were always there in time have not given up)
        assert torch.equal(out[~kept], want[~kept]) and torch.equal(lse[~kept], want_lse[~kept])


# ---- values that are not finite and are seen: the infinity, or NaN where one is NaN or both infinities meet
SEEN = [(hq, dtype, d) for hq in (2, 8, 16, 24, 32, 64) for dtype, d in ((BF, 128), (HF, 128), (BF, 64), (HF, 64))]   # 4 to 128 rows


@pytest.mark.parametrize("hq,dtype,d", SEEN)
@pytest.mark.parametrize("ctx", [[300, 1029, 130], [20000, 5, 130]])
def test_attention_gives_the_infinities_that_a_row_sees(hq, dtype, d, ctx):
    c = Attn(80, ctx, [4, 3, 4], hq, 2, d, 16, dtype, dtype)
    clean, clean_lse = c.call()
    c.check(clean, clean_lse)
    inf = float("inf")

    def put(b, key, column, value):
        c.cache.v[int(c.table[b, key // 16]), :, key % 16, column::5] = value

    # request 0: in full tiles of the context, far from and near its end; request 2: in a node and in the partial tile
    first, second = 37, ctx[0] - 180
    put(0, first, 0, inf), put(0, second, 1, -inf), put(0, first, 2, inf), put(0, second, 2, -inf), put(0, second, 3, float("nan"))
    put(2, ctx[2] + 1, 0, inf), put(2, ctx[2] - 1, 1, -inf)
    out, lse = c.call()
    assert torch.equal(lse, clean_lse)
    assert (out[:4, :, 0::5] == inf).all() and (out[:4, :, 1::5] == -inf).all()
    assert torch.isnan(out[:4, :, 2::5]).all() and torch.isnan(out[:4, :, 3::5]).all() and torch.equal(out[:4, :, 4::5], clean[:4, :, 4::5])
    assert torch.equal(out[4:7], clean[4:7])
    sees = torch.tensor(c.seen[2][:, 1], device="cuda")
    assert (out[7:][sees][:, :, 0::5] == inf).all() and torch.equal(out[7:][~sees][:, :, 0::5], clean[7:][~sees][:, :, 0::5])
    assert (out[7:, :, 1::5] == -inf).all() and all(torch.equal(out[7:, :, i::5], clean[7:, :, i::5]) for i in (2, 3, 4))


@pytest.mark.parametrize("hq,dtype,d", SEEN)
def test_attention_gives_an_infinity_of_small_probability(hq, dtype, d):
    """e^-30 of the largest: f16 rounds such a probability to zero, fp32 does not."""
    c = Attn(81, [700], [4], hq, 2, d, 16, dtype, dtype)
    c.cache.k.zero_(), c.q.fill_(1.0)
    page, at = int(c.table[0, 203 // 16]), 203 % 16
    c.cache.k[page, :, at] = -30.0 / (c.scale * d)
    clean, _ = c.call()
    c.cache.v[page, :, at, ::3] = float("inf")
    out, lse = c.call()
    assert (out[:, :, ::3] == float("inf")).all() and torch.isfinite(lse).all()
    assert torch.equal(out[:, :, 1::3], clean[:, :, 1::3])


@pytest.mark.parametrize("hq,dtype,ctype,d", [x for x in PATHS if x[2] == E4] + [(32, BF, E4, 128)])
@pytest.mark.parametrize("k_scale", [1e-45, 1e-38])
def test_attention_with_scales_below_fp32(hq, dtype, ctype, d, k_scale):
    """Keys whose scale times the softmax's is 0 in fp32 have equal scores; keys that a row does not see stay out."""
    c = Attn(82, [300, 0, 20], [4, 3, 4], hq, 2, d, 16, dtype, ctype, masks="random")
    c.cache.k_scale.fill_(k_scale)
    c.check(*c.call())
    c.q *= 2.0 ** -14                                # (bf16 rows enter f16 times a power of two)
    c.check(*c.call())


@pytest.mark.parametrize("m,n,k,group,dtype", [(m, 1000, 2048, g, t) for m in (1, 8, 9, 32) for g in (32, 64, 128) for t in (BF, HF)])
def test_w4_linear_takes_every_zero(m, n, k, group, dtype):
    """Zeros of 0 to 255, not those of a code alone, in every kernel; bit for bit with x of one element at a time, for
    which nothing is rounded."""
    w = w4_case(83 + m, n, k, group, False, dtype)
    w = api.W4Weights(w.q, w.scale, torch.arange(n * (k // group), device="cuda").remainder(256).to(torch.uint8).view(n, -1))
    x = torch.randn((m, k), generator=gen(m), device="cuda").to(dtype)
    y = torch.empty((m, n), dtype=F32, device="cuda")
    api.w4_linear(w, x, y)
    want, tol = w4_want(w, x)
    assert_close(host(y), want, tol + half_step(F32) * np.abs(want))
    weight = OA.w4_weight(w.q.cpu().numpy(), host(w.scale), w.zero.cpu().numpy(), group)
    for first in (0, 77, k - m):
        x.zero_()
        x[torch.arange(m), torch.arange(first, first + m)] = 1.0
        api.w4_linear(w, x, y)
        assert np.array_equal(host(y), weight[:, first:first + m].T)


@pytest.mark.parametrize("m", [1, 8, 9, 32])
@pytest.mark.parametrize("group", [32, 128])
def test_w4_linear_products_are_exact_at_the_ends_of_bf16(m, group):
    """Elements of 2^-100 and scales just below 2^121: one element a token, so that the scale's product alone is rounded."""
    n, k = 500, 1024
    w = w4_case(84, n, k, group, True, BF)
    top = 2.0 ** 120 * (1 + 127 / 128)
    w.scale.copy_(torch.where(torch.rand(w.scale.shape, generator=gen(1), device="cuda") < 0.5, top, 1.0).to(BF))
    x = torch.zeros((m, k), dtype=BF, device="cuda")
    at = torch.randint(0, k, (m,), generator=gen(2), device="cuda")
    x[torch.arange(m, device="cuda"), at] = (2.0 ** -100 * (1 + torch.randint(0, 128, (m,), generator=gen(3), device="cuda") / 128)).to(BF)
    y = torch.empty((m, n), dtype=F32, device="cuda")
    api.w4_linear(w, x, y)
    want, _ = w4_want(w, x)
    assert_close(host(y), want, half_step(F32) * np.abs(want))
    x *= 2.0 ** 100
    w.scale.fill_(2.0 ** -100)
    api.w4_linear(w, x, y)
    want, _ = w4_want(w, x)
    assert_close(host(y), want, half_step(F32) * np.abs(want))


@pytest.mark.parametrize("hq,dtype,d", SEEN)
def test_attention_infinities_without_a_mask_and_on_bad_pages(hq, dtype, d):
    """Chains without a mask; infinities on a page that no row sees any more stay out."""
    c = Attn(85, [600, 40], [4, 2], hq, 2, d, 32, dtype, dtype, masks="chain")
    clean, clean_lse = c.call()
    inf, t = float("inf"), c.table
    c.cache.v[int(t[0, 3]), :, 5, ::4] = -inf
    c.cache.v[int(t[1, 40 // 32]), :, 40 % 32, 1::4] = inf       # node 0 of request 1: seen by both rows
    c.cache.v[int(t[1, 41 // 32]), :, 41 % 32, 2::4] = inf       # node 1: by itself
    out, lse = c.call(mask=None)
    assert torch.equal(lse, clean_lse)
    assert (out[:4, :, ::4] == -inf).all() and all(torch.equal(out[:4, :, i::4], clean[:4, :, i::4]) for i in (1, 2, 3))
    assert (out[4:, :, 1::4] == inf).all() and all(torch.equal(out[4:, :, i::4], clean[4:, :, i::4]) for i in (0, 3))
    assert (out[5, :, 2::4] == inf).all() and torch.equal(out[4, :, 2::4], clean[4, :, 2::4])
    table = t.copy()
    table[0, 3] = -1
    hidden, _ = c.call(mask=None, table=table, status=i32([0]))
    assert torch.isfinite(hidden[:4]).all()
