"""GPU parity of the linear-attention sub-layer (rows of requests, trees, accepted paths, norms between sub-layers)
against the float64 oracle.

Tolerances, derived from the arithmetic the entry points promise, u = 2^-24 (fp32) and 2^-8 (bf16) being half a step:
* a state after n rows: a row's update rounds the decayed state, the product and their sum and the factor e^g, at most 4 u of the
  magnitudes then in the state, and these decay with it: 4 u `chain`. Rows taken together in chunks: a factor e^(sum of g) is off
  by at most 2^-21, a sum of tensor-core products in at most 32 chained additions by 2^-18 of the magnitudes, and the
  additions between chunks are fewer than those between rows: 2^-18 `size` + 4 u `chain` covers both.
* an output: the same error of what it reads, and for rows taken together one rounding of each term to bf16 (the scores
  beside the values, and the state): 2^-8 `bound`; trees: terms in 16 bits and the rest in 16 more: 2^-14 `bound`; then its own
  rounding to bf16, 2^-8 of itself.
* norms: sums of at most 16,384 squares by at most 64 chained additions of a thread and 20 between threads, the root, the
  products: below 128 u of the magnitudes, half of it through the root; then the output's own rounding. A sum that is off by
  its own rounding moves x by as much.
"""

import numpy as np
import pytest
import torch

from moe_decode_weight_gb300 import api
from oracle import linear as OL

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def host(t):
    return t.detach().to(torch.float64).cpu().numpy()


def assert_close(got, want, tol, what=""):
    got = np.asarray(got, np.float64)
    bad = ~((np.abs(got - want) <= tol) | ((got == want) & np.isinf(want)))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], np.asarray(want)[bad][:4])


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Inputs of requests with the given rows, q, k and v as slices of one buffer's rows, and three more rows behind the last."""

    def __init__(self, seed, lens, hk=2, h=4, d=128, steps=True, fresh=(), inplace=True, rate=0.3, lead=0, tail=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.h, self.d, self.hk = lens, h, d, hk
        n, b = sum(lens), len(lens)
        self.t, self.b = lead + n + tail, b
        self.start = np.concatenate([[lead], lead + np.cumsum(lens)])
        buf = torch.randn((self.t, (2 * hk + h) * d + 24), generator=g, device="cuda").to(BF)
        self.q = buf[:, 8:8 + hk * d].unflatten(1, (hk, d))
        self.k = buf[:, 8 + hk * d:8 + 2 * hk * d].unflatten(1, (hk, d))
        self.v = buf[:, 8 + 2 * hk * d:8 + (2 * hk + h) * d].unflatten(1, (h, d))
        self.g = -rate * torch.rand((self.t, h), generator=g, device="cuda") if steps else -rate * torch.rand(h, generator=g, device="cuda")
        slots = 2 * b + 2
        self.pool = torch.randn((slots, h, d, d), generator=g, device="cuda")
        order = np.random.RandomState(seed).permutation(slots)
        self.slot_in = [-1 if i in fresh else int(order[i]) for i in range(b)]
        self.slot_out = [int(order[i] if inplace else order[b + i]) for i in range(b)]
        self.out = torch.full((self.t, h, d), 7.0, dtype=BF, device="cuda")
        self.new = max(max(lens), 1)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rows(self, b):
        at = slice(int(self.start[b]), int(self.start[b + 1]))
        g = self.g[at] if self.g.dim() == 2 else self.g.expand(at.stop - at.start, self.h)
        return at, host(self.q[at]), host(self.k[at]), host(self.v[at]), host(g)

    def before(self, b, pool):
        s = self.slot_in[b]
        return np.zeros((self.h, self.d, self.d)) if s < 0 else pool[s]

    def call(self, new=None, scale=None, stream=None, **kw):
        st = api.LinearState(self.pool)
        new = new or self.new
        n = api.mdw_linear_attention_workspace_bytes(st, self.b, self.t, self.hk, new)
        ws = torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
        a = dict(start=i32(self.start.tolist()), slot_in=i32(self.slot_in), slot_out=i32(self.slot_out)) | kw
        api.mdw_linear_attention(st, self.q, self.k, self.v, self.g, self.out, a["start"], a["slot_in"], a["slot_out"], new, ws,
                                 scale=scale, status=self.status, stream=stream)

    def tree(self, masks, new=None, **kw):
        a = dict(start=i32(self.start.tolist()), slot_in=i32(self.slot_in)) | kw
        m = None if masks is None else torch.from_numpy(np.array(masks, dtype=np.uint64).view(np.int64)).cuda()
        api.mdw_linear_tree_attention(api.LinearState(self.pool), self.q, self.k, self.v, self.g, self.out, a["start"], a["slot_in"],
                                      new or self.new, tree_mask=m, status=self.status)

    def advance(self, accepted, new=None, **kw):
        a = dict(start=i32(self.start.tolist()), slot_in=i32(self.slot_in), slot_out=i32(self.slot_out)) | kw
        m = torch.from_numpy(np.array(accepted, dtype=np.uint64).view(np.int64)).cuda()
        api.mdw_linear_state_advance(api.LinearState(self.pool), self.k, self.v, self.g, a["start"], m, a["slot_in"], a["slot_out"],
                                     new or self.new, status=self.status)


def check_rows(c, pool0, scale=None, skip=()):
    """Outputs, states, and that nothing else was written."""
    scale = c.d ** -0.5 if scale is None else scale
    pool, out = host(c.pool), host(c.out)
    written = set()
    for b in range(c.b):
        at, q, k, v, g = c.rows(b)
        if b in skip:
            assert (out[at] == 7).all()
            continue
        o, s, bound, size, chain = OL.linear_attention(c.before(b, pool0), q, k, v, g, scale)
        assert_close(out[at], o, half_step(BF) * np.abs(o) + (2.0 ** -8 + 2.0 ** -17) * bound + abs(scale) * 4 * U * np.einsum(
            "nhi,hij->nhj", np.repeat(np.abs(q), c.h // c.hk, 1), chain), ("out", b))
        if c.slot_out[b] >= 0:
            assert_close(pool[c.slot_out[b]], s, 2.0 ** -18 * size + 4 * U * chain, ("state", b))
            written.add(c.slot_out[b])
    for s in range(len(pool)):
        if s not in written:
            assert np.array_equal(pool[s], pool0[s]), ("slot", s)
    assert (out[:c.start[0]] == 7).all() and (out[c.start[-1]:] == 7).all()


LENS = [[1], [1, 1, 1, 1, 1], [4, 0, 1, 7], [8, 9, 16, 17], [15, 31, 33, 1, 63], [64, 65, 127, 1], [128, 129, 0, 2], [255, 256, 257],
        [300, 5, 700], [16, 1, 0, 12], [13, 15, 2, 9, 0, 16, 14]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("hk,h,d,steps", [(2, 4, 128, True), (1, 3, 64, False), (3, 3, 128, False), (2, 2, 64, True)])
def test_rows(lens, hk, h, d, steps):
    c = Case(sum(lens), lens, hk, h, d, steps, fresh=(1,), inplace=len(lens) % 2 == 0)
    before = host(c.pool)
    c.call()
    check_rows(c, before)
    assert int(c.status) == 0


@pytest.mark.parametrize("n,h,d,rate", [(2500, 1, 128, 0.01), (1537, 2, 64, 0.001), (1100, 2, 128, 30.0)])
def test_long_prompts(n, h, d, rate):
    """Slow decays, over which every row still counts at the end, and fast ones, whose products underflow."""
    c = Case(n, [n], h, h, d, True, rate=rate)
    before = host(c.pool)
    c.call()
    check_rows(c, before)


@pytest.mark.parametrize("new", [1, 16, 17, 64, 100, 129, 1000, 1 << 20])
def test_a_bound_above_the_rows_changes_no_result_beyond_rounding(new):
    lens = [min(n, new) for n in (3, 17, 90)]
    c = Case(5, lens, 2, 4, 64)
    before = host(c.pool)
    c.call(new=new)
    check_rows(c, before)


@pytest.mark.parametrize("lens", [[5, 2, 30], [200, 140], [16, 12]], ids=str)
def test_decays_that_forget(lens):
    """A decay of 0 forgets what was before, and the rows after it count on."""
    c = Case(3, lens, 2, 2, 128)
    c.g[int(c.start[0]) + 2] = -float("inf")
    c.g[int(c.start[1]) - 1, 0] = -float("inf")
    c.g[int(c.start[1]), 1] = -1e30
    c.g[int(c.start[1]) + 1] = 0.0
    before = host(c.pool)
    c.call()
    check_rows(c, before)
    assert torch.isfinite(c.out).all() and torch.isfinite(c.pool).all()


@pytest.mark.parametrize("scale", [1.0, -2.5, 0.0])
def test_scale(scale):
    c = Case(4, [3, 150], 2, 2, 64)
    before = host(c.pool)
    c.call(scale=scale)
    check_rows(c, before, scale)


@pytest.mark.parametrize("lens", [[2, 0, 3], [140, 0, 1, 200], [14, 0, 3]], ids=str)
def test_states_not_stored_copied_and_elsewhere(lens):
    c = Case(6, lens, 1, 2, 128, inplace=False, fresh=(0,))
    c.slot_out[0] = -1
    before = host(c.pool)
    c.call()
    check_rows(c, before)
    # a request without rows copies its state (zeros from no slot)
    c.slot_in[1] = -1
    before = host(c.pool)
    c.out.fill_(7)
    c.call()
    check_rows(c, before)
    assert not c.pool[c.slot_out[1]].any()


def test_two_requests_may_read_one_slot():
    for lens in ([3, 4], [150, 130]):
        c = Case(7, lens, 2, 2, 64, inplace=False)
        c.slot_in[1] = c.slot_in[0]
        before = host(c.pool)
        c.call()
        check_rows(c, before)


@pytest.mark.parametrize("lens", [[4, 3, 2, 5], [140, 3, 200, 150], [14, 3, 12, 5]], ids=str)
@pytest.mark.parametrize("fault,skip", [("out", (0, 2)), ("in", (0,)), ("high", (1,)), ("low", (2,)), ("rows", (3,)), ("back", (1, 2))])
def test_bad_requests_are_skipped(lens, fault, skip):
    c = Case(8, lens, 2, 2, 64, inplace=False)
    start = c.start.copy()
    if fault == "out":                                      # two requests store to one slot
        c.slot_out[2] = c.slot_out[0]
    elif fault == "in":                                     # one reads what another stores
        c.slot_in[0] = c.slot_out[2]
    elif fault == "high":
        c.slot_in[1] = len(c.pool)
    elif fault == "low":
        c.slot_out[2] = -2
    elif fault == "rows":                                   # rows behind the last
        start[-1] = c.t + 1
    else:                                                   # rows that run backwards, and the next request's that are then too many
        start[2] = start[1] - 1
        c.new = max(lens)
        skip = (1,) if start[3] - start[2] <= c.new else (1, 2)
    before = host(c.pool)
    c.call(start=i32(start.tolist()))
    assert int(c.status) == 7
    pool, out = host(c.pool), host(c.out)
    for b in range(c.b):
        at, q, k, v, g = c.rows(b)
        if b in skip:
            if fault != "back":
                assert (out[at] == 7).all()
        elif fault != "back" or b != 2:
            o, s, bound, size, chain = OL.linear_attention(c.before(b, before), q, k, v, g, c.d ** -0.5)
            assert_close(out[at][:1], o[:1], half_step(BF) * np.abs(o[:1]) + 2.0 ** -7 * bound[:1])
            assert_close(pool[c.slot_out[b]], s, 2.0 ** -18 * size + 4 * U * chain)
    if fault in ("out", "in"):
        assert np.array_equal(pool[c.slot_out[0]], before[c.slot_out[0]])


def test_too_many_rows_are_refused_on_the_device():
    for lens, new in (([3, 9], 4), ([100, 300], 200)):
        c = Case(9, lens, 1, 1, 64)
        before = host(c.pool)
        c.call(new=new)
        assert int(c.status) == 7
        assert (host(c.out)[c.start[1]:] == 7).all()
        assert np.array_equal(host(c.pool)[c.slot_out[1]], before[c.slot_out[1]])


@pytest.mark.parametrize("what", ["q", "k", "v"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("lens,row", [([6, 3], 4), ([6, 3], 0), ([16, 3], 4), ([13, 5], 12), ([300, 140], 190), ([140, 20], 0), ([129, 3], 128)], ids=str)
def test_values_that_are_not_finite_reach_no_earlier_row(what, value, lens, row):
    c = Case(10, lens, 2, 2, 128, lead=2)
    clean = Case(10, lens, 2, 2, 128, lead=2)
    at = int(c.start[0]) + row
    {"q": c.q, "k": c.k, "v": c.v}[what][at, 1, 5] = value
    # rows outside the requests hold anything
    for t in (c.q, c.k, c.v):
        t[:2] = value
        t[int(c.start[-1]):] = value
    before = host(c.pool)
    c.call()
    clean.call()
    got, want = host(c.out), host(clean.out)
    rest = np.ones(c.t, bool)
    rest[at:at + 1 if what == "q" else int(c.start[1])] = False
    assert np.array_equal(got[rest], want[rest])            # earlier rows and other requests: bit for bit
    assert np.array_equal(got[:, 0], want[:, 0])            # the other head
    row_now = got[at, 1]
    if what == "v":
        assert not np.isfinite(row_now[5]) and np.array_equal(np.delete(got[:, 1], 5, 1), np.delete(want[:, 1], 5, 1))
        assert not np.isfinite(got[at:int(c.start[1]), 1, 5]).any()
    else:
        assert not np.isfinite(row_now).all()
    pool = host(c.pool)
    assert np.array_equal(pool[c.slot_out[1]], host(clean.pool)[c.slot_out[1]])
    if what == "q":
        assert np.array_equal(pool, host(clean.pool))
    elif what == "v":
        assert not np.isfinite(pool[c.slot_out[0], 1, :, 5]).all()
        assert np.isfinite(np.delete(pool[c.slot_out[0], 1], 5, 1)).all()
    else:
        assert not np.isfinite(pool[c.slot_out[0], 1, 5]).any()
        assert np.isfinite(np.delete(pool[c.slot_out[0], 1], 5, 0)).all()
    assert np.isfinite(before).all()


@pytest.mark.parametrize("lens", [[1, 3], [700, 1, 130], [16, 2, 13]], ids=str)
def test_calls_repeat_bit_for_bit(lens):
    results = []
    for _ in range(3):
        c = Case(11, lens, 2, 4, 128)
        c.call()
        results.append((c.out, c.pool))
    assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(r, results[0]))


@pytest.mark.parametrize("lens", [[2, 3], [400, 1, 130], [12, 0, 15]], ids=str)
def test_captured_calls_on_a_stream_of_their_own(lens):
    """Two captured calls with workspaces of their own replay on new inputs, as eager calls give them."""
    a, b = Case(12, lens, 2, 2, 128), Case(13, lens, 2, 2, 128)
    args = []
    for c in (a, b):
        st = api.LinearState(c.pool)
        n = api.mdw_linear_attention_workspace_bytes(st, c.b, c.t, c.hk, c.new)
        args.append((st, c.q, c.k, c.v, c.g, c.out, i32(c.start.tolist()), i32(c.slot_in), i32(c.slot_out), c.new,
                     torch.empty(n, dtype=torch.uint8, device="cuda")))
    saved = [c.pool.clone() for c in (a, b)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for x in args:
            api.mdw_linear_attention(*x)
    a.q.copy_(b.q)
    for c, p in zip((a, b), saved):
        c.pool.copy_(p)
    graph.replay()
    torch.cuda.synchronize()
    for c, p in zip((a, b), saved):
        out, pool = c.out.clone(), c.pool.clone()
        c.pool.copy_(p)
        c.call()
        assert torch.equal(out, c.out) and torch.equal(pool, c.pool)


def test_expanded_decays_and_single_rows():
    """Decays of all rows from one row, as a tensor without a row stride; one row whose stride says nothing."""
    c = Case(14, [5, 40], 2, 2, 64, steps=False)
    before = host(c.pool)
    c.g = c.g.expand(c.t, c.h)
    c.call()
    check_rows(c, before)
    c = Case(15, [1], 2, 2, 64, tail=0)
    before = host(c.pool)
    c.call()
    check_rows(c, before)


def test_strided_slots():
    c = Case(16, [4, 130], 2, 2, 64)
    full = torch.full((len(c.pool), 3, 64, 64), 5.0, device="cuda")
    full[:, :2] = c.pool
    c.pool = full[:, :2]
    before = host(c.pool)
    c.call()
    check_rows(c, before)
    assert (full[:, 2] == 5).all()


def test_slots_beyond_4_gigabytes():
    """A pool whose last slot starts behind 2^32 bytes."""
    d, h = 128, 64
    slots = (1 << 32) // (h * d * d * 4) + 2
    c = Case(17, [3, 140], h, h, d)
    pool = torch.empty((slots, h, d, d), device="cuda")
    pool[-2:] = c.pool[:2]
    c.pool = pool
    c.slot_in, c.slot_out = [slots - 1, slots - 2], [slots - 1, slots - 2]
    before = [host(pool[s]) for s in c.slot_in]
    c.call()
    for b in range(2):
        at, q, k, v, g = c.rows(b)
        _, s, _, size, chain = OL.linear_attention(before[b], q, k, v, g, 1.0)
        assert_close(host(pool[c.slot_out[b]]), s, 2.0 ** -18 * size + 4 * U * chain)


@pytest.mark.parametrize("lens", [[1024], [1025, 3], [1500, 0, 1200], [13 * 128 + 1, 17], [2 * 2048 + 77]], ids=str)
@pytest.mark.parametrize("h,d", [(1, 128), (2, 64)])
def test_segments_of_every_length(lens, h, d):
    """Requests long enough to be cut into segments, of 4 chunks and on, stored to the slots that they were read from."""
    c = Case(sum(lens), lens, h, h, d, True, rate=0.01)
    before = host(c.pool)
    c.call()
    check_rows(c, before)


@pytest.mark.parametrize("lens", [[5, 200], [130, 1]], ids=str)
def test_outputs_off_32_byte_boundaries(lens):
    c = Case(18, lens, 2, 2, 128)
    buf = torch.full((c.t, 2 * 128 + 24), 7.0, dtype=BF, device="cuda")
    c.out = buf[:, 8:8 + 256].unflatten(1, (2, 128))
    before = host(c.pool)
    c.call()
    check_rows(c, before)
    assert (buf[:, :8] == 7).all() and (buf[:, 264:] == 7).all()


@pytest.mark.parametrize("b", [300, 4096])
def test_many_requests(b):
    lens = [(1, 0, 2, 17, 1, 16, 130, 1)[i * 5 % 8] if i < 300 else i % 2 for i in range(b)]
    c = Case(19, lens, 1, 1, 64)
    before = host(c.pool)
    c.call()
    check_rows(c, before)
    assert int(c.status) == 0


def test_workspace_of_two_captured_calls():
    """One workspace serves captured calls that replay one after the other, in either order."""
    a, b = Case(20, [1300, 2, 140], 2, 2, 64), Case(21, [200, 40], 2, 2, 64, inplace=False)
    ws = torch.empty(max(api.mdw_linear_attention_workspace_bytes(api.LinearState(c.pool), c.b, c.t, c.hk, c.new) for c in (a, b)),
                     dtype=torch.uint8, device="cuda")
    saved = [c.pool.clone() for c in (a, b)]
    args = [(api.LinearState(c.pool), c.q, c.k, c.v, c.g, c.out, i32(c.start.tolist()), i32(c.slot_in), i32(c.slot_out), c.new, ws) for c in (a, b)]
    torch.cuda.synchronize()
    graphs = []
    for x in args:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            api.mdw_linear_attention(*x)
    for order in ((0, 1), (1, 0), (0, 0)):
        for i in order:
            c = (a, b)[i]
            c.pool.copy_(saved[i])
            c.out.fill_(7)
            graphs[i].replay()
            torch.cuda.synchronize()
            check_rows(c, host(saved[i]))


@pytest.mark.parametrize("lens", [[300, 2], [1500]], ids=str)
def test_a_wait_that_runs_out(lens):
    """With a budget of one cycle the first wait of a block gives up: a status word, no fault, and the next call is right."""
    c = Case(22, lens, 2, 2, 128)
    previous = api.mdw_debug_set_spin_budget(1)
    try:
        c.call()
    finally:
        api.mdw_debug_set_spin_budget(previous)
    torch.cuda.synchronize()
    assert int(c.status) == 6                                  # MDW_ERR_TIMEOUT
    c = Case(22, lens, 2, 2, 128)
    before = host(c.pool)
    c.call()
    check_rows(c, before)
    assert int(c.status) == 0


@pytest.mark.parametrize("h,d,lens", [(40, 64, [16, 3, 12, 0] * 5), (32, 128, [1, 14, 15] * 4)], ids=str)
def test_windows_of_many_heads(h, d, lens):
    """More units than blocks, with requests without rows and from empty states among them."""
    c = Case(23, lens, h // 2, h, d, fresh=(0, 3, 4), inplace=False)
    before = host(c.pool)
    c.call(new=16)
    check_rows(c, before)
    assert int(c.status) == 0


def test_a_state_of_many_windows():
    """Errors of 80 windows of 16 rows, with decays so slow that all of them count."""
    n, d = 80, 64
    c = Case(24, [16 * n], 1, 1, d, rate=0.0005, tail=0)
    first = host(c.pool)
    for i in range(n):
        at = slice(16 * i, 16 * i + 16)
        st = api.LinearState(c.pool)
        ws = torch.empty(api.mdw_linear_attention_workspace_bytes(st, 1, 16, 1, 16), dtype=torch.uint8, device="cuda")
        api.mdw_linear_attention(st, c.q[at], c.k[at], c.v[at], c.g[at], c.out[at], i32([0, 16]), i32(c.slot_in), i32(c.slot_out), 16, ws)
    check_rows(c, first)


# ------------------------------------------------------------------------------ trees


def random_masks(rng, n):
    m = []
    for i in range(n):
        p = int(rng.integers(-1, i)) if i else -1
        m.append((m[p] if p >= 0 else 0) | 1 << i)
    return m


@pytest.mark.parametrize("lens", [[1], [4], [1, 7, 8, 9, 0], [16, 3, 15, 17], [33, 64, 63, 31, 2, 48]], ids=str)
@pytest.mark.parametrize("hk,h,d,steps", [(2, 4, 128, True), (1, 3, 64, False), (2, 2, 128, False), (3, 3, 64, True)])
@pytest.mark.parametrize("chain", [False, True])
def test_trees(lens, hk, h, d, steps, chain):
    c = Case(sum(lens) + h, lens, hk, h, d, steps, fresh=(2,), rate=1.0, lead=1)
    rng = np.random.default_rng(sum(lens))
    masks = [m for n in lens for m in random_masks(rng, n)]
    dirty = [(m | (int(rng.integers(0, 1 << 30)) << 34 & ~((2 << j) - 1))) & ~(1 << j if rng.random() < 0.5 else 0) & (1 << 64) - 1
             for n, at in zip(lens, np.cumsum([0] + lens)) for j, m in enumerate(masks[at:at + n])]
    before = c.pool.clone()
    c.tree(None if chain else [0] + dirty + [0] * 3)
    out, at = host(c.out), 0
    for b, n in enumerate(lens):
        rows, q, k, v, g = c.rows(b)
        m = [(2 << j) - 1 for j in range(n)] if chain else masks[at:at + n]
        at += n
        o, bound = OL.tree_attention(c.before(b, host(before)), q, k, v, g, m, d ** -0.5)
        assert_close(out[rows], o, half_step(BF) * np.abs(o) + 2.0 ** -14 * bound, b)
    assert torch.equal(c.pool, before) and int(c.status) == 0
    assert (out[:1] == 7).all() and (out[c.start[-1]:] == 7).all()


def test_tree_refuses_bad_requests_and_keeps_the_others():
    c = Case(20, [5, 6, 70, 3], 2, 2, 64)
    c.slot_in[0] = len(c.pool)
    c.tree(None, new=64)
    assert int(c.status) == 7
    out = host(c.out)
    for b in (0, 2):
        assert (out[c.rows(b)[0]] == 7).all()
    for b in (1, 3):
        rows, q, k, v, g = c.rows(b)
        o, bound = OL.tree_attention(c.before(b, host(c.pool)), q, k, v, g, [(2 << j) - 1 for j in range(len(q))], 0.125)
        assert_close(out[rows], o, half_step(BF) * np.abs(o) + 2.0 ** -14 * bound)


@pytest.mark.parametrize("what", ["q", "k", "v"])
@pytest.mark.parametrize("n", [6, 40])
def test_tree_values_that_are_not_finite_reach_only_what_comes_after(what, n):
    c, clean = Case(21, [n, 3], 2, 2, 64), Case(21, [n, 3], 2, 2, 64)
    masks = random_masks(np.random.default_rng(4), n) + [1, 3, 5] + [0] * 3
    {"q": c.q, "k": c.k, "v": c.v}[what][2, 1, 5] = float("inf")
    for t in (c.q, c.k, c.v):
        t[int(c.start[-1]):] = float("nan")
    c.tree(masks)
    clean.tree(masks)
    got, want = host(c.out), host(clean.out)
    after = [i for i in range(n) if (masks[i] >> 2 & 1 if what != "q" else i == 2)]
    rest = [i for i in range(c.t) if i not in after]
    assert np.array_equal(got[rest], want[rest]) and np.array_equal(got[:, 0], want[:, 0])
    for i in after:
        assert not np.isfinite(got[i, 1, 5] if what == "v" else got[i, 1]).all()


def test_tree_forgets_at_a_decay_of_zero():
    c = Case(22, [20], 1, 2, 128)
    c.g[3], c.g[7, 1] = -float("inf"), -1e30
    masks = random_masks(np.random.default_rng(5), 20)
    c.tree(masks + [0] * 3)
    rows, q, k, v, g = c.rows(0)
    o, bound = OL.tree_attention(host(c.pool)[c.slot_in[0]], q, k, v, g, masks, 128 ** -0.5)
    assert_close(host(c.out)[rows], o, half_step(BF) * np.abs(o) + 2.0 ** -14 * bound)


# ------------------------------------------------------------------------------ accepted paths


@pytest.mark.parametrize("lens", [[1], [4, 7, 0, 16], [64, 63, 20, 33, 2]], ids=str)
@pytest.mark.parametrize("hk,h,d,steps,inplace", [(2, 4, 128, True, True), (1, 3, 64, False, False), (40, 40, 64, True, False)])
def test_advance(lens, hk, h, d, steps, inplace):
    c = Case(sum(lens), lens, hk, h, d, steps, fresh=(1,), inplace=inplace, lead=2)
    rng = np.random.default_rng(1)
    accepted = [int(rng.integers(0, 1 << 63)) << 1 | 1 for _ in lens]          # (bits behind the rows are not looked at)
    accepted[-1] = 0
    before = host(c.pool)
    c.advance(accepted)
    pool = host(c.pool)
    for b in range(c.b):
        _, q, k, v, g = c.rows(b)
        s, size = OL.advance(c.before(b, before), k, v, g, accepted[b])
        assert_close(pool[c.slot_out[b]], s, 4 * U * (len(k) + 1) * size, b)
    for s in set(range(len(pool))) - set(c.slot_out):
        assert np.array_equal(pool[s], before[s])
    assert int(c.status) == 0


def test_advance_refuses_slots_in_conflict():
    c = Case(24, [4, 4, 4], 2, 2, 64, inplace=False)
    c.slot_in[1] = c.slot_out[0]
    before = host(c.pool)
    c.advance([3, 3, 3])
    assert int(c.status) == 7
    pool = host(c.pool)
    assert np.array_equal(pool[c.slot_out[1]], before[c.slot_out[1]])
    for b in (0, 2):
        _, _, k, v, g = c.rows(b)
        s, size = OL.advance(c.before(b, before), k, v, g, 3)
        assert_close(pool[c.slot_out[b]], s, 8 * U * size)


def test_advance_of_a_whole_chain_is_the_state_of_its_rows():
    a, b = Case(25, [9, 3], 2, 4, 128), Case(25, [9, 3], 2, 4, 128)
    a.call()
    b.advance([(1 << 9) - 1, 7])
    assert torch.equal(a.pool, b.pool)


# ------------------------------------------------------------------------------ norms between sub-layers


def norm_case(seed, t, w, x=BF, y=None, group=None, post=True, kind="none", rows=True, res=None, pre=True, pad=0, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def make(shape, dtype, scale=1.0):
        full = torch.randn((*shape[:-1], shape[-1] + pad + shift), generator=g, device="cuda").mul(scale).to(dtype)
        return full[..., shift:shift + shape[-1]]

    a = dict(y=make((t, w), y or x, 3.0), post_weight=make((group or w,), x).add(1).contiguous() if post else None, group=group,
             gate=None if kind == "none" else make((t, w), x, 2.0) if rows else make((w,), x, 2.0).contiguous(), gate_kind=kind, residual=None if res is None else make((t, w), res, 5.0), pre_weight=make((w,), x).add(1).contiguous() if pre else None)
    sum_type = res or x
    a["sum"] = torch.full((t + 1, w + pad + shift), 9.0, dtype=sum_type, device="cuda")[:t, shift:shift + w]
    a["x"] = torch.full((t + 1, w + pad + shift), 9.0, dtype=x, device="cuda")[:t, shift:shift + w] if pre else None
    return a


def check_norm(a, want_y=None, want_r=None, branch_scale=1.0, residual_scale=1.0, eps=1e-6, got_sum=None, got_x=None):
    y = host(a["y"]) if want_y is None else want_y
    r = None if a["residual"] is None else host(a["residual"]) if want_r is None else want_r
    n = lambda t: None if t is None else host(t)  # noqa: E731
    s, size = OL.block_sum(y, n(a["post_weight"]), a["group"], n(a["gate"]), a["gate_kind"], r, branch_scale, residual_scale, eps)
    got = host(a["sum"]) if got_sum is None else got_sum
    step = half_step(a["sum"].dtype)
    assert_close(got, s, step * np.abs(s) + 128 * U * size + 2.0 ** -24, "sum")
    if a["x"] is not None:
        # x is of the sum as it is stored
        x = OL.rmsnorm(got, host(a["pre_weight"]), eps)
        assert_close(host(a["x"]) if got_x is None else got_x, x, (half_step(a["x"].dtype) + 128 * U) * np.abs(x) + 2.0 ** -24, "x")


@pytest.mark.parametrize("w", [1, 2, 7, 8, 64, 100, 128, 255, 256, 264, 1000, 2560, 4104, 8192, 8200, 16383, 16384])
@pytest.mark.parametrize("t", [1, 5])
def test_norm_widths(t, w):
    for x, y, res, kind, rows in ((BF, None, BF, "none", True), (HF, F32, None, "sigmoid", True), (BF, F32, F32, "silu", False),
                                  (HF, None, F32, "mul", True)):
        a = norm_case(w + t, t, w, x, y, None, True, kind, rows, res)
        api.mdw_block_norm(**a, branch_scale=0.5, residual_scale=-0.75, eps=1e-5)
        check_norm(a, branch_scale=0.5, residual_scale=-0.75, eps=1e-5)


@pytest.mark.parametrize("group,w", [(64, 64), (64, 192), (128, 128), (128, 2560), (64, 8320), (128, 16384)])
@pytest.mark.parametrize("pre,res", [(False, None), (True, BF)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (3, 1)])
def test_norm_of_heads(group, w, pre, res, pad, shift):
    a = norm_case(w, 9, w, BF, None, group, True, "sigmoid", True, res, pre, pad, shift)
    api.mdw_block_norm(**a)
    check_norm(a)


@pytest.mark.parametrize("pad,shift", [(8, 0), (5, 0), (7, 3), (0, 8), (16, 8)])
@pytest.mark.parametrize("w", [512, 513, 2560])
def test_norm_strides_and_alignment(w, pad, shift):
    """Rows at any place; what lies between them stays."""
    a = norm_case(w + pad, 6, w, HF, None, None, True, "silu", True, HF, True, pad, shift)
    api.mdw_block_norm(**a)
    check_norm(a)
    for t in (a["sum"], a["x"]):
        base = t._base
        assert (base[:, :shift] == 9).all() and (base[:, shift + w:] == 9).all() and (base[6:] == 9).all()


@pytest.mark.parametrize("post,kind,res,pre", [(False, "none", None, False), (False, "mul", BF, False), (False, "none", BF, True),
                                               (True, "none", None, True), (False, "sigmoid", None, True)])
def test_norm_parts(post, kind, res, pre):
    a = norm_case(1, 7, 1000, BF, None, None, post, kind, True, res, pre)
    api.mdw_block_norm(**a, branch_scale=2.0)
    check_norm(a, branch_scale=2.0)


@pytest.mark.parametrize("kind", ["mul", "sigmoid", "silu"])
def test_norm_gates_of_all_sizes(kind):
    """Gates whose exponentials overflow or vanish: a product with the gate alone would be infinite times zero."""
    values = [-3e38, -1e5, -200.0, -89.0, -88.0, -30.0, -1e-30, 0.0, 1e-30, 30.0, 88.0, 200.0, 1e5, 3e38]
    a = norm_case(2, 3, 16 * len(values), post=False, kind=kind, pre=False)
    a["y"].clamp_(-0.5, 0.5)
    a["y"][:, ::2] *= 1.0 if kind == "mul" else -1.0
    a["gate"].copy_(torch.tensor(values, device="cuda").repeat_interleave(16).to(BF).expand(3, -1))
    with np.errstate(over="ignore"):
        api.mdw_block_norm(**a)
        check_norm(a)
    if kind == "silu":
        b = norm_case(2, 1, 16, post=False, kind=kind, pre=False)
        b["y"].fill_(2.0 ** 100)
        b["gate"].fill_(-2.0 ** 100)
        api.mdw_block_norm(**b)
        assert (b["sum"] == 0).all()


def test_norm_without_the_sum():
    a = norm_case(2, 3, 640, BF, None, None, True, "none", True, BF, True)
    b = dict(a)
    api.mdw_block_norm(**a)
    b["sum"], b["x"] = None, torch.empty_like(a["x"])
    api.mdw_block_norm(**b)
    assert torch.equal(a["x"], b["x"])


@pytest.mark.parametrize("w", [1000, 2560, 129])
def test_norm_in_place(w):
    a = norm_case(3, 11, w, BF, None, None, True, "silu", True, BF, True)
    y, r = host(a["y"]), host(a["residual"])
    a["sum"], a["x"] = a["residual"], a["y"]
    api.mdw_block_norm(**a)
    check_norm(a, want_y=y, want_r=r)
    a = norm_case(4, 11, w, BF, None, None, True, "mul", False, None, False)
    y = host(a["y"])
    a["sum"] = a["y"]
    api.mdw_block_norm(**a)
    check_norm(a, want_y=y)


def test_norm_rows_are_apart_and_zeros_stay():
    a = norm_case(5, 300, 256, BF, None, None, True, "none", True, BF, True)
    a["y"][3], a["residual"][3] = 0, 0
    a["y"][7, 11] = float("nan")
    a["y"][9, 11] = float("inf")
    api.mdw_block_norm(**a)
    keep = [i for i in range(300) if i not in (7, 9)]
    assert not a["sum"][3].any() and not a["x"][3].any()
    assert torch.isnan(a["x"][7]).all() and not torch.isfinite(a["sum"][9]).all()
    b = {k: v[keep] if isinstance(v, torch.Tensor) and v.dim() == 2 else v for k, v in a.items()}
    check_norm(b)


def test_norm_refuses_mixed_types():
    a = norm_case(6, 2, 64, BF, None, None, True, "none", True, BF, True)
    for key, t in (("post_weight", a["post_weight"].half()), ("x", a["x"].half()), ("residual", a["residual"].float())):
        with pytest.raises(api.MdwError):
            api.mdw_block_norm(**(a | {key: t}))


def test_norm_captured_on_a_stream_of_its_own():
    a = norm_case(7, 33, 2560, BF, None, None, True, "sigmoid", True, F32, True)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        api.mdw_block_norm(**a)
    a["y"].mul_(2)
    a["residual"].add_(1)
    graph.replay()
    torch.cuda.synchronize()
    check_norm(a)


# ------------------------------------------------------------------------------ together


def test_a_window_with_trees_as_a_program_runs_it():
    """Norm, int4 projection, plan of the trees, tree attention, gated norm of the heads, output projection, residual and next
    norm; then the accepted paths' states, and the next token from them. Each step is checked on what the steps before gave."""
    d, hk, h, width, b = 128, 2, 4, 512, 3
    g = torch.Generator(device="cuda").manual_seed(30)
    lens = [5, 1, 9]
    t, pad = sum(lens), 1                                        # at most 32 tokens a window
    rows = (2 * hk + 2 * h) * d
    codes = lambda n, k: torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    scales = lambda n, k: (torch.rand((n, k // 128), generator=g, device="cuda") * 0.01 + 0.002).to(BF)  # noqa: E731
    w_in, w_out = api.W4Weights(codes(rows, width), scales(rows, width)), api.W4Weights(codes(width, h * d), scales(width, h * d))
    resid = torch.randn((t + pad, width), generator=g, device="cuda").to(BF)
    ones = lambda n: (torch.rand(n, generator=g, device="cuda") + 0.5).to(BF)  # noqa: E731
    w_pre, w_head, w_post = ones(width), ones(d), ones(width)
    decay = -torch.rand(h, generator=g, device="cuda")
    pool = torch.randn((b + 1, h, d, d), generator=g, device="cuda")
    state, slots = api.LinearState(pool), i32([2, 0, 3])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(3)
    parents = np.concatenate([[-1 if i == 0 else int(rng.integers(0, i)) for i in range(n)] for n in lens] + [[0] * pad])

    x = torch.empty_like(resid)
    api.mdw_block_norm(resid, None, pre_weight=w_pre, x=x)
    assert_close(host(x), OL.rmsnorm(host(resid), host(w_pre), 1e-6), 2.0 ** -8 * np.abs(host(x)) * 1.01 + 1e-6)
    proj = torch.empty((t + pad, rows), dtype=BF, device="cuda")
    api.w4_linear(w_in, x, proj, status=status)
    q, k, v, gate = (proj[:, a * d:z * d] for a, z in ((0, hk), (hk, 2 * hk), (2 * hk, 2 * hk + h), (2 * hk + h, 2 * hk + 2 * h)))
    q, k, v = q.unflatten(1, (hk, d)), k.unflatten(1, (hk, d)), v.unflatten(1, (h, d))
    start, mask = torch.empty(b + 1, dtype=torch.int32, device="cuda"), torch.empty(t + pad, dtype=torch.int64, device="cuda")
    api.mdw_kv_plan(i32([40, 7, 0]), i32(lens), 16, 64, torch.zeros((b, 8), dtype=torch.int32, device="cuda"), i32(list(range(64))), start,
                    torch.empty(t + pad, dtype=torch.int64, device="cuda"), torch.empty(t + pad, dtype=torch.int32, device="cuda"),
                    torch.empty(1, dtype=torch.int32, device="cuda"), parents=i32(parents.tolist()), tree_mask=mask, status=status)
    o = torch.zeros((t + pad, h, d), dtype=BF, device="cuda")
    api.mdw_linear_tree_attention(state, q, k, v, decay, o, start, slots, 16, tree_mask=mask, status=status)
    begin, masks = [0, 5, 6, 15], mask.cpu().numpy().view(np.uint64)
    for i in range(b):
        at = slice(begin[i], begin[i + 1])
        want, bound = OL.tree_attention(host(pool)[int(slots[i])], host(q[at]), host(k[at]), host(v[at]),
                                        np.repeat(host(decay)[None], lens[i], 0), masks[at], d ** -0.5)
        assert_close(host(o[at]), want, 2.0 ** -8 * np.abs(want) + 2.0 ** -14 * bound)
    y = torch.empty((t + pad, h * d), dtype=BF, device="cuda")
    api.mdw_block_norm(o.flatten(1), y, post_weight=w_head, group=d, gate=gate, gate_kind="sigmoid")
    want, size = OL.block_sum(host(o.flatten(1)), host(w_head), d, host(gate), "sigmoid")
    assert_close(host(y), want, 2.0 ** -8 * np.abs(want) + 128 * U * size + 1e-7)
    z = torch.empty((t + pad, width), dtype=F32, device="cuda")
    api.w4_linear(w_out, y, z, status=status)
    after, nx = torch.empty_like(resid), torch.empty_like(resid)
    api.mdw_block_norm(z, after, post_weight=w_post, residual=resid, pre_weight=w_pre, x=nx)
    want, size = OL.block_sum(host(z), host(w_post), residual=host(resid))
    assert_close(host(after), want, 2.0 ** -8 * np.abs(want) + 128 * U * size + 1e-7)
    assert_close(host(nx), OL.rmsnorm(host(after), host(w_pre), 1e-6), 2.0 ** -8 * np.abs(host(nx)) * 1.01 + 1e-6)

    # the accepted paths: a node's mask is the way to it
    chosen = [3, 0, 8]
    accepted = mask[torch.tensor([begin[i] + chosen[i] for i in range(b)], device="cuda")].contiguous()
    before = host(pool)
    api.mdw_linear_state_advance(state, k, v, decay, start, accepted, slots, slots, 16, status=status)
    for i in range(b):
        at = slice(begin[i], begin[i + 1])
        want, size = OL.advance(before[int(slots[i])], host(k[at]), host(v[at]), np.repeat(host(decay)[None], lens[i], 0),
                                masks[begin[i] + chosen[i]])
        assert_close(host(pool)[int(slots[i])], want, 64 * U * size)
    # and the next token of each request from them
    before = host(pool)
    ws = torch.empty(api.mdw_linear_attention_workspace_bytes(state, b, b, hk, 1), dtype=torch.uint8, device="cuda")
    o = torch.empty((b, h, d), dtype=BF, device="cuda")
    api.mdw_linear_attention(state, q[:b], k[:b], v[:b], decay, o, i32([0, 1, 2, 3]), slots, slots, 1, ws, status=status)
    for i in range(b):
        want, s, bound, size, chain = OL.linear_attention(before[int(slots[i])], host(q[i:i + 1]), host(k[i:i + 1]), host(v[i:i + 1]),
                                                          host(decay)[None], d ** -0.5)
        assert_close(host(o[i:i + 1]), want, 2.0 ** -7 * np.abs(want) + 2.0 ** -7 * bound)
        assert_close(host(pool)[int(slots[i])], s, 2.0 ** -18 * size)
    assert int(status) == 0


@pytest.mark.parametrize("power", [-28, 20, 28])
@pytest.mark.parametrize("d", [64, 128])
def test_prompts_of_large_and_small_values(power, d):
    """q, k and v of 2^power each, and decays that pass 2^-60 within a chunk: the terms are of 2^(3 power), which the range at the
    declaration allows, and the tolerances are relative to them."""
    c = Case(26, [300, 17, 128], 2, 2, d, True, rate=0.8)
    for t in (c.q, c.k, c.v):
        t.mul_(2.0 ** power)
    c.pool.mul_(2.0 ** (2 * power))
    before = host(c.pool)
    c.call()
    check_rows(c, before)


@pytest.mark.parametrize("scale", [2.0 ** -110, -2.0 ** -70, 2.0 ** 100])
def test_scales_of_all_sizes(scale):
    """The factor that is left for a row's outputs and a small or large scale: neither product may leave fp32."""
    c = Case(27, [150, 3, 40], 2, 2, 64, True, rate=0.8)
    before = host(c.pool)
    c.call(scale=scale)
    check_rows(c, before, scale)


# ------------------------------------------------------------------------------ more units than blocks


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def test_segments_of_more_units_than_blocks():
    """Pieces and segments whose number passes the blocks'."""
    h, lens = 32, [3000, 1100, 40, 300]
    c = Case(30, lens, 8, h, 64, True, rate=0.02)
    chunks = [-(-n // 128) for n in lens]
    segments = chunks[0] // max(4, -(-sum(chunks) * h // sms()))
    assert segments > 1 and 3 * (segments - 1) * h > sms() and (segments + 3) * h > sms()
    before = host(c.pool)
    c.call()
    check_rows(c, before)


@pytest.mark.parametrize("t", [(1 << 31) - 1, (1 << 31) - 3])
def test_norm_of_as_many_rows_as_an_int32_holds(t):
    y = torch.empty((t, 1), dtype=BF, device="cuda").normal_()
    out = torch.empty_like(y)
    api.mdw_block_norm(y, out)
    assert torch.equal(y, out)


@pytest.mark.parametrize("y", [BF, F32])
@pytest.mark.parametrize("w", [640, 1003])
def test_norm_of_a_sum_that_is_not_stored(y, w):
    """Without sum and residual nothing is rounded before x."""
    a = norm_case(8, 5, w, BF, y, None, True, "sigmoid", True, None, True)
    a["sum"] = None
    api.mdw_block_norm(**a)
    s, _ = OL.block_sum(host(a["y"]), host(a["post_weight"]), None, host(a["gate"]), "sigmoid")
    x = OL.rmsnorm(s, host(a["pre_weight"]), 1e-6)
    # s is off by 128 u of its magnitude, its root mean square by as much, and x is rounded once
    assert_close(host(a["x"]), x, (half_step(BF) + 256 * U) * np.abs(x) + 2.0 ** -24)


@pytest.mark.parametrize("kind", ["sigmoid", "silu"])
def test_norm_gates_far_below_zero_in_an_fp32_sum(kind):
    """In units of u = 2^-24: the exponential 4, what is left of its argument 1, one plus it 1, the reciprocal 2, the products with y, the gate
    and the scale 3, the store 1: 12."""
    n = 4096
    a = dict(y=norm_case(9, 2, n, F32)["y"], sum=torch.empty((2, n), device="cuda"), gate_kind=kind,
             gate=torch.linspace(-80, 10, n, device="cuda").to(BF).expand(2, n).contiguous())
    api.mdw_block_norm(**a, branch_scale=0.7)
    s, _ = OL.block_sum(host(a["y"]), None, None, host(a["gate"]), kind, branch_scale=np.float64(np.float32(0.7)))
    assert_close(host(a["sum"]), s, 12 * U * np.abs(s))


# ------------------------------------------------------------------------------ each kernel at its own precision


def check_precision(c, pool0, rows_of_norm=64):
    """Outputs by the kernel that a call takes (see the end of the first docstring):
    * rows one by one (a bound below 12; requests of up to 16 rows of a call with longer ones): fp32. The sum over a column of the state has at most
      8 additions of a thread, 2 between lanes and 8 between warps, and the scale: 20 u `bound`, beside what the state itself is off by.
    * a bound of 12 to 16: scores and state as two bf16 numbers, off by 2^-7 (what the first one leaves) times 2^-8: 2^-15, doubled for the
      exponentials and sums.
    * chunks: an output's own rounding, and one of its terms to bf16 each. A rounding is uniform within half a step, so its root mean square is at
      most 2^-8 / sqrt(3) of the value; terms and output are independent of each other: sqrt(2) of that, 0.0032, of the norm. 0.004, of the
      norm over some rows of a head, among which those that start a segment."""
    out, scale = host(c.out), c.d ** -0.5
    for b in range(c.b):
        at, q, k, v, g = c.rows(b)
        if not len(q):
            continue
        o, s, bound, size, chain = OL.linear_attention(c.before(b, pool0), q, k, v, g, scale)
        if len(q) > 16:
            for h in range(c.h):
                for first in range(0, max(len(q) - rows_of_norm + 1, 1), rows_of_norm):
                    part = slice(first, first + rows_of_norm)
                    norm = np.linalg.norm(o[part, h])
                    assert np.linalg.norm(out[at][part, h] - o[part, h]) <= 0.004 * norm, (b, h, first)
            continue
        tol = 2.0 ** -14 * bound if 12 <= c.new <= 16 else 20 * U * bound + scale * 4 * U * np.einsum("nhi,hij->nhj", np.repeat(np.abs(q), c.h // c.hk, 1), chain)
        assert_close(out[at], o, half_step(BF) * np.abs(o) + 1.01 * tol, b)


@pytest.mark.parametrize("lens", [[1], [1, 5, 11, 8], [16, 3, 12, 0, 9], [300, 16, 5, 17], [1025, 3], [1500, 0, 1200]], ids=str)
@pytest.mark.parametrize("h,d,rate", [(2, 64, 0.3), (2, 128, 0.02), (1, 128, 2.0)])
def test_precision_of_each_kernel(lens, h, d, rate):
    c = Case(sum(lens) + 1, lens, 1, h, d, True, rate=rate)
    before = host(c.pool)
    c.call()
    check_precision(c, before)


@pytest.mark.parametrize("lens", [[4, 3, 2, 5], [140, 3, 200, 150], [14, 3, 12, 5]], ids=str)
@pytest.mark.parametrize("fault,skip", [("out", (0, 2)), ("in", (0,)), ("high", (1,)), ("low", (2,)), ("rows", (3,))])
def test_a_bad_request_changes_nothing_of_the_others(lens, fault, skip):
    """The others' rows and states are those of a call without the fault, bit for bit; a skipped one's rows and slot stay."""
    c, clean = Case(28, lens, 2, 2, 64, inplace=False), Case(28, lens, 2, 2, 64, inplace=False)
    start, to = c.start.copy(), list(c.slot_out)
    if fault == "out":
        c.slot_out[2] = c.slot_out[0]
    elif fault == "in":
        c.slot_in[0] = c.slot_out[2]
    elif fault == "high":
        c.slot_in[1] = len(c.pool)
    elif fault == "low":
        c.slot_out[2] = -2
    else:
        start[-1] = c.t + 1
    before = c.pool.clone()
    c.call(start=i32(start.tolist()))
    clean.call()
    assert int(c.status) == 7 and int(clean.status) == 0
    want, pool = clean.out.clone(), clean.pool.clone()
    for b in skip:
        want[int(c.start[b]):int(c.start[b + 1])] = 7
        pool[to[b]] = before[to[b]]
    assert torch.equal(c.out, want) and torch.equal(c.pool, pool)


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def alone(c, b, run):
    """The outputs and the pool of a call with request b only, whose bound, rows and state are the same."""
    at = slice(int(c.start[b]), int(c.start[b + 1]))
    one = Case(0, [at.stop - at.start], c.hk, c.h, c.d, tail=0)
    one.q, one.k, one.v, one.g = c.q[at], c.k[at], c.v[at], c.g[at]
    one.pool, one.slot_in, one.slot_out, one.new = c.pool.clone(), [c.slot_in[b]], [c.slot_out[b]], c.new
    run(one)
    return one.out, one.pool


@pytest.mark.parametrize("h,d,lens", [(64, 64, [130, 17, 300, 1, 256, 40, 129]), (40, 128, [150, 260, 20, 0, 129, 33, 128])], ids=str)
@pytest.mark.parametrize("odd", [False, True])
def test_prompts_of_more_units_than_blocks(h, d, lens, odd):
    """Blocks of the chunk kernel that take several units: as each request alone gives them, values that are not finite among them."""
    c = Case(29, lens, h // 2, h, d, True, fresh=(2,), inplace=False, lead=1)
    assert sum(n > 16 for n in lens) * h > sms()
    if odd:
        c.v[int(c.start[0]) + 60, 3, 7] = float("inf")
        c.k[int(c.start[1]) + 2, 2, 1] = float("nan")
        c.v[int(c.start[5]) + 1, :, 9] = float("nan")
    before = c.pool.clone()
    whole = Case(29, lens, h // 2, h, d, True, fresh=(2,), inplace=False, lead=1)
    whole.q, whole.k, whole.v, whole.pool = c.q, c.k, c.v, c.pool.clone()
    whole.call()
    for b, n in enumerate(lens):
        if n:
            out, pool = alone(c, b, lambda one: one.call(new=c.new))
            assert torch.equal(bits(whole.out[int(c.start[b]):int(c.start[b + 1])]), bits(out)), b
            assert torch.equal(bits(whole.pool[c.slot_out[b]]), bits(pool[c.slot_out[b]])), b
    if not odd:
        check_rows(whole, host(before))
        check_precision(whole, host(before))


@pytest.mark.parametrize("h,d,most,each", [(32, 128, 16, 2), (64, 64, 16, 4), (32, 128, 32, 2), (64, 64, 32, 4), (20, 128, 64, 1), (32, 64, 64, 2)])
def test_trees_of_more_units_than_blocks(h, d, most, each):
    """The same for each number of tiles of the trees' kernel, `each` of whose blocks fit an SM."""
    rng = np.random.default_rng(most + d)
    b = each * sms() // h + 3
    lens = [most] + [int(rng.integers(0, most + 1)) for _ in range(b - 1)]
    assert b * h > each * sms()
    c = Case(31, lens, h // 2, h, d, True, fresh=(3,), rate=1.0, lead=1)
    masks = [[1] * c.start[0]] + [random_masks(rng, n) for n in lens]
    for i in (1, b // 2, b - 1):
        if lens[i]:
            c.v[int(c.start[i]) + lens[i] // 2, ::3, 5] = float("inf")
    before = c.pool.clone()
    c.tree([m for r in masks for m in r] + [0] * 3)
    assert torch.equal(c.pool, before) and int(c.status) == 0
    assert (c.out[:1] == 7).all() and (c.out[int(c.start[-1]):] == 7).all()
    for i, n in enumerate(lens):
        if n:
            out, _ = alone(c, i, lambda one: one.tree(masks[i + 1], new=most))
            assert torch.equal(bits(c.out[int(c.start[i]):int(c.start[i + 1])]), bits(out)), i
    rows, q, k, v, g = c.rows(0)
    few = min(lens[0], 16)
    o, bound = OL.tree_attention(c.before(0, host(before)), q[:few], k[:few], v[:few], g[:few], masks[1][:few], d ** -0.5)
    assert_close(host(c.out)[rows][:few], o, half_step(BF) * np.abs(o) + 2.0 ** -14 * bound)
