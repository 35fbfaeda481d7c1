"""Refusals of the linear-attention sub-layer's entry points: every call here fails a host-side check before any
CUDA call, so the placeholder addresses are never touched."""

import pytest
import torch

from moe_decode_weight_gb300 import api
from test_boundary import FAKE, _define

BF, HF, F32 = api.DT_BF16, api.DT_F16, api.DT_F32


def _state(**kw):
    s = api.LinearStateC(api.MDW_MAGIC, api.FMT_LINEAR_STATE, 5, 4, 128, 0, 4 * 128 * 128, FAKE)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _lin(s=None, **kw):
    a = dict(b=2, t=9, hq=2, new=5, q=FAKE, ldq=256, k=FAKE, ldk=256, v=FAKE, ldv=512, g=FAKE, ldd=4, out=FAKE, ldo=512, start=FAKE, i=FAKE,
             o=FAKE, scale=0.1, status=None, ws=FAKE, n=1 << 40) | kw
    return api.lib().mdw_linear_attention(s or _state(), a["b"], a["t"], a["hq"], a["new"], a["q"], a["ldq"], a["k"], a["ldk"], a["v"],
                                          a["ldv"], a["g"], a["ldd"], a["out"], a["ldo"], a["start"], a["i"], a["o"], a["scale"],
                                          a["status"], a["ws"], a["n"], None)


def _tree(s=None, **kw):
    a = dict(b=2, t=9, hq=2, new=5, q=FAKE, ldq=256, k=FAKE, ldk=256, v=FAKE, ldv=512, g=FAKE, ldd=4, out=FAKE, ldo=512, start=FAKE, i=FAKE,
             mask=None, scale=0.1, status=None) | kw
    return api.lib().mdw_linear_tree_attention(s or _state(), a["b"], a["t"], a["hq"], a["new"], a["q"], a["ldq"], a["k"], a["ldk"],
                                               a["v"], a["ldv"], a["g"], a["ldd"], a["out"], a["ldo"], a["start"], a["i"], a["mask"],
                                               a["scale"], a["status"], None)


def _advance(s=None, **kw):
    a = dict(b=2, t=9, hq=2, new=5, k=FAKE, ldk=256, v=FAKE, ldv=512, g=FAKE, ldd=4, start=FAKE, acc=FAKE, i=FAKE, o=FAKE, status=None) | kw
    return api.lib().mdw_linear_state_advance(s or _state(), a["b"], a["t"], a["hq"], a["new"], a["k"], a["ldk"], a["v"], a["ldv"], a["g"],
                                              a["ldd"], a["start"], a["acc"], a["i"], a["o"], a["status"], None)


def test_limits_match_the_header():
    assert api.MAX_NORM_WIDTH == _define("MDW_MAX_NORM_WIDTH")


@pytest.mark.parametrize("field,value,code", [
    ("magic", 0, 3), ("fmt", api.FMT_KV_PAGED, 3), ("num_slots", 0, 2), ("heads", 0, 2), ("heads", 1025, 2), ("head_dim", 96, 2),
    ("head_dim", 256, 2), ("slot_stride", 4 * 128 * 128 - 4, 1), ("slot_stride", 4 * 128 * 128 + 2, 1), ("slot_stride", (1 << 32) + 4, 1),
    ("s", None, 1), ("s", FAKE + 8, 1)])
def test_state_handle_is_checked(field, value, code):
    s = _state(**{field: value})
    assert _lin(s) == _tree(s) == _advance(s) == code
    assert api.lib().mdw_linear_attention_workspace_bytes(s, 2, 9, 2, 5) == 0


COMMON = [(dict(b=0), 1), (dict(b=api.MAX_REQUESTS + 1), 1), (dict(t=0), 1), (dict(t=0x7fff0001), 2), (dict(new=0), 1), (dict(hq=0), 1),
          (dict(hq=3), 1), (dict(k=None), 1), (dict(k=FAKE + 8), 1), (dict(ldk=248), 1), (dict(ldk=257), 1), (dict(v=FAKE + 2), 1),
          (dict(ldv=504), 1), (dict(g=None), 1), (dict(g=FAKE + 2), 1), (dict(ldd=3), 1), (dict(ldd=-4), 1), (dict(start=None), 1),
          (dict(start=FAKE + 2), 1), (dict(i=None), 1), (dict(i=FAKE + 1), 1), (dict(status=FAKE + 2), 1)]
ROWS = [(dict(q=None), 1), (dict(q=FAKE + 8), 1), (dict(ldq=248), 1), (dict(ldq=260), 1), (dict(out=None), 1), (dict(ldo=504), 1),
        (dict(ldo=516), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1)]


@pytest.mark.parametrize("kw,code", COMMON + ROWS + [(dict(o=None), 1), (dict(o=FAKE + 2), 1), (dict(ws=None), 1), (dict(ws=FAKE + 8), 1),
                                                     (dict(n=15), 4)])
def test_linear_attention_rejects(kw, code):
    assert _lin(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + ROWS + [(dict(new=65), 1), (dict(mask=FAKE + 4), 1)])
def test_tree_rejects(kw, code):
    assert _tree(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [(dict(new=65), 1), (dict(acc=None), 1), (dict(acc=FAKE + 4), 1), (dict(o=None), 1)])
def test_advance_rejects(kw, code):
    assert _advance(**kw) == code


def test_one_key_head_serves_a_bounded_number_of_value_heads():
    s = _state(heads=65, slot_stride=65 * 128 * 128)
    assert _lin(s, hq=1, ldv=65 * 128, ldo=65 * 128, ldd=65) == 1


@pytest.mark.parametrize("kw,code", [
    (dict(t=0), 1), (dict(w=0), 1), (dict(w=16385, ldy=16385, lds=16385, group=16385), 2), (dict(dt=F32), 3), (dict(yd=HF), 3), (dict(sd=HF), 3),
    (dict(sd=0), 3), (dict(y=None), 1), (dict(y=FAKE + 1), 1), (dict(ldy=255), 1), (dict(yd=F32, y=FAKE + 2), 1), (dict(post=FAKE + 1), 1),
    (dict(group=32), 2), (dict(group=96), 2), (dict(w=200, group=64), 2), (dict(gate=FAKE), 1), (dict(kind=1), 1), (dict(gate=FAKE, kind=4), 1),
    (dict(gate=FAKE, kind=-1), 1), (dict(gate=FAKE, kind=2, ldg=255), 1), (dict(gate=FAKE + 1, kind=2), 1), (dict(bs=float("inf")), 1),
    (dict(rs=float("nan")), 1), (dict(res=FAKE + 1), 1), (dict(res=FAKE, ldr=255), 1), (dict(sum=None), 1), (dict(sum=FAKE + 1), 1),
    (dict(lds=255), 1), (dict(sd=F32, sum=FAKE + 2), 1), (dict(pre=FAKE), 1), (dict(x=FAKE, ldx=256), 1), (dict(pre=FAKE, x=FAKE, ldx=255), 1),
    (dict(pre=FAKE + 1, x=FAKE, ldx=256), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1)])
def test_norm_rejects(kw, code):
    a = dict(t=2, w=256, dt=BF, y=FAKE, ldy=256, yd=BF, post=None, group=256, gate=None, ldg=0, kind=0, bs=1.0, res=None, ldr=0, rs=1.0,
             sum=FAKE, lds=256, sd=BF, pre=None, x=None, ldx=0, eps=1e-6) | kw
    assert api.lib().mdw_block_norm(a["t"], a["w"], a["dt"], a["y"], a["ldy"], a["yd"], a["post"], a["group"], a["gate"], a["ldg"], a["kind"],
                                    a["bs"], a["res"], a["ldr"], a["rs"], a["sum"], a["lds"], a["sd"], a["pre"], a["x"], a["ldx"], a["eps"],
                                    None) == code


def test_binding_refuses_host_tensors_and_unknown_gates():
    with pytest.raises(api.MdwError) as e:
        api.LinearState(torch.zeros((1, 1, 64, 64)))
    assert e.value.code == 1
    with pytest.raises(api.MdwError):
        api.LinearState(torch.zeros((1, 64, 64)))
    y = torch.zeros((1, 64), dtype=torch.bfloat16)
    with pytest.raises(api.MdwError):
        api.mdw_block_norm(y, y)
    with pytest.raises(api.MdwError):
        api.mdw_block_norm(y, y, gate=y, gate_kind="tanh")
