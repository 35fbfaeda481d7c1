"""Refusals of the attention sub-layer's entry points: every call here fails a host-side check before
any CUDA call, so the placeholder addresses are never touched."""

import pytest
import torch

from moe_decode_weight_gb300 import api
from test_boundary import FAKE, _define

BF, HF, F32, E4 = api.DT_BF16, api.DT_F16, api.DT_F32, api.DT_E4M3


def _w4(**kw):
    w = api.W4WeightsC(api.MDW_MAGIC, api.FMT_INT4_GROUP, 100, 2560, 128, BF, FAKE, FAKE, None)
    for k, v in kw.items():
        setattr(w, k, v)
    return w


def _cache(**kw):
    c = api.KVCacheC(api.MDW_MAGIC, api.FMT_KV_PAGED, BF, 10, 16, 4, 128, 0, 4 * 16 * 128, FAKE, FAKE, None, None)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_limits_match_the_header():
    assert api.MAX_REQUESTS == _define("MDW_MAX_REQUESTS")
    assert api.MAX_TREE == _define("MDW_MAX_TREE") and api.MAX_GROUP == _define("MDW_MAX_GROUP")


@pytest.mark.parametrize("field,value,code", [
    ("magic", 0, 3), ("fmt", api.FMT_MXFP4, 3), ("dtype", F32, 3), ("group", 16, 2), ("group", 256, 2), ("n", 0, 2),
    ("k", 2592, 2), ("k", 0, 2), ("q", FAKE + 8, 1), ("q", None, 1), ("scale", None, 1), ("scale", FAKE + 8, 1), ("zero", FAKE + 8, 1)])
def test_w4_rejects_weights(field, value, code):
    assert api.lib().w4_linear(_w4(**{field: value}), 1, FAKE, 2560, FAKE, 100, BF, None, None, 0, None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(m=0), 1), (dict(m=33), 1), (dict(x=None), 1), (dict(x=FAKE + 2), 1), (dict(ldx=2552), 1), (dict(ldx=2561), 1),
    (dict(y=FAKE + 1), 1), (dict(y=None), 1), (dict(ldy=99), 1), (dict(yd=HF), 3), (dict(yd=0), 3), (dict(yd=F32, y=FAKE + 2), 1),
    (dict(bias=FAKE + 1), 1), (dict(res=FAKE + 1, ldr=100), 1), (dict(res=FAKE, ldr=99), 1), (dict(status=FAKE + 2), 1)])
def test_w4_rejects_arguments(kw, code):
    a = dict(m=1, x=FAKE, ldx=2560, y=FAKE, ldy=100, yd=BF, bias=None, res=None, ldr=0, status=None) | kw
    assert api.lib().w4_linear(_w4(), a["m"], a["x"], a["ldx"], a["y"], a["ldy"], a["yd"], a["bias"], a["res"], a["ldr"], a["status"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(b=0), 1), (dict(b=api.MAX_REQUESTS + 1), 1), (dict(t=0), 1), (dict(pages=0), 1), (dict(width=0), 1), (dict(free=-1), 1),
    (dict(page=8), 2), (dict(page=512), 2), (dict(page=48), 2), (dict(width=1 << 28), 2), (dict(ctx=None), 1), (dict(ctx=FAKE + 2), 1),
    (dict(table=None), 1), (dict(pfree=None), 1), (dict(parents=FAKE + 1), 1), (dict(start=None), 1), (dict(slot=FAKE + 4), 1),
    (dict(pos=None), 1), (dict(mask=FAKE + 4), 1), (dict(taken=None), 1), (dict(status=FAKE + 1), 1)])
def test_plan_rejects(kw, code):
    a = dict(b=2, ctx=FAKE, new=FAKE, page=16, pages=9, table=FAKE, width=4, pfree=FAKE, free=3, parents=None, t=8, start=FAKE,
             slot=FAKE, pos=FAKE, mask=None, taken=FAKE, status=None) | kw
    assert api.lib().mdw_kv_plan(a["b"], a["ctx"], a["new"], a["page"], a["pages"], a["table"], a["width"], a["pfree"], a["free"],
                                 a["parents"], a["t"], a["start"], a["slot"], a["pos"], a["mask"], a["taken"], a["status"], None) == code


CACHE_FAULTS = [
    ("magic", 0, 3), ("fmt", api.FMT_FP8, 3), ("dtype", F32, 3), ("page_size", 8, 2), ("page_size", 24, 2), ("page_size", 512, 2),
    ("num_pages", 0, 2), ("kv_heads", 0, 2), ("head_dim", 96, 2), ("k", None, 1), ("v", FAKE + 8, 1), ("page_stride", 4 * 16 * 128 - 8, 1),
    ("page_stride", 4 * 16 * 128 + 4, 1), ("k_scale", FAKE, 1), ("dtype", E4, 1)]


@pytest.mark.parametrize("field,value,code", CACHE_FAULTS)
def test_cache_handle_is_checked(field, value, code):
    lib, c = api.lib(), _cache(**{field: value})
    assert lib.mdw_kv_write(c, 1, FAKE, 512, FAKE, 512, BF, FAKE, None, None) == code
    assert lib.mdw_tree_attention_workspace_bytes(c, 1, 4, 8, 4) == 0
    assert lib.mdw_tree_attention(c, 1, 4, 8, 4, FAKE, 1024, BF, FAKE, 1024, None, FAKE, 4, FAKE, FAKE, None, 0.1, None, FAKE,
                                  1 << 40, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(t=0), 1), (dict(dt=HF), 3), (dict(dt=F32), 3), (dict(k=FAKE + 8), 1), (dict(v=None), 1), (dict(ldk=504), 1), (dict(ldv=513), 1),
    (dict(slot=None), 1), (dict(slot=FAKE + 4), 1), (dict(status=FAKE + 2), 1)])
def test_write_rejects(kw, code):
    a = dict(t=2, k=FAKE, ldk=512, v=FAKE, ldv=512, dt=BF, slot=FAKE, status=None) | kw
    assert api.lib().mdw_kv_write(_cache(), a["t"], a["k"], a["ldk"], a["v"], a["ldv"], a["dt"], a["slot"], a["status"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(b=0), 1), (dict(b=api.MAX_REQUESTS + 1), 1), (dict(t=0), 1), (dict(new=0), 1), (dict(new=65), 1), (dict(hq=6), 1),
    (dict(hq=4 * 65), 1), (dict(dt=HF), 3), (dict(dt=E4), 3), (dict(q=FAKE + 8), 1), (dict(ldq=1016), 1), (dict(ldq=1028), 1),
    (dict(out=None), 1), (dict(ldo=1016), 1), (dict(lse=FAKE + 2), 1), (dict(table=None), 1), (dict(width=0), 2), (dict(width=1 << 28), 2),
    (dict(ctx=None), 1), (dict(start=FAKE + 1), 1), (dict(mask=FAKE + 4), 1), (dict(status=FAKE + 2), 1), (dict(scale=0.0), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(ws=FAKE + 8), 1), (dict(nbytes=15), 4)])
def test_attention_rejects(kw, code):
    a = dict(b=1, t=4, hq=8, new=4, q=FAKE, ldq=1024, dt=BF, out=FAKE, ldo=1024, lse=None, table=FAKE, width=4, ctx=FAKE, start=FAKE,
             mask=None, scale=0.1, status=None, ws=FAKE, nbytes=1 << 40) | kw
    assert api.lib().mdw_tree_attention(_cache(), a["b"], a["t"], a["hq"], a["new"], a["q"], a["ldq"], a["dt"], a["out"], a["ldo"],
                                        a["lse"], a["table"], a["width"], a["ctx"], a["start"], a["mask"], a["scale"], a["status"],
                                        a["ws"], a["nbytes"], None) == code


def test_binding_refuses_host_tensors():
    with pytest.raises(api.MdwError) as e:
        api.W4Weights(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 1), dtype=torch.bfloat16))
    assert e.value.code == 1
    with pytest.raises(api.MdwError):
        api.KVCache(torch.zeros((1, 1, 16, 64)), torch.zeros((1, 1, 16, 64)))
    with pytest.raises(api.MdwError):
        api.mdw_kv_plan(*(torch.zeros(1, dtype=torch.int32),) * 2, 16, 1, *(torch.zeros((1, 1), dtype=torch.int32),) * 6)


@pytest.mark.parametrize("n", [(1 << 31) - 255, (1 << 31) - 1])
def test_w4_rejects_features_whose_tiles_pass_int32(n):
    assert api.lib().w4_linear(_w4(n=n, k=128), 1, FAKE, 128, FAKE, n, BF, None, None, 0, None, None) == 2


@pytest.mark.parametrize("m", [1, 8])
@pytest.mark.parametrize("k", [(1 << 31) - 128, (1 << 31) - 224])
def test_w4_rejects_elements_whose_units_pass_int32(m, k):
    k = k // 32 * 32
    assert api.lib().w4_linear(_w4(n=1, k=k, group=32), m, FAKE, k, FAKE, 1, BF, None, None, 0, None, None) == 2


@pytest.mark.parametrize("page,width", [(16, (1 << 27) - 1), (256, (1 << 23) - 1), (256, (1 << 23) - 255)])
def test_attention_rejects_tables_whose_tiles_pass_int32(page, width):
    c = _cache(page_size=page, page_stride=4 * page * 128)
    assert api.lib().mdw_tree_attention(c, 1, 4, 8, 4, FAKE, 1024, BF, FAKE, 1024, None, FAKE, width, FAKE, FAKE, None, 0.1, None,
                                        FAKE, 1 << 40, None) == 2
