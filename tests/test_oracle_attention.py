"""Pins of the attention sub-layer's oracle against torch operations and closed forms (CPU)."""

import numpy as np
import pytest
import torch

from oracle import attention as OA


def test_w4_weight_against_unpacked_codes():
    rng = np.random.default_rng(0)
    code = rng.integers(0, 16, (6, 128))
    q = (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8)
    scale, zero = rng.normal(size=(6, 4)), rng.integers(0, 16, (6, 4))
    want = (code - np.repeat(zero, 32, 1)) * np.repeat(scale, 32, 1)
    assert np.array_equal(OA.w4_weight(q, scale, zero, 32), want)
    assert np.array_equal(OA.w4_weight(q, scale, None, 32), (code - 8) * np.repeat(scale, 32, 1))
    x = rng.normal(size=(3, 128))
    got = OA.w4_linear(q, scale, zero, 32, x, bias=np.ones(6), residual=np.full((3, 6), 2.0))
    assert np.allclose(got, x @ want.T + 3.0, rtol=1e-13)


@pytest.mark.parametrize("group", [1, 5])
def test_tree_attention_against_torch(group):
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((3, 2 * group, 8), (9, 2, 8), (9, 2, 8)))
    seen = torch.rand((3, 9), generator=g) > 0.4
    seen[:, 0] = True
    kk, vv = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    want = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), kk.transpose(0, 1), vv.transpose(0, 1),
                                                            attn_mask=seen, scale=0.3).transpose(0, 1)
    out, lse, _, _ = OA.tree_attention(q.numpy(), k.numpy(), v.numpy(), seen.numpy(), 0.3)
    assert np.allclose(out, want.numpy(), rtol=1e-12, atol=1e-13)
    z = torch.einsum("nhd,khd->nhk", q, kk).mul(0.3).masked_fill(~seen[:, None], -np.inf)
    assert np.allclose(lse, torch.logsumexp(z, -1).numpy(), rtol=1e-12)


def test_tree_attention_of_a_row_that_sees_nothing():
    out, lse, _, _ = OA.tree_attention(np.ones((1, 2, 4)), np.full((3, 1, 4), np.nan), np.ones((3, 1, 4)), np.zeros((1, 3), bool), 1.0)
    assert not out.any() and np.all(lse == -np.inf)


def test_plan_of_a_worked_example():
    # two requests, pages of 16: request 0 fills its page and takes one, request 1 starts empty
    p = OA.kv_plan([15, 0], [3, 2], 16, 8, [[5, -1], [-1, -1]], [2, 7, 1], 6, parents=[-1, 0, 0, -1, 0, 0])
    assert p["table"].tolist() == [[5, 2], [7, -1]] and p["start"].tolist() == [0, 3, 5] and p["taken"] == 2
    assert p["slot"].tolist() == [95, 32, 33, 112, 113, -1]
    assert p["pos"].tolist() == [15, 16, 16, 0, 1, -1]
    assert p["mask"].tolist() == [0b1, 0b11, 0b101, 0b1, 0b11, 0] and not p["bad"]
    assert OA.kv_plan([31], [2], 16, 8, [[5, 4]], [2], 6)["fail"]
    assert OA.kv_plan([0], [2], 16, 8, [[5, 4]], [2], 6, parents=[-1, 1, 0, 0, 0, 0])["bad"]


def test_write_rounds_to_e4m3():
    rows = np.array([[[1.0, -3.3, 500.0, 1e-4]]], np.float32)
    out = OA.kv_write(np.zeros((2, 1, 16, 4), np.uint8), np.concatenate([rows, rows]), [17, -1], 16, [0.5])
    want = torch.tensor([2.0, -6.6, 448.0, 2e-4]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert out[1, 0, 1].tolist() == want.tolist() and not out[0].any()
