"""Pins of the router and FP8 oracles (CPU): torch's casts, brute force and closed forms."""

import itertools

import numpy as np
import pytest
import torch

from oracle import fp8 as O
from oracle import router as R
from oracle.formats import e4m3_decode


def test_codes_are_torchs_cast():
    rng = np.random.default_rng(1)
    q = np.concatenate([rng.standard_normal(4000) * s for s in (1e-3, 0.02, 1.0, 60.0)]).astype(np.float32)
    grid = e4m3_decode(np.arange(0x7F))
    q = np.clip(np.concatenate([q, (grid[1:] + grid[:-1]) / 2, grid, -grid]), -448, 448).astype(np.float32)
    want = torch.from_numpy(q).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(O.e4m3(q.astype(np.float64)), want)


@pytest.mark.parametrize("block_rows,shape", [(1, (3, 300)), (128, (130, 144)), (1, (2, 16))])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantiser_against_torch(block_rows, shape, pow2):
    g = torch.Generator().manual_seed(2)
    h = torch.randn(shape, generator=g) * 3
    h[0, :16] = 0
    codes, s = O.quantize(h.double().numpy(), block_rows, pow2)
    for i, j in itertools.product(range(s.shape[0]), range(s.shape[1])):
        block = h[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
        a = block.abs().max()
        if a == 0:
            assert s[i, j] == 1
            continue
        if pow2:
            assert np.log2(s[i, j]) % 1 == 0 and a <= 448 * s[i, j] and a > 224 * s[i, j]
        else:
            assert s[i, j] == float(a / torch.tensor(448.0))
        want = (block / float(s[i, j])).clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
        assert np.array_equal(codes[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128], want)
    back = O.dequant(codes, s, block_rows)
    assert np.all(np.abs(back - h.numpy()) <= np.maximum(2.0**-4 * np.abs(h.numpy()), 2.0**-10 * O.spread(s, shape, block_rows)) * 1.0001)


def test_product_of_ones():
    a, w = np.ones((3, 256)), np.full((5, 256), 0.5)
    y, mags = O.product(O.fake_quant(a), O.fake_quant(w))
    assert np.allclose(y, 128.0, rtol=1e-7) and np.array_equal(y, mags)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (4, 2, 1), (4, 2, 2), (2, 1, 2)])
def test_router_against_torch(score, bias, groups, top_groups, group_top):
    g = torch.Generator().manual_seed(3)
    z = torch.randn(20, 16, generator=g, dtype=torch.float64)
    b = torch.randn(16, generator=g, dtype=torch.float64) * 0.2 if bias else None
    s = torch.softmax(z, -1) if score == "softmax" else torch.sigmoid(z)
    c = s + b if bias else s
    value = c.view(20, groups, -1).topk(group_top, -1).values.sum(-1)
    keep = torch.zeros(20, groups, dtype=torch.bool).scatter_(1, value.topk(top_groups, -1).indices, True)
    masked = torch.where(keep.repeat_interleave(16 // groups, 1), c, -torch.inf)
    ids = masked.topk(3, -1).indices
    w = s.gather(1, ids)
    got_ids, got_w = R.route(z.numpy(), None if b is None else b.numpy(), 3, score, scale=2.0, groups=groups,
                             top_groups=top_groups, group_top=group_top)
    assert np.array_equal(got_ids, ids.numpy())
    assert np.allclose(got_w, (2.0 * w / w.sum(-1, keepdim=True)).numpy(), rtol=1e-12)
    _, raw = R.route(z.numpy(), None if b is None else b.numpy(), 3, score, renorm=False, groups=groups,
                     top_groups=top_groups, group_top=group_top)
    assert np.allclose(raw, w.numpy(), rtol=1e-12)


def test_router_special_rows():
    inf, nan = np.inf, np.nan
    ids, w = R.route([[-inf] * 4, [nan, 1, -inf, 1], [inf, 0, inf, 5], [2, 2, 2, 2]], None, 3, "softmax")
    assert ids.tolist() == [[-1, -1, -1], [1, 3, -1], [0, 2, 3], [0, 1, 2]]
    assert np.allclose(w, [[0, 0, 0], [0.5, 0.5, 0], [0.5, 0.5, 0], [1 / 3] * 3])
    ids, w = R.route([[0, 0, 0, 0]], [nan, -inf, inf, 0.1], 3, "sigmoid", scale=3.0)
    assert ids.tolist() == [[2, 3, -1]] and np.allclose(w, [[1.5, 1.5, 0]])
    ids, w = R.route([[-1000, -1001, -2000]], None, 2, "sigmoid")
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.e)]])
    # groups: one without experts is never taken, one with a single expert counts with it
    ids, _ = R.route([[nan, nan, -3, nan, 1, 0]], None, 2, "sigmoid", groups=3, top_groups=2, group_top=2)
    assert ids.tolist() == [[4, 5]]
