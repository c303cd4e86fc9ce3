"""Pins of the FP4 activation oracle (CPU): against torch casts, fractions and closed forms."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fp4, quant
from oracle.formats import e2m1_decode, e4m3_decode, e8m0_decode

NV, MX = quant.NVFP4, quant.MXFP4


def test_row_scale_is_the_least_power_of_two():
    rng = np.random.default_rng(1)
    h = rng.standard_normal((200, 32)) * np.exp(rng.uniform(-20, 20, (200, 1)))
    h[0] = 0
    h[1] = 0
    h[1, 3] = 2688.0 * 2.0**-5  # exactly at a power: that power, not the next
    h[2, :] = 0
    h[2, 5] = -np.nextafter(2688.0 * 2.0**-5, np.inf)
    gs = fp4.row_gs(h)
    assert gs[0] == 1.0 and gs[1] == 2.0**-5 and gs[2] == 2.0**-4
    for g, row in zip(gs[3:], h[3:]):
        top = Fraction(float(np.abs(row).max()))
        assert Fraction(float(g)) * 2688 >= top > Fraction(float(g)) * 2688 / 2
    assert fp4.row_gs(np.full((1, 16), 1e-60))[0] == 2.0**-126


@pytest.mark.parametrize("fmt", [NV, MX])
def test_blocks_match_the_weight_quantiser(fmt):
    """Row by row the codes and scales are the weight quantiser's, given its global scale."""
    w = np.random.default_rng(2).standard_normal((1, 24, 64)).astype(np.float32) * 0.02
    codes, scales, gs = quant.quantize(w, fmt)
    if fmt == NV:
        assert np.float32(fp4.matrix_gs(w[0])) == gs[0]
    c, s = fp4.quantize_rows(w[0].astype(np.float64), fmt, None if gs is None else gs[0])
    assert np.array_equal(c, quant.unpack_nibbles(codes[0])) and np.array_equal(s, scales[0])


@pytest.mark.parametrize("fmt", [NV, MX])
def test_error_bound_and_idempotence(fmt):
    h = np.random.default_rng(3).standard_normal((40, 96))
    v, gs = fp4.fake_quant(h, fmt)
    v = v * gs[:, None]
    g = quant.GROUP[fmt]
    amax = np.repeat(np.abs(h.reshape(40, -1, g)).max(-1), g, axis=1)
    # half of the widest step (2 of 6) of a scale up to 2x (MXFP4) or 17/16 (E4M3 rounding) the needed
    # one; or, below 6, the saturation of a block whose scale rounded down by 1/17
    assert np.all(np.abs(v - h) <= amax / 6 * (2.0 if fmt == MX else 17 / 16) + 1e-12)
    v2, gs2 = fp4.fake_quant(v, fmt)
    if fmt == MX:
        assert np.array_equal(v2, v)


def test_tiles_are_the_documented_permutation():
    s = torch.arange(2 * 200 * 10, dtype=torch.int64).remainder(251).to(torch.uint8).view(2, 200, 10)
    pad = torch.zeros(2, 256, 12, dtype=torch.uint8)
    pad[:, :200, :10] = s
    want = pad.view(2, 2, 4, 32, 3, 4).permute(0, 1, 4, 3, 2, 5)
    assert np.array_equal(fp4.tile_scales(s.numpy()), want.numpy())


def test_product_of_exact_integers():
    """Powers of two and small integers: every product exact, checked against a python loop."""
    rng = np.random.default_rng(4)
    codes = rng.integers(0, 16, (5, 64)).astype(np.uint8)
    scales = rng.integers(120, 134, (5, 2)).astype(np.uint8)
    a = fp4.dequant_rows(codes, scales, MX)
    w = rng.integers(0, 16, (3, 64)).astype(np.uint8)
    ws = rng.integers(120, 134, (3, 2)).astype(np.uint8)
    got, mags = fp4.product(a, np.ones(5), quant.pack_nibbles(w), ws, None, MX)
    for t in range(5):
        for n in range(3):
            terms = [Fraction(float(e2m1_decode(codes[t, k]))) * Fraction(float(e8m0_decode(scales[t, k // 32])))
                     * Fraction(float(e2m1_decode(w[n, k]))) * Fraction(float(e8m0_decode(ws[n, k // 32])))
                     for k in range(64)]
            assert Fraction(float(got[t, n])) == sum(terms)
            assert Fraction(float(mags[t, n])) == sum(abs(x) for x in terms)


def test_layer_with_one_expert_is_an_mlp():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 32))
    w13 = rng.standard_normal((1, 64, 32)).astype(np.float32) * 0.2
    w2 = rng.standard_normal((1, 32, 32)).astype(np.float32) * 0.2
    c13, s13, g13 = quant.quantize(w13, NV)
    c2, s2, g2 = quant.quantize(w2, NV)
    ids, wts = np.zeros((3, 1), dtype=np.int32), np.ones((3, 1), dtype=np.float32)
    out = fp4.fused_moe_a4(x, c13, s13, g13, c2, s2, g2, ids, wts, "silu", NV, 1)
    xv, xg = fp4.fake_quant(x, NV)
    a = torch.from_numpy(xv * xg[:, None]) @ torch.from_numpy(quant.dequant(c13[0], s13[0], NV, g13[0])).T
    a = a.to(torch.bfloat16).double()
    h = (torch.nn.functional.silu(a[:, :32]) * a[:, 32:]).numpy()
    hv, hg = fp4.fake_quant(h, NV)
    y = torch.from_numpy(hv * hg[:, None]) @ torch.from_numpy(quant.dequant(c2[0], s2[0], NV, g2[0])).T
    assert np.allclose(out, y.to(torch.bfloat16).double().numpy(), rtol=2**-7, atol=1e-6)
    dropped = fp4.fused_moe_a4(x, c13, s13, g13, c2, s2, g2, ids - 1, wts, "silu", NV, 1)
    assert not dropped.any()
    assert np.all(e4m3_decode(s13) >= 0)
