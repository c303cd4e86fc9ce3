"""Block-scaled FP4 activations and the FP4 x FP4 products, restated in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The pages have no counterpart (their layer keeps activations in 16 bits); the
number formats are those of ``formats.py``.  What is fixed here:

* a row of h is cut along K into blocks of 16 (NVFP4) or 32 (MXFP4);
* NVFP4: s = e4m3_rn_satfinite(amax_block / (6 gs)), c = e2m1_rn_sat(h / (s gs)),
  c = 0 where s gs = 0; gs per row is the least power of two 2^j, j >= -126,
  with amax_row <= 6 * 448 * 2^j (1 for a zero row), per matrix
  amax / (6 * 448) in float32;
* MXFP4: s = 2^j, j the least (>= -127) with amax_block <= 6 * 2^j;
* the product out[t][n] = gs_a[t] gs_w sum_k (c s)_a (c s)_w, exact.
"""

from __future__ import annotations

import numpy as np

from .formats import bf16_rn, e2m1_decode, e2m1_rn_sat, e4m3_decode, e4m3_rn_satfinite, e8m0_decode
from .moe import activation_fn
from .quant import GROUP, MXFP4, dequant
from .routing import local_experts


def _least_pow2_exponent(amax, unit, lowest):
    """Least integer j >= lowest with amax <= unit * 2^j, elementwise (amax > 0)."""
    j = np.ceil(np.log2(np.maximum(amax, 1e-300) / unit)).astype(np.int64)
    j = np.where(np.ldexp(unit, j - 1) >= amax, j - 1, j)  # the logarithm may round either way
    j = np.where(np.ldexp(unit, j) < amax, j + 1, j)
    return np.maximum(j, lowest)


def row_gs(h):
    """Per-row global scales of h [R, K]: powers of two."""
    amax = np.abs(h).max(axis=-1)
    return np.where(amax > 0, np.ldexp(1.0, _least_pow2_exponent(amax, 2688.0, -126)), 1.0)


def matrix_gs(h):
    """The global scale of a whole matrix, as the float32 the operator returns."""
    amax = np.abs(h).max()
    return float(np.float32(amax / 2688.0)) if amax > 0 else 1.0


def quotients(h, fmt, gs=None):
    """(scale ratios [R, B] before rounding or None, scale bytes [R, B], code quotients [R, K])."""
    h = np.asarray(h, dtype=np.float64)
    r, k = h.shape
    b = h.reshape(r, k // GROUP[fmt], GROUP[fmt])
    amax = np.abs(b).max(axis=-1)
    if fmt == MXFP4:
        ratio = None
        s = np.where(amax > 0, _least_pow2_exponent(amax, 6.0, -127) + 127, 0).astype(np.uint8)
        d = e8m0_decode(s)
    else:
        g = np.broadcast_to(np.asarray(gs, dtype=np.float64), (r,))[:, None]
        ratio = amax / (6.0 * g)
        s = e4m3_rn_satfinite(ratio)
        d = e4m3_decode(s) * g
    q = np.where(d[..., None] > 0, b / np.where(d > 0, d, 1.0)[..., None], 0.0)
    return ratio, s, q.reshape(r, k)


def quantize_rows(h, fmt, gs=None):
    """(codes [R, K] 0..15, scale bytes [R, K/g]) of h with the given global scales."""
    _, s, q = quotients(h, fmt, gs)
    zero = np.repeat(e8m0_decode(s) * 0 if fmt == MXFP4 else e4m3_decode(s), GROUP[fmt], axis=1) == 0
    codes = e2m1_rn_sat(q)
    if fmt != MXFP4:
        codes = np.where(zero, 0, codes)
    return codes.astype(np.uint8), s


def dequant_rows(codes, scales, fmt):
    """scale * e2m1(code), without global scales."""
    sv = e8m0_decode(scales) if fmt == MXFP4 else e4m3_decode(scales)
    return e2m1_decode(codes) * np.repeat(sv, GROUP[fmt], axis=1)


def fake_quant(h, fmt):
    """h through the format with per-row global scales: (scale * code values, gs per row)."""
    gs = np.ones(h.shape[0]) if fmt == MXFP4 else row_gs(h)
    codes, s = quantize_rows(h, fmt, None if fmt == MXFP4 else gs)
    return dequant_rows(codes, s, fmt), gs


def tile_scales(scales):
    """Row-major scales [E, R, B] -> tiles [E, ceil(R/128), ceil(B/4), 32, 4, 4], zero-padded (a plain loop)."""
    e, r, b = scales.shape
    out = np.zeros((e, -(-r // 128), -(-b // 4), 32, 4, 4), dtype=np.uint8)
    for row in range(r):
        for blk in range(b):
            out[:, row // 128, blk // 4, row % 32, row % 128 // 32, blk % 4] = scales[:, row, blk]
    return out


def product(a, gs_a, w_codes, w_scales, w_gs, fmt):
    """a [R, K] dequantised (without gs), one weight matrix -> (out [R, N], sum of |terms| [R, N])."""
    w = dequant(w_codes, w_scales, fmt)
    g = np.asarray(gs_a, dtype=np.float64).reshape(-1, 1) * (1.0 if w_gs is None else float(w_gs))
    return a @ w.T * g, np.abs(a) @ np.abs(w).T * np.abs(g)


def fused_moe_a4(x, w13, s13, gs13, w2, s2, gs2, topk_ids, topk_weights, act, fmt, num_global_experts,
                 expert_map=None, swiglu=None):
    """The MoE layer with 4-bit activations: x and h quantised by rows, FC1 and every route's FC2 output
    rounded to bf16, the routes of a token summed and rounded once."""
    x = np.asarray(x, dtype=np.float64)
    e_l, n1 = w13.shape[:2]
    inter = w2.shape[2] * 2
    loc = local_experts(topk_ids, num_global_experts, e_l, expert_map)
    out = np.zeros(x.shape)
    xa, xg = fake_quant(x, fmt)
    for e in range(e_l):
        t, j = np.nonzero(loc == e)
        if not len(t):
            continue
        g13 = None if gs13 is None else gs13[e]
        g2 = None if gs2 is None else gs2[e]
        a = bf16_rn(product(xa[t], xg[t], w13[e], s13[e], g13, fmt)[0])
        h, hg = fake_quant(activation_fn(a, act, inter, swiglu), fmt)
        y = bf16_rn(product(h, hg, w2[e], s2[e], g2, fmt)[0])
        np.add.at(out, t, np.asarray(topk_weights, dtype=np.float64)[t, j][:, None] * y)
    return bf16_rn(out)
