"""Block-scaled FP8 operands, their products and the layer of them, restated in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The pages have no counterpart.  What is fixed here:

* blocks of 128 along K, one row (activations) or 128 rows (weights) high;
* s = amax / 448 rounded to float32, or the least power of two with
  amax <= 448 s; at least 2^-126; 1 where amax is 0;
* code = E4M3 of the quotient h / s rounded to float32, nearest even, saturating;
* a product sums sa sw a w over K exactly.
"""

from __future__ import annotations

import numpy as np

from .formats import bf16_rn, e4m3_decode, e4m3_rn_satfinite
from .fp4 import _least_pow2_exponent
from .moe import activation_fn
from .routing import local_experts

BLOCK = 128


def block_amax(h, block_rows=1):
    """Largest magnitudes [ceil(R / block_rows), ceil(K / 128)] of h [R, K]."""
    r, k = h.shape
    return np.array([[np.abs(h[i:i + block_rows, j:j + BLOCK]).max() for j in range(0, k, BLOCK)]
                     for i in range(0, r, block_rows)]).reshape(-(-r // block_rows), -(-k // BLOCK))


def scales(h, block_rows=1, pow2=False):
    """The scales as the float32 values the operator holds."""
    a = block_amax(np.asarray(h, dtype=np.float64), block_rows)
    if pow2:
        return np.where(a > 0, np.ldexp(1.0, _least_pow2_exponent(a, 448.0, -126)), 1.0)
    return np.where(a > 0, np.maximum((a / 448.0).astype(np.float32).astype(np.float64), 2.0**-126), 1.0)


def spread(s, shape, block_rows=1):
    """A block's scale at each of its elements."""
    return np.repeat(np.repeat(s, block_rows, axis=0), BLOCK, axis=1)[: shape[0], : shape[1]]


def e4m3(q):
    """The value of the code nearest to q (already rounded to float32), with its sign."""
    return np.copysign(e4m3_decode(e4m3_rn_satfinite(np.abs(q))), q)


def quantize(h, block_rows=1, pow2=False):
    """(code values [R, K], scales): the operand is their product."""
    h = np.asarray(h, dtype=np.float64)
    s = scales(h, block_rows, pow2)
    q = (h / spread(s, h.shape, block_rows)).astype(np.float32).astype(np.float64)
    return e4m3(q), s


def dequant(codes, s, block_rows=1):
    return codes * spread(s, codes.shape, block_rows)


def fake_quant(h, pow2=False):
    return dequant(*quantize(h, 1, pow2))


def product(a, w):
    """(a w^T, sum of the terms' magnitudes) of dequantised operands."""
    return a @ w.T, np.abs(a) @ np.abs(w).T


def fused_moe_fp8(x, w13, w2, topk_ids, topk_weights, act, num_global_experts, expert_map=None, swiglu=None):
    """The layer on dequantised weights w13 [E, N1, H], w2 [E, H, I]: x and h quantised by rows, FC1 kept in full,
    every route's FC2 output rounded to bf16, the routes of a token summed and rounded once."""
    x = np.asarray(x, dtype=np.float64)
    loc = local_experts(topk_ids, num_global_experts, w13.shape[0], expert_map)
    out = np.zeros(x.shape)
    xa = fake_quant(x)
    for e in range(w13.shape[0]):
        t, j = np.nonzero(loc == e)
        if len(t):
            h = fake_quant(activation_fn(xa[t] @ w13[e].T, act, w2.shape[2], swiglu))
            np.add.at(out, t, np.asarray(topk_weights, dtype=np.float64)[t, j][:, None] * bf16_rn(h @ w2[e].T))
    return bf16_rn(out)
