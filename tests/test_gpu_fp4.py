"""GPU tests of the FP4 operators (b4_fp4_*, b4_fused_moe_a4) against the float64 oracle.

Quantisation: codes, scales and global scales equal the oracle's bit for bit, except where the exact quotient lies
within 2^-21 of a rounding tie (the operator divides in fp32; its quotient is off by at most 2^-23 for d rounded and
2^-24 for the division).  With 8- or 11-bit inputs and power-of-two global scales no quotient can come that close
without being the tie itself, so those cases allow nothing.  Products: bf16 / f16 / f32 rounding of the output plus the
tensor core's fp32 accumulation, at most 2^-22 of the terms' magnitude for each of the K / 16 partial sums.
"""

import numpy as np
import pytest
import torch

import workloads as W
from gpu_util import assert_parity, bf16_to_np, dev
from oracle import fp4 as O
from oracle import moe as M
from oracle import quant as Q
from oracle import routing as R
from oracle.formats import e2m1_decode, e2m1_rn_sat, e4m3_decode, e8m0_decode

pytestmark = pytest.mark.gpu

NV, MX = W.NV, W.MX
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ROUND = {BF: 2.0**-8, HF: 2.0**-11, F32: 2.0**-24}  # relative half-ulp of each output type, upper bounds


@pytest.fixture(scope="module")
def b4():
    import w4a16_moe_gb300 as mod

    return mod


def _np(t):
    return t.detach().double().cpu().numpy()


def _randn(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def _unpack(codes, k):
    return Q.unpack_nibbles(codes.cpu().numpy()[..., : k // 2])


def _untile(tiles, rows, blocks):
    """[.., R tiles, K tiles, 32, 4, 4] -> [.., rows, blocks]."""
    t = tiles.cpu().numpy()
    t = np.moveaxis(t, (-5, -2, -3, -4, -1), (-5, -4, -3, -2, -1))  # row tile, row/32, row%32, k tile, block
    return t.reshape(*t.shape[:-5], t.shape[-5] * 128, -1)[..., :rows, :blocks]


def _weights(fmt, e, n, k, seed):
    """Oracle-quantised weights: checkpoint arrays and device operands (codes padded to ld, tiled scales)."""
    w = (np.random.default_rng(seed).standard_normal((e, n, k)) * 0.02).astype(np.float32)
    codes, scales, gs = Q.quantize(w, fmt)
    ld = -(-(k // 2) // 16) * 16
    padded = np.full((e, n, ld), 0xA5, dtype=np.uint8)  # bytes past K/2 must not matter
    padded[..., : k // 2] = codes
    return (codes, scales, gs), (dev(padded), dev(O.tile_scales(scales)), None if gs is None else dev(gs))


def _assert_product(got, want, mags, k, dtype, what=""):
    tol = ROUND[dtype] * np.abs(want) + (k / 16 + 4) * 2.0**-22 * mags + (2.0**-25 if dtype == HF else 0)
    err = np.abs(got - want)
    assert np.all(err <= tol), f"{what}: worst excess {np.max(err - tol):.3e}"


# ------------------------------------------------------------- quantisation


def _act_np(x, act):
    if act is None:
        return x
    return M.activation_fn(x, act, x.shape[1] // (1 if act == "relu2" else 2), W.Workload("x", NV, 1, 1, 1, 1, 1, "silu", ()).swiglu)


def _check_quantised(codes, scales, gs, h, fmt, gs_mode, exact):
    """codes [R, K], scale bytes [R, B], gs [R] against the oracle on h [R, K]."""
    ratio, s, q = O.quotients(h, fmt, gs)
    g = Q.GROUP[fmt]
    near_s = np.zeros(s.shape, bool)
    near_q = np.zeros(q.shape, bool)
    if not exact:
        if fmt == NV:
            grid = e4m3_decode(np.arange(0x7F))
            ties = (grid[1:] + grid[:-1]) / 2
            near_s = (np.abs(ratio[..., None] / ties - 1) < 2.0**-21).any(-1)
        ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
        near_q = (np.abs(np.abs(q)[..., None] / ties - 1) < 2.0**-21).any(-1)
    assert np.array_equal(scales[~near_s], s[~near_s])
    want = e2m1_rn_sat(q)
    if fmt == NV:
        want = np.where(np.repeat(s, g, axis=1) == 0, 0, want)
    ok = near_q | np.repeat(near_s, g, axis=1) | (codes == want)
    assert ok.all(), np.argwhere(~ok)[:5]
    assert np.abs(codes.astype(int) - want.astype(int))[near_q & ~np.repeat(near_s, g, axis=1)].max(initial=0) <= 1


QUANT = [
    # fmt, dtype, groups, m, k, gs mode, act
    (NV, BF, 1, 1, 16, "row", None),
    (NV, BF, 1, 1, 4096, "row", None),
    (NV, BF, 1, 130, 80, "row", None),      # K tail inside a scale tile, rows across a row tile
    (NV, HF, 1, 7, 8208, "row", None),      # more than two chunks a thread
    (NV, F32, 2, 33, 1040, "row", None),
    (NV, BF, 3, 129, 48, "tensor", None),
    (NV, F32, 2, 65, 272, "tensor", None),
    (NV, BF, 2, 5, 336, "given", None),
    (NV, BF, 1, 9, 288, "row", "relu2"),
    (MX, BF, 1, 1, 32, "none", None),
    (MX, BF, 1, 37, 2880, "none", None),
    (MX, HF, 2, 131, 160, "none", None),
    (MX, F32, 1, 3, 8224, "none", None),
    (MX, BF, 1, 9, 288, "none", "relu2"),
]


@pytest.mark.parametrize("layout", ["tiles", "rows"])
@pytest.mark.parametrize("fmt,dtype,groups,m,k,mode,act", QUANT)
def test_quantise_matches_the_oracle(b4, fmt, dtype, groups, m, k, mode, act, layout):
    x = _randn((groups, m, k), m * k + groups, dtype) * torch.exp(_randn((groups, m, 1), 5, F32)).to(dtype)
    x[0, m // 2] = 0  # a zero row
    x[..., :16] *= 2.0**-12  # a block far below its row
    modes = {"none": b4.GS_NONE, "row": b4.GS_ROW, "tensor": b4.GS_TENSOR, "given": b4.GS_GIVEN}
    cfg = b4.Fp4Config(m=m, k=k, num_groups=groups, format=b4.FORMATS[fmt], x_dtype=dtype, gs_mode=modes[mode],
                       activation=b4.ACTIVATIONS.get(act),
                       scale_layout=b4.SCALES_TILED if layout == "tiles" else b4.SCALES_ROWS)
    codes, scales, gs = b4.fp4_empty(cfg, "cuda")
    codes.fill_(0xEE), scales.fill_(0xEE)
    if mode == "given":
        gs.copy_(torch.tensor([0.013, 0.0007])[:groups])
    values = torch.empty(groups, m, k, dtype=dtype, device="cuda")
    b4.fp4_quantize(cfg, x.cuda(), codes, scales, gs, values=values)
    torch.cuda.synchronize()
    c = _unpack(codes, k)
    sc = scales.cpu().numpy() if layout == "rows" else _untile(scales, m, k // Q.GROUP[fmt])
    h = _np(x)
    for e in range(groups):
        he = _act_np(h[e], act)
        g = None
        if mode == "row":
            g = _np(gs)[e]
            assert np.array_equal(g, O.row_gs(he))
        elif mode == "tensor":
            g = np.full(m, _np(gs)[e])
            assert g[0] == O.matrix_gs(he)
        elif mode == "given":
            g = np.full(m, _np(gs)[e])
        exact = act is None and (mode in ("none", "row")) and dtype != F32 or fmt == MX and act is None
        _check_quantised(c[e], sc[e], g, he, fmt, mode, exact)
        # values: the code times the fp32 step s gs, each product rounded to fp32, then to x's type
        step = (e4m3_decode if fmt == NV else e8m0_decode)(sc[e]).astype(np.float32)
        if g is not None:
            step = step * g.astype(np.float32)[:, None]
        v = e2m1_decode(c[e]).astype(np.float32) * np.repeat(step, Q.GROUP[fmt], axis=1)
        assert torch.equal(values[e].cpu(), torch.from_numpy(v).to(dtype))
    if layout == "tiles":  # the padding of a stack's tiles is zero
        full = np.moveaxis(scales.cpu().numpy(), (-5, -2, -3, -4, -1), (-5, -4, -3, -2, -1))
        full = full.reshape(groups, full.shape[1] * 128, -1)
        assert not full[:, m:].any() and not full[:, :, k // Q.GROUP[fmt]:].any()


@pytest.mark.parametrize("act", ["silu", "swiglu_oai"])
def test_gated_quantise_is_within_a_step(b4, act):
    """The gated prologue's exponential is approximate: values are within half a code step plus its error."""
    m, k = 50, 352
    x = _randn((m, 2 * k), 8, BF, 2.0)
    cfg = b4.Fp4Config(m=m, k=k, activation=b4.ACTIVATIONS[act])
    codes, scales, gs = b4.fp4_empty(cfg, "cuda")
    values = torch.empty(m, k, dtype=BF, device="cuda")
    b4.fp4_quantize(cfg, x.cuda(), codes, scales, gs, values=values)
    h = _act_np(_np(x), act)
    s = np.repeat(e4m3_decode(_untile(scales, m, k // 16)[0]), 16, axis=1) * _np(gs)[0][:, None]
    # half of the widest step (6 - 4), or the 1/17 by which a scale may round down below amax / 6; bf16 values
    assert np.all(np.abs(_np(values) - h) <= s * (1 + 1e-3) + ROUND[BF] * np.abs(h))


def test_special_values(b4):
    """NaN and infinities: where they go and that they stay in their row or block."""
    inf, nan = float("inf"), float("nan")
    x = _randn((6, 96), 3, BF)
    x[0, 5], x[1, 40], x[2, 70] = nan, inf, -inf
    x[3] = 0
    x[4] = 2.0**-130  # subnormal in bf16 (below 2^-126)
    for fmt, mode in ((b4.NVFP4, b4.GS_ROW), (b4.NVFP4, b4.GS_GIVEN), (b4.MXFP4, b4.GS_NONE)):
        cfg = b4.Fp4Config(m=6, k=96, format=fmt, gs_mode=mode)
        codes, scales, gs = b4.fp4_empty(cfg, "cuda")
        if mode == b4.GS_GIVEN:
            gs.fill_(2.0**-9)
        values = torch.empty(6, 96, dtype=BF, device="cuda")
        b4.fp4_quantize(cfg, x.cuda(), codes, scales, gs, values=values)
        v = _np(values)
        block = 32 if fmt == b4.MXFP4 else 16
        assert not v[3].any()
        assert np.isfinite(v[5]).all() and np.abs(v[5] - _np(x)[5]).max() < 0.6
        if mode == b4.GS_ROW:  # the row's scale is not finite: so is every value, and every product with it
            assert np.isnan(v[:3]).all()
            assert np.isnan(_np(gs)[0][:3]).all() and _np(gs)[0][3] == 1 and _np(gs)[0][4] == 2.0**-126
        else:
            bad = np.zeros(96, bool)
            bad[:block] = True
            assert np.isnan(v[0][bad]).all() and np.isfinite(v[0][~bad]).all()
            b1, b2 = 40 // block, 70 // block
            top = 6 * 448 * 2.0**-9 if fmt == b4.NVFP4 else inf  # saturated; MXFP4's 6 2^127 passes the type's range
            assert v[1, 40] == top and v[2, 70] == -top
            for r, b in ((1, b1), (2, b2)):
                out = np.ones(96, bool)
                out[b * block:(b + 1) * block] = False
                assert np.isfinite(v[r][out]).all()
        if fmt == b4.MXFP4:
            assert np.all(np.abs(v[4] - 2.0**-130) <= 2.0**-130)


@pytest.mark.parametrize("act", [None, "silu", "relu2"])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_nan_and_infinity_of_every_type(b4, dtype, act):
    """By row: rows with a NaN or an infinity, of either sign and in any place of a chunk, give NaN, and only they;
    the other rows' bits do not depend on them."""
    m, k = 36, 80
    x = _randn((m, 2 * k if act == "silu" else k), 5, dtype)
    clean = x.clone()
    bad = []
    for i, v in enumerate((float("nan"), float("inf"), -float("inf"))):
        for j, col in enumerate((0, 1, 15, 16, 47, 78, 79)):
            r = 1 + 8 * i + j
            x[r, col] = v
            if not (act == "relu2" and v < 0):  # ReLU of -inf is 0
                bad.append(r)
    good = [r for r in range(m) if r not in bad]
    cfg = b4.Fp4Config(m=m, k=k, x_dtype=dtype, activation=b4.ACTIVATIONS.get(act))
    outs = []
    for rows in (x, clean):
        codes, scales, gs = b4.fp4_empty(cfg, "cuda")
        values = torch.empty(m, k, dtype=dtype, device="cuda")
        b4.fp4_quantize(cfg, rows.cuda(), codes, scales, gs, values=values)
        outs.append((codes[..., : k // 2], gs.reshape(-1), values))  # (bytes past K / 2 are padding)
    assert torch.isnan(outs[0][1][bad]).all() and torch.isnan(outs[0][2][bad]).all()
    same = [r for r in good if torch.equal(x[r], clean[r])]
    assert len(same) >= m - 21
    for a, b in zip(*outs):
        assert torch.equal(a[..., same, :] if a.dim() > 1 else a[same], b[..., same, :] if b.dim() > 1 else b[same])
    assert torch.isfinite(outs[0][2][good]).all()


def test_given_scale_that_is_far_off(b4):
    """Saturation at 6 * 448 gs, all-zero blocks below it, and scales outside the reciprocal's safe range."""
    x = _randn((4, 64), 4, F32)
    for g in (2.0**-40, 2.0**40, 2.0**-119, 1e-38):
        cfg = b4.Fp4Config(m=4, k=64, gs_mode=b4.GS_GIVEN, x_dtype=F32)
        codes, scales, gs = b4.fp4_empty(cfg, "cuda")
        gs.fill_(g)
        values = torch.empty(4, 64, dtype=F32, device="cuda")
        b4.fp4_quantize(cfg, x.cuda(), codes, scales, gs, values=values)
        g32 = float(gs[0])
        v = _np(values)
        if g < 1:
            sat = np.abs(_np(x)) >= 6 * 448 * g32
            assert sat.all() and np.array_equal(v, np.float32(np.sign(_np(x)) * 6 * np.float32(448 * g32)))
        else:
            assert not v.any()


@pytest.mark.parametrize("dtype,shift,stride", [(BF, 0, 88), (BF, 1, 83), (HF, 3, 96), (F32, 1, 81), (BF, 8, 80)])
def test_strided_and_unaligned_rows(b4, dtype, shift, stride):
    m, k = 21, 80
    base = _randn((m * stride + 16,), 9, dtype).cuda()
    x = base[shift:shift + m * stride].view(m, stride)[:, :k]
    dense = b4.Fp4Config(m=m, k=k, x_dtype=dtype)
    strided = b4.Fp4Config(m=m, k=k, x_dtype=dtype, x_stride=stride)
    a, b = b4.fp4_empty(dense, "cuda"), b4.fp4_empty(strided, "cuda")
    b4.fp4_quantize(dense, x.contiguous(), *a)
    b4.fp4_quantize(strided, x, *b)
    for u, v in zip(a, b):
        assert torch.equal(u[..., : k // 2] if u is a[0] else u, v[..., : k // 2] if v is b[0] else v)


def test_gather_and_ragged_scales(b4):
    """Rows gathered through an index, groups of every kind: the tiles of group e start at offsets[e] / 128 + e."""
    k, tokens, div = 96, 40, 3
    counts = [0, 1, 130, 0, 127, 128, 3, 0]
    m = sum(counts) + 5
    off = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    rows = np.random.default_rng(6).integers(0, tokens * div, m).astype(np.int32)
    rows[3], rows[10] = -1, tokens * div + 7  # a zero row each
    x = _randn((tokens, k), 7, BF)
    cfg = b4.Fp4Config(m=m, k=k, num_groups=len(counts), row_div=div)
    codes, scales, gs = b4.fp4_empty(cfg, "cuda", ragged=True)
    codes.fill_(0xEE), gs.fill_(7.0)
    b4.fp4_quantize(cfg, x.cuda(), codes, scales, gs, rows=dev(rows), offsets=dev(off))
    c, g = _unpack(codes, k), _np(gs)
    src = rows // div
    h = np.where((rows < 0)[:, None] | (src >= tokens)[:, None], 0.0, _np(x)[np.clip(src, 0, tokens - 1)])
    tiles = scales.cpu().numpy()
    for e, n in enumerate(counts):
        if not n:
            continue
        lo = off[e]
        t0 = lo // 128 + e
        part = torch.from_numpy(tiles[t0:t0 + -(-n // 128)])
        sc = _untile(part[None], n, k // 16)[0]
        assert np.array_equal(g[lo:lo + n], O.row_gs(h[lo:lo + n]))
        _check_quantised(c[lo:lo + n], sc, g[lo:lo + n], h[lo:lo + n], NV, "row", True)
    assert np.all(g[off[-1]:] == 7.0) and np.all(codes.cpu().numpy()[off[-1]:] == 0xEE)  # not written


@pytest.mark.parametrize("fmt", [NV, MX])
def test_tile_scales(b4, fmt):
    g = Q.GROUP[fmt]
    src = np.random.default_rng(1).integers(0, 127, (3, 150, 7)).astype(np.uint8)
    cfg = b4.Fp4Config(m=150, k=7 * g, num_groups=3, format=b4.FORMATS[fmt])
    assert np.array_equal(b4.fp4_tile_scales(cfg, dev(src)).cpu().numpy(), O.tile_scales(src))


def test_quantised_weights_feed_the_w4a16_layer(b4):
    """Row-major codes and scales are the checkpoint layout: equal to the oracle's quantiser, and accepted by
    prepare_weights and the dense W4A16 layer."""
    n, k = 256, 512
    w = _randn((1, n, k), 12, F32, 0.02)
    cfg = b4.Fp4Config(m=n, k=k, gs_mode=b4.GS_TENSOR, x_dtype=F32, scale_layout=b4.SCALES_ROWS)
    codes, scales, gs = b4.fp4_empty(cfg, "cuda")
    b4.fp4_quantize(cfg, w.cuda(), codes, scales, gs)
    lc = b4.linear_config(5, n, k)
    pw, ps = b4.prepare_linear_weights(lc, codes, scales)
    x = _randn((5, k), 13, BF)
    out = torch.empty(5, n, dtype=BF, device="cuda")
    ws = torch.empty(b4.linear_workspace_bytes(lc), dtype=torch.uint8, device="cuda")
    b4.linear(lc, x.cuda(), pw, ps, gs, out, ws)
    torch.cuda.synchronize()
    oc, osc, ogs = Q.quantize(w.numpy(), NV)
    assert (codes.cpu().numpy() == oc).mean() > 0.9999 and ogs[0] == float(gs[0])
    from oracle import linear as L

    assert_parity(bf16_to_np(out), L.linear(_np(x), oc, osc, ogs, NV), "quantised weights in the W4A16 layer")


# ------------------------------------------------------------------ product


def _operand(b4, cfg, fmt, h, ragged_offsets=None):
    """Oracle-quantised rows h [R, K] as a device operand with tiles placed by the documented rule."""
    gs = None if fmt == MX else O.row_gs(h)
    codes, s = O.quantize_rows(h, fmt, gs)
    packed = np.full((h.shape[0], cfg.ld), 0x5A, dtype=np.uint8)
    packed[:, : cfg.k // 2] = Q.pack_nibbles(codes)
    kt = -(-cfg.k // (4 * Q.GROUP[fmt]))
    if ragged_offsets is None:
        e = cfg.num_groups
        tiles = O.tile_scales(s.reshape(e, cfg.m, -1))
    else:
        tiles = np.full((cfg.m // 128 + cfg.num_groups, kt, 32, 4, 4), 0x7F if fmt == NV else 0xFF, dtype=np.uint8)
        for e in range(cfg.num_groups):
            lo, hi = ragged_offsets[e], ragged_offsets[e + 1]
            if hi > lo:
                t = O.tile_scales(s[None, lo:hi])[0]
                live = np.zeros((t.shape[0] * 128, 1), bool)
                live[: hi - lo] = True  # rows past the group stay NaN: they must not matter
                live = np.moveaxis(live.reshape(-1, 4, 32), 1, 2)[:, None, :, :, None]
                at = tiles[lo // 128 + e: lo // 128 + e + t.shape[0]]
                at[...] = np.where(live, t, at)
    a = O.dequant_rows(codes, s, fmt)
    return a, gs, (dev(packed), dev(tiles), None if gs is None else dev(gs.astype(np.float32)))


DENSE = [
    # fmt, groups, m, n, k, out dtype
    (NV, 1, 1, 1, 16, BF),
    (NV, 1, 1, 128, 64, F32),
    (NV, 1, 1, 300, 4096, BF),
    (NV, 1, 16, 129, 48, HF),
    (NV, 1, 17, 127, 272, F32),
    (NV, 1, 64, 256, 1040, BF),
    (NV, 1, 65, 100, 256, BF),       # the wide unit, one live scale tile
    (NV, 1, 193, 131, 528, F32),     # a second wide unit of one row, half a tile in
    (NV, 1, 400, 257, 320, BF),
    (NV, 3, 70, 130, 112, BF),       # a stack
    (MX, 1, 1, 5, 32, BF),
    (MX, 1, 3, 1440, 2880, BF),
    (MX, 1, 37, 129, 96, F32),
    (MX, 1, 200, 64, 160, HF),
    (MX, 2, 200, 130, 288, BF),
    # one unit shared by a cluster along K (its parts of 16 rows: one, three, four)
    (MX, 1, 16, 200, 4096, HF),
    (NV, 1, 40, 100, 4112, BF),
    (NV, 1, 64, 70, 4096, F32),
    (NV, 2, 5, 130, 2048, BF),
    # pairs of SMs, units of 128 rows, then of 256
    (NV, 1, 520, 2571, 272, F32),
    (MX, 1, 520, 2576, 160, BF),
    (NV, 3, 300, 1500, 112, BF),
    (NV, 1, 1030, 2568, 1296, BF),
    (MX, 1, 1030, 2568, 160, HF),
    (MX, 2, 700, 2603, 96, BF),
    # pairs, more than two rounds of units of 128 rows and of 256
    (NV, 1, 100, 40000, 80, BF),
    (MX, 1, 1030, 8000, 96, HF),
    # the last units of 256 rows in halves, one of them ragged
    (NV, 1, 1970, 2500, 80, BF),
    (MX, 2, 1000, 2500, 96, F32),
]


@pytest.mark.parametrize("fmt,groups,m,n,k,dtype", DENSE)
def test_product_matches_the_oracle(b4, fmt, groups, m, n, k, dtype):
    cfg = b4.Fp4Config(m=m, n=n, k=k, num_groups=groups, format=b4.FORMATS[fmt], out_dtype=dtype)
    h = _np(_randn((groups * m, k), 17, BF))
    a, ga, ad = _operand(b4, cfg, fmt, h)
    (codes, scales, gs), wd = _weights(fmt, groups, n, k, 18)
    out = torch.full((groups * m, n), float("nan"), dtype=dtype, device="cuda")
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    b4.fp4_matmul(cfg, *ad, *wd, out, device_status=status)
    got = _np(out)
    assert not status.any()
    for e in range(groups):
        rows = slice(e * m, (e + 1) * m)
        want, mags = O.product(a[rows], np.ones(m) if ga is None else ga[rows], codes[e], scales[e],
                               None if gs is None else gs[e], fmt)
        _assert_product(got[rows], want, mags, k, dtype, f"group {e}")


def test_product_with_given_scales_and_output_stride(b4):
    m, n, k = 50, 70, 64
    h = _np(_randn((m, k), 21, BF))
    codes, s = O.quantize_rows(h, NV, 0.01)
    a = O.dequant_rows(codes, s, NV)
    cfg = b4.Fp4Config(m=m, n=n, k=k, gs_mode=b4.GS_GIVEN, out_stride=91)
    (wc, wsc, wg), wd = _weights(NV, 1, n, k, 22)
    buf = torch.full((m, 91), 7.0, dtype=BF, device="cuda")
    b4.fp4_matmul(cfg, dev(Q.pack_nibbles(codes)), dev(O.tile_scales(s[None])), torch.tensor([0.01]).cuda(), *wd,
                  buf[:, :n])
    want, mags = O.product(a, np.full(m, np.float32(0.01)), wc[0], wsc[0], wg[0], NV)
    _assert_product(_np(buf[:, :n]), want, mags, k, BF)
    assert torch.all(buf[:, n:] == 7.0)


def test_nan_scale_reaches_its_row_only(b4):
    m, n, k = 20, 40, 64
    cfg = b4.Fp4Config(m=m, n=n, k=k, out_dtype=F32)
    h = _np(_randn((m, k), 23, BF))
    _, _, (codes, tiles, gs) = _operand(b4, cfg, NV, h)
    tiles[0, 0, 0, 5, 0, 2] = 0x7F  # row 5, third block
    (_, _, _), wd = _weights(NV, 1, n, k, 24)
    out = torch.empty(m, n, dtype=F32, device="cuda")
    b4.fp4_matmul(cfg, codes, tiles, gs, *wd, out)
    got = _np(out)
    assert np.isnan(got[5]).all() and np.isfinite(np.delete(got, 5, 0)).all()


RAGGED = [
    (NV, [3], 96, 80, 5),
    (NV, [0, 1, 64, 65, 0, 130, 7, 0], 200, 272, 9),      # pairs, one unit of two rows past 128
    (NV, [0, 400, 193, 1, 192, 0], 130, 64, 3),           # wide units
    (NV, [0, 0, 0], 40, 64, 6),                           # nothing live
    (NV, [2] * 64 + [0] * 960, 40, 64, 0),                # as many groups as there can be
    (MX, [5, 0, 300, 127, 129], 150, 96, 4),
    (MX, [1] * 30, 70, 160, 2),
    (NV, [1, 0, 2, 5], 130, 2048, 2),                     # split along K
    (NV, [100, 0, 128, 129, 65], 300, 528, 3),            # pairs, units of 128 rows
    (MX, [400, 300, 0, 193], 270, 288, 7),                # pairs, units of 256 rows
    (NV, [0, 1, 65, 0, 130, 7] + [0] * 10, 200, 272, 9),  # a small mean: units of 64 rows at 0 and 64 of a scale tile
    (MX, [70, 5] + [0] * 8, 150, 96, 3),
    (NV, [300, 0, 129, 256, 70, 1, 385], 700, 80, 4),     # units of 256 rows from three places at once
]


@pytest.mark.parametrize("scatter", [False, True])
@pytest.mark.parametrize("fmt,counts,n,k,spare", RAGGED)
def test_ragged_product(b4, fmt, counts, n, k, spare, scatter):
    e = len(counts)
    m = sum(counts) + spare
    off = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    cfg = b4.Fp4Config(m=m, n=n, k=k, num_groups=e, format=b4.FORMATS[fmt], out_dtype=F32)
    h = _np(_randn((m, k), 31, BF))
    a, ga, ad = _operand(b4, cfg, fmt, h, off)
    few = min(e, 64)
    (codes, scales, gs), (wc, wt, wg) = _weights(fmt, few, n, k, 32)
    rep = -(-e // few)
    wd = (wc.repeat(rep, 1, 1)[:e], wt.repeat(rep, 1, 1, 1, 1, 1)[:e], None if wg is None else wg.repeat(rep)[:e])
    out = torch.full((m, n), 7.0, device="cuda")
    to = None
    if scatter:
        to = np.random.default_rng(33).permutation(m).astype(np.int32)
        to[:2] = (-1, m)  # dropped
    b4.fp4_matmul(cfg, *ad, *(None if w is None else w.contiguous() for w in wd), out, offsets=dev(off),
                  out_rows=None if to is None else dev(to))
    got = _np(out)
    seen = np.zeros(m, bool)
    for g in range(e):
        lo, hi = off[g], off[g + 1]
        if hi == lo:
            continue
        want, mags = O.product(a[lo:hi], np.ones(hi - lo) if ga is None else ga[lo:hi], codes[g % few],
                               scales[g % few], None if gs is None else gs[g % few], fmt)
        dest = np.arange(lo, hi) if to is None else to[lo:hi]
        ok = (dest >= 0) & (dest < m)
        _assert_product(got[dest[ok]], want[ok], mags[ok], k, F32, f"group {g}")
        seen[dest[ok]] = True
    assert np.all(got[~seen] == (7.0 if scatter else 0.0))


# ------------------------------------------------ quantisation and product


LINEAR = [(NV, BF, 1, 300, 272, None), (NV, F32, 70, 130, 80, None), (MX, HF, 37, 129, 160, None),
          (NV, BF, 33, 128, 176, "silu"), (MX, BF, 33, 128, 160, "swiglu_oai"), (NV, BF, 5, 200, 336, "relu2")]


@pytest.mark.parametrize("fmt,dtype,m,n,k,act", LINEAR)
def test_linear(b4, fmt, dtype, m, n, k, act):
    """The composite call: against the oracle, bitwise equal to its two parts, on another stream and in a graph."""
    gated = act in ("silu", "swiglu_oai")
    cfg = b4.Fp4Config(m=m, n=n, k=k, format=b4.FORMATS[fmt], x_dtype=dtype, activation=b4.ACTIVATIONS.get(act))
    x = _randn((m, 2 * k if gated else k), 41, dtype).cuda()
    (codes, scales, gs), wd = _weights(fmt, 1, n, k, 42)
    out = torch.empty(m, n, dtype=BF, device="cuda")
    ws = torch.empty(b4.fp4_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    b4.fp4_linear(cfg, x, *wd, out, ws)
    torch.cuda.synchronize()
    b4.check_status(ws)
    a, ga = O.fake_quant(_act_np(_np(x), act), fmt)
    want = O.product(a, ga, codes[0], scales[0], None if gs is None else gs[0], fmt)[0]
    assert_parity(_np(out), want, "fp4_linear")

    parts = b4.fp4_empty(cfg, "cuda")
    again = torch.empty_like(out)
    b4.fp4_quantize(cfg, x, *parts)
    b4.fp4_matmul(cfg, *parts, *wd, again)
    assert torch.equal(out, again)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    again.zero_()
    stream.wait_stream(torch.cuda.current_stream())
    b4.fp4_linear(cfg, x, *wd, again, ws, stream=stream)
    stream.synchronize()
    assert torch.equal(out, again)

    again.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b4.fp4_linear(cfg, x, *wd, again, ws)
    again.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, again)


FEW = [
    # fmt, x dtype, out dtype, m, n, k, act, gs mode, x shift, row padding
    (NV, BF, BF, 1, 130, 4096, None, "row", 0, 0), (NV, F32, F32, 2, 1, 16, None, "row", 0, 0),
    (NV, HF, HF, 3, 257, 1040, None, "row", 3, 9), (NV, BF, F32, 4, 128, 2320, None, "row", 1, 2),
    (NV, F32, BF, 5, 90, 528, None, "row", 1, 5), (NV, BF, BF, 4, 200, 208, None, "given", 0, 8),
    (MX, BF, HF, 2, 150, 2880, None, "none", 0, 0), (MX, F32, F32, 3, 40, 32, None, "none", 1, 0),
    (MX, HF, BF, 4, 129, 288, None, "none", 5, 1), (NV, BF, BF, 3, 140, 1424, "silu", "row", 0, 0),
    (NV, HF, F32, 4, 60, 80, "swiglu_oai", "row", 2, 4), (MX, BF, BF, 2, 30, 96, "silu", "none", 1, 1),
    (NV, F32, F32, 2, 70, 272, "relu2", "given", 0, 0),
]


@pytest.mark.parametrize("fmt,dtype,odtype,m,n,k,act,mode,shift,pad", FEW)
def test_linear_of_few_rows(b4, fmt, dtype, odtype, m, n, k, act, mode, shift, pad):
    """Few rows are quantised by the product's own kernel: the same bits as the two calls, an infinite and a NaN
    row among them, from strided and unaligned rows, and nothing written past the output's rows."""
    width = 2 * k if act in ("silu", "swiglu_oai") else k
    stride = width + pad
    base = _randn((m * stride + shift,), 43, dtype).cuda()
    x = base[shift:].view(m, stride)[:, :width]
    if m > 2:
        x[1, width // 2] = float("inf")
        x[2, 0] = float("nan")
    cfg = b4.Fp4Config(m=m, n=n, k=k, format=b4.FORMATS[fmt], x_dtype=dtype, out_dtype=odtype, x_stride=stride,
                       out_stride=n + pad, activation=b4.ACTIVATIONS.get(act), gs_mode=getattr(b4, "GS_" + mode.upper()))
    gs = torch.full((1,), 2.0**-8, device="cuda") if mode == "given" else None
    _, wd = _weights(fmt, 1, n, k, 44)
    parts = b4.fp4_empty(cfg, "cuda")
    if mode == "given":
        parts[2].copy_(gs)
    b4.fp4_quantize(cfg, x, *parts)
    want, got = (torch.full((m + 1, n + pad), 7.0, dtype=odtype, device="cuda") for _ in range(2))
    b4.fp4_matmul(cfg, *parts, *wd, want[:m, :n])
    ws = torch.empty(b4.fp4_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    b4.fp4_linear(cfg, x, *wd, got[:m, :n], ws, **({} if gs is None else {"x_gs": gs}))
    b4.check_status(ws)
    torch.testing.assert_close(got, want, rtol=0, atol=0, equal_nan=True)
    assert torch.isfinite(got[0]).all() and torch.all(got[m] == 7.0) and torch.all(got[:, n:] == 7.0)


@pytest.mark.parametrize("fmt,k", [(NV, 80), (NV, 2064), (MX, 2048)])
@pytest.mark.parametrize("counts", [[1] * 8, [8], [0, 3, 0, 0, 4], [0, 0], [2, 1, 5]])
def test_grouped_linear_of_few_rows(b4, fmt, k, counts):
    """As above for a few gathered rows by group, in place and scattered: groups empty, of one row and of all."""
    n, e, tokens, div = 140, len(counts), 5, 2
    m = 8
    off = dev(np.concatenate(([0], np.cumsum(counts))).astype(np.int32))
    rows = dev(np.array([3, 0, 9, -1, 4, 11, 1, 8], dtype=np.int32))  # -1 and 11 / 2 are no token: zero rows
    to = dev(np.array([5, 2, -1, 0, 8, 7, 1, 3], dtype=np.int32))     # -1 and 8 are dropped
    x = _randn((tokens, k), 45, BF).cuda()
    cfg = b4.Fp4Config(m=m, n=n, k=k, num_groups=e, format=b4.FORMATS[fmt], row_div=div)
    _, wd = _weights(fmt, e, n, k, 46)
    parts = b4.fp4_empty(cfg, "cuda", ragged=True)
    b4.fp4_quantize(cfg, x, *parts, rows=rows, offsets=off)
    ws = torch.empty(b4.fp4_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    for out_rows in (None, to):
        want, got = (torch.full((m, n), 7.0, dtype=BF, device="cuda") for _ in range(2))
        b4.fp4_matmul(cfg, *parts, *wd, want, offsets=off, out_rows=out_rows)
        b4.fp4_linear(cfg, x, *wd, got, ws, rows=rows, offsets=off, out_rows=out_rows)
        b4.check_status(ws)
        assert torch.equal(got, want) and torch.isfinite(got).all()


def test_grouped_linear_from_packed_routes(b4):
    """Routes packed by b4_route_pack (drops included), rows gathered, outputs by expert."""
    wl = W.WORKLOADS["mxfp4"].scaled(hidden=160, inter=96, experts=7)
    m, k, e = 45, 160, wl.num_local_experts
    ids, _ = W.routing(wl, m, 3)
    em = W.expert_map(wl)
    counts, off, routes = R.route_pack(ids, wl.num_global_experts, e, em)
    mc = b4.MoEConfig(m, wl.top_k, wl.num_global_experts, e, 160, 96, format=b4.MXFP4, expert_map=dev(em))
    dcounts, doff = torch.empty(e, dtype=torch.int32, device="cuda"), torch.empty(e + 1, dtype=torch.int32, device="cuda")
    droutes = torch.empty(routes.shape[0], dtype=torch.int32, device="cuda")
    b4.route_pack(mc, dev(ids), dcounts, doff, droutes)
    rows = m * wl.top_k
    cfg = b4.Fp4Config(m=rows, n=100, k=k, num_groups=e, format=b4.MXFP4, row_div=wl.top_k)
    x = _randn((m, k), 51, BF)
    (codes, scales, _), wd = _weights(MX, e, 100, k, 52)
    out = torch.full((rows, 100), 9.0, dtype=BF, device="cuda")
    ws = torch.empty(b4.fp4_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    b4.fp4_linear(cfg, x.cuda(), *wd, out, ws, rows=droutes, offsets=doff)
    got = _np(out)
    a, _ = O.fake_quant(_np(x), MX)
    for g in range(e):
        t = routes[off[g]:off[g + 1]] // wl.top_k
        want, mags = O.product(a[t], np.ones(len(t)), codes[g], scales[g], None, MX)
        _assert_product(got[off[g]:off[g + 1]], want, mags, k, BF, f"expert {g}")
    assert not got[off[-1]:].any() and off[-1] < rows


def test_operand_beyond_32_bit_offsets(b4):
    """x, codes and out of more than 2^31 bytes: every repeat of a 1000-row pattern gives the same rows."""
    period, reps, k, n = 1000, 1060, 4096, 1030
    x1 = _randn((period, k), 61, BF).cuda()
    x = x1.repeat(reps, 1)
    m = period * reps
    (_, _, _), wd = _weights(NV, 1, n, k, 62)
    cfg = b4.Fp4Config(m=m, n=n, k=k)
    out = torch.empty(m, n, dtype=BF, device="cuda")
    ws = torch.empty(b4.fp4_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    b4.fp4_linear(cfg, x, *wd, out, ws)
    small = b4.Fp4Config(m=period, n=n, k=k)
    want = torch.empty(period, n, dtype=BF, device="cuda")
    b4.fp4_linear(small, x1, *wd, want, ws)
    assert m * k // 2 > 2**31 and m * n * 2 > 2**31
    assert torch.all(out.view(reps, period, n) == want)


# ------------------------------------------------------------- whole layer


LAYERS = [("tiny", W.WORKLOADS["tiny"], 4), ("decode", W.WORKLOADS["decode"].scaled(hidden=512, inter=384, experts=16), 1),
          ("small", W.WORKLOADS["small"].scaled(hidden=512, inter=352, experts=16), 64),
          ("oai", W.WORKLOADS["small"].scaled(hidden=256, inter=192, experts=8).with_act("swiglu_oai", (1.702, 1.0, 0.4)), 33),
          ("mxfp4", W.WORKLOADS["mxfp4"].scaled(hidden=352, inter=160, experts=7), 65)]


@pytest.mark.parametrize("name,wl,m", LAYERS, ids=[c[0] for c in LAYERS])
def test_layer_with_4bit_activations(b4, name, wl, m):
    x_bits, x = W.activations(wl, m, 71)
    ids, wts = W.routing(wl, m, 71)
    em = W.expert_map(wl)
    w13, w2 = W.float_weights(wl, 71)
    c13, s13, g13 = Q.quantize(w13, wl.fmt)
    c2, s2, g2 = Q.quantize(w2, wl.fmt)
    want = O.fused_moe_a4(x, c13, s13, g13, c2, s2, g2, ids, wts, wl.act, wl.fmt, wl.num_global_experts, em,
                          wl.swiglu)
    dem = None if em is None else dev(em)
    cfg = b4.MoEConfig(m, wl.top_k, wl.num_global_experts, wl.num_local_experts, wl.hidden, wl.inter,
                       format=b4.FORMATS[wl.fmt], expert_map=dem, swiglu_alpha=wl.swiglu[0], swiglu_beta=wl.swiglu[1],
                       swiglu_limit=wl.swiglu[2])
    act = b4.ACTIVATIONS[wl.act]

    def operand(c, s, g):
        t = b4.fp4_tile_scales(b4.Fp4Config(m=c.shape[1], k=2 * c.shape[2], num_groups=c.shape[0],
                                            format=b4.FORMATS[wl.fmt]), dev(s))
        return dev(c), t, None if g is None else dev(g)

    a13, a2 = operand(c13, s13, g13), operand(c2, s2, g2)
    ws = torch.empty(b4.fused_moe_a4_workspace_bytes(cfg, act), dtype=torch.uint8, device="cuda")
    args = (cfg, dev(x_bits).view(BF), *a13, *a2, dev(ids), dev(wts), act)
    outs = []
    for _ in range(2):
        out = torch.full((m, wl.hidden), float("nan"), dtype=BF, device="cuda")
        b4.fused_moe_a4(*args, out, ws)
        torch.cuda.synchronize()
        b4.check_status(ws)
        outs.append(out)
    assert_parity(bf16_to_np(outs[0]), want, name)
    assert torch.equal(outs[0], outs[1])  # no atomics: the same bits
    if wl.drop_globals or wl.invalid_frac:
        none = torch.full_like(args[8], -1)  # every route dropped: zeros
        out = torch.full((m, wl.hidden), float("nan"), dtype=BF, device="cuda")
        b4.fused_moe_a4(*args[:8], none, args[9], act, out, ws)
        assert not out.any()


@pytest.mark.parametrize("fmt,groups,m,n,k", [(NV, 3, 70, 130, 112), (NV, 2, 5, 130, 2048), (NV, 3, 300, 1500, 112),
                                              (MX, 2, 700, 2603, 96)])
def test_scatter_of_a_stack(b4, fmt, groups, m, n, k):
    """out_rows of a stack has an entry for each of its groups * m rows and may name any of them."""
    rows = groups * m
    cfg = b4.Fp4Config(m=m, n=n, k=k, num_groups=groups, format=b4.FORMATS[fmt])
    _, _, ad = _operand(b4, cfg, fmt, _np(_randn((rows, k), 81, BF)))
    _, wd = _weights(fmt, groups, n, k, 82)
    plain, got = (torch.full((rows, n), 7.0, dtype=BF, device="cuda") for _ in range(2))
    b4.fp4_matmul(cfg, *ad, *wd, plain)
    to = np.random.default_rng(83).permutation(rows).astype(np.int32)
    to[1], to[m] = -1, rows  # dropped
    b4.fp4_matmul(cfg, *ad, *wd, got, out_rows=dev(to))
    want = torch.full_like(plain, 7.0)
    kept = (to >= 0) & (to < rows)
    want[torch.from_numpy(to[kept]).long().cuda()] = plain[torch.from_numpy(np.flatnonzero(kept)).cuda()]
    assert (to[kept] >= m).any() and torch.equal(got, want)
