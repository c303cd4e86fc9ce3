"""GPU tests of the FP8 operators (b4_fp8_*, b4_fused_moe_fp8) against the float64 oracle.

Quantisation: F32 scales are the float32 of amax / 448 and POW2 scales exact, bit for bit, without an activation; behind
one, amax is off by the activation's error.  Codes are the oracle's but where the exact quotient lies within NEAR of a tie
between two of them without being it: the kernel's quotient is rounded once from 46 bits (2^-24), the oracle's float32
likewise, so 2^-22 is enough; behind a gated activation its relative error 2^-21 + |alpha g| 2^-23 (|g| < 2^4 here: 2^-18.4)
counts too, so 2^-18.  POW2 quotients of 16-bit x are exact: nothing is allowed there.

Products: half a unit of the output's type, plus fp32 accumulation: each of the K / 32 instructions and of the K / 128
promotions (two roundings each, the scales' product one more) is off by at most 2^-22 of the terms' magnitude.
"""

import numpy as np
import pytest
import torch

import workloads as W
from gpu_util import assert_parity, bf16_to_np, dev
from oracle import fp8 as O
from oracle import moe as M
from oracle import router as R
from oracle import routing as P
from oracle.formats import e4m3_decode

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ROUND = {BF: 2.0**-8, HF: 2.0**-11, F32: 2.0**-24}
OAI = W.WORKLOADS["small"].swiglu


@pytest.fixture(scope="module")
def b4():
    import w4a16_moe_gb300 as mod

    return mod


def _np(t):
    return t.detach().double().cpu().numpy()


def _randn(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def _weights(e, n, k, seed):
    """Codes [E, N, K], scales [E, ceil(N/128), ceil(K/128)] and the dequantised matrices in float64."""
    g = torch.Generator().manual_seed(seed)
    codes = (torch.randn(e, n, k, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = (torch.rand(e, -(-n // 128), -(-k // 128), generator=g) + 0.5) * 2e-4
    full = np.stack([O.dequant(_np(codes[i].float()), _np(s[i]), 128) for i in range(e)])
    return codes.cuda(), s.cuda(), full


def _operand(x):
    """x [R, K] quantised by the oracle, on the device, and dequantised."""
    codes, s = O.quantize(x)
    c = torch.from_numpy(codes).to(torch.float8_e4m3fn)
    return c.cuda(), torch.from_numpy(s).float().cuda(), O.dequant(codes, s)


def _assert_product(got, want, mags, k, dtype, what=""):
    steps = k / 32 + 3 * -(-k // 128) + 4
    tol = ROUND[dtype] * np.abs(want) + steps * 2.0**-22 * mags + (2.0**-25 if dtype == HF else 0)
    err = np.abs(got - want)
    assert got.shape == want.shape and np.all(err <= tol), f"{what}: worst excess {np.max(err - tol):.3e}"


# ------------------------------------------------------------- quantisation


def _check_quantised(codes, scales, h, block_rows, pow2, near):
    """near None: equal."""
    s = _np(scales)
    want_s = O.scales(h, block_rows, pow2)
    if near is None or near <= 2.0**-22:
        assert np.array_equal(s, want_s)
    elif pow2:
        assert np.all((s == want_s) | (s == 2 * want_s) | (2 * s == want_s)) and np.mean(s != want_s) < 0.01
    else:
        assert np.all(np.abs(s - want_s) <= near * want_s)
    q = (h / O.spread(s, h.shape, block_rows)).astype(np.float32).astype(np.float64)
    got, want = _np(codes.float()), O.e4m3(q)
    bad = got != want
    if near is None:
        assert not bad.any()
        return
    lo, hi = np.minimum(got, want), np.maximum(got, want)
    tie = np.abs(np.abs(q) - np.abs(lo + hi) / 2) <= near * np.abs(q)
    neighbours = np.abs(hi - lo) <= np.maximum(np.abs(q) * 2.0**-3 * 1.01, 2.0**-9)
    assert np.all(~bad | (tie & neighbours)), np.argwhere(bad & ~tie)[:5]


ROWS = [  # dtype, m, k, groups, act
    (BF, 1, 16, 1, None), (BF, 5, 128, 1, None), (BF, 130, 80, 2, None), (HF, 7, 272, 3, None), (F32, 33, 4096, 1, None),
    (BF, 1, 4096, 1, None), (BF, 700, 2048, 1, None), (F32, 260, 1008, 2, None),
    (BF, 40, 352, 1, "silu"), (HF, 9, 128, 2, "swiglu_oai"), (F32, 3, 1408, 1, "silu"), (BF, 20, 144, 1, "relu2"),
]


@pytest.mark.parametrize("dtype,m,k,groups,act", ROWS)
@pytest.mark.parametrize("pow2", [False, True])
def test_quantise_rows(b4, dtype, m, k, groups, act, pow2):
    gated = act in ("silu", "swiglu_oai")
    x = _randn((groups * m, 2 * k if gated else k), 11, dtype)
    x[0, : k // 2] = 0
    cfg = b4.Fp8Config(m=m, k=k, num_groups=groups, x_dtype=dtype, activation=b4.ACTIVATIONS.get(act),
                       scale_mode=b4.FP8_SCALE_POW2 if pow2 else b4.FP8_SCALE_F32)
    codes, scales = b4.fp8_empty(cfg, "cuda")
    values = torch.empty(groups * m, k, dtype=dtype, device="cuda")
    b4.fp8_quantize(cfg, x.cuda(), codes, scales, values=values)
    h = _np(x) if act is None else M.activation_fn(_np(x), act, k, OAI)
    near = 2.0**-18 if gated else None if pow2 and dtype != F32 and act is None else 2.0**-22
    codes, scales = codes.view(-1, k), scales.view(groups * m, -1)
    if act == "relu2":  # the fp32 square is rounded: the oracle's h with it
        h = np.float32(np.maximum(_np(x), 0)) ** 2
        h = h.astype(np.float64)
    _check_quantised(codes, scales, h, 1, pow2, near)
    want = (codes.float() * scales.repeat_interleave(128, 1)[:, :k]).to(dtype)
    assert torch.equal(values, want)


@pytest.mark.parametrize("dtype,m,k,groups", [(BF, 128, 128, 1), (F32, 200, 336, 3), (HF, 1, 16, 2), (F32, 129, 128, 1)])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantise_blocks(b4, dtype, m, k, groups, pow2):
    x = _randn((groups, m, k), 12, dtype, 0.02)
    x[0, :, :16] = 0
    cfg = b4.Fp8Config(m=m, k=k, num_groups=groups, x_dtype=dtype, block_rows=128,
                       scale_mode=b4.FP8_SCALE_POW2 if pow2 else b4.FP8_SCALE_F32)
    codes, scales = b4.fp8_empty(cfg, "cuda")
    assert scales.shape == (groups, -(-m // 128), -(-k // 128))
    values = torch.empty_like(x, device="cuda")
    b4.fp8_quantize(cfg, x.cuda(), codes, scales, values=values)
    for g in range(groups):
        _check_quantised(codes[g], scales[g], _np(x[g]), 128, pow2, None if pow2 and dtype != F32 else 2.0**-22)
        full = scales[g].repeat_interleave(128, 0)[:m].repeat_interleave(128, 1)[:, :k]
        assert torch.equal(values[g], (codes[g].float() * full).to(dtype))


def test_exact_ties_and_extreme_blocks(b4):
    """Quotients on ties go to the even code; tiny, huge, zero, infinite and NaN blocks."""
    grid = e4m3_decode(np.arange(0x7F))
    ties = np.concatenate([(grid[1:] + grid[:-1]) / 2, grid])[:250]
    x = np.zeros((8, 256), dtype=np.float32)
    x[0, :250], x[0, [127, 255]] = ties, 448.0           # scale 1
    x[1, :250], x[1, [127, 255]] = -ties * 2.0**20, 448.0 * 2.0**20
    x[2, :250], x[2, [127, 255]] = ties * 2.0**-110, 448.0 * 2.0**-110
    x[3, :128] = 1e-42                                   # below the least scale
    x[4, :128] = 3e38
    x[5, 3], x[6, 200] = np.inf, np.nan
    for pow2 in (False, True):
        cfg = b4.Fp8Config(m=8, k=256, x_dtype=F32, scale_mode=b4.FP8_SCALE_POW2 if pow2 else b4.FP8_SCALE_F32)
        codes, scales = b4.fp8_empty(cfg, "cuda")
        b4.fp8_quantize(cfg, torch.from_numpy(x).cuda(), codes, scales)
        codes, scales = codes[0], scales[0]
        ok = [0, 1, 2, 3, 4, 7]
        _check_quantised(codes[ok], scales[ok], x[ok].astype(np.float64), 1, pow2, None)
        c, s = _np(codes.float()), _np(scales)
        assert np.isnan(s[5, 0]) and np.isnan(c[5, :128]).all() and s[5, 1] == 1 and not c[5, 128:].any()
        assert np.isnan(s[6, 1]) and np.isnan(c[6, 128:]).all() and s[6, 0] == 1


def test_quantise_gathered_rows(b4):
    """Rows through an index, with entries that name none, rows past the last group left alone, rows apart and off 16 bytes."""
    m, k, div = 13, 144, 3
    base = _randn((20, k + 5), 13, BF).cuda()
    for off in (0, 1):
        x = base[:, off:off + k]
        rows = np.array([0, 59, 7, -1, 30, 61, 3, 3, 58, 12, 1, 2, 4], dtype=np.int32)
        offsets = np.array([0, 4, 4, 11], dtype=np.int32)
        cfg = b4.Fp8Config(m=m, k=k, num_groups=3, row_div=div, x_stride=k + 5)
        codes, scales = b4.fp8_empty(cfg, "cuda", ragged=True)
        codes.view(torch.uint8).fill_(0x11)
        scales.fill_(7.0)
        b4.fp8_quantize(cfg, x, codes, scales, rows=dev(rows), offsets=dev(offsets))
        h = np.stack([_np(x)[r // div] if 0 <= r // div < 20 else np.zeros(k) for r in rows[:11]])
        _check_quantised(codes[:11], scales[:11], h, 1, False, 2.0**-22)
        assert torch.all(codes.view(torch.uint8)[11:] == 0x11) and torch.all(scales[11:] == 7.0)


# ----------------------------------------------------------------- products


DENSE = [  # out dtype, m, n, k
    (BF, 1, 128, 128), (BF, 1, 4096, 4096), (BF, 2, 100, 144), (F32, 3, 1, 16), (HF, 16, 130, 272), (BF, 17, 384, 2880),
    (BF, 33, 1440, 1040), (F32, 64, 257, 512), (BF, 100, 200, 336), (BF, 129, 640, 1408), (HF, 300, 1030, 656),
    (BF, 256, 2816, 2048), (BF, 520, 770, 4096), (BF, 1111, 1536, 528),
]


@pytest.mark.parametrize("odtype,m,n,k", DENSE)
def test_matmul(b4, odtype, m, n, k):
    a, sa, full = _operand(_np(_randn((m, k), 21, BF)))
    w, sw, wfull = _weights(1, n, k, 22)
    cfg = b4.Fp8Config(m=m, n=n, k=k, out_dtype=odtype)
    out = torch.full((m + 1, n), 7.0, dtype=odtype, device="cuda")
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    b4.fp8_matmul(cfg, a, sa, w, sw, out[:m], device_status=status)
    want, mags = O.product(full, wfull[0])
    _assert_product(_np(out[:m]), want, mags, k, odtype)
    assert torch.all(out[m] == 7.0) and not status.any()
    again = torch.empty_like(out[:m])
    b4.fp8_matmul(cfg, a.view(torch.uint8), sa, w.view(torch.uint8), sw, again)
    assert torch.equal(again, out[:m])


@pytest.mark.parametrize("odtype", [BF, HF, F32])
@pytest.mark.parametrize("m,pad,off", [(3, 8, 0), (150, 3, 0), (70, 24, 1), (300, 16, 8)])
def test_output_rows_apart(b4, odtype, m, pad, off):
    n, k = 200, 256
    a, sa, full = _operand(_np(_randn((m, k), 23, BF)))
    w, sw, wfull = _weights(1, n, k, 24)
    cfg = b4.Fp8Config(m=m, n=n, k=k, out_dtype=odtype, out_stride=n + pad)
    base = torch.full((m * (n + pad) + off + 64,), 7.0, dtype=odtype, device="cuda")
    view = base[off:off + m * (n + pad)].view(m, n + pad)
    b4.fp8_matmul(cfg, a, sa, w, sw, view[:, :n])
    want, mags = O.product(full, wfull[0])
    _assert_product(_np(view[:, :n]), want, mags, k, odtype)
    assert torch.all(view[:, n:] == 7.0) and torch.all(base[:off] == 7.0) and torch.all(base[off + view.numel():] == 7.0)


@pytest.mark.parametrize("groups,m,n,k", [(3, 70, 130, 112), (2, 5, 257, 2048), (3, 300, 500, 144)])
def test_stack_and_scatter(b4, groups, m, n, k):
    rows = groups * m
    a, sa, full = _operand(_np(_randn((rows, k), 25, BF)))
    w, sw, wfull = _weights(groups, n, k, 26)
    cfg = b4.Fp8Config(m=m, n=n, k=k, num_groups=groups)
    plain, got = (torch.full((rows, n), 7.0, dtype=BF, device="cuda") for _ in range(2))
    b4.fp8_matmul(cfg, a, sa, w, sw, plain)
    for g in range(groups):
        want, mags = O.product(full[g * m:(g + 1) * m], wfull[g])
        _assert_product(_np(plain[g * m:(g + 1) * m]), want, mags, k, BF)
    to = np.random.default_rng(27).permutation(rows).astype(np.int32)
    to[1], to[m] = -1, rows  # dropped
    b4.fp8_matmul(cfg, a, sa, w, sw, got, out_rows=dev(to))
    want = torch.full_like(plain, 7.0)
    kept = (to >= 0) & (to < rows)
    want[torch.from_numpy(to[kept]).long().cuda()] = plain[torch.from_numpy(np.flatnonzero(kept)).cuda()]
    assert torch.equal(got, want)


RAGGED = [  # counts, rows past the last group, n, k
    ([1] * 8, 0, 1536, 1024), ([0, 3, 0, 0, 4], 2, 140, 80), ([0, 0], 5, 100, 64), ([130, 0, 1, 257, 64], 7, 300, 528),
    ([33, 17, 129, 128, 300, 2], 3, 640, 400), ([5], 0, 130, 2048), ([257, 128, 129, 511, 384], 9, 1300, 272), ([1024, 3], 0, 128, 144), ([700, 1, 40], 0, 256, 640), ([0], 1, 16, 16),
]


@pytest.mark.parametrize("counts,tail,n,k", RAGGED)
@pytest.mark.parametrize("odtype", [BF, F32])
def test_grouped(b4, counts, tail, n, k, odtype):
    e, m = len(counts), sum(counts) + tail
    off = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    a, sa, full = _operand(_np(_randn((m, k), 31, BF)))
    if tail:  # what lies past the last group must not matter
        a.view(torch.uint8)[off[-1]:] = 0x7F
        sa[off[-1]:] = float("nan")
    w, sw, wfull = _weights(e, n, k, 32)
    cfg = b4.Fp8Config(m=m, n=n, k=k, num_groups=e, out_dtype=odtype)
    out = torch.full((m + 1, n), 7.0, dtype=odtype, device="cuda")
    b4.fp8_matmul(cfg, a, sa, w, sw, out[:m], offsets=dev(off))
    got = _np(out)
    for g in range(e):
        want, mags = O.product(full[off[g]:off[g + 1]], wfull[g])
        _assert_product(got[off[g]:off[g + 1]], want, mags, k, odtype, f"group {g}")
    assert not got[off[-1]:m].any() and np.all(got[m] == 7.0)
    to = np.random.default_rng(33).permutation(m).astype(np.int32)
    scattered = torch.full((m, n), 7.0, dtype=odtype, device="cuda")
    b4.fp8_matmul(cfg, a, sa, w, sw, scattered, offsets=dev(off), out_rows=dev(to))
    want = torch.full((m, n), 7.0, dtype=odtype, device="cuda")
    live = off[-1]
    want[torch.from_numpy(to[:live]).long().cuda()] = out[:live]
    assert torch.equal(scattered, want)


LINEAR = [  # x dtype, out dtype, m, n, k, act, shift, pad
    (BF, BF, 1, 4096, 4096, None, 0, 0), (BF, BF, 4, 384, 2048, None, 0, 0), (HF, F32, 3, 130, 80, None, 1, 3), (F32, HF, 8, 100, 1024, None, 0, 4),
    (BF, BF, 2, 257, 1408, "silu", 0, 8), (BF, BF, 37, 1440, 2880, None, 0, 0), (BF, BF, 130, 200, 144, "relu2", 0, 0),
    (F32, F32, 260, 140, 272, "swiglu_oai", 1, 1), (BF, BF, 300, 512, 512, None, 0, 0), (BF, BF, 12, 640, 4096, None, 0, 0),
]


@pytest.mark.parametrize("dtype,odtype,m,n,k,act,shift,pad", LINEAR)
@pytest.mark.parametrize("pow2", [False, True])
def test_linear_is_the_two_calls(b4, dtype, odtype, m, n, k, act, shift, pad, pow2):
    """The same bits as quantisation and product, an infinite and a NaN row among them, from strided and unaligned
    rows, and nothing written past the output's rows."""
    width = 2 * k if act in ("silu", "swiglu_oai") else k
    stride = width + pad
    base = _randn((m * stride + shift,), 43, dtype).cuda()
    x = base[shift:].view(m, stride)[:, :width]
    if m > 2:
        x[1, width // 2] = float("inf")
        x[2, 0] = float("nan")
    cfg = b4.Fp8Config(m=m, n=n, k=k, x_dtype=dtype, out_dtype=odtype, x_stride=stride, out_stride=n + pad,
                       activation=b4.ACTIVATIONS.get(act), scale_mode=b4.FP8_SCALE_POW2 if pow2 else b4.FP8_SCALE_F32)
    w, sw, wfull = _weights(1, n, k, 44)
    codes, scales = b4.fp8_empty(cfg, "cuda")
    b4.fp8_quantize(cfg, x, codes, scales)
    want, got = (torch.full((m + 1, n + pad), 7.0, dtype=odtype, device="cuda") for _ in range(2))
    b4.fp8_matmul(cfg, codes, scales, w, sw, want[:m, :n])
    ws = torch.empty(b4.fp8_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    b4.fp8_linear(cfg, x, w, sw, got[:m, :n], ws)
    b4.check_status(ws)
    torch.testing.assert_close(got, want, rtol=0, atol=0, equal_nan=True)
    assert torch.isfinite(got[0]).all() and torch.all(got[m] == 7.0) and torch.all(got[:, n:] == 7.0)
    full = O.dequant(_np(codes[0, :1].float()), _np(scales[0, :1]))
    _assert_product(_np(got[:1, :n]), *O.product(full, wfull[0]), k, odtype)
    if m > 2:
        assert torch.isnan(got[2, :n]).all()
        # (the clamped swiglu limits an infinite up)
        assert torch.isfinite(got[1, :n]).all() if act == "swiglu_oai" else torch.isnan(got[1, :n]).all()


@pytest.mark.parametrize("k", [80, 2064])
@pytest.mark.parametrize("counts", [[1] * 8, [8], [0, 3, 0, 0, 4], [0, 0], [2, 1, 5]])
def test_grouped_linear_of_few_rows(b4, k, counts):
    """A few gathered rows by group, in place and scattered: groups empty, of one row and of all."""
    n, e, tokens, div, m = 140, len(counts), 5, 2, 8
    off = dev(np.concatenate(([0], np.cumsum(counts))).astype(np.int32))
    rows = dev(np.array([3, 0, 9, -1, 4, 11, 1, 8], dtype=np.int32))  # -1 and 11 / 2 are no token: zero rows
    to = dev(np.array([5, 2, -1, 0, 8, 7, 1, 3], dtype=np.int32))     # -1 and 8 are dropped
    x = _randn((tokens, k), 45, BF).cuda()
    cfg = b4.Fp8Config(m=m, n=n, k=k, num_groups=e, row_div=div)
    w, sw, wfull = _weights(e, n, k, 46)
    codes, scales = b4.fp8_empty(cfg, "cuda", ragged=True)
    b4.fp8_quantize(cfg, x, codes, scales, rows=rows, offsets=off)
    ws = torch.empty(b4.fp8_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    for out_rows in (None, to):
        want, got = (torch.full((m, n), 7.0, dtype=BF, device="cuda") for _ in range(2))
        b4.fp8_matmul(cfg, codes, scales, w, sw, want, offsets=off, out_rows=out_rows)
        b4.fp8_linear(cfg, x, w, sw, got, ws, rows=rows, offsets=off, out_rows=out_rows)
        b4.check_status(ws)
        assert torch.equal(got, want) and torch.isfinite(got).all()
        if out_rows is None:
            full, o = O.dequant(_np(codes.float()), _np(scales)), off.cpu().numpy()
            for g in range(e):
                y, mags = O.product(full[o[g]:o[g + 1]], wfull[g])
                _assert_product(_np(got)[o[g]:o[g + 1]], y, mags, k, BF)


def test_operand_beyond_32_bit_offsets(b4):
    """x, codes and out of more than 2^31 bytes: every repeat of a 1000-row pattern gives the same rows."""
    period, reps, k, n = 1000, 1060, 4096, 1030
    x1 = _randn((period, k), 61, BF).cuda()
    x = x1.repeat(reps, 1)
    m = period * reps
    w, sw, _ = _weights(1, n, k, 62)
    cfg = b4.Fp8Config(m=m, n=n, k=k)
    out = torch.empty(m, n, dtype=BF, device="cuda")
    ws = torch.empty(b4.fp8_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    b4.fp8_linear(cfg, x, w, sw, out, ws)
    small = b4.Fp8Config(m=period, n=n, k=k)
    want = torch.empty(period, n, dtype=BF, device="cuda")
    b4.fp8_linear(small, x1, w, sw, want, ws)
    assert m * k > 2**31 and m * n * 2 > 2**31
    assert torch.all(out.view(reps, period, n) == want)


# --------------------------------------------------- layer, from logits on


LAYERS = [  # workload, tokens, router
    (W.WORKLOADS["tiny"], 4, dict()),
    (W.WORKLOADS["decode"].scaled(hidden=512, inter=384, experts=16), 1, dict(score="sigmoid", scale=2.5)),
    (W.WORKLOADS["small"].scaled(hidden=512, inter=352, experts=16), 64, dict(score="sigmoid", bias=True, groups=4, top_groups=3, group_top=2)),
    (W.WORKLOADS["small"].scaled(hidden=256, inter=192, experts=8).with_act("swiglu_oai", (1.702, 1.0, 0.4)), 33, dict(renorm=False)),
    (W.WORKLOADS["mxfp4"].scaled(hidden=352, inter=160, experts=7), 65, dict(bias=True)),
    (W.WORKLOADS["small"].scaled(hidden=256, inter=160, experts=8), 700, dict()),
    # h quantised by FC1's own kernel: groups of hundreds of rows, whole blocks of h
    (W.WORKLOADS["small"].scaled(hidden=256, inter=384, experts=8), 700, dict()),
    (W.WORKLOADS["small"].scaled(hidden=272, inter=256, experts=8).with_act("swiglu_oai", (1.702, 1.0, 0.4)), 450, dict(score="sigmoid", bias=True)),
    (W.WORKLOADS["decode"].scaled(hidden=400, inter=384, experts=16), 700, dict()),
    (W.WORKLOADS["mxfp4"].scaled(hidden=352, inter=128, experts=7), 600, dict()),
]


def _layer(b4, wl, m, seed):
    w13, w2 = W.float_weights(wl, seed)
    full, ops = [], []
    for w in (w13, w2):
        e, n, k = w.shape
        cfg = b4.Fp8Config(m=n, k=k, num_groups=e, x_dtype=F32, block_rows=128)
        codes, scales = b4.fp8_empty(cfg, "cuda")
        b4.fp8_quantize(cfg, dev(w.astype(np.float32)), codes, scales)
        full.append(np.stack([O.dequant(*O.quantize(w[i].astype(np.float32), 128), 128) for i in range(e)]))
        ops += [codes, scales]
    em = W.expert_map(wl)
    cfg = b4.MoEConfig(m, wl.top_k, wl.num_global_experts, wl.num_local_experts, wl.hidden, wl.inter,
                       expert_map=None if em is None else dev(em), swiglu_alpha=wl.swiglu[0], swiglu_beta=wl.swiglu[1],
                       swiglu_limit=wl.swiglu[2])
    act = b4.ACTIVATIONS[wl.act]
    ws = torch.empty(b4.fused_moe_fp8_workspace_bytes(cfg, act), dtype=torch.uint8, device="cuda")
    return full, ops, em, cfg, act, ws


@pytest.mark.parametrize("wl,m,router", LAYERS, ids=[f"{c[0].name}-{c[0].inter}-{c[1]}" for c in LAYERS])
def test_layer_from_logits(b4, wl, m, router):
    """Weights quantised, experts chosen, the layer run: by the framework's calls alone, twice, and from a graph."""
    x_bits, x = W.activations(wl, m, 71)
    router = dict(router)
    score, has_bias = router.pop("score", "softmax"), router.pop("bias", False)
    z = _randn((m, wl.num_global_experts), 72, F32, 1.5)
    bias = _randn((wl.num_global_experts,), 73, F32, 0.1) if has_bias else None
    full, ops, em, cfg, act, ws = _layer(b4, wl, m, 71)
    ids, wts = R.route(_np(z), None if bias is None else _np(bias), wl.top_k, score, **router)
    want = O.fused_moe_fp8(x, *full, ids, wts, wl.act, wl.num_global_experts, em, wl.swiglu)
    rcfg = b4.RouterConfig(m, wl.num_global_experts, wl.top_k, score=b4.SCORES[score], dtype=F32,
                           renormalize=router.get("renorm", True), scale=router.get("scale", 1.0),
                           num_groups=router.get("groups", 1), top_groups=router.get("top_groups"),
                           group_top=router.get("group_top", 1))
    dids = torch.empty(m, wl.top_k, dtype=torch.int32, device="cuda")
    dw = torch.empty(m, wl.top_k, device="cuda")
    z, xd = z.cuda(), dev(x_bits).view(BF)
    bias = None if bias is None else bias.cuda()

    def run(out):
        b4.route_topk(rcfg, z, dids, dw, bias=bias)
        b4.fused_moe_fp8(cfg, xd, *ops, dids, dw, act, out, ws)

    outs = [torch.full((m, wl.hidden), float("nan"), dtype=BF, device="cuda") for _ in range(3)]
    for out in outs[:2]:
        run(out)
        torch.cuda.synchronize()
        b4.check_status(ws)
    assert np.array_equal(dids.cpu().numpy(), ids)
    assert_parity(bf16_to_np(outs[0]), want, wl.name)
    assert torch.equal(outs[0], outs[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(outs[2])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2])
    dids.fill_(-1)  # every route dropped: zeros
    b4.fused_moe_fp8(cfg, xd, *ops, dids, dw, act, outs[2], ws)
    assert not outs[2].any()


def test_ids_of_the_router_serve_the_other_layers(b4):
    """The 4-bit layer reads the router's outputs, written just before on the same stream."""
    from gpu_util import DeviceLayer, host_layer, oracle_out

    wl = W.WORKLOADS["tiny"]
    hl = host_layer(wl, 4, 3)
    z = _randn((4, wl.num_global_experts), 74, BF, 1.5)
    hl.ids, hl.wts = R.route(_np(z), None, wl.top_k, "softmax")
    layer = DeviceLayer(hl)
    cfg = b4.RouterConfig(4, wl.num_global_experts, wl.top_k)
    layer.ids, layer.wts = torch.empty(4, wl.top_k, dtype=torch.int32, device="cuda"), torch.empty(4, wl.top_k, device="cuda")
    b4.route_topk(cfg, z.cuda(), layer.ids, layer.wts)
    layer.run()
    assert_parity(layer.result(), oracle_out(hl))


def test_packed_routes(b4):
    """Routes packed by b4_route_pack (drops included), rows gathered, outputs by expert."""
    wl = W.WORKLOADS["mxfp4"].scaled(hidden=160, inter=96, experts=7)
    m, k, e = 45, 160, wl.num_local_experts
    ids, _ = W.routing(wl, m, 3)
    em = W.expert_map(wl)
    _, off, routes = P.route_pack(ids, wl.num_global_experts, e, em)
    mc = b4.MoEConfig(m, wl.top_k, wl.num_global_experts, e, 160, 96, format=b4.MXFP4, expert_map=dev(em))
    dcounts, doff = torch.empty(e, dtype=torch.int32, device="cuda"), torch.empty(e + 1, dtype=torch.int32, device="cuda")
    droutes = torch.empty(routes.shape[0], dtype=torch.int32, device="cuda")
    b4.route_pack(mc, dev(ids), dcounts, doff, droutes)
    rows = m * wl.top_k
    cfg = b4.Fp8Config(m=rows, n=100, k=k, num_groups=e, row_div=wl.top_k)
    x = _randn((m, k), 51, BF)
    w, sw, wfull = _weights(e, 100, k, 52)
    out = torch.full((rows, 100), 9.0, dtype=BF, device="cuda")
    ws = torch.empty(b4.fp8_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    b4.fp8_linear(cfg, x.cuda(), w, sw, out, ws, rows=droutes, offsets=doff)
    got, a = _np(out), O.fake_quant(_np(x))
    for g in range(e):
        want, mags = O.product(a[routes[off[g]:off[g + 1]] // wl.top_k], wfull[g])
        # (a code next to a tie may differ: one step of 2^-3 of an element each; the test's seed has none)
        _assert_product(got[off[g]:off[g + 1]], want, mags, k, BF, f"expert {g}")
    assert not got[off[-1]:].any() and off[-1] < rows
