"""GPU tests of the forms of the FP4 operators beside those of test_gpu_fp4.py: long rows behind an activation (their
chunks are read a second time), one global scale per matrix behind an activation, stacks with a row stride, and the
layer with 4-bit activations at full size and in a CUDA graph.

Gated rows: the exponential and the reciprocal are approximate, so values are held to a step of their codes: half of
the widest one (6 - 4), which is also more than the 6/17 by which a block's scale may round down below amax / 6; a
per-matrix scale to 2^-16, the largest element's own error at |alpha g| <= 20 (the argument of the exponential rounds to
2^-24 |alpha g| log2 e, the two approximations to 2^-22 each) with room for the fp32 products."""

import numpy as np
import pytest
import torch

import test_gpu_fp4 as T
import workloads as W
from gpu_util import assert_parity, bf16_to_np, dev, host_layer
from oracle import fp4 as O
from oracle import quant as Q
from oracle.formats import e4m3_decode, e8m0_decode

pytestmark = pytest.mark.gpu

NV, MX, BF, HF, F32 = T.NV, T.MX, T.BF, T.HF, T.F32


@pytest.fixture(scope="module")
def b4():
    import w4a16_moe_gb300 as mod

    return mod


EXACT = [
    # fmt, dtype, groups, m, k, gs mode, act: rows longer than a block's threads hold, scales per matrix
    (NV, BF, 2, 3, 4400, "row", "relu2"),
    (NV, BF, 1, 5, 2064, "given", "relu2"),
    (MX, BF, 1, 3, 4128, "none", "relu2"),
    (NV, BF, 3, 65, 272, "tensor", "relu2"),
    (NV, BF, 2, 3, 4400, "tensor", "relu2"),
]


@pytest.mark.parametrize("layout", ["tiles", "rows"])
@pytest.mark.parametrize("fmt,dtype,groups,m,k,mode,act", EXACT)
def test_quantise_behind_relu2(b4, fmt, dtype, groups, m, k, mode, act, layout):
    T.test_quantise_matches_the_oracle(b4, fmt, dtype, groups, m, k, mode, act, layout)


@pytest.mark.parametrize("act", ["silu", "swiglu_oai"])
@pytest.mark.parametrize("fmt,dtype,mode,groups,m,k", [
    (NV, BF, "row", 1, 9, 4400), (NV, HF, "row", 2, 3, 2064), (MX, BF, "none", 1, 5, 4128), (MX, F32, "none", 2, 3, 288),
    (NV, BF, "tensor", 2, 37, 272), (NV, F32, "tensor", 1, 3, 4400),
])
def test_gated_quantise(b4, fmt, dtype, mode, groups, m, k, act):
    x = T._randn((groups, m, 2 * k), 91, dtype, 2.0)
    cfg = b4.Fp4Config(m=m, k=k, num_groups=groups, format=b4.FORMATS[fmt], x_dtype=dtype,
                       activation=b4.ACTIVATIONS[act], gs_mode=getattr(b4, "GS_" + mode.upper()))
    codes, scales, gs = b4.fp4_empty(cfg, "cuda")
    values = torch.empty(groups, m, k, dtype=dtype, device="cuda")
    b4.fp4_quantize(cfg, x.cuda(), codes, scales, gs, values=values)
    sc = T._untile(scales, m, k // Q.GROUP[fmt])
    for e in range(groups):
        h = T._act_np(T._np(x[e]), act)
        if mode == "tensor":
            assert abs(float(gs[e]) / O.matrix_gs(h) - 1) < 2.0**-16
        step = np.repeat((e8m0_decode if fmt == MX else e4m3_decode)(sc[e]), Q.GROUP[fmt], axis=1)
        if mode != "none":
            step = step * (T._np(gs)[e][:, None] if mode == "row" else float(gs[e]))
        assert np.all(np.abs(T._np(values[e]) - h) <= step * (1 + 1e-3) + T.ROUND[dtype] * np.abs(h))


@pytest.mark.parametrize("fmt,mode,act", [(NV, "row", None), (NV, "tensor", None), (MX, "none", None), (NV, "tensor", "silu"),
                                          (NV, "row", "silu")])
@pytest.mark.parametrize("dtype,pad", [(BF, 16), (F32, 3)])
def test_stack_with_a_row_stride(b4, fmt, mode, act, dtype, pad):
    """Matrices whose rows are further apart than they are long: the bits of the same matrices side by side."""
    groups, m, k = 3, 35, 160
    width = 2 * k if act else k
    kw = dict(m=m, k=k, num_groups=groups, format=b4.FORMATS[fmt], x_dtype=dtype, activation=b4.ACTIVATIONS.get(act),
              gs_mode=getattr(b4, "GS_" + mode.upper()))
    x = T._randn((groups * m, width + pad), 92, dtype).cuda()[:, :width]
    x[:, 0] *= torch.arange(1, groups * m + 1, device="cuda").to(dtype)  # every matrix has a largest element of its own
    outs = []
    for cfg, src in ((b4.Fp4Config(**kw), x.contiguous()), (b4.Fp4Config(x_stride=width + pad, **kw), x)):
        codes, scales, gs = b4.fp4_empty(cfg, "cuda")
        values = torch.empty(groups * m, k, dtype=dtype, device="cuda")
        b4.fp4_quantize(cfg, src, codes, scales, gs, values=values)
        outs.append((codes[..., : k // 2], scales, gs, values))
    for a, b in zip(*outs):
        assert a is b is None or torch.equal(a, b)
    if mode == "tensor":
        assert len(set(outs[0][2].tolist())) == groups


@pytest.mark.parametrize("fmt,m,act", [(NV, 3, "silu"), (NV, 1, "relu2"), (MX, 4, "swiglu_oai"), (NV, 70, "silu")])
def test_linear_behind_an_activation_with_long_rows(b4, fmt, m, act):
    """The composite call, in one launch or two, against its parts."""
    n, k = 140, 4416
    cfg = b4.Fp4Config(m=m, n=n, k=k, format=b4.FORMATS[fmt], activation=b4.ACTIVATIONS[act])
    x = T._randn((m, k if act == "relu2" else 2 * k), 93, BF).cuda()
    _, wd = T._weights(fmt, 1, n, k, 94)
    parts = b4.fp4_empty(cfg, "cuda")
    want, got = (torch.empty(m, n, dtype=BF, device="cuda") for _ in range(2))
    b4.fp4_quantize(cfg, x, *parts)
    b4.fp4_matmul(cfg, *parts, *wd, want)
    ws = torch.empty(b4.fp4_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    b4.fp4_linear(cfg, x, *wd, got, ws)
    b4.check_status(ws)
    assert torch.isfinite(got).all() and torch.equal(got, want)


FULL = [("small", W.WORKLOADS["small"], (1, 64, 2048)), ("mxfp4", W.WORKLOADS["mxfp4"], (1, 512)),
        ("relu2", W.WORKLOADS["small"].with_act("relu2"), (16, 1200))]


@pytest.mark.parametrize("name,wl,ms", FULL, ids=[c[0] for c in FULL])
def test_layer_at_full_size_and_in_a_graph(b4, name, wl, ms):
    """The layer at a framework's own sizes (groups of one row, of dozens, of hundreds): some of its tokens against the
    oracle, and the same bits from a captured graph."""
    few = 3
    hl = host_layer(wl, max(ms), 95, weights="random")
    em = None if hl.em is None else dev(hl.em)
    act, fmt = b4.ACTIVATIONS[wl.act], b4.FORMATS[wl.fmt]

    def operand(c, s, g):
        t = b4.Fp4Config(m=c.shape[1], k=2 * c.shape[2], num_groups=c.shape[0], format=fmt)
        return dev(c), b4.fp4_tile_scales(t, dev(s)), None if g is None else dev(g)

    w = operand(hl.c13, hl.s13, hl.g13) + operand(hl.c2, hl.s2, hl.g2)
    stream = torch.cuda.Stream()
    for m in ms:
        cfg = b4.MoEConfig(m, wl.top_k, wl.num_global_experts, wl.num_local_experts, wl.hidden, wl.inter, format=fmt,
                           expert_map=em)
        ws = torch.empty(b4.fused_moe_a4_workspace_bytes(cfg, act), dtype=torch.uint8, device="cuda")
        x, ids, wts = dev(hl.x_bits[:m]).view(BF), dev(hl.ids[:m]), dev(hl.wts[:m])
        out = torch.full((m, wl.hidden), float("nan"), dtype=BF, device="cuda")
        torch.cuda.synchronize()
        b4.fused_moe_a4(cfg, x, *w, ids, wts, act, out, ws, stream=stream)
        stream.synchronize()
        b4.check_status(ws)
        tok = np.unique(np.linspace(0, m - 1, few).astype(int))
        want = O.fused_moe_a4(hl.x[tok], hl.c13, hl.s13, hl.g13, hl.c2, hl.s2, hl.g2, hl.ids[tok], hl.wts[tok], wl.act,
                              wl.fmt, wl.num_global_experts, hl.em, wl.swiglu)
        assert_parity(bf16_to_np(out)[tok], want, f"{name} m={m}")
        eager = out.clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            b4.fused_moe_a4(cfg, x, *w, ids, wts, act, out, ws, stream=stream)
        for _ in range(3):
            out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager)


@pytest.mark.parametrize("m", [2, 40])
@pytest.mark.parametrize("act", ["silu", "relu2"])
def test_layer_whose_rows_of_codes_are_padded(b4, act, m):
    """hidden and inter odd multiples of 16: the codes' rows end 8 bytes before the next begin."""
    wl = W.Workload("odd", NV, 5, 5, 2, 336, 176, act, (m,))
    (c13, s13, g13), w13 = T._weights(NV, 5, wl.n1, 336, 96)
    (c2, s2, g2), w2 = T._weights(NV, 5, 336, 176, 97)
    x_bits, x = W.activations(wl, m, 98)
    ids, wts = W.routing(wl, m, 98)
    cfg = b4.MoEConfig(m, 2, 5, 5, 336, 176)
    ws = torch.empty(b4.fused_moe_a4_workspace_bytes(cfg, b4.ACTIVATIONS[act]), dtype=torch.uint8, device="cuda")
    out = torch.full((m, 336), float("nan"), dtype=BF, device="cuda")
    b4.fused_moe_a4(cfg, dev(x_bits).view(BF), *w13, *w2, dev(ids), dev(wts), b4.ACTIVATIONS[act], out, ws)
    torch.cuda.synchronize()
    b4.check_status(ws)
    want = O.fused_moe_a4(x, c13, s13, g13, c2, s2, g2, ids, wts, act, NV, 5)
    assert_parity(bf16_to_np(out), want, f"padded codes m={m}")


@pytest.mark.parametrize("mode", ["given", "tensor"])
def test_zero_blocks_under_a_scale_of_zero(b4, mode):
    """A global scale of 0 (calibrated on nothing but zeros; or amax / 2688 below fp32's least number) makes every value
    0, the zero blocks' too, and the products with them."""
    m, n, k = 3, 40, 96
    x = torch.zeros(m, k)
    x[1, 40] = 1.0 if mode == "given" else 1e-42
    cfg = b4.Fp4Config(m=m, n=n, k=k, x_dtype=F32, out_dtype=F32, gs_mode=getattr(b4, "GS_" + mode.upper()))
    codes, scales, gs = b4.fp4_empty(cfg, "cuda")
    gs.zero_()
    values = torch.full((m, k), float("nan"), device="cuda")
    b4.fp4_quantize(cfg, x.cuda(), codes, scales, gs, values=values)
    assert float(gs[0]) == 0 and not values.any() and not codes[..., : k // 2].any()
    sc = T._untile(scales, m, k // 16)[0]
    assert np.isfinite(e4m3_decode(sc)).all() and not np.delete(sc.reshape(-1), 1 * (k // 16) + 40 // 16).any()
    _, wd = T._weights(NV, 1, n, k, 99)
    out = torch.full((m, n), float("nan"), device="cuda")
    b4.fp4_matmul(cfg, codes, scales, gs, *wd, out)
    assert not out.any()
    if mode == "given":
        ws = torch.empty(b4.fp4_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
        out.fill_(float("nan"))
        b4.fp4_linear(cfg, x.cuda(), *wd, out, ws, x_gs=gs)
        assert not out.any()


@pytest.mark.parametrize("m", [2, 40, 300])
def test_calls_behind_copies_and_fills_in_a_graph(b4, m):
    """A captured call whose stream did a copy and a fill before it (nodes that are no kernels)."""
    n, k = 300, 272
    cfg = b4.Fp4Config(m=m, n=n, k=k)
    src = T._randn((2, m, k), 100, BF).cuda()
    x, out = torch.empty(m, k, dtype=BF, device="cuda"), torch.empty(m, n, dtype=BF, device="cuda")
    parts, prod = b4.fp4_empty(cfg, "cuda"), torch.empty_like(out)
    _, wd = T._weights(NV, 1, n, k, 101)
    ws = torch.empty(b4.fp4_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    picked = src[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(picked)
        out.zero_()
        b4.fp4_linear(cfg, x, *wd, out, ws)
        x.copy_(picked)
        prod.zero_()
        b4.fp4_quantize(cfg, x, *parts)
        b4.fp4_matmul(cfg, *parts, *wd, prod)
    want = torch.empty_like(out)
    for i in (0, 1):
        picked.copy_(src[i])
        b4.fp4_linear(cfg, src[i], *wd, want, ws)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(prod, want)
