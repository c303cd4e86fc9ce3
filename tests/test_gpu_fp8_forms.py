"""GPU tests of the FP8 operators where calls follow, overlap or repeat one another, and at their largest sizes.

Results of the same call are compared bit for bit; against the float64 oracle, and between calls whose sums are cut along K
differently, with the tolerances of test_gpu_fp8.py.
"""

import numpy as np
import pytest
import torch

import workloads as W
from gpu_util import assert_parity, bf16_to_np, dev
from oracle import fp8 as O
from test_gpu_fp8 import BF, F32, _assert_product, _layer, _np, _operand, _randn, _weights, b4  # noqa: F401

pytestmark = pytest.mark.gpu


def _linear(b4, m, n, k, seed):
    cfg = b4.Fp8Config(m=m, n=n, k=k)
    w, sw, _ = _weights(1, n, k, seed)
    return cfg, w, sw, torch.empty(b4.fp8_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("m,n,k", [(3, 520, 2064), (40, 300, 1040), (200, 260, 400), (700, 640, 784)])
def test_two_streams_and_two_graphs(b4, m, n, k):  # noqa: F811
    """Two calls at once on streams and workspaces of their own, eager and as graphs replayed with new inputs."""
    calls = [_linear(b4, m, n, k, 81), _linear(b4, m, n, k, 82)]
    x = [_randn((m, k), 83 + i, BF).cuda() for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty(m, n, dtype=BF, device="cuda") for _ in range(2)]

    def want(i):
        cfg, w, sw, _ = calls[i]
        codes, scales = b4.fp8_empty(cfg, "cuda")
        out = torch.empty(m, n, dtype=BF, device="cuda")
        b4.fp8_quantize(cfg, x[i], codes, scales)
        b4.fp8_matmul(cfg, codes, scales, w, sw, out)
        return out

    def check():
        torch.cuda.synchronize()
        for i in range(2):
            b4.check_status(calls[i][3])
            assert torch.equal(outs[i], want(i))

    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            cfg, w, sw, ws = calls[i]
            b4.fp8_linear(cfg, x[i], w, sw, outs[i], ws, stream=streams[i])
    check()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        cfg, w, sw, ws = calls[i]
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            for _ in range(3):
                b4.fp8_linear(cfg, x[i], w, sw, outs[i], ws)
    for r in range(3):
        for i in range(2):
            x[i].copy_(_randn((m, k), 90 + 2 * r + i, BF))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        check()


@pytest.mark.parametrize("m", [1, 30, 200, 600])
def test_weights_quantised_right_before(b4, m):  # noqa: F811
    """The product's weights come from the call just before it (kernels of one stream start under one another)."""
    n, k = 2816, 2048
    weights = _randn((n, k), 91, F32, 0.05).cuda()
    x = _randn((m, k), 92, BF).cuda()
    wcfg = b4.Fp8Config(m=n, k=k, x_dtype=F32, block_rows=128)
    cfg = b4.Fp8Config(m=m, n=n, k=k)
    codes, scales = b4.fp8_empty(wcfg, "cuda")
    ws = torch.empty(b4.fp8_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    want, got = (torch.empty(m, n, dtype=BF, device="cuda") for _ in range(2))
    b4.fp8_quantize(wcfg, weights, codes, scales)
    torch.cuda.synchronize()
    b4.fp8_linear(cfg, x, codes, scales, want, ws)
    for _ in range(10):
        codes.view(torch.uint8).fill_(0x7F)
        scales.fill_(float("nan"))
        b4.fp8_quantize(wcfg, weights, codes, scales)
        b4.fp8_linear(cfg, x, codes, scales, got, ws)
        assert torch.equal(got, want)


@pytest.mark.parametrize("m,k", [(3, 512), (200, 512), (600, 512)])
def test_scales_at_odd_addresses(b4, m, k):  # noqa: F811
    """Scales of whole quadruples of blocks that do not start on 16 bytes."""
    n = 300
    a, sa, full = _operand(_np(_randn((m, k), 93, BF)))
    w, sw, wfull = _weights(1, n, k, 94)

    def moved(t):
        base = torch.full((t.numel() + 1,), float("nan"), device="cuda")
        base[1:] = t.flatten()
        return base[1:].view(t.shape)

    cfg = b4.Fp8Config(m=m, n=n, k=k)
    want, got = (torch.empty(m, n, dtype=BF, device="cuda") for _ in range(2))
    b4.fp8_matmul(cfg, a, sa, w, sw, want)
    b4.fp8_matmul(cfg, a, moved(sa), w, moved(sw), got)
    assert torch.equal(got, want)
    _assert_product(_np(want), *O.product(full, wfull[0]), k, BF)


def _random_weights(n, k):
    codes = torch.randint(0, 0x7F, (n, k), dtype=torch.uint8, device="cuda")
    return codes, torch.rand(1, -(-n // 128), -(-k // 128), device="cuda") * 1e-4


@pytest.mark.parametrize("m", [2, 40, 300])
def test_weights_beyond_32_bit_offsets(b4, m):  # noqa: F811
    """The last of 2^20 weight rows, past 2^32 bytes, against a call of these alone."""
    n, k, part = 2**20, 4112, 256
    w, sw = _random_weights(n, k)
    a, sa, _ = _operand(_np(_randn((m, k), 95, BF)))
    out = torch.empty(m, n, dtype=BF, device="cuda")
    few = torch.empty(m, part, device="cuda")
    b4.fp8_matmul(b4.Fp8Config(m=m, n=n, k=k), a, sa, w[None], sw, out)
    b4.fp8_matmul(b4.Fp8Config(m=m, n=part, k=k, out_dtype=F32), a, sa, w[None, -part:].contiguous(),
                  sw[:, -2:].contiguous(), few)
    wfull = O.dequant(_np(w[-part:].view(torch.float8_e4m3fn).float()), _np(sw[0, -2:]), 128)
    want, mags = O.product(O.dequant(_np(a.float()), _np(sa)), wfull)
    _assert_product(_np(out[:, -part:]), want, mags, k, BF)
    _assert_product(_np(few), want, mags, k, F32)


@pytest.mark.parametrize("odtype", [BF, F32])
def test_output_beyond_32_bit_elements(b4, odtype):  # noqa: F811
    """Outputs of more than 2^31 elements: the last rows against a call of these alone."""
    m, n, k, part = 2100, 2**20, 16, 600
    w, sw = _random_weights(n, k)
    a, sa, _ = _operand(_np(_randn((m, k), 96, BF)))
    out = torch.empty(m, n, dtype=odtype, device="cuda")
    b4.fp8_matmul(b4.Fp8Config(m=m, n=n, k=k, out_dtype=odtype), a, sa, w[None], sw, out)
    few = torch.empty(part, n, dtype=odtype, device="cuda")
    b4.fp8_matmul(b4.Fp8Config(m=part, n=n, k=k, out_dtype=odtype), a[-part:].contiguous(), sa[-part:].contiguous(), w[None],
                  sw, few)
    assert m * n > 2**31 and torch.equal(out[-part:], few)


WL = W.WORKLOADS["small"]
FORMS = [  # workload, tokens: h by FC1's own kernel (gated, an odd number of blocks; ReLU^2), and in 32 bits through memory
    (WL.scaled(hidden=272, inter=384, experts=8), 600), (WL.scaled(hidden=272, inter=128, experts=8), 600),
    (W.WORKLOADS["decode"].scaled(hidden=256, inter=128, experts=8), 600), (WL.scaled(hidden=256, inter=160, experts=8), 600),
    (WL.scaled(hidden=256, inter=384, experts=8), 12), (WL.scaled(hidden=256, inter=384, experts=8), 1),
]


@pytest.mark.parametrize("wl,m", FORMS, ids=[f"{c[0].name}-{c[0].inter}-{c[1]}" for c in FORMS])
def test_layer_of_few_experts_padding_and_repeats(b4, wl, m):  # noqa: F811
    """Experts without rows, a token's expert twice, a padded batch, a NaN token, new inputs in a replayed graph."""
    e, top = wl.num_global_experts, wl.top_k
    x_bits, x = W.activations(wl, m, 97)
    full, ops, em, cfg, act, ws = _layer(b4, wl, m, 97)
    rng = np.random.default_rng(98)
    ids = rng.choice(np.array([1, 4, e - 1]), size=(m, top)).astype(np.int32)
    wts = rng.random((m, top)).astype(np.float32)
    live = max(m - 7, 1)
    ids[live:] = -1
    want = O.fused_moe_fp8(x, *full, ids, wts, wl.act, e, em, wl.swiglu)
    xd, dids, dw = dev(x_bits).view(BF), dev(ids), dev(wts)
    out, again = (torch.full((m, wl.hidden), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    b4.fused_moe_fp8(cfg, xd, *ops, dids, dw, act, out, ws)
    torch.cuda.synchronize()
    b4.check_status(ws)
    assert_parity(bf16_to_np(out), want, wl.name)
    assert not out[live:].any()
    # a token of NaNs leaves the others' bits as they are; and what lies in dropped rows does not matter
    bad = xd.clone()
    bad[0] = float("nan")
    bad[live:] = float("inf")
    b4.fused_moe_fp8(cfg, bad, *ops, dids, dw, act, again, ws)
    assert torch.isnan(again[0]).all() and torch.equal(again[1:], out[1:])
    # captured, then replayed with other tokens on a stream of its own
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        b4.fused_moe_fp8(cfg, bad, *ops, dids, dw, act, again, ws)
    bad.copy_(xd)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph.replay()
    stream.synchronize()
    b4.check_status(ws)
    assert torch.equal(again, out)


def test_router_pads_the_layer(b4):  # noqa: F811
    """num_tokens at the router: the layer's rows from there on are zero, the others those of the whole batch's experts."""
    wl, m, live = WL.scaled(hidden=256, inter=160, experts=16), 40, 23
    x_bits, _ = W.activations(wl, m, 99)
    _, ops, _, cfg, act, ws = _layer(b4, wl, m, 99)
    z = _randn((m, 16), 100, BF, 1.5)
    z[live:] = float("nan")
    z = z.cuda()
    ids, wts = torch.empty(m, wl.top_k, dtype=torch.int32, device="cuda"), torch.empty(m, wl.top_k, device="cuda")
    rcfg = b4.RouterConfig(m, 16, wl.top_k)
    outs = [torch.empty(m, wl.hidden, dtype=BF, device="cuda") for _ in range(2)]
    count = torch.tensor([live], dtype=torch.int32, device="cuda")
    for out, n in zip(outs, (count, None)):  # (rows of NaN choose nothing either)
        b4.route_topk(rcfg, z, ids, wts, num_tokens=n)
        b4.fused_moe_fp8(cfg, dev(x_bits).view(BF), *ops, ids, wts, act, out, ws)
    assert torch.equal(*outs) and not outs[0][live:].any() and outs[0][:live].any(dim=1).all()
