"""Refusals of the FP4 operators that keep a launch inside its buffers or from a wrong reading of them (CPU: every one
of them comes before any device is looked up)."""

import ctypes

import pytest
import torch

BF = torch.bfloat16


@pytest.fixture(scope="module")
def b4():
    import __graft_entry__

    __graft_entry__._build_module().build()
    import w4a16_moe_gb300 as mod

    return mod


@pytest.fixture()
def addr():
    buf = ctypes.create_string_buffer(1 << 12)
    return (ctypes.addressof(buf) + 255) // 256 * 256, buf


def _weights(n, k, groups=1):
    """Zero weights as a product takes them: codes, tiled scales, global scales."""
    ld = -(-(k // 2) // 16) * 16
    return (torch.zeros(groups, n, ld, dtype=torch.uint8),
            torch.zeros(groups, -(-n // 128), -(-k // 64), 32, 4, 4, dtype=torch.uint8), torch.ones(groups))


@pytest.mark.parametrize("m", [0, 4])
def test_product_refuses_row_major_scales(b4, addr, m):
    """The product reads whole tiles: scales in the checkpoint's layout are too short for it."""
    a = addr[0]
    cfg = b4.Fp4Config(m=m, k=64, n=8, scale_layout=b4.SCALES_ROWS)
    st = b4.raw_lib().b4_fp4_matmul(cfg._ref, a, a, a, a, a, a, None, None, a, None, None)
    assert st == b4.B4_ERR_INVALID_ARGUMENT and "tiled scales" in b4.last_error()
    if m == 0:
        return
    codes, scales, gs = b4.fp4_empty(cfg, "cpu")
    assert scales.numel() == 16  # of the 512 bytes of a tile
    with pytest.raises((b4.B4Error, ValueError), match="tiled scales"):
        b4.fp4_matmul(cfg, codes, scales, gs, *_weights(8, 64), torch.zeros(4, 8, dtype=BF), stream=_NoStream)


class _NoStream:
    cuda_stream = None


def test_tiling_refuses_a_row_major_config(b4, addr):
    """b4_fp4_scale_bytes of such a config is the source's size, less than the tiles that would be written."""
    a = addr[0]
    cfg = b4.Fp4Config(m=1, k=64, scale_layout=b4.SCALES_ROWS)
    assert b4.fp4_scale_bytes(cfg) == 4
    st = b4.raw_lib().b4_fp4_tile_scales(cfg._ref, a, a, None)
    assert st == b4.B4_ERR_INVALID_ARGUMENT and "tiled scales" in b4.last_error()


@pytest.mark.parametrize("fmt,mode", [(0, "ROW"), (0, "TENSOR"), (1, "NONE")])
def test_empty_calls_are_accepted(b4, fmt, mode):
    """No rows: every buffer of rows is empty, its address null, and nothing is launched."""
    cfg = b4.Fp4Config(m=0, k=64, n=8, format=fmt, gs_mode=getattr(b4, "GS_" + mode))
    x, parts = torch.zeros(0, 64, dtype=BF), b4.fp4_empty(cfg, "cpu")
    b4.fp4_quantize(cfg, x, *parts, values=torch.zeros_like(x), stream=_NoStream)
    w = _weights(8, 64)
    w = w[:2] + (w[2] if fmt == 0 else None,)
    out = torch.zeros(0, 8, dtype=BF)
    b4.fp4_matmul(cfg, *parts, *w, out, stream=_NoStream)
    if mode != "TENSOR":
        ws = torch.zeros(b4.fp4_linear_workspace_bytes(cfg), dtype=torch.uint8)
        b4.fp4_linear(cfg, x, *w, out, ws, stream=_NoStream)


@pytest.mark.parametrize("x", [torch.zeros(63, dtype=BF), torch.zeros(1, 62, dtype=BF), torch.zeros(0, 64, dtype=BF)])
def test_gather_needs_a_row_to_gather_from(b4, x):
    """An x shorter than one row bounds gathered rows by 0, which the library takes for no bound."""
    cfg = b4.Fp4Config(m=4, k=64, n=8)
    rows = torch.tensor([0, -1, 5, 100], dtype=torch.int32)
    with pytest.raises(ValueError, match="not one row"):
        b4.fp4_quantize(cfg, x, *b4.fp4_empty(cfg, "cpu"), rows=rows, stream=_NoStream)
    ws = torch.zeros(b4.fp4_linear_workspace_bytes(cfg), dtype=torch.uint8)
    with pytest.raises(ValueError, match="not one row"):
        b4.fp4_linear(cfg, x, *_weights(8, 64), torch.zeros(4, 8, dtype=BF), ws, rows=rows, stream=_NoStream)
    none = b4.Fp4Config(m=0, k=64, n=8)
    b4.fp4_quantize(none, x, *b4.fp4_empty(none, "cpu"), rows=rows[:0], stream=_NoStream)  # nothing to gather


def _layer(b4, hidden=352, inter=160, act=0, m=3, top_k=2, experts=5, fmt=0):
    """Config and valid arguments of the layer with 4-bit activations."""
    cfg = b4.MoEConfig(m, top_k, experts, experts, hidden, inter, format=fmt)
    n1 = inter if act == b4.RELU2 else 2 * inter
    kt = (lambda k: -(-k // 64)) if fmt == 0 else (lambda k: -(-k // 128))
    ld = lambda k: -(-(k // 2) // 16) * 16  # noqa: E731
    args = dict(
        x=torch.zeros(m, hidden, dtype=BF), w13=torch.zeros(experts, n1, ld(hidden), dtype=torch.uint8),
        s13=torch.zeros(experts, -(-n1 // 128), kt(hidden), 32, 4, 4, dtype=torch.uint8),
        gs13=torch.ones(experts) if fmt == 0 else None,
        w2=torch.zeros(experts, hidden, ld(inter), dtype=torch.uint8),
        s2=torch.zeros(experts, -(-hidden // 128), kt(inter), 32, 4, 4, dtype=torch.uint8),
        gs2=torch.ones(experts) if fmt == 0 else None, topk_ids=torch.zeros(m, top_k, dtype=torch.int32),
        topk_weights=torch.ones(m, top_k), activation=act, out=torch.zeros(m, hidden, dtype=BF),
        workspace=torch.zeros(0, dtype=torch.uint8))  # too small: a call that passes the binding ends there
    return cfg, args


@pytest.mark.parametrize("act,fmt", [(0, 0), (1, 0), (2, 1)])
def test_layer_refuses_short_buffers(b4, act, fmt):
    """Every buffer of the layer is as large as the kernels read it; one element less is named and refused."""
    cfg, args = _layer(b4, act=act, fmt=fmt)
    with pytest.raises(b4.B4Error) as ei:
        b4.fused_moe_a4(cfg, **args, stream=_NoStream)
    assert ei.value.status == b4.B4_ERR_INVALID_ARGUMENT  # (no workspace at all)
    for name, t in args.items():
        if isinstance(t, torch.Tensor) and name != "workspace":
            with pytest.raises(ValueError, match=rf"^{name} needs {t.numel()} elements, got {t.numel() - 1}$"):
                b4.fused_moe_a4(cfg, **{**args, name: t.reshape(-1)[:-1]}, stream=_NoStream)
            with pytest.raises(TypeError, match=f"^{name} must be"):
                b4.fused_moe_a4(cfg, **{**args, name: t.to(torch.int16)}, stream=_NoStream)
    with pytest.raises(TypeError, match="^w13 must be"):
        b4.fused_moe_a4(cfg, **{**args, "w13": None}, stream=_NoStream)


@pytest.mark.parametrize("hidden,inter,name", [(336, 160, "w13"), (352, 176, "w2")])
def test_layer_refuses_a_checkpoints_unpadded_codes(b4, hidden, inter, name):
    """K % 32 == 16: the kernels' rows of codes are 8 bytes further apart than the checkpoint's."""
    cfg, args = _layer(b4, hidden, inter)
    unpadded = args[name][..., :-8].contiguous()
    assert unpadded.shape[-1] == (hidden if name == "w13" else inter) // 2
    with pytest.raises(ValueError, match=f"^{name} needs"):
        b4.fused_moe_a4(cfg, **{**args, name: unpadded}, stream=_NoStream)


@pytest.mark.parametrize("fmt,n,k", [(0, 128, 64), (0, 256, 192), (1, 128, 256)])
def test_scales_that_were_not_tiled_are_refused(b4, fmt, n, k):
    """Where a matrix fills its tiles, row-major scales have the tiles' size: they are told by their shape."""
    cfg = b4.Fp4Config(m=128, n=n, k=k, num_groups=2, format=fmt)
    parts = b4.fp4_empty(cfg, "cpu")
    codes, gs = torch.zeros(2, n, k // 2, dtype=torch.uint8), torch.ones(2) if fmt == 0 else None
    rows = torch.zeros(2, n, cfg.blocks, dtype=torch.uint8)
    tiles = torch.zeros(2, n // 128, k // (64 if fmt == 0 else 128), 32, 4, 4, dtype=torch.uint8)
    assert rows.numel() == tiles.numel()
    out = torch.zeros(256, n, dtype=BF)
    with pytest.raises(ValueError, match="^w_scales has the row-major shape"):
        b4.fp4_matmul(cfg, *parts, codes, rows, gs, out, stream=_NoStream)
    with pytest.raises(ValueError, match="^a_scales has the row-major shape"):
        b4.fp4_matmul(cfg, parts[0], parts[1].view(2, 128, cfg.blocks), parts[2], codes, tiles, gs, out, stream=_NoStream)
    lin = b4.Fp4Config(m=4, n=n, k=k, format=fmt)
    ws = torch.zeros(b4.fp4_linear_workspace_bytes(lin), dtype=torch.uint8)
    with pytest.raises(ValueError, match="^w_scales has the row-major shape"):
        b4.fp4_linear(lin, torch.zeros(4, k, dtype=BF), codes[:1], rows[:1], None if gs is None else gs[:1],
                      torch.zeros(4, n, dtype=BF), ws, stream=_NoStream)
    cfg, args = _layer(b4, hidden=256, inter=128, fmt=fmt)
    for name, n, k in (("s13", 256, 256), ("s2", 256, 128)):
        bad = torch.zeros(5, n, k // (16 if fmt == 0 else 32), dtype=torch.uint8)
        assert bad.numel() == args[name].numel()
        with pytest.raises(ValueError, match=f"^{name} has the row-major shape"):
            b4.fused_moe_a4(cfg, **{**args, name: bad}, stream=_NoStream)
        flat = {**args, name: args[name].view(-1)}  # tiles in another shape are tiles
        with pytest.raises(b4.B4Error):
            b4.fused_moe_a4(cfg, **flat, stream=_NoStream)


def _passes_the_binding(call):
    """A call on CPU tensors that the binding lets through ends at the library's device check."""
    import w4a16_moe_gb300 as b4

    with pytest.raises(b4.B4Error) as ei:
        call()
    return ei.value.status in (b4.B4_ERR_UNSUPPORTED_DEVICE, b4.B4_ERR_CUDA)


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the calls it lets through would reach the GPU")


@no_gpu
def test_an_x_of_longer_rows_is_refused(b4):
    """A contiguous x whose rows are longer than the config's would be read as more and shorter rows."""
    cfg = b4.Fp4Config(m=4, k=64, n=8)
    ws = torch.zeros(b4.fp4_linear_workspace_bytes(cfg) + 256, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:]
    idx = torch.zeros(4, dtype=torch.int32)

    def quant(x, c=cfg, **kw):
        return b4.fp4_quantize(c, x, *b4.fp4_empty(c, "cpu"), stream=_NoStream, **kw)

    def linear(x, **kw):
        return b4.fp4_linear(cfg, x, *_weights(8, 64), torch.zeros(4, 8, dtype=BF), ws, stream=_NoStream, **kw)

    for x in (torch.zeros(4, 128, dtype=BF), torch.zeros(2, 4, 80, dtype=BF)):
        for call in (quant, linear):
            with pytest.raises(ValueError, match="^x has rows of"):
                call(x)
            with pytest.raises(ValueError, match="^x has rows of"):
                call(x, rows=idx)
    # the config's elements in any contiguous shape, more rows than needed, the stride said, one flat row
    for x in (torch.zeros(4, 64), torch.zeros(9, 64), torch.zeros(2, 128), torch.zeros(4, 4, 16), torch.zeros(256),
              torch.zeros(1, 512), torch.zeros(2, 3, 64)):
        assert _passes_the_binding(lambda: quant(x.to(BF))) and _passes_the_binding(lambda: linear(x.to(BF)))
    assert _passes_the_binding(lambda: quant(torch.zeros(4, 128, dtype=BF), b4.Fp4Config(m=4, k=64, x_stride=128)))
    assert _passes_the_binding(lambda: quant(torch.zeros(4, 128, dtype=BF)[:, :64], b4.Fp4Config(m=4, k=64, x_stride=128)))
    assert _passes_the_binding(lambda: quant(torch.zeros(2, 4, 64, dtype=BF), b4.Fp4Config(m=4, k=64, num_groups=2)))
    assert _passes_the_binding(lambda: quant(torch.zeros(7, 64, dtype=BF), rows=idx))


def test_the_layers_rows_are_the_configs(b4):
    cfg, args = _layer(b4)
    for name in ("x", "out"):
        with pytest.raises(ValueError, match=f"^{name} has rows of 400 elements, the config rows of 352$"):
            b4.fused_moe_a4(cfg, **{**args, name: torch.zeros(3, 400, dtype=BF)}, stream=_NoStream)
        for t in (torch.zeros(7, 352, dtype=BF), torch.zeros(1056, dtype=BF), torch.zeros(2, 528, dtype=BF)):
            with pytest.raises(b4.B4Error):  # passes: a larger buffer, the layer's elements in another shape
                b4.fused_moe_a4(cfg, **{**args, name: t}, stream=_NoStream)


@no_gpu
def test_an_out_of_longer_rows_is_refused(b4):
    """As for x: a stack's output [groups, m, width] with a width that is not the config's."""
    cfg = b4.Fp4Config(m=4, k=64, n=8, num_groups=2)

    def product(out, c=cfg):
        return b4.fp4_matmul(c, *b4.fp4_empty(c, "cpu"), *_weights(8, 64, 2), out, stream=_NoStream)

    with pytest.raises(ValueError, match="^out has rows of 16 elements"):
        product(torch.zeros(2, 4, 16, dtype=BF))
    for shape in ((2, 4, 8), (3, 4, 8), (64,), (2, 2, 16), (2, 4, 2, 4), (8, 8)):
        assert _passes_the_binding(lambda: product(torch.zeros(*shape, dtype=BF)))
    wide = b4.Fp4Config(m=4, k=64, n=8, num_groups=2, out_stride=16)
    assert _passes_the_binding(lambda: product(torch.zeros(2, 4, 16, dtype=BF), wide))


@no_gpu
def test_each_refusal_is_its_own(b4):
    """Each malformed argument is refused for what it is, where the same call with it mended passes the binding."""
    cfg = b4.Fp4Config(m=4, k=64, n=8)
    parts = b4.fp4_empty(cfg, "cpu")
    quant = dict(x=torch.zeros(4, 64, dtype=BF), codes=parts[0], scales=parts[1], gs=parts[2],
                 values=torch.zeros(4, 64, dtype=BF), rows=torch.zeros(4, dtype=torch.int32))
    w = _weights(8, 64)
    product = dict(a_codes=parts[0], a_scales=parts[1], a_gs=parts[2], w_codes=w[0], w_scales=w[1], w_gs=w[2],
                   out=torch.zeros(4, 8, dtype=BF), out_rows=torch.zeros(4, dtype=torch.int32))

    def call(f, base, **kw):
        return f(cfg, **{**base, **kw}, stream=_NoStream)

    assert _passes_the_binding(lambda: call(b4.fp4_quantize, quant))
    assert _passes_the_binding(lambda: call(b4.fp4_quantize, quant, rows=None))
    assert _passes_the_binding(lambda: call(b4.fp4_matmul, product))
    x, out = quant["x"], product["out"]
    for kw, error, text in (
            (dict(x=x.float()), TypeError, "x must be torch.bfloat16"), (dict(x=x[:3], rows=None), ValueError, "x holds 3 rows, 4 needed"),
            (dict(x=x.t()), ValueError, "x must be contiguous, or two-dimensional"),
            (dict(x=torch.zeros(4, 80, dtype=BF)[:, :64]), ValueError, "x must be contiguous, or two-dimensional"),
            (dict(codes=parts[0][:, :2].contiguous()), ValueError, "codes needs 128 elements, got 64"),
            (dict(codes=parts[0].to(torch.int8)), TypeError, "codes must be torch.uint8"),
            (dict(scales=parts[1].view(-1)[:511]), ValueError, "scales needs 512 elements, got 511"),
            (dict(gs=parts[2].view(-1)[:3]), ValueError, "gs needs 4 elements, got 3"),
            (dict(values=quant["values"][:3]), ValueError, "values needs 256 elements, got 192"),
            (dict(rows=torch.zeros(4, dtype=torch.int64)), TypeError, "rows must be torch.int32"),
            (dict(rows=torch.zeros(3, dtype=torch.int32)), ValueError, "rows needs 4 elements, got 3"),
            (dict(offsets=torch.zeros(1, dtype=torch.int32)), ValueError, "offsets needs 2 elements, got 1")):
        with pytest.raises(error, match=text):
            call(b4.fp4_quantize, quant, **kw)
    for kw, error, text in (
            (dict(w_codes=w[0][:, :7].contiguous()), ValueError, "w_codes needs 256 elements, got 224"),
            (dict(w_scales=w[1].view(-1)[:256]), ValueError, "w_scales needs 512 elements, got 256"),
            (dict(w_gs=w[2][:0]), ValueError, "w_gs needs 1 elements, got 0"),
            (dict(out=out[:3]), ValueError, "out needs 4 rows of 8 elements"),
            (dict(out=out.t().contiguous().t()), ValueError, "out rows must be contiguous"),
            (dict(out=torch.zeros(4, 7, dtype=BF)), ValueError, "out rows must be contiguous and out_stride"),
            (dict(out=out.float()), TypeError, "out must be torch.bfloat16"),
            (dict(out_rows=torch.zeros(3, dtype=torch.int32)), ValueError, "out_rows needs 4 elements, got 3"),
            (dict(device_status=torch.zeros(1, dtype=torch.int32)), ValueError, "device_status needs 2 elements, got 1")):
        with pytest.raises(error, match=text):
            call(b4.fp4_matmul, product, **kw)
