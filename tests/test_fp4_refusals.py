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
