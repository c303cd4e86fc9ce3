"""Host-side contract of the FP4 operators (CPU): sizes and refusals, none of which touch a device."""

import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def b4():
    import __graft_entry__

    __graft_entry__._build_module().build()
    import w4a16_moe_gb300 as mod

    return mod


def _addr(n=1 << 12):
    buf = ctypes.create_string_buffer(n + 256)
    return buf, (ctypes.addressof(buf) + 255) // 256 * 256


def test_config_struct_matches_the_header(b4):
    text = open(os.path.join(ROOT, "include", "b4moe.h")).read()
    body = re.search(r"typedef struct b4_fp4_config \{(.*?)\} b4_fp4_config;", text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = [f for decl in re.findall(r"\w+ ([\w, ]+);", body) for f in re.findall(r"\w+", decl)]
    assert [f[0] for f in b4._Fp4Config._fields_] == fields
    assert b4._Fp4Config.x_stride.offset == 64 and ctypes.sizeof(b4._Fp4Config) == 80
    for enum, names in (("b4_fp4_gs", {"NONE": b4.GS_NONE, "GIVEN": b4.GS_GIVEN, "ROW": b4.GS_ROW, "TENSOR": b4.GS_TENSOR}),
                        ("b4_dtype", {"BF16": 0, "F16": 1, "F32": 2}),
                        ("b4_fp4_scale_layout", {"TILED": b4.SCALES_TILED, "ROWS": b4.SCALES_ROWS})):
        vals = re.search(r"typedef enum %s \{(.*?)\}" % enum, text, re.S).group(1)
        assert {k.split("_")[-1]: int(v) for k, v in re.findall(r"(\w+)\s*=\s*(\d+)", vals)} == names


def test_sizes(b4):
    cfg = b4.Fp4Config(m=130, k=80, num_groups=3)
    assert cfg.ld == 48 and b4.fp4_codes_bytes(cfg) == 3 * 130 * 48
    assert b4.fp4_scale_bytes(cfg) == 3 * 2 * 2 * 512  # two row tiles, two tiles of 64 K
    assert b4.fp4_codes_bytes(cfg, ragged=True) == 130 * 48
    assert b4.fp4_scale_bytes(cfg, ragged=True) == (1 + 3) * 2 * 512
    mx = b4.Fp4Config(m=128, k=2880, format=b4.MXFP4)
    assert b4.fp4_scale_bytes(mx) == 23 * 512 and mx.gs_mode == b4.GS_NONE
    rows = b4.Fp4Config(m=130, k=80, num_groups=3, scale_layout=b4.SCALES_ROWS)
    assert b4.fp4_scale_bytes(rows) == 3 * 130 * 5
    codes, scales, gs = b4.fp4_empty(cfg, "cpu")
    assert codes.shape == (3, 130, 48) and scales.shape == (3, 2, 2, 32, 4, 4) and gs.shape == (3, 130)
    for m in range(0, 300, 7):  # the ragged rule always has room for every split of m rows
        c = b4.Fp4Config(m=m, k=16, num_groups=5)
        for cuts in ([0, 0, m, m, m, m], [0, m // 5, m // 2, m // 2, m - m // 7, m], [0, 1, 2, 3, 4, m]):
            cuts = sorted(min(x, m) for x in cuts)
            end = 0
            for e in range(5):
                t0 = cuts[e] // 128 + e
                assert t0 >= end
                end = t0 + -(-(cuts[e + 1] - cuts[e]) // 128)
            assert end * 512 <= b4.fp4_scale_bytes(c, ragged=True)


@pytest.mark.parametrize("kw,fragment", [
    (dict(m=-1), "m ="), (dict(k=24), "k ="), (dict(k=0), "k ="), (dict(k=48, format=1), "k ="),
    (dict(num_groups=0), "num_groups"), (dict(num_groups=1025), "num_groups"), (dict(format=5), "format"),
    (dict(activation=9), "activation"), (dict(gs_mode=7), "gs_mode"), (dict(gs_mode=0), "gs_mode"),
    (dict(format=1, gs_mode=2), "gs_mode"), (dict(row_div=0), "row_div"), (dict(x_stride=10), "x_stride"),
    (dict(scale_layout=4), "scale_layout"), (dict(x_rows=-3), "x_rows"),
    (dict(activation=2, swiglu=(1.0, 0.0, 0.0)), "swiglu"), (dict(activation=0, x_stride=80), "x_stride"),
])
def test_bad_shapes_are_refused(b4, kw, fragment):
    base = dict(m=4, k=64, n=8)
    base.update(kw)
    cfg = b4.Fp4Config(**base)
    with pytest.raises(b4.B4Error) as ei:
        b4.fp4_linear_workspace_bytes(cfg)
    assert ei.value.status == b4.B4_ERR_INVALID_ARGUMENT and fragment in str(ei.value)


@pytest.mark.parametrize("kw", [dict(n=0), dict(n=(1 << 20) + 1), dict(out_stride=7)])
def test_bad_outputs_are_refused(b4, kw):
    base = dict(m=4, k=64, n=8)
    base.update(kw)
    with pytest.raises(b4.B4Error):
        b4.fp4_linear_workspace_bytes(b4.Fp4Config(**base))


def test_calls_refuse_before_any_device(b4):
    lib = b4.raw_lib()
    keep, a = _addr()
    bad = b4.B4_ERR_INVALID_ARGUMENT

    def quant(c, x=a, rows=None, off=None, gs=a, codes=a, scales=a, values=None):
        return lib.b4_fp4_quantize(c._ref, x, rows, off, gs, codes, scales, values, None)

    nv, mx = b4.Fp4Config(m=4, k=64, n=8), b4.Fp4Config(m=4, k=64, n=8, format=b4.MXFP4)
    assert quant(nv, x=None) == bad and "null" in b4.last_error()
    assert quant(nv, gs=None) == bad and quant(mx) == bad
    assert quant(nv, codes=a + 8) == bad and quant(nv, scales=a + 4) == bad and quant(nv, values=a + 2) == bad
    assert quant(nv, x=a + 1) == bad and quant(nv, rows=a + 2) == bad
    assert quant(b4.Fp4Config(m=4, k=64, gs_mode=b4.GS_TENSOR), rows=a) == bad
    assert quant(b4.Fp4Config(m=0, k=64), x=None, codes=None, scales=None) == b4.B4_OK

    def mm(c, ac=a, asc=a, ag=a, wc=a, wsc=a, wg=a, off=None, to=None, out=a, st=None):
        return lib.b4_fp4_matmul(c._ref, ac, asc, ag, wc, wsc, wg, off, to, out, st, None)

    assert mm(nv, out=None) == bad and mm(nv, ag=None) == bad and mm(nv, wg=None) == bad and mm(nv, wc=None) == bad
    assert mm(mx) == bad and mm(mx, ag=None) == bad and "global scale" in b4.last_error()
    assert mm(nv, ac=a + 8) == bad and mm(nv, wsc=a + 8) == bad and mm(nv, out=a + 1) == bad and mm(nv, st=a + 2) == bad
    assert mm(b4.Fp4Config(m=0, k=64, n=8), None, None) == b4.B4_OK
    assert mm(b4.Fp4Config(m=1 << 25, k=64, n=8, num_groups=1024)) == bad

    def linear(c, xg=None, off=None, ws=a, nbytes=1 << 12, wg=a):
        return lib.b4_fp4_linear(c._ref, a, xg, None, off, a, a, wg, None, a, ws, nbytes, None)

    assert linear(b4.Fp4Config(m=4, k=64, n=8, num_groups=2)) == bad and "offsets" in b4.last_error()
    assert linear(b4.Fp4Config(m=4, k=64, n=8, gs_mode=b4.GS_TENSOR)) == bad
    assert linear(b4.Fp4Config(m=4, k=64, n=8, scale_layout=b4.SCALES_ROWS)) == bad
    assert linear(b4.Fp4Config(m=4, k=64, n=8, gs_mode=b4.GS_GIVEN)) == bad and linear(nv, xg=a) == bad
    assert linear(nv, ws=a + 16) == bad and linear(nv, ws=None) == bad
    assert linear(nv, nbytes=64) == b4.B4_ERR_WORKSPACE_TOO_SMALL
    assert linear(b4.Fp4Config(m=0, k=64, n=8)) == b4.B4_OK
    del keep


def test_layer_refuses_before_any_device(b4):
    lib = b4.raw_lib()
    keep, a = _addr()
    cfg = b4.MoEConfig(4, 2, 8, 8, 256, 512)
    need = b4.fused_moe_a4_workspace_bytes(cfg, b4.SILU)
    assert need > b4.fused_moe_a4_workspace_bytes(cfg, b4.RELU2) > 0
    assert b4.fused_moe_a4_workspace_bytes(b4.MoEConfig(3, 2, 8, 8, 256, 512), b4.SILU) == need

    def call(c, act=b4.SILU, x=a, g=a, ws=a, nbytes=1 << 40, out=a):
        c = c._c()
        return lib.b4_fused_moe_a4(ctypes.byref(c), x, a, a, g, a, a, g, a, a, act, out, ws, nbytes, None)

    assert call(cfg, x=None) == b4.B4_ERR_INVALID_ARGUMENT and call(cfg, g=None) == b4.B4_ERR_INVALID_ARGUMENT
    assert call(cfg, act=7) == b4.B4_ERR_INVALID_ARGUMENT and call(cfg, out=a + 2) == b4.B4_ERR_INVALID_ARGUMENT
    assert call(cfg, nbytes=need - 1) == b4.B4_ERR_WORKSPACE_TOO_SMALL
    assert call(b4.MoEConfig(0, 2, 8, 8, 256, 512)) == b4.B4_OK
    with pytest.raises(b4.B4Error):
        b4.fused_moe_a4_workspace_bytes(b4.MoEConfig(4, 0, 8, 8, 256, 512), b4.SILU)
    del keep


def test_python_refuses_short_or_mistyped_tensors(b4):
    cfg = b4.Fp4Config(m=4, k=64, n=8)
    codes, scales, gs = b4.fp4_empty(cfg, "cpu")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        b4.fp4_quantize(cfg, x.float(), codes, scales, gs)
    with pytest.raises(ValueError):
        b4.fp4_quantize(cfg, x[:3], codes, scales, gs)
    with pytest.raises(ValueError):
        b4.fp4_quantize(cfg, x, codes[:, :2].contiguous(), scales, gs)
    with pytest.raises(ValueError):
        b4.fp4_quantize(cfg, x.t(), codes, scales, gs)
    with pytest.raises(ValueError):
        b4.fp4_quantize(cfg, torch.zeros(4, 80, dtype=torch.bfloat16)[:, :64], codes, scales, gs)
    with pytest.raises(TypeError):
        b4.fp4_quantize(cfg, x, codes, scales, gs, rows=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        b4.fp4_quantize(cfg, x, codes, scales, gs, rows=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        b4.Fp4Config(m=4, k=64, x_dtype=torch.int8)
    w = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), torch.ones(1)
    out = torch.zeros(4, 8, dtype=torch.bfloat16)
    for args in ((codes, scales, gs, w[0][:7], w[1], w[2], out), (codes, scales, gs, w[0], w[1][:256], w[2], out),
                 (codes, scales, gs, *w, out[:3]), (codes, scales, gs, *w, out.t().contiguous().t()),
                 (codes, scales, gs, *w, torch.zeros(4, 7, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            b4.fp4_matmul(cfg, *args)
    with pytest.raises(TypeError):
        b4.fp4_matmul(cfg, codes, scales, gs, *w, out.float())
