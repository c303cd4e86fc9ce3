"""Host-side contract of the routing and FP8 operators (CPU): sizes and refusals, none of which touch a device."""

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


def _fields(text, name):
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    return [f for decl in re.findall(r"\w+ ([\w, ]+);", body) for f in re.findall(r"\w+", decl)]


def test_structs_and_enums_match_the_header(b4):
    text = open(os.path.join(ROOT, "include", "b4moe.h")).read()
    assert [f[0] for f in b4._Fp8Config._fields_] == _fields(text, "b4_fp8_config")
    assert [f[0] for f in b4._RouteConfig._fields_] == _fields(text, "b4_route_config")
    assert b4._Fp8Config.x_stride.offset == 56 and ctypes.sizeof(b4._Fp8Config) == 72
    assert b4._RouteConfig.logits_stride.offset == 40 and ctypes.sizeof(b4._RouteConfig) == 48
    for enum, names in (("b4_score", {"SOFTMAX": b4.SOFTMAX, "SIGMOID": b4.SIGMOID}),
                        ("b4_fp8_scale", {"F32": b4.FP8_SCALE_F32, "POW2": b4.FP8_SCALE_POW2})):
        vals = re.search(r"typedef enum %s \{(.*?)\}" % enum, text, re.S).group(1)
        assert {k.split("_")[-1]: int(v) for k, v in re.findall(r"(\w+)\s*=\s*(\d+)", vals)} == names


ROUTE_BAD = [
    (dict(m=-1), "m ="), (dict(num_experts=0), "num_experts"), (dict(num_experts=1025), "num_experts"), (dict(top_k=0), "top_k"),
    (dict(top_k=33, num_experts=64), "top_k"), (dict(top_k=17), "top_k"), (dict(num_groups=0), "num_groups"),
    (dict(num_groups=3), "num_groups"), (dict(num_groups=64, num_experts=64), "num_groups"), (dict(num_groups=4, top_groups=0), "top_groups"),
    (dict(num_groups=4, top_groups=5), "top_groups"), (dict(num_groups=8, top_groups=1, top_k=4), "top_groups"), (dict(group_top=0), "group_top"),
    (dict(group_top=3), "group_top"), (dict(score=2), "score"), (dict(scale=float("nan")), "scale"),
    (dict(scale=float("inf")), "scale"), (dict(stride=15), "logits_stride"),
]


@pytest.mark.parametrize("kw,fragment", ROUTE_BAD)
def test_bad_routing_is_refused(b4, kw, fragment):
    base = dict(m=4, num_experts=16, top_k=2)
    base.update(kw)
    cfg = b4.RouterConfig(**base)
    _, a = _addr()
    assert b4.raw_lib().b4_route_topk(cfg._ref, a, None, None, a, a, None) == b4.B4_ERR_INVALID_ARGUMENT
    assert fragment in b4.last_error()


def test_routing_refuses_pointers_and_tensors(b4):
    lib, bad = b4.raw_lib(), b4.B4_ERR_INVALID_ARGUMENT
    keep, a = _addr()
    cfg = b4.RouterConfig(4, 16, 2)
    assert lib.b4_route_topk(None, a, None, None, a, a, None) == bad
    for args in ((None, None, None, a, a), (a, None, None, None, a), (a, None, None, a, None)):
        assert lib.b4_route_topk(cfg._ref, *args, None) == bad and "null" in b4.last_error()
    for args in ((a + 1, None, None, a, a), (a, a + 2, None, a, a), (a, None, a + 1, a, a), (a, None, None, a + 2, a),
                 (a, None, None, a, a + 1)):
        assert lib.b4_route_topk(cfg._ref, *args, None) == bad and "misaligned" in b4.last_error()
    cfg._struct.logits_dtype = 3
    assert lib.b4_route_topk(cfg._ref, a, None, None, a, a, None) == bad and "logits_dtype" in b4.last_error()
    assert lib.b4_route_topk(b4.RouterConfig(0, 16, 2)._ref, None, None, None, None, None, None) == b4.B4_OK
    with pytest.raises(TypeError):
        b4.RouterConfig(4, 16, 2, dtype=torch.float64)
    cfg = b4.RouterConfig(4, 16, 2)
    ids, w = torch.empty(4, 2, dtype=torch.int32), torch.empty(4, 2)
    with pytest.raises(TypeError, match="logits"):
        b4.route_topk(cfg, torch.empty(4, 16), ids, w)
    with pytest.raises(ValueError, match="CUDA"):
        b4.route_topk(cfg, torch.empty(4, 16, dtype=torch.bfloat16), ids, w)


FP8_BAD = [
    (dict(m=-1), "m ="), (dict(m=(1 << 25) + 1), "m ="), (dict(k=24), "k ="), (dict(k=0), "k ="), (dict(k=1 << 17), "k ="),
    (dict(num_groups=0), "num_groups"), (dict(num_groups=1025), "num_groups"), (dict(activation=9), "activation"),
    (dict(scale_mode=2), "scale_mode"), (dict(block_rows=2), "block_rows"), (dict(block_rows=128), "block_rows"),
    (dict(row_div=0), "row_div"), (dict(x_stride=10), "x_stride"), (dict(x_rows=-3), "x_rows"),
    (dict(activation=2, swiglu=(1.0, 0.0, 0.0)), "swiglu"), (dict(activation=2, swiglu=(float("nan"), 0.0, 1.0)), "swiglu"),
    (dict(activation=0, x_stride=80), "x_stride"), (dict(n=0), "n ="), (dict(n=(1 << 20) + 1), "n ="), (dict(out_stride=7), "out_stride"),
]


@pytest.mark.parametrize("kw,fragment", FP8_BAD)
def test_bad_shapes_are_refused(b4, kw, fragment):
    base = dict(m=4, k=64, n=8)
    base.update(kw)
    with pytest.raises(b4.B4Error) as ei:
        b4.fp8_linear_workspace_bytes(b4.Fp8Config(**base))
    assert ei.value.status == b4.B4_ERR_INVALID_ARGUMENT and fragment in str(ei.value)


def test_calls_refuse_before_any_device(b4):
    lib, bad = b4.raw_lib(), b4.B4_ERR_INVALID_ARGUMENT
    keep, a = _addr()
    c = b4.Fp8Config(m=4, k=64, n=8)

    def quant(c=c, x=a, rows=None, off=None, codes=a, scales=a, values=None):
        return lib.b4_fp8_quantize(c._ref, x, rows, off, codes, scales, values, None)

    for kw in (dict(x=None), dict(codes=None), dict(scales=None)):
        assert quant(**kw) == bad and "null" in b4.last_error()
    for kw in (dict(codes=a + 8), dict(values=a + 8)):
        assert quant(**kw) == bad and "16-byte" in b4.last_error()
    for kw in (dict(x=a + 1), dict(scales=a + 2), dict(rows=a + 1), dict(off=a + 2)):
        assert quant(**kw) == bad and "misaligned" in b4.last_error()
    blocks = b4.Fp8Config(m=4, k=64, block_rows=128)
    for kw in (dict(rows=a), dict(off=a)):
        assert quant(blocks, **kw) == bad and "128 rows" in b4.last_error()
    assert quant(b4.Fp8Config(m=1 << 25, k=64, num_groups=1024)) == bad and "row index" in b4.last_error()
    assert quant(b4.Fp8Config(m=0, k=64), x=None) == b4.B4_OK

    def matmul(c=c, ac=a, asc=a, wc=a, wsc=a, off=None, to=None, out=a, status=None):
        return lib.b4_fp8_matmul(c._ref, ac, asc, wc, wsc, off, to, out, status, None)

    for kw in (dict(ac=None), dict(asc=None), dict(wc=None), dict(wsc=None), dict(out=None)):
        assert matmul(**kw) == bad and "null" in b4.last_error()
    for kw in (dict(ac=a + 8), dict(wc=a + 4)):
        assert matmul(**kw) == bad and "16-byte" in b4.last_error()
    for kw in (dict(asc=a + 2), dict(wsc=a + 1), dict(off=a + 1), dict(to=a + 2), dict(out=a + 1), dict(status=a + 2)):
        assert matmul(**kw) == bad and "misaligned" in b4.last_error()
    assert matmul(blocks) == bad and "block_rows" in b4.last_error()
    assert matmul(b4.Fp8Config(m=0, k=64)) == b4.B4_OK

    def linear(c=c, x=a, rows=None, off=None, wc=a, wsc=a, to=None, out=a, ws=a, n=1 << 30):
        return lib.b4_fp8_linear(c._ref, x, rows, off, wc, wsc, to, out, ws, n, None)

    for kw in (dict(x=None), dict(out=None), dict(ws=None), dict(wc=None), dict(wsc=None)):
        assert linear(**kw) == bad and "null" in b4.last_error()
    assert linear(ws=a + 16) == bad and "256-byte" in b4.last_error()
    assert linear(b4.Fp8Config(m=4, k=64, n=8, num_groups=2)) == bad and "without offsets" in b4.last_error()
    assert linear(n=16) == b4.B4_ERR_WORKSPACE_TOO_SMALL
    for kw in (dict(x=a + 1), dict(rows=a + 1), dict(off=a + 2), dict(to=a + 2), dict(out=a + 1)):
        assert linear(**kw) == bad and "misaligned" in b4.last_error()


def test_layer_refusals_and_sizes(b4):
    lib, bad = b4.raw_lib(), b4.B4_ERR_INVALID_ARGUMENT
    keep, a = _addr()
    sizes = {m: b4.fused_moe_fp8_workspace_bytes(b4.MoEConfig(m, 2, 8, 8, 256, 512), b4.SILU) for m in (33, 64, 65)}
    assert sizes[33] == sizes[64] < sizes[65]  # by the power-of-two capacity
    # the format and the path are not read
    assert b4.fused_moe_fp8_workspace_bytes(b4.MoEConfig(64, 2, 8, 8, 256, 512, format=b4.MXFP4, path=b4.PATH_DECODE), b4.SILU) == sizes[64]
    for kw in (dict(hidden=40), dict(inter=24), dict(top_k=0), dict(num_local_experts=7)):
        cfg = b4.MoEConfig(**{**dict(m=4, top_k=2, num_global_experts=8, num_local_experts=8, hidden=256, inter=512), **kw})
        with pytest.raises(b4.B4Error):
            b4.fused_moe_fp8_workspace_bytes(cfg, b4.SILU)
    c = b4.MoEConfig(4, 2, 8, 8, 256, 512)._c()

    def layer(x=a, w13=a, s13=a, w2=a, s2=a, ids=a, wts=a, act=0, out=a, ws=a, n=1 << 30, cfg=c):
        return lib.b4_fused_moe_fp8(ctypes.byref(cfg), x, w13, s13, w2, s2, ids, wts, act, out, ws, n, None)

    for name in ("x", "w13", "s13", "w2", "s2", "ids", "wts", "out", "ws"):
        assert layer(**{name: None}) == bad and "null" in b4.last_error()
    for kw in (dict(x=a + 8), dict(out=a + 8), dict(w13=a + 8), dict(s2=a + 2), dict(ids=a + 2), dict(ws=a + 16)):
        assert layer(**kw) == bad and "align" in b4.last_error()
    assert layer(n=100) == b4.B4_ERR_WORKSPACE_TOO_SMALL
    assert layer(act=7) == bad
    assert lib.b4_fused_moe_fp8(None, a, a, a, a, a, a, a, 0, a, a, 1 << 30, None) == bad


def test_binding_refuses_small_or_wide_tensors(b4):
    """Sizes are looked at before anything is launched (CPU tensors: the device is refused first, so the helpers are called)."""
    cfg = b4.Fp8Config(m=4, k=64, n=200, num_groups=2)
    codes, scales = torch.zeros(2, 200, 64, dtype=torch.float8_e4m3fn), torch.zeros(2, 2, 1)
    assert b4._fp8_weights(cfg, codes, scales) == (codes.data_ptr(), scales.data_ptr())
    for c, s, what in ((codes[:1], scales, "w_codes"), (codes, scales[:, :1], "w_scales"), (codes, scales[:1], "w_scales"),
                       (torch.zeros(2, 200, 80, dtype=torch.uint8), scales, "w_codes"), (codes, torch.zeros(2, 2, 3), "w_scales"),
                       (codes.transpose(1, 2), scales, "w_codes")):
        with pytest.raises(ValueError, match=what):
            b4._fp8_weights(cfg, c, s)
    with pytest.raises(TypeError, match="w_scales"):
        b4._fp8_weights(cfg, codes, scales.double())
    with pytest.raises(TypeError, match="w_codes"):
        b4._fp8_weights(cfg, codes.float(), scales)
    for call in (lambda x: b4.fp8_quantize(cfg, x, codes, scales), lambda x: b4.fp8_linear(cfg, x, codes, scales, x, codes)):
        with pytest.raises(ValueError, match="CUDA"):
            call(torch.zeros(4, 64, dtype=torch.bfloat16))
    r = b4.RouterConfig(4, 16, 2)
    with pytest.raises(ValueError, match="topk_ids"):
        b4._route_out(torch.zeros(3, 2, dtype=torch.int32), torch.int32, r, "topk_ids")
    with pytest.raises(ValueError, match="rows of 3"):
        b4._route_out(torch.zeros(4, 3, dtype=torch.int32), torch.int32, r, "topk_ids")
    empty = b4.fp8_empty(b4.Fp8Config(m=130, k=144, num_groups=3, block_rows=128), "cpu")
    assert empty[0].shape == (3, 130, 144) and empty[1].shape == (3, 2, 2) and empty[0].dtype is torch.float8_e4m3fn
