"""What the binding of the routing and FP8 operators refuses, operand by operand (CPU).

The library is replaced by a recorder, so that a call that is let through is seen and nothing runs.
"""

import glob
import os
import re

import pytest
import torch

BF, F32, U8, I32, E4M3 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.float8_e4m3fn


@pytest.fixture
def b4(monkeypatch):
    import __graft_entry__

    __graft_entry__._build_module().build()
    import w4a16_moe_gb300 as mod

    calls = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *args: calls.append(name) or 0

    monkeypatch.setattr(mod, "_lib", Recorder())
    monkeypatch.setattr(mod, "_launch_stream", lambda stream, t, name: (0, t.get_device()))
    mod.calls = calls
    yield mod
    del mod.calls


def _entries(b4):
    """Entry point -> (call, its tensors by name)."""
    m, k, n, kb, top = 4, 272, 200, 3, 2
    q, blocks, p, r = (b4.Fp8Config(m=m, k=k), b4.Fp8Config(m=n, k=k, x_dtype=F32, block_rows=128), b4.Fp8Config(m=m, k=k, n=n),
                       b4.RouterConfig(m, 16, top))
    layer = b4.MoEConfig(m, top, 8, 8, 272, 144)

    def z(*shape, dtype=F32):
        return torch.zeros(*shape, dtype=dtype)

    w = dict(w_codes=z(1, n, k, dtype=E4M3), w_scales=z(1, 2, kb))
    return {
        "route_topk": (lambda **t: b4.route_topk(r, **t), dict(logits=z(m, 16, dtype=BF), topk_ids=z(m, top, dtype=I32),
                       topk_weights=z(m, top), bias=z(16), num_tokens=z(1, dtype=I32))),
        "fp8_quantize": (lambda **t: b4.fp8_quantize(q, **t), dict(x=z(m, k, dtype=BF), codes=z(m, k, dtype=E4M3), scales=z(m, kb),
                         values=z(m, k, dtype=BF), rows=z(m, dtype=I32), offsets=z(2, dtype=I32))),
        "fp8_quantize blocks": (lambda **t: b4.fp8_quantize(blocks, **t), dict(x=z(n, k), codes=z(n, k, dtype=U8), scales=z(2, kb),
                                values=z(n, k))),
        "fp8_matmul": (lambda **t: b4.fp8_matmul(p, **t), dict(a_codes=z(m, k, dtype=E4M3), a_scales=z(m, kb), **w, out=z(m, n, dtype=BF),
                       offsets=z(2, dtype=I32), out_rows=z(m, dtype=I32), device_status=z(2, dtype=I32))),
        "fp8_linear": (lambda **t: b4.fp8_linear(p, **t), dict(x=z(m, k, dtype=BF), **w, out=z(m, n, dtype=BF), workspace=z(9, dtype=U8),
                       rows=z(m, dtype=I32), offsets=z(2, dtype=I32), out_rows=z(m, dtype=I32))),
        "fused_moe_fp8": (lambda **t: b4.fused_moe_fp8(layer, activation=b4.SILU, **t),
                          dict(x=z(m, 272, dtype=BF), w13=z(8, 288, 272, dtype=E4M3), s13=z(8, 3, 3), w2=z(8, 272, 144, dtype=U8),
                               s2=z(8, 3, 2), topk_ids=z(m, top, dtype=I32), topk_weights=z(m, top), out=z(m, 272, dtype=BF),
                               workspace=z(9, dtype=U8))),
    }


ROWS = [("route_topk", "topk_ids"), ("route_topk", "topk_weights"), ("fp8_quantize", "codes"), ("fp8_quantize", "scales"),
        ("fp8_quantize", "values"), ("fp8_quantize blocks", "codes"), ("fp8_quantize blocks", "scales"),
        ("fp8_quantize blocks", "values"), ("fp8_matmul", "a_codes"), ("fp8_matmul", "a_scales"), ("fp8_matmul", "w_codes"),
        ("fp8_matmul", "w_scales"), ("fp8_linear", "w_codes"), ("fp8_linear", "w_scales"), ("fused_moe_fp8", "x"),
        ("fused_moe_fp8", "out"), ("fused_moe_fp8", "w13"), ("fused_moe_fp8", "s13"), ("fused_moe_fp8", "w2"),
        ("fused_moe_fp8", "s2"), ("fused_moe_fp8", "topk_ids"), ("fused_moe_fp8", "topk_weights")]


@pytest.mark.parametrize("entry,name", ROWS)
def test_rows_longer_than_the_configs_are_refused(b4, entry, name):
    """A contiguous tensor of longer rows would be read or written at another pitch; one of more rows is fine."""
    call, tensors = _entries(b4)[entry]
    call(**tensors)
    assert len(b4.calls) == 1
    t = tensors[name]
    wide = torch.zeros(*t.shape[:-1], t.shape[-1] + 16, dtype=t.dtype)
    with pytest.raises(ValueError, match=rf"^{name} has rows of {t.shape[-1] + 16} "):
        call(**{**tensors, name: wide})
    assert len(b4.calls) == 1
    call(**{**tensors, name: torch.zeros(t.shape[0] + 1, *t.shape[1:], dtype=t.dtype)})
    call(**{**tensors, name: torch.zeros(t.numel() + 5, dtype=t.dtype)})
    assert len(b4.calls) == 3


class Elsewhere(torch.Tensor):
    """A tensor of another device."""

    def get_device(self):
        return 1


PLACES = [(entry, name) for entry, names in {
    "route_topk": "topk_ids topk_weights bias num_tokens", "fp8_quantize": "codes scales values rows offsets",
    "fp8_matmul": "a_scales w_codes w_scales out offsets out_rows device_status",
    "fp8_linear": "w_codes w_scales out workspace rows offsets out_rows",
    "fused_moe_fp8": "w13 s13 w2 s2 topk_ids topk_weights out workspace"}.items() for name in names.split()]


@pytest.mark.parametrize("entry,name", PLACES)
def test_tensors_of_another_device_are_refused(b4, entry, name):
    """Each but the first, whose device is the call's."""
    call, tensors = _entries(b4)[entry]
    with pytest.raises(ValueError, match=rf"^{name} is on "):
        call(**{**tensors, name: tensors[name].as_subclass(Elsewhere)})
    first = next(iter(tensors))
    with pytest.raises(ValueError, match=" is on "):  # the other way round: it alone is there
        call(**{**tensors, first: tensors[first].as_subclass(Elsewhere)})
    assert not b4.calls
    call(**tensors)
    assert len(b4.calls) == 1


def test_an_expert_map_of_another_device_is_refused(b4):
    _, tensors = _entries(b4)["fused_moe_fp8"]
    em = torch.zeros(8, dtype=I32)
    for t, what in ((em.as_subclass(Elsewhere), "expert_map is on "), (em[:7], "expert_map needs 8")):
        with pytest.raises(ValueError, match=what):
            b4.fused_moe_fp8(b4.MoEConfig(4, 2, 8, 8, 272, 144, expert_map=t), activation=b4.SILU, **tensors)
    b4.fused_moe_fp8(b4.MoEConfig(4, 2, 8, 8, 272, 144, expert_map=em), activation=b4.SILU, **tensors)
    assert len(b4.calls) == 1


@pytest.mark.parametrize("entry,name", [("route_topk", "logits"), ("fp8_quantize", "x"), ("fp8_linear", "out"),
                                        ("fp8_matmul", "out"), ("fused_moe_fp8", "w13"), ("fused_moe_fp8", "topk_ids")])
def test_a_missing_tensor_is_named(b4, monkeypatch, entry, name):
    call, tensors = _entries(b4)[entry]
    if name == next(iter(tensors)):
        monkeypatch.undo()
    with pytest.raises(TypeError, match=f"{name} must be a torch tensor"):
        call(**{**tensors, name: None})


def test_gathering_from_more_rows_than_an_index_reaches(b4):
    """Every entry of rows names a row of such an x: no bound (a bound of the row count cut to 32 bits would drop some)."""
    rows = torch.zeros(4, dtype=I32)
    for make in (b4.Fp8Config, b4.Fp4Config):
        for n, bound in ((1000, 1000), (2**31 - 1, 2**31 - 1), (2**31, 0), (2**32 + 5, 0)):
            cfg = make(m=4, k=16)
            b4._fp4_x(cfg, torch.empty(n, 16, dtype=BF, device="meta"), rows, False, type(cfg._struct))
            bounded = cfg._gather[1]._obj if cfg._gather[1] is not None else cfg._struct
            assert bounded.x_rows == bound


def test_no_copy_is_multicast():
    """A copy into several CTAs may only read this GPU's memory, which the address of an operand does not tell."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a16_moe_gb300", "csrc")
    files = glob.glob(os.path.join(csrc, "*.cu*"))
    assert files
    for f in files:
        text = re.sub(r'"\s*"', "", open(f).read())  # (an instruction may be several literals)
        assert not re.search(r"cp\.async\.bulk[^;]*multicast", text), f
