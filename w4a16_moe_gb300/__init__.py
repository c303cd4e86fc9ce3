"""GB300 (sm_103a) fused W4A16 mixture-of-experts layer.

A thin Python binding over the C ABI of ``libb4moe.so`` (``include/b4moe.h``):
argument marshalling only -- every step of the layer runs in the library's
CUDA kernels.  Tensors are torch CUDA tensors (torch serves as the device
allocator and stream provider); their data pointers are handed to the C
entry points as plain addresses.

The library must be built first (``python w4a16_moe_gb300/build.py`` or
``__graft_entry__.build()``); importing this package without it raises.
"""

from __future__ import annotations

import ctypes
import dataclasses
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libb4moe.so")

B4_OK = 0
B4_ERR_INVALID_ARGUMENT = 1
B4_ERR_UNSUPPORTED_DEVICE = 2
B4_ERR_WORKSPACE_TOO_SMALL = 3
B4_ERR_CUDA = 4
B4_ERR_TIMEOUT = 5

NVFP4 = 0
MXFP4 = 1
SILU = 0
RELU2 = 1
SWIGLU_OAI = 2
PATH_AUTO = 0
PATH_DECODE = 1
PATH_GROUPED = 2
DECODE_MAX_M = 64
NOALLOC_SCRATCH_BYTES = 64 << 20
FORMATS = {"nvfp4_e4m3_k16": NVFP4, "mxfp4_e8m0_k32": MXFP4}
ACTIVATIONS = {"silu": SILU, "relu2": RELU2, "swiglu_oai": SWIGLU_OAI}
# FP4 operators: element types, global-scale modes and scale layouts
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
GS_NONE = 0
GS_GIVEN = 1
GS_ROW = 2
GS_TENSOR = 3
SCALES_TILED = 0
SCALES_ROWS = 1
# the gpt-oss models' clamped-swiglu parameters (alpha, beta, limit)
SWIGLU_OAI_DEFAULTS = (1.702, 1.0, 7.0)


class B4Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_string(status)}: {message}")
        self.status = status


class _Config(ctypes.Structure):
    _fields_ = [
        ("m", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("num_global_experts", ctypes.c_int32),
        ("num_local_experts", ctypes.c_int32),
        ("hidden", ctypes.c_int32),
        ("inter", ctypes.c_int32),
        ("format", ctypes.c_int32),
        ("path", ctypes.c_int32),
        ("expert_map", ctypes.c_void_p),
        ("swiglu_alpha", ctypes.c_float),
        ("swiglu_beta", ctypes.c_float),
        ("swiglu_limit", ctypes.c_float),
    ]


class _Fp4Config(ctypes.Structure):
    _fields_ = [
        ("m", ctypes.c_int32),
        ("n", ctypes.c_int32),
        ("k", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("format", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("activation", ctypes.c_int32),
        ("gs_mode", ctypes.c_int32),
        ("scale_layout", ctypes.c_int32),
        ("row_div", ctypes.c_int32),
        ("x_rows", ctypes.c_int32),
        ("swiglu_alpha", ctypes.c_float),
        ("swiglu_beta", ctypes.c_float),
        ("swiglu_limit", ctypes.c_float),
        ("x_stride", ctypes.c_int64),
        ("out_stride", ctypes.c_int64),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python w4a16_moe_gb300/build.py` "
            "(there is no CPU or Python fallback for this layer)"
        )
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    S = ctypes.c_size_t
    I32 = ctypes.c_int32
    CP = ctypes.POINTER(_Config)
    FP = ctypes.POINTER(_Fp4Config)
    sigs = {
        "b4_route_capacity_tokens": (I32, [I32]),
        "b4_workspace_bytes": (S, [CP, I32]),
        "b4_prepared_sizes": (I32, [CP, I32, I32, ctypes.POINTER(S), ctypes.POINTER(S)]),
        "b4_prepare_weights": (I32, [CP, I32, I32, P, P, P, P, P]),
        "b4_route_pack": (I32, [CP, P, P, P, P, P]),
        "b4_fused_moe": (I32, [CP, P, P, P, P, P, P, P, P, P, I32, P, P, S, P]),
        "b4_fused_moe_noalloc": (I32, [CP, P, P, P, P, P, P, P, P, P, I32, P, P, P]),
        "b4_linear_workspace_bytes": (S, [CP]),
        "b4_linear": (I32, [CP, P, P, P, P, P, P, S, P]),
        "b4_check_status": (I32, [P, P]),
        "b4_wait_self_test": (I32, [P, S, ctypes.c_uint32, P]),
        "b4_set_timing_events": (I32, [ctypes.POINTER(P), I32]),
        "b4_set_trace": (I32, [P, S]),
        "b4_fp4_codes_bytes": (S, [FP, I32]),
        "b4_fp4_scale_bytes": (S, [FP, I32]),
        "b4_fp4_quantize": (I32, [FP, P, P, P, P, P, P, P, P]),
        "b4_fp4_tile_scales": (I32, [FP, P, P, P]),
        "b4_fp4_matmul": (I32, [FP, P, P, P, P, P, P, P, P, P, P, P]),
        "b4_fp4_linear_workspace_bytes": (S, [FP]),
        "b4_fp4_linear": (I32, [FP, P, P, P, P, P, P, P, P, P, P, S, P]),
        "b4_fused_moe_a4_workspace_bytes": (S, [CP, I32]),
        "b4_fused_moe_a4": (I32, [CP, P, P, P, P, P, P, P, P, P, I32, P, P, S, P]),
        "b4_status_string": (ctypes.c_char_p, [I32]),
        "b4_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()
EXPORTED = (
    "b4_route_capacity_tokens",
    "b4_workspace_bytes",
    "b4_prepared_sizes",
    "b4_prepare_weights",
    "b4_route_pack",
    "b4_fused_moe",
    "b4_fused_moe_noalloc",
    "b4_linear_workspace_bytes",
    "b4_linear",
    "b4_check_status",
    "b4_wait_self_test",
    "b4_set_timing_events",
    "b4_set_trace",
    "b4_fp4_codes_bytes",
    "b4_fp4_scale_bytes",
    "b4_fp4_quantize",
    "b4_fp4_tile_scales",
    "b4_fp4_matmul",
    "b4_fp4_linear_workspace_bytes",
    "b4_fp4_linear",
    "b4_fused_moe_a4_workspace_bytes",
    "b4_fused_moe_a4",
    "b4_status_string",
    "b4_last_error",
)


def status_string(status: int) -> str:
    return _lib.b4_status_string(int(status)).decode()


def last_error() -> str:
    return _lib.b4_last_error().decode()


def _check(status: int):
    if status != B4_OK:
        raise B4Error(status, last_error())


@dataclasses.dataclass
class MoEConfig:
    """Shape of one fused MoE call (mirrors ``b4_moe_config``)."""

    m: int
    top_k: int
    num_global_experts: int
    num_local_experts: int
    hidden: int
    inter: int
    format: int = NVFP4
    path: int = PATH_AUTO
    expert_map: torch.Tensor | None = None  # int32 CUDA tensor [E_g] or None
    # read for the SWIGLU_OAI activation only
    swiglu_alpha: float = SWIGLU_OAI_DEFAULTS[0]
    swiglu_beta: float = SWIGLU_OAI_DEFAULTS[1]
    swiglu_limit: float = SWIGLU_OAI_DEFAULTS[2]

    def _c(self) -> _Config:
        em = 0
        if self.expert_map is not None:
            _need(self.expert_map, torch.int32, "expert_map")
            em = self.expert_map.data_ptr()
        return _Config(self.m, self.top_k, self.num_global_experts, self.num_local_experts,
                       self.hidden, self.inter, self.format, self.path, em,
                       self.swiglu_alpha, self.swiglu_beta, self.swiglu_limit)


def _need(t, dtype, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


# torch's handle of a device's current stream without building a Stream object (2 - 3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(stream, t):
    """Handle of ``stream``, or of the current stream of the tensor's device."""
    if stream is not None:
        return stream.cuda_stream
    device = t.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, got {device}")
    return _stream(None) if _raw_stream is None else _raw_stream(device.index)


def route_capacity_tokens(m: int) -> int:
    return int(_lib.b4_route_capacity_tokens(int(m)))


def workspace_bytes(cfg: MoEConfig, activation: int) -> int:
    c = cfg._c()
    n = _lib.b4_workspace_bytes(ctypes.byref(c), int(activation))
    if n == 0:
        raise B4Error(B4_ERR_INVALID_ARGUMENT, last_error())
    return int(n)


def prepared_sizes(cfg: MoEConfig, which: int, activation: int):
    c = cfg._c()
    cb, sb = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(_lib.b4_prepared_sizes(ctypes.byref(c), int(which), int(activation), ctypes.byref(cb), ctypes.byref(sb)))
    return int(cb.value), int(sb.value)


def prepare_weights(cfg: MoEConfig, which: int, activation: int, src_codes, src_scales, dst_codes=None,
                    dst_scales=None, stream=None):
    """Checkpoint layout -> serving layout.  Allocates the outputs with torch when not given."""
    _need(src_codes, torch.uint8, "src_codes")
    _need(src_scales, torch.uint8, "src_scales")
    cb, sb = prepared_sizes(cfg, which, activation)
    dev = src_codes.device
    if dst_codes is None:
        dst_codes = torch.empty(cb, dtype=torch.uint8, device=dev)
    if dst_scales is None:
        dst_scales = torch.empty(sb, dtype=torch.uint8, device=dev)
    c = cfg._c()
    _check(_lib.b4_prepare_weights(ctypes.byref(c), int(which), int(activation), _ptr(src_codes), _ptr(src_scales),
                                   _ptr(dst_codes), _ptr(dst_scales), _stream(stream)))
    return dst_codes, dst_scales


def route_pack(cfg: MoEConfig, topk_ids, counts, offsets, sorted_routes, stream=None):
    _need(topk_ids, torch.int32, "topk_ids")
    for t, n in ((counts, "counts"), (offsets, "offsets"), (sorted_routes, "sorted_routes")):
        _need(t, torch.int32, n)
    c = cfg._c()
    _check(_lib.b4_route_pack(ctypes.byref(c), _ptr(topk_ids), _ptr(counts), _ptr(offsets), _ptr(sorted_routes),
                              _stream(stream)))


def fused_moe(cfg: MoEConfig, x, w13, s13, gs13, w2, s2, gs2, topk_ids, topk_weights, activation, out, workspace,
              stream=None):
    """Enqueue the fused layer; ``out`` [m, H] bf16 is written in full."""
    _need(x, torch.bfloat16, "x")
    _need(out, torch.bfloat16, "out")
    _need(topk_ids, torch.int32, "topk_ids")
    _need(topk_weights, torch.float32, "topk_weights")
    _need(workspace, torch.uint8, "workspace")
    for t, n in ((w13, "w13"), (s13, "s13"), (w2, "w2"), (s2, "s2")):
        _need(t, torch.uint8, n)
    for t, n in ((gs13, "gs13"), (gs2, "gs2")):
        if t is not None:
            _need(t, torch.float32, n)
    c = cfg._c()
    _check(_lib.b4_fused_moe(ctypes.byref(c), _ptr(x), _ptr(w13), _ptr(s13), _ptr(gs13), _ptr(w2), _ptr(s2),
                             _ptr(gs2), _ptr(topk_ids), _ptr(topk_weights), int(activation), _ptr(out),
                             _ptr(workspace), workspace.numel(), _stream(stream)))


def fused_moe_noalloc(cfg: MoEConfig, x, w13, s13, gs13, w2, s2, gs2, topk_ids, topk_weights, activation, out,
                      device_status=None, stream=None):
    """``fused_moe`` for callers that cannot allocate: the scratch is the library's
    static device array of ``NOALLOC_SCRATCH_BYTES``; larger shapes are refused.
    ``device_status`` (optional int32 CUDA tensor of 2) receives the call's
    device status word.  Calls that overlap on the GPU race on the shared array."""
    _need(x, torch.bfloat16, "x")
    _need(out, torch.bfloat16, "out")
    _need(topk_ids, torch.int32, "topk_ids")
    _need(topk_weights, torch.float32, "topk_weights")
    for t, n in ((w13, "w13"), (s13, "s13"), (w2, "w2"), (s2, "s2")):
        _need(t, torch.uint8, n)
    for t, n in ((gs13, "gs13"), (gs2, "gs2")):
        if t is not None:
            _need(t, torch.float32, n)
    if device_status is not None:
        _need(device_status, torch.int32, "device_status")
        if device_status.numel() < 2:
            raise ValueError("device_status needs 2 elements")
    c = cfg._c()
    _check(_lib.b4_fused_moe_noalloc(ctypes.byref(c), _ptr(x), _ptr(w13), _ptr(s13), _ptr(gs13), _ptr(w2), _ptr(s2),
                                     _ptr(gs2), _ptr(topk_ids), _ptr(topk_weights), int(activation), _ptr(out),
                                     _ptr(device_status), _stream(stream)))


def linear_config(m: int, n: int, k: int, format: int = NVFP4, path: int = PATH_AUTO) -> MoEConfig:
    """Shape of a dense W4A16 linear call: out [m, n] = x [m, k] . W[n, k]^T
    (one expert, top-1, inter = n, hidden = k; ``b4_linear`` in b4moe.h)."""
    return MoEConfig(m=m, top_k=1, num_global_experts=1, num_local_experts=1, hidden=k, inter=n, format=format,
                     path=path)


def linear_workspace_bytes(cfg: MoEConfig) -> int:
    c = cfg._c()
    n = _lib.b4_linear_workspace_bytes(ctypes.byref(c))
    if n == 0:
        raise B4Error(B4_ERR_INVALID_ARGUMENT, last_error())
    return int(n)


def prepare_linear_weights(cfg: MoEConfig, src_codes, src_scales, stream=None):
    """W [n, k] (codes [n, k/2], scales [n, k/g]; a leading expert axis of 1 is
    optional) -> the serving layout ``linear`` reads (the non-gated FC1 layout)."""
    return prepare_weights(cfg, 0, RELU2, src_codes, src_scales, stream=stream)


def linear(cfg: MoEConfig, x, w, s, gs, out, workspace, stream=None):
    """Enqueue the dense W4A16 linear layer; ``out`` [m, n] bf16 is written in full."""
    _need(x, torch.bfloat16, "x")
    _need(out, torch.bfloat16, "out")
    _need(workspace, torch.uint8, "workspace")
    _need(w, torch.uint8, "w")
    _need(s, torch.uint8, "s")
    if gs is not None:
        _need(gs, torch.float32, "gs")
    c = cfg._c()
    _check(_lib.b4_linear(ctypes.byref(c), _ptr(x), _ptr(w), _ptr(s), _ptr(gs), _ptr(out), _ptr(workspace),
                          workspace.numel(), _stream(stream)))


# ------------------------------------------------------- FP4 x FP4 operators


class Fp4Config:
    """Shape of one call of the FP4 operators (``b4_fp4_config`` in b4moe.h); read-only once made.

    ``m`` rows (per matrix of a stack, or the row capacity with ``offsets``), ``n`` outputs, ``k`` quantised
    columns.  ``activation``: None, or SILU / RELU2 / SWIGLU_OAI applied to x first.  ``gs_mode`` defaults to
    GS_ROW for NVFP4 and GS_NONE for MXFP4.
    """

    def __init__(self, m, k, n=1, num_groups=1, format=NVFP4, x_dtype=torch.bfloat16, out_dtype=torch.bfloat16,
                 activation=None, gs_mode=None, scale_layout=SCALES_TILED, row_div=1, x_rows=0,
                 swiglu=SWIGLU_OAI_DEFAULTS, x_stride=0, out_stride=0):
        for t, name in ((x_dtype, "x_dtype"), (out_dtype, "out_dtype")):
            if t not in DTYPES:
                raise TypeError(f"{name} must be one of {list(DTYPES)}, got {t}")
        if gs_mode is None:
            gs_mode = GS_ROW if format == NVFP4 else GS_NONE
        self.m, self.k, self.n, self.num_groups = int(m), int(k), int(n), int(num_groups)
        self.format, self.gs_mode, self.x_dtype, self.out_dtype = format, gs_mode, x_dtype, out_dtype
        self.scale_layout = scale_layout
        self.gated = activation in (SILU, SWIGLU_OAI)
        self.width = 2 * self.k if self.gated else self.k
        self.x_stride = int(x_stride) or self.width
        self.out_stride = int(out_stride) or self.n
        self.ld = (self.k // 2 + 15) // 16 * 16
        self.blocks = self.k // (16 if format == NVFP4 else 32)
        self._struct = _Fp4Config(self.m, self.n, self.k, self.num_groups, format, DTYPES[x_dtype], DTYPES[out_dtype],
                                  -1 if activation is None else activation, gs_mode, scale_layout, int(row_div),
                                  int(x_rows), *swiglu, int(x_stride), int(out_stride))
        self._ref = ctypes.byref(self._struct)
        self._elements = (self.m * self.num_groups * self.x_stride, self.m * self.x_stride)  # of x: a stack's, ragged
        self._sizes = {}
        self._gather = (-1, None)

    def rows(self, ragged):
        return self.m if ragged else self.m * self.num_groups

    def _operand(self, ragged):
        """(rows, code bytes, scale bytes, global scales) of the quantised operand."""
        s = self._sizes.get(ragged)
        if s is None:
            n = self.rows(ragged)
            gs = {GS_NONE: 0, GS_ROW: n}.get(self.gs_mode, self.num_groups)
            s = self._sizes[ragged] = (n, n * self.ld, fp4_scale_bytes(self, ragged), gs)
        return s

    def _weight_sizes(self):
        """(code bytes, scale bytes, shape of row-major scales) of the weights."""
        s = self._sizes.get("w")
        if s is None:
            s = self._sizes["w"] = _stack_sizes(self.num_groups, self.n, self.k, self.format)
        return s


def _wider(t, pitch):
    """Whether a contiguous tensor has several rows that are longer than the config's, so that read in one go its rows
    would not be the config's.  (Callers ask it of tensors that hold more than the config's elements.)"""
    shape = t.shape
    return len(shape) > 1 and shape[-1] > pitch and shape[-1] != t.numel()


def _fp4_x(cfg, x, rows, ragged):
    """x as the config describes it: a 2-D view of rows, or any contiguous shape with that many elements.
    Returns the call's config: with gathered rows, bounded by the rows x holds."""
    if x.dtype is not cfg.x_dtype:
        raise TypeError(f"x must be {cfg.x_dtype}, got {x.dtype}")
    if x.is_contiguous():
        have = x.numel()
        if rows is None and have == cfg._elements[ragged]:
            return cfg._ref
        n = 0 if have < cfg.width else (have - cfg.width) // cfg.x_stride + 1
        if _wider(x, cfg.x_stride):
            raise ValueError(f"x has rows of {x.shape[-1]} elements, the config rows of {cfg.x_stride} (x_stride)")
    else:
        if x.dim() != 2 or x.stride(1) != 1 or x.stride(0) != cfg.x_stride:
            raise ValueError("x must be contiguous, or two-dimensional with rows x_stride elements apart")
        n = x.shape[0]
        if x.shape[1] < cfg.width:
            raise ValueError(f"x rows need {cfg.width} elements, got {x.shape[1]}")
    if rows is None:
        if n < cfg.rows(ragged):
            raise ValueError(f"x holds {n} rows, {cfg.rows(ragged)} needed")
    elif n == 0 and cfg.m:  # (a bound of 0 rows would be none)
        raise ValueError(f"x holds not one row of {cfg.width} elements to gather from")
    elif not 0 < cfg._struct.x_rows <= n:
        bounded = cfg._gather
        if bounded[0] != n:
            c = _Fp4Config.from_buffer_copy(cfg._struct)
            c.x_rows = n
            bounded = cfg._gather = (n, ctypes.byref(c))
        return bounded[1]
    return cfg._ref


_U8, _I32, _F32, _Tensor = torch.uint8, torch.int32, torch.float32, torch.Tensor


def _fp4_buffer(t, dtype, n, name):
    """Address of a contiguous tensor of at least n elements (None stays None)."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.numel() >= n and t.is_contiguous():
        return t.data_ptr()
    if t is None:
        return None
    _need(t, dtype, name)
    raise ValueError(f"{name} needs {n} elements, got {t.numel()}")


def _fp4_tiles(t, nbytes, name, shape):
    """Address of tiled scales.  ``shape`` is that of the same scales row by row, [matrices, rows, K / g], as a
    checkpoint holds them: they have the same size where the matrices fill their tiles, and are told by it (rows of
    512 scales are left alone: that may be a view of the tiles)."""
    if (isinstance(t, _Tensor) and t.dtype is _U8 and t.numel() >= nbytes and t.is_contiguous()
            and (t.dim() != 3 or t.shape != shape or shape[2] == 512)):
        return t.data_ptr()
    if _fp4_buffer(t, _U8, nbytes, name) is None:
        return None
    raise ValueError(f"{name} has the row-major shape of a checkpoint's scales; "
                     "tiled scales are needed (fp4_tile_scales)")


def fp4_codes_bytes(cfg: Fp4Config, ragged=False) -> int:
    n = _lib.b4_fp4_codes_bytes(cfg._ref, int(ragged))
    if n == 0 and cfg.m:
        raise B4Error(B4_ERR_INVALID_ARGUMENT, last_error())
    return int(n)


def fp4_scale_bytes(cfg: Fp4Config, ragged=False) -> int:
    n = _lib.b4_fp4_scale_bytes(cfg._ref, int(ragged))
    if n == 0 and cfg.m:
        raise B4Error(B4_ERR_INVALID_ARGUMENT, last_error())
    return int(n)


def fp4_empty(cfg: Fp4Config, device, ragged=False):
    """Output buffers of ``fp4_quantize``: codes [.., ld], scales (tiles [.., k tiles, 32, 4, 4] or rows) and gs
    ([groups, m] per row, [groups] otherwise, None for MXFP4)."""
    g = 16 if cfg.format == NVFP4 else 32
    lead = () if ragged else (cfg.num_groups,)
    codes = torch.empty(*lead, cfg.m, cfg.ld, dtype=torch.uint8, device=device)
    nbytes = fp4_scale_bytes(cfg, ragged)
    if cfg.scale_layout == SCALES_ROWS:
        scales = torch.empty(*lead, cfg.m, cfg.k // g, dtype=torch.uint8, device=device)
    else:
        kt = -(-cfg.k // (4 * g))
        scales = torch.empty(*lead, nbytes // (512 * kt * (1 if ragged else cfg.num_groups)), kt, 32, 4, 4,
                             dtype=torch.uint8, device=device)
    gs = None
    if cfg.gs_mode == GS_ROW:
        gs = torch.empty(*lead, cfg.m, dtype=torch.float32, device=device)
    elif cfg.gs_mode != GS_NONE:
        gs = torch.empty(cfg.num_groups, dtype=torch.float32, device=device)
    return codes, scales, gs


def fp4_quantize(cfg: Fp4Config, x, codes, scales, gs=None, values=None, rows=None, offsets=None, stream=None):
    """Enqueue the quantisation of x rows into ``codes``, ``scales`` and ``gs`` (an input with GS_GIVEN).

    x: rows of the config's width, x_stride elements apart, or a contiguous tensor of any shape that holds exactly the
    config's elements.  ``rows`` gathers from x's rows (entries that name none give zero rows)."""
    ragged = offsets is not None
    n, code_bytes, scale_bytes, gs_n = cfg._operand(ragged)
    st = _lib.b4_fp4_quantize(
        _fp4_x(cfg, x, rows, ragged), x.data_ptr(), rows if rows is None else _fp4_buffer(rows, _I32, n, "rows"),
        _fp4_buffer(offsets, _I32, cfg.num_groups + 1, "offsets") if ragged else None,
        gs if gs is None else _fp4_buffer(gs, _F32, gs_n, "gs"), _fp4_buffer(codes, _U8, code_bytes, "codes"),
        _fp4_buffer(scales, _U8, scale_bytes, "scales"),
        values if values is None else _fp4_buffer(values, cfg.x_dtype, n * cfg.k, "values"), _stream_of(stream, x))
    if st:
        _check(st)


def fp4_tile_scales(cfg: Fp4Config, src, dst=None, stream=None):
    """Row-major scales [groups, m, k/g] of a checkpoint -> the tiles the product reads."""
    g = 16 if cfg.format == NVFP4 else 32
    if cfg.scale_layout != SCALES_TILED:
        raise ValueError("fp4_tile_scales writes tiles: the config's scale_layout must be SCALES_TILED")
    need = fp4_scale_bytes(cfg)
    if dst is None:
        kt = -(-cfg.k // (4 * g))
        dst = torch.empty(cfg.num_groups, -(-cfg.m // 128), kt, 32, 4, 4, dtype=torch.uint8, device=src.device)
    _check(_lib.b4_fp4_tile_scales(cfg._ref, _fp4_buffer(src, torch.uint8, cfg.rows(False) * (cfg.k // g), "src"),
                                   _fp4_buffer(dst, torch.uint8, need, "dst"), _stream(stream)))
    return dst


def _fp4_out(cfg, out, rows):
    if out.dtype is not cfg.out_dtype:
        raise TypeError(f"out must be {cfg.out_dtype}, got {out.dtype}")
    shape = out.shape
    if len(shape) == 2:
        if rows and (out.stride(1) != 1 or (shape[0] > 1 and out.stride(0) != cfg.out_stride)):
            raise ValueError("out rows must be contiguous and out_stride elements apart")
        ok = shape[0] >= rows and shape[1] >= cfg.n
    else:
        if not out.is_contiguous():
            raise ValueError("out must be contiguous, or two-dimensional with rows out_stride elements apart")
        if out.numel() != rows * cfg.out_stride and _wider(out, cfg.out_stride):
            raise ValueError(f"out has rows of {shape[-1]} elements, the config rows of {cfg.out_stride} (out_stride)")
        ok = rows == 0 or out.numel() >= (rows - 1) * cfg.out_stride + cfg.n
    if not ok:
        raise ValueError(f"out needs {rows} rows of {cfg.n} elements")
    return out.data_ptr()


def fp4_matmul(cfg: Fp4Config, a_codes, a_scales, a_gs, w_codes, w_scales, w_gs, out, offsets=None, out_rows=None,
               device_status=None, stream=None):
    """Enqueue the product of two quantised operands (``b4_fp4_matmul``)."""
    n, code_bytes, scale_bytes, gs_n = cfg._operand(offsets is not None)
    w_bytes, ws_bytes, ws_rows = cfg._weight_sizes()
    st = _lib.b4_fp4_matmul(
        cfg._ref, _fp4_buffer(a_codes, _U8, code_bytes, "a_codes"),
        _fp4_tiles(a_scales, scale_bytes, "a_scales", (cfg.num_groups, cfg.m, cfg.blocks)),
        a_gs if a_gs is None else _fp4_buffer(a_gs, _F32, gs_n, "a_gs"),
        _fp4_buffer(w_codes, _U8, w_bytes, "w_codes"), _fp4_tiles(w_scales, ws_bytes, "w_scales", ws_rows),
        w_gs if w_gs is None else _fp4_buffer(w_gs, _F32, cfg.num_groups, "w_gs"),
        offsets if offsets is None else _fp4_buffer(offsets, _I32, cfg.num_groups + 1, "offsets"),
        out_rows if out_rows is None else _fp4_buffer(out_rows, _I32, n, "out_rows"), _fp4_out(cfg, out, n),
        device_status if device_status is None else _fp4_buffer(device_status, _I32, 2, "device_status"),
        _stream_of(stream, a_codes))
    if st:
        _check(st)


def fp4_linear_workspace_bytes(cfg: Fp4Config) -> int:
    n = _lib.b4_fp4_linear_workspace_bytes(cfg._ref)
    if n == 0:
        raise B4Error(B4_ERR_INVALID_ARGUMENT, last_error())
    return int(n)


def fp4_linear(cfg: Fp4Config, x, w_codes, w_scales, w_gs, out, workspace, x_gs=None, rows=None, offsets=None,
               out_rows=None, stream=None):
    """Enqueue quantisation of x and the product with the quantised weights: ``out`` [m, n].

    With ``offsets`` [groups + 1] the rows are grouped by expert; ``rows`` gathers them from x (row i of the
    operand is x row rows[i] // row_div) and ``out_rows`` scatters the result.
    """
    m = cfg.m
    w_bytes, ws_bytes, ws_rows = cfg._weight_sizes()
    ragged = offsets is not None
    st = _lib.b4_fp4_linear(
        _fp4_x(cfg, x, rows, ragged), x.data_ptr(),
        x_gs if x_gs is None else _fp4_buffer(x_gs, _F32, cfg.num_groups, "x_gs"),
        rows if rows is None else _fp4_buffer(rows, _I32, m, "rows"),
        _fp4_buffer(offsets, _I32, cfg.num_groups + 1, "offsets") if ragged else None,
        _fp4_buffer(w_codes, _U8, w_bytes, "w_codes"), _fp4_tiles(w_scales, ws_bytes, "w_scales", ws_rows),
        w_gs if w_gs is None else _fp4_buffer(w_gs, _F32, cfg.num_groups, "w_gs"),
        out_rows if out_rows is None else _fp4_buffer(out_rows, _I32, m, "out_rows"), _fp4_out(cfg, out, m),
        _fp4_buffer(workspace, _U8, 0, "workspace"), workspace.numel(), _stream_of(stream, x))
    if st:
        _check(st)


def fused_moe_a4_workspace_bytes(cfg: MoEConfig, activation: int) -> int:
    c = cfg._c()
    n = _lib.b4_fused_moe_a4_workspace_bytes(ctypes.byref(c), int(activation))
    if n == 0:
        raise B4Error(B4_ERR_INVALID_ARGUMENT, last_error())
    return int(n)


def _stack_sizes(e, n, k, format):
    """(code bytes, scale bytes, shape of row-major scales) of a stack of e quantised [n, k] matrices."""
    g = 16 if format == NVFP4 else 32
    return e * n * ((k // 2 + 15) // 16 * 16), 512 * e * -(-n // 128) * -(-k // (4 * g)), (e, n, k // g)


@functools.lru_cache(maxsize=64)
def _layer_sizes(e, h, i, format, activation):
    """The sizes of W13 and of W2."""
    return _stack_sizes(e, i if activation == RELU2 else 2 * i, h, format) + _stack_sizes(e, h, i, format)


def fused_moe_a4(cfg: MoEConfig, x, w13, s13, gs13, w2, s2, gs2, topk_ids, topk_weights, activation, out, workspace,
                 stream=None):
    """The fused layer with 4-bit activations (``b4_fused_moe_a4``): weights as quantised operands
    (``fp4_quantize``, or checkpoint codes with ``fp4_tile_scales``: rows of codes are K/2 bytes rounded up to 16
    apart, so a checkpoint's codes are used as they are where hidden and inter are multiples of 32); ``out`` [m, H]
    bf16 is written in full."""
    e, m, h, i = cfg.num_local_experts, cfg.m, cfg.hidden, cfg.inter
    w13_bytes, s13_bytes, s13_rows, w2_bytes, s2_bytes, s2_rows = _layer_sizes(e, h, i, cfg.format, activation)
    rows, routes = m * h, m * cfg.top_k
    xp, op = _fp4_buffer(x, torch.bfloat16, rows, "x"), _fp4_buffer(out, torch.bfloat16, rows, "out")
    w13p, s13p = _fp4_buffer(w13, _U8, w13_bytes, "w13"), _fp4_tiles(s13, s13_bytes, "s13", s13_rows)
    w2p, s2p = _fp4_buffer(w2, _U8, w2_bytes, "w2"), _fp4_tiles(s2, s2_bytes, "s2", s2_rows)
    idp = _fp4_buffer(topk_ids, _I32, routes, "topk_ids")
    wtp = _fp4_buffer(topk_weights, _F32, routes, "topk_weights")
    _need(workspace, _U8, "workspace")
    if None in (xp, op, w13p, s13p, w2p, s2p, idp, wtp):
        for t, name in ((x, "x"), (out, "out"), (topk_ids, "topk_ids"), (topk_weights, "topk_weights"), (w13, "w13"),
                        (s13, "s13"), (w2, "w2"), (s2, "s2")):
            if t is None:
                raise TypeError(f"{name} must be a torch tensor")
    for t, name in ((x, "x"), (out, "out")):
        if t.numel() != rows and _wider(t, h):
            raise ValueError(f"{name} has rows of {t.shape[-1]} elements, the config rows of {h}")
    c = cfg._c()
    st = _lib.b4_fused_moe_a4(ctypes.byref(c), xp, w13p, s13p, _fp4_buffer(gs13, _F32, e, "gs13"), w2p, s2p,
                              _fp4_buffer(gs2, _F32, e, "gs2"), idp, wtp, int(activation), op, workspace.data_ptr(),
                              workspace.numel(), _stream(stream))
    if st:
        _check(st)


def fused_moe_raw(cfg: MoEConfig, ptrs: dict, activation: int, workspace_ptr: int, workspace_bytes_: int,
                  stream_handle: int) -> int:
    """The C call with raw addresses (host code that manages its own pointers); returns the status."""
    c = cfg._c()
    return int(_lib.b4_fused_moe(ctypes.byref(c), ptrs["x"], ptrs["w13"], ptrs["s13"], ptrs.get("gs13"), ptrs["w2"],
                                 ptrs["s2"], ptrs.get("gs2"), ptrs["topk_ids"], ptrs["topk_weights"], int(activation),
                                 ptrs["out"], workspace_ptr, workspace_bytes_, stream_handle))


_timing_keepalive = None


def set_timing_events(events):
    """Per-kernel timing: a list of torch.cuda.Event(enable_timing=True), or None to stop."""
    global _timing_keepalive
    if events is None:
        _timing_keepalive = None
        _check(_lib.b4_set_timing_events(None, 0))
        return
    for e in events:  # torch creates the CUDA event at its first record
        if not e.cuda_event:
            e.record(torch.cuda.current_stream())
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _timing_keepalive = arr
    _check(_lib.b4_set_timing_events(arr, len(events)))


def set_trace(buffer):
    """Kernel timeline (see b4_set_trace): an int64 CUDA tensor of >= 32768 entries, or None."""
    if buffer is None:
        _check(_lib.b4_set_trace(None, 0))
    else:
        _need(buffer, torch.int64, "trace buffer")
        _check(_lib.b4_set_trace(buffer.data_ptr(), buffer.numel() * 8))


def check_status(workspace, stream=None):
    _check(_lib.b4_check_status(_ptr(workspace), _stream(stream)))


def wait_self_test(workspace, limit_us, stream=None):
    """Enqueue the bounded-wait diagnostic (b4_wait_self_test): a wait that no
    arrival completes runs out after limit_us and leaves B4_ERR_TIMEOUT in the
    workspace's status word (read it with check_status)."""
    _need(workspace, torch.uint8, "workspace")
    _check(_lib.b4_wait_self_test(_ptr(workspace), workspace.numel(), int(limit_us), _stream(stream)))


def raw_lib():
    """The loaded ctypes library (for tests of the C ABI itself)."""
    return _lib
