"""Cases of the FP4 operators: block-scaled quantisation, the FP4 x FP4 product, and the product
grouped by expert with ragged sizes.

``own`` False computes the plain forms (elementary torch operations in 32 bits, rounded once at the
end); ``own`` True makes a user's calls of ``w4a16_moe_gb300``.

Formulas.  A row of x (bf16, f16 or f32), after the prologue h = x, silu(g) u, max(x, 0)^2 or the
clamped swiglu, is cut along K into blocks of 16 (NVFP4) or 32 (MXFP4):

    NVFP4   s = e4m3(amax_block / (6 gs)),  d = s gs,  c = e2m1(h / d)  (c = 0 where d = 0)
            gs per row: 2^j, j >= -126 the least with amax_row <= 6 448 2^j; per matrix: amax / (6 448);
            1 where amax is 0
    MXFP4   s = 2^k, k the least with amax_block <= 6 2^k,  c = e2m1(h / s)

with round-to-nearest-even saturating conversions.  The product of two such operands is
out[t][n] = gs_a[t] gs_w sum_k (c s)_a[t][k] (c s)_w[n][k]; grouped, the rows offsets[e] ..
offsets[e + 1] meet the weights of expert e, and rows past offsets[E] are zero.

Weights arrive as a checkpoint of this family holds them: codes [E, N, K/2], two a byte with the even
element in the low nibble, and scales in 512-byte tiles of 128 rows x 4 scales,
[E][ceil(N / 128)][ceil(K / 4g)][32][4][4] (row % 32, row / 32 % 4, scale), zero-padded.
"""

import math

import torch

own = False

NV, MX = "nvfp4_e4m3_k16", "mxfp4_e8m0_k32"
GROUP = {NV: 16, MX: 32}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
OAI = (1.702, 1.0, 7.0)


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one token's activations, quantised with its own global scale: decode latency
        dict(name="quantize_token", op="quantize", fmt=NV, dtype="bf16", groups=1, m=1, k=4096, gs="row"),
        # a prefill's activations
        dict(name="quantize_prefill", op="quantize", fmt=NV, dtype="bf16", groups=1, m=2048, k=4096, gs="row"),
        # fp32 master weights of 16 experts (E64 H2048 I1408 layer) into NVFP4, one global scale per expert
        dict(name="quantize_weights_nv", op="quantize", fmt=NV, dtype="f32", groups=16, m=2816, k=2048, gs="tensor"),
        # the W2 stack of a 28-expert MXFP4 layer, K not a multiple of 128
        dict(name="quantize_weights_mx", op="quantize", fmt=MX, dtype="bf16", groups=28, m=2880, k=1440, gs="none"),
        # a dense projection, one token: weight-stream latency
        dict(name="linear_token", op="linear", fmt=NV, dtype="bf16", m=1, n=4096, k=4096, act="none"),
        # a ragged batch of requests, scale tail along K
        dict(name="linear_batch_mx", op="linear", fmt=MX, dtype="bf16", m=37, n=1440, k=2880, act="none"),
        # the down projection behind a SwiGLU: [gate | up] rows in, quantised h inside
        dict(name="linear_gated", op="linear", fmt=NV, dtype="bf16", m=2048, n=2048, k=1408, act="silu"),
        # prefill through a dense projection
        dict(name="linear_prefill", op="linear", fmt=NV, dtype="bf16", m=4096, n=4096, k=4096, act="none"),
        # FC1 of a 128-expert layer, one token: eight experts of one row
        dict(name="grouped_token", op="grouped", fmt=NV, m=1, n=1536, k=4096, experts=128, top_k=8, hot=0, drop=0),
        # small batch with eight hot experts: groups of zero to dozens of rows
        dict(name="grouped_batch", op="grouped", fmt=NV, m=64, n=2816, k=2048, experts=64, top_k=6, hot=8, drop=0),
        # MXFP4, 32 global experts of which 28 are local, some routes invalid
        dict(name="grouped_mx", op="grouped", fmt=MX, m=512, n=2880, k=2880, experts=28, top_k=4, hot=0, drop=4),
        # prefill of the hot-expert layer: ragged groups of hundreds of rows
        dict(name="grouped_prefill", op="grouped", fmt=NV, m=2048, n=2816, k=2048, experts=64, top_k=6, hot=8, drop=0),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    v = max(step, int(round(v / step)) * step)
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(("quantize", "linear", "linear", "grouped", "grouped"))
    fmt = rng.choice((NV, MX))
    g = GROUP[fmt]
    if op == "quantize":
        groups = rng.choice((1, 1, _log(rng, 1, 32)))
        k = _log(rng, 64, 8192, g)
        m = _log(rng, 1, min(8192, max(2, 90_000_000 // (groups * k))))
        gs = "none" if fmt == MX else rng.choice(("row", "tensor"))
        return dict(op=op, fmt=fmt, dtype=rng.choice(("bf16", "bf16", "f16", "f32")), groups=groups, m=m, k=k, gs=gs)
    if op == "linear":
        n, k = _log(rng, 48, 4096), _log(rng, 64, 4096, g)
        return dict(op=op, fmt=fmt, dtype=rng.choice(("bf16", "bf16", "f16", "f32")), m=_log(rng, 1, 4096), n=n, k=k,
                    act=rng.choice(("none", "none", "silu", "relu2", "swiglu_oai")))
    experts = _log(rng, 2, 128)
    n, k = _log(rng, 64, 2880), _log(rng, 64, 2880, g)
    experts = max(1, min(experts, 400_000_000 // (n * k)))
    top_k = rng.randint(1, min(8, experts))
    m = max(1, min(_log(rng, 1, 2048), 12000 // top_k, int(5e10 / (top_k * n * k))))
    return dict(op=op, fmt=fmt, m=m, n=n, k=k, experts=experts, top_k=top_k, hot=rng.choice((0, 0, experts // 8)),
                drop=rng.choice((0, 0, 3)))


# ----------------------------------------------------------------- inputs


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1_000_003 + salt) % (1 << 62))
    return g


def _x(case, rows, cols, seed):
    """Activations: N(0, 1) with channels of different size; weights: N(0, 0.02)."""
    g = _gen(seed, 1)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    if case["op"] == "quantize" and case["gs"] in ("tensor", "none"):
        x *= 0.02
    else:
        x *= torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    return x.to(DTYPES[case.get("dtype", "bf16")])


def _cdiv(a, b):
    return (a + b - 1) // b


def _weights(case, experts, seed):
    """Codes [E, N, ld] (ld = K/2 rounded up to 16), tiled scales and global scales of random FP4 weights."""
    g, n, k = GROUP[case["fmt"]], case["n"], case["k"]
    gen = _gen(seed, 2)
    ld = _cdiv(k // 2, 16) * 16
    codes = torch.randint(0, 256, (experts, n, ld), generator=gen, device="cuda", dtype=torch.uint8)
    lo, hi = (0x68, 0x7F) if case["fmt"] == NV else (117, 125)  # 64 .. 448; 2^-10 .. 2^-3
    sc = torch.randint(lo, hi, (experts, n, k // g), generator=gen, device="cuda", dtype=torch.uint8)
    gs = None
    if case["fmt"] == NV:
        gs = 0.02 * 3.0 / (6.0 * 448.0) * (1.0 + 0.1 * torch.rand(experts, generator=gen, device="cuda"))
    return codes, _tile(sc), gs


def _tile(sc):
    """Row-major scales [E, N, K/g] -> [E, ceil(N/128), ceil(K/4g), 32, 4, 4], zero-padded."""
    e, n, b = sc.shape
    p = torch.zeros(e, _cdiv(n, 128) * 128, _cdiv(b, 4) * 4, dtype=sc.dtype, device=sc.device)
    p[:, :n, :b] = sc
    return p.view(e, -1, 4, 32, _cdiv(b, 4), 4).permute(0, 1, 4, 3, 2, 5).contiguous()


def _untile(t, n, b):
    e, rt, kt = t.shape[:3]
    return t.permute(0, 1, 4, 3, 2, 5).reshape(e, rt * 128, kt * 4)[:, :n, :b]


def _routing(case, seed):
    """Top-k routing packed by expert: offsets [E + 1], routes sorted by expert (stable), -1 past the valid ones."""
    e, k, m = case["experts"], case["top_k"], case["m"]
    gen = _gen(seed, 3)
    logits = torch.randn(m, e + case["drop"], generator=gen, device="cuda")
    if case["hot"]:
        logits[:, : case["hot"]] += 2.0
    ids = torch.topk(logits, k, dim=-1).indices.reshape(-1)  # ids from e on are not local: dropped
    order = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=e + case["drop"])[:e]
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    valid = torch.arange(m * k, device="cuda") < offsets[-1]
    routes = torch.where(valid, order, -1).to(torch.int32)
    return offsets, routes, max(1, int(counts.max())), torch.nonzero(counts).flatten()


def prepare(case, seed):
    s = {"case": case}
    if case["op"] == "quantize":
        s["x"] = _x(case, case["groups"] * case["m"], case["k"], seed).view(case["groups"], case["m"], case["k"])
    elif case["op"] == "linear":
        cols = 2 * case["k"] if case["act"] in ("silu", "swiglu_oai") else case["k"]
        s["x"] = _x(case, case["m"], cols, seed)
        s["w"] = _weights(case, 1, seed)
    else:
        s["x"] = _x(case, case["m"], case["k"], seed)
        s["w"] = _weights(case, case["experts"], seed)
        s["offsets"], s["routes"], s["most"], s["used"] = _routing(case, seed)
    return s


# ------------------------------------------------------------ plain forms


def _e2m1(q):
    """The E2M1 value nearest to q, ties to the even mantissa, saturating at 6."""
    a = q.abs()
    v = (0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75) + 1.0 * (a > 2.5)
         + 1.0 * (a >= 3.5) + 2.0 * (a > 5.0))
    return torch.where(q < 0, -v, v)


def _act_plain(x, act):
    x = x.float()
    if act == "none":
        return x
    if act == "relu2":
        r = torch.clamp_min(x, 0.0)
        return r * r
    g, u = x[..., : x.shape[-1] // 2], x[..., x.shape[-1] // 2:]
    if act == "silu":
        return g / (1.0 + torch.exp(-g)) * u
    alpha, beta, limit = OAI
    g, u = torch.clamp(g, max=limit), torch.clamp(u, -limit, limit)
    return g / (1.0 + torch.exp(-alpha * g)) * (u + beta)


def _quantize_plain(h, fmt, gs_mode):
    """h [G, m, K] f32 -> (E2M1 values [G, m, K/g, g], scales [G, m, K/g], gs [G, m] or [G] or None)."""
    b = h.view(*h.shape[:2], -1, GROUP[fmt])
    amax = b.abs().amax(-1)
    if fmt == MX:
        f, ex = torch.frexp(amax)  # amax = f 2^ex, f in [0.5, 1): amax <= 6 2^k from k = ex - 3 (f <= 0.75) on
        k = torch.where(amax > 0, ex - 3 + (f > 0.75), -127).clamp(-127, 127)
        s = torch.ldexp(torch.ones_like(amax), k)
        return _e2m1(torch.ldexp(b, -k[..., None])), s, None
    if gs_mode == "row":
        f, ex = torch.frexp(amax.amax(-1))  # 6 448 = 0.65625 2^12
        gs = torch.ldexp(torch.ones_like(f), torch.where(f > 0, (ex - 12 + (f > 0.65625)).clamp(min=-126), 0))
        gb = gs[:, :, None]
    else:
        top = amax.amax((-1, -2))
        gs = torch.where(top > 0, top / torch.full_like(top, 6.0 * 448.0), torch.ones_like(top))
        gb = gs[:, None, None]
    s = torch.clamp(amax / (6.0 * gb), max=448.0).to(torch.float8_e4m3fn).float()
    d = s * gb
    q = torch.where(d[..., None] > 0, b / torch.where(d > 0, d, torch.ones_like(d))[..., None], 0.0)
    return _e2m1(q), s, gs


def _dequant_plain(codes, tiles, fmt, n, k):
    """e2m1(code) * scale of [E, N, K] weights, without the global scale."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=codes.device)
    c = codes[:, :, : k // 2]
    v = torch.stack((table[(c & 15).long()], table[(c >> 4).long()]), -1).view(c.shape[0], n, k // GROUP[fmt], -1)
    s = _untile(tiles, n, k // GROUP[fmt])
    if fmt == NV:
        s = s.contiguous().view(torch.float8_e4m3fn).float()
    else:
        s = torch.ldexp(torch.ones((), device=s.device), s.int() - 127)
    return (v * s[..., None]).view(c.shape[0], n, k)


def _run_plain(s):
    case = s["case"]
    fmt = case["fmt"]
    if case["op"] == "quantize":
        c, sc, gs = _quantize_plain(s["x"].float(), fmt, case["gs"])
        if gs is None:
            return {"values": (c * sc[..., None]).view(s["x"].shape).to(s["x"].dtype)}
        d = sc * (gs[:, :, None] if case["gs"] == "row" else gs[:, None, None])
        return {"values": (c * d[..., None]).view(s["x"].shape).to(s["x"].dtype), "gs": gs,
                "scales": _tile(sc.to(torch.float8_e4m3fn).view(torch.uint8)).view(torch.float8_e4m3fn)}
    codes, tiles, gw = s["w"]
    if case["op"] == "linear":
        w = _dequant_plain(codes, tiles, fmt, case["n"], case["k"])
        c, sc, gs = _quantize_plain(_act_plain(s["x"], case["act"])[None], fmt, "row")
        a = (c * sc[..., None]).view(case["m"], case["k"])
        y = a @ w[0].T
        if gs is not None:
            y = y * (gs[0][:, None] * gw)
        return y.to(torch.bfloat16)
    # grouped: rows of one expert side by side, padded to the longest group; experts without rows left out
    off, routes, most, used = s["offsets"].long(), s["routes"], s["most"], s["used"]
    w = _dequant_plain(codes[used], tiles[used], fmt, case["n"], case["k"])
    c, sc, gs = _quantize_plain(s["x"].float()[None], fmt, "row")
    a = (c * sc[..., None]).view(case["m"], case["k"])
    rows = routes.shape[0]
    pos = torch.arange(rows, device=routes.device)
    live = pos < off[-1]
    e = torch.clamp(torch.searchsorted(off[1:], pos, right=True), max=case["experts"] - 1)
    groups = used.shape[0]
    slot = torch.where(live, torch.searchsorted(used, e) * most + (pos - off[e]), groups * most)
    token = torch.clamp(routes, min=0).long() // case["top_k"]
    pad = torch.zeros(groups * most + 1, case["k"], device=a.device)
    pad[slot] = a[token]
    y = torch.bmm(pad[:-1].view(groups, most, case["k"]), w.transpose(1, 2)).view(-1, case["n"])
    y = torch.cat((y, torch.zeros(1, case["n"], device=y.device)))[slot]
    if gs is not None:
        y = y * (gs[0][token] * gw[e])[:, None]
    return torch.where(live[:, None], y, 0.0).to(torch.bfloat16)


# ---------------------------------------------------- the framework's calls


def _run_own(s):
    import w4a16_moe_gb300 as b4

    case = s["case"]
    if "plan" not in s:  # what a program keeps: the call's shape, its output buffers and workspace
        fmt = b4.FORMATS[case["fmt"]]
        if case["op"] == "quantize":
            mode = {"row": b4.GS_ROW, "tensor": b4.GS_TENSOR, "none": b4.GS_NONE}[case["gs"]]
            cfg = b4.Fp4Config(m=case["m"], k=case["k"], num_groups=case["groups"], format=fmt, gs_mode=mode,
                               x_dtype=s["x"].dtype)
            codes, scales, gs = b4.fp4_empty(cfg, "cuda")
            s["plan"] = (cfg, codes, scales, gs, torch.empty_like(s["x"]))
        else:
            grouped = case["op"] == "grouped"
            cfg = b4.Fp4Config(m=s["routes"].shape[0] if grouped else case["m"], n=case["n"], k=case["k"],
                               num_groups=case["experts"] if grouped else 1, format=fmt, x_dtype=s["x"].dtype,
                               gs_mode=b4.GS_ROW if case["fmt"] == NV else b4.GS_NONE,
                               activation=b4.ACTIVATIONS.get(case.get("act")), row_div=case.get("top_k", 1))
            ws = torch.empty(b4.fp4_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
            s["plan"] = (cfg, torch.empty(cfg.m, cfg.n, dtype=torch.bfloat16, device="cuda"), ws)
    if case["op"] == "quantize":
        cfg, codes, scales, gs, values = s["plan"]
        b4.fp4_quantize(cfg, s["x"], codes, scales, gs, values=values)
        if gs is None:
            return {"values": values}
        return {"values": values, "gs": gs, "scales": scales.view(torch.float8_e4m3fn)}
    cfg, out, ws = s["plan"]
    codes, tiles, gw = s["w"]
    if case["op"] == "linear":
        b4.fp4_linear(cfg, s["x"], codes, tiles, gw, out, ws)
    else:
        b4.fp4_linear(cfg, s["x"], codes, tiles, gw, out, ws, rows=s["routes"], offsets=s["offsets"])
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------- accounting


def work(case):
    g, k = GROUP[case["fmt"]], case["k"]
    fp4 = lambda rows: rows * (k / 2 + k / g)  # noqa: E731  codes and scales
    if case["op"] == "quantize":
        rows = case["groups"] * case["m"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * rows * k * size + fp4(rows), "flops": 4 * rows * k}  # x in; values, codes, scales out
    n = case["n"]
    if case["op"] == "linear":
        cols = 2 * k if case["act"] in ("silu", "swiglu_oai") else k
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["m"] * cols * size + fp4(n) + 2 * case["m"] * n, "flops": 2 * case["m"] * n * k}
    rows = case["m"] * case["top_k"]
    every = case["experts"] + case["drop"]
    used = case["experts"] * (1 - (1 - case["top_k"] / every) ** case["m"])  # experts that get a row, about
    return {"bytes": 2 * case["m"] * k + used * fp4(n) + 2 * rows * n,
            "flops": 2 * rows * case["experts"] / every * n * k}


# ------------------------------------------------------- 64-bit definition


def _grid64(v, grid):
    """Round v >= 0 to the nearest of an ascending grid whose odd entries have odd mantissas; saturates."""
    i = torch.searchsorted(grid, v).clamp(1, len(grid) - 1)
    lo, hi = grid[i - 1], grid[i]
    up = (v - lo > hi - v) | ((v - lo == hi - v) & (i % 2 == 0))
    return torch.where(up, hi, lo)


def _quant64(h, fmt, gs_mode):
    """Dequantised h [G, m, K] without gs, the E4M3 scales [G, m, K/g] and gs [G, m] or [G], from the definition."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=h.device)
    parts = h.reshape(h.shape[0], h.shape[1], h.shape[2] // GROUP[fmt], GROUP[fmt])
    amax = parts.abs().max(-1).values
    if fmt == MX:
        e = torch.ceil(torch.log2(torch.clamp(amax, min=1e-300) / 6.0))
        e = torch.where(torch.exp2(e - 1) * 6.0 >= amax, e - 1, e)  # the logarithm may be a rounding too high
        e = torch.where(torch.exp2(e) * 6.0 < amax, e + 1, e).clamp(-127, 127)
        s, gs = torch.exp2(e), None
        unit = s
    else:
        if gs_mode == "tensor":
            whole = amax.flatten(1).max(1).values[:, None].expand(amax.shape[:2])
            # an fp32 output of the operator: the scales and codes are chosen against the value it holds
            gs = torch.where(whole > 0, whole / 2688.0, 1.0).float().double()
        else:
            top = amax.max(-1).values
            j = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 2688.0))
            j = torch.where(torch.exp2(j - 1) * 2688.0 >= top, j - 1, j)
            j = torch.where(torch.exp2(j) * 2688.0 < top, j + 1, j).clamp(min=-126)
            gs = torch.where(top > 0, torch.exp2(j), 1.0)
        e4m3 = torch.arange(0, 127, device=h.device, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        s = _grid64(amax / (6.0 * gs[..., None]), e4m3)
        unit = s * gs[..., None]
    q = _grid64(torch.where(unit[..., None] > 0, parts.abs() / torch.where(unit > 0, unit, 1.0)[..., None], 0.0), grid)
    return (torch.sign(parts) * q * s[..., None]).reshape(h.shape), s, gs


def _act64(x, act):
    if act == "none":
        return x
    if act == "relu2":
        return torch.where(x > 0, x * x, 0.0)
    g, u = x.chunk(2, -1)
    alpha, beta, limit = OAI if act == "swiglu_oai" else (1.0, 0.0, math.inf)
    g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    return g * torch.sigmoid(alpha * g) * (u + beta)


def _weights64(codes, tiles, fmt, n, k):
    """One matrix [n, k] from its bits: sign, two exponent bits and one of mantissa; E4M3 likewise; E8M0 2^(s - 127)."""
    c = torch.empty(n, k, dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = codes[:, : k // 2] % 16, codes[:, : k // 2] // 16
    e, f = c // 2 % 4, c % 2
    v = torch.where(e > 0, (1 + f / 2.0).double() * torch.exp2((e - 1).double()), f.double() / 2) * (1 - 2 * (c // 8)).double()
    row = torch.arange(n, device=c.device)[:, None]
    col = torch.arange(k, device=c.device)[None, :] // GROUP[fmt]
    b = tiles[row // 128, col // 4, row % 32, row % 128 // 32, col % 4].long()
    if fmt == MX:
        return v * torch.exp2(b.double() - 127)
    e, f = b // 8, b % 8
    return v * torch.where(e > 0, (1 + f / 8.0).double() * torch.exp2((e - 7).double()), f.double() / 8 * 2.0**-6)


def exact(case, seed):
    s = prepare(case, seed)
    fmt = case["fmt"]
    if case["op"] == "quantize":
        v, sc, gs = _quant64(s["x"].double(), fmt, case["gs"])
        if gs is None:
            return {"values": v}
        per = gs if case["gs"] == "row" else gs[:, 0]
        return {"values": v * gs[..., None], "gs": per, "scales": _tile(sc)}
    codes, tiles, gw = s["w"]
    n, k = case["n"], case["k"]
    if case["op"] == "linear":
        w = _weights64(codes[0], tiles[0], fmt, n, k)
        a, _, gs = _quant64(_act64(s["x"].double(), case["act"])[None], fmt, "row")
        y = a[0] @ w.T
        return y if gs is None else y * gs[0][:, None] * gw.double()
    a, _, gs = _quant64(s["x"].double()[None], fmt, "row")
    off = s["offsets"].tolist()
    token = s["routes"].clamp(min=0).long() // case["top_k"]
    y = torch.zeros(s["routes"].shape[0], n, dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            w = _weights64(codes[e], tiles[e], fmt, n, k)
            t = token[lo:hi]
            part = a[0][t] @ w.T
            y[lo:hi] = part if gs is None else part * gs[0][t][:, None] * gw[e].double()
    return y
