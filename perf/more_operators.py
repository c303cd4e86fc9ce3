"""Cases of the routing and FP8 operators: choice of experts, 8-bit block quantisation, the product of
two such operands (dense and grouped by expert), and the mixture-of-experts layer of them.

``own`` False computes the plain forms (elementary torch operations, rounded once at the end); ``own``
True makes a user's calls of ``w4a16_moe_gb300``.

Formulas.

Routing.  For the logits z of a token over E experts, s = softmax(z) or sigmoid(z), c = s + bias (without a
bias the order is that of z).  With groups, the E experts are cut into equal neighbouring groups, a group
counts with its largest c or with the sum of its two largest, and only the best groups' experts stay.  The
top_k experts are those of the largest c, in descending order; ties go to the lowest index.  Their weights
are s, divided by their sum where renormalised, times a constant.

Quantisation.  A row of h = x, silu(g) u, max(x, 0)^2 or the clamped swiglu is cut along K into blocks of 128,
and each block has one fp32 scale (weights: one for 128 rows x 128 columns):

    s = amax / 448, or the least power of two with amax <= 448 s (1 where amax is 0),  c = e4m3(h / s)

the quotients rounded to fp32, then to the nearest 8-bit value, ties to even.

Product.  out[t][n] = sum over blocks b of sa[t][b] sw[n / 128][b] sum over k in b of a[t][k] w[n][k]; grouped,
the rows offsets[e] .. offsets[e + 1] meet the weights of expert e, and rows past offsets[E] are zero.

Layer.  Routing; h = act(x W13^T) of the chosen experts, quantised; out[t] = sum_j weight_j (h W2^T) of route j.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
OAI = (1.702, 1.0, 7.0)
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases


def listed():
    return [
        # the router of a 128-expert layer in a decode step: latency
        dict(name="route_token", op="route", m=1, experts=128, top_k=8, dtype="bf16", score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0),
        # a ragged decode batch, sigmoid scores with a balance bias, eight groups of which four stay
        dict(name="route_batch", op="route", m=93, experts=256, top_k=8, dtype="f32", score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5),
        # the same router over the prompts of a prefill batch
        dict(name="route_prefill", op="route", m=16384, experts=256, top_k=8, dtype="bf16", score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5),
        # a prefill's activations, a scale per 128 of each row
        dict(name="quantize_prefill", op="quantize", dtype="bf16", groups=1, m=8192, k=4096, block_rows=1, pow2=False),
        # fp32 master weights of 16 experts (E64 H2048 I1408 layer), a scale per 128 x 128
        dict(name="quantize_weights", op="quantize", dtype="f32", groups=16, m=2816, k=2048, block_rows=128, pow2=False),
        # a dense projection, one token: weight-stream latency
        dict(name="linear_token", op="linear", dtype="bf16", m=1, n=4096, k=4096, act="none", pow2=False),
        # prefill through a dense projection
        dict(name="linear_prefill", op="linear", dtype="bf16", m=4096, n=4096, k=4096, act="none", pow2=False),
        # FC1 of a 128-expert layer, one token: eight experts of one row
        dict(name="grouped_token", op="grouped", m=1, n=1536, k=4096, experts=128, top_k=8, hot=0, drop=0),
        # 32 global experts of which 28 are local, sizes that fill no tile, some routes invalid
        dict(name="grouped_ragged", op="grouped", m=509, n=2880, k=2880, experts=28, top_k=4, hot=0, drop=4),
        # prefill of a layer with eight popular experts: groups of hundreds of rows
        dict(name="grouped_prefill", op="grouped", m=2048, n=2816, k=2048, experts=64, top_k=6, hot=8, drop=0),
        # the whole layer from router logits on, a decode batch
        dict(name="moe_batch", op="moe", m=64, hidden=2048, inter=1408, experts=64, top_k=6, act="silu", score="softmax",
             bias=False, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0, hot=8),
        # and a prefill
        dict(name="moe_prefill", op="moe", m=2048, hidden=2048, inter=1408, experts=64, top_k=6, act="silu",
             score="sigmoid", bias=True, groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5, hot=0),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def _draw_route(rng, experts, top_k):
    groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts % g == 0])
    top_groups = rng.randint(1, groups)
    if top_groups * (experts // groups) < top_k:
        top_groups = groups
    return dict(score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                group_top=rng.choice((1, 2)), renorm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)))


def draw(rng):
    op = rng.choice(("route", "route", "quantize", "linear", "linear", "grouped", "grouped", "moe"))
    if op == "route":
        experts = _log(rng, 4, 512, rng.choice((1, 4, 8)))
        m, top_k = _log(rng, 1, 16384), rng.randint(1, min(16, experts))
        m = min(m, max(1, 16384 * 256 // experts))
        return dict(op=op, m=m, experts=experts, top_k=top_k, dtype=rng.choice(("bf16", "f16", "f32")),
                    **_draw_route(rng, experts, top_k))
    if op == "quantize":
        groups = rng.choice((1, 1, _log(rng, 1, 32)))
        k = _log(rng, 64, 8192, 16)
        m = _log(rng, 1, min(8192, max(2, 33_000_000 // (groups * k))))
        return dict(op=op, dtype=rng.choice(("bf16", "bf16", "f16", "f32")), groups=groups, m=m, k=k,
                    block_rows=rng.choice((1, 1, 128)), pow2=rng.random() < 0.3)
    if op == "linear":
        n, k = _log(rng, 48, 4096), _log(rng, 64, 4096, 16)
        return dict(op=op, dtype=rng.choice(("bf16", "bf16", "f16", "f32")), m=_log(rng, 1, 4096), n=n, k=k,
                    act=rng.choice(("none", "none", "silu", "relu2", "swiglu_oai")), pow2=rng.random() < 0.3)
    experts = _log(rng, 2, 128)
    if op == "grouped":
        n, k = _log(rng, 64, 2880), _log(rng, 64, 2880, 16)
        experts = max(1, min(experts, 360_000_000 // (n * k)))
        top_k = rng.randint(1, min(8, experts))
        m = max(1, min(_log(rng, 1, 2048), 12000 // top_k, int(7e10 / (top_k * n * k))))
        return dict(op=op, m=m, n=n, k=k, experts=experts, top_k=top_k, hot=rng.choice((0, 0, experts // 8)),
                    drop=rng.choice((0, 0, 3)))
    hidden, inter = _log(rng, 64, 2048, 64), _log(rng, 32, 1408, 32)
    top_k = rng.randint(1, min(6, experts))
    experts = max(top_k, min(experts, 500_000_000 // (3 * hidden * inter)))
    m = max(1, min(_log(rng, 1, 2048), int(1e11 / (3 * top_k * hidden * inter))))
    return dict(op=op, m=m, hidden=hidden, inter=inter, experts=experts, top_k=top_k,
                act=rng.choice(("silu", "relu2", "swiglu_oai")), hot=rng.choice((0, 0, experts // 8)),
                **_draw_route(rng, experts, top_k))


# ----------------------------------------------------------------- inputs


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1_000_003 + salt) % (1 << 62))
    return g


def _cdiv(a, b):
    return (a + b - 1) // b


def _x(case, rows, cols, seed):
    """Activations: N(0, 1) with channels of different size; weights to quantise: N(0, 0.02)."""
    g = _gen(seed, 1)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    if case.get("block_rows") == 128:
        x *= 0.02
    else:
        x *= torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    return x.to(DTYPES[case.get("dtype", "bf16")])


def _weights(experts, n, k, seed, salt=2):
    """Codes [E, N, K] as a checkpoint holds them (values of about N(0, 0.02)), scales [E, ceil(N/128), ceil(K/128)]."""
    gen = _gen(seed, salt)
    codes = torch.empty(experts, n, k, dtype=E4M3, device="cuda")
    step = max(1, 200_000_000 // (n * k))
    for e in range(0, experts, step):
        part = codes[e : e + step]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(100.0).clamp_(-448.0, 448.0))
    scales = torch.rand(experts, _cdiv(n, 128), _cdiv(k, 128), generator=gen, device="cuda") + 0.5
    return codes, scales * (0.02 / 100.0)


def _logits(case, seed):
    z = torch.randn(case["m"], case["experts"], generator=_gen(seed, 4), device="cuda") * 1.5
    if case.get("hot"):
        z[:, : case["hot"]] += 2.0
    bias = None
    if case["bias"]:
        bias = 0.1 * torch.randn(case["experts"], generator=_gen(seed, 5), device="cuda")
    return z.to(DTYPES[case.get("dtype", "bf16")]), bias


def _pack(ids, experts):
    """Offsets [E + 1] and routes sorted by expert (stable), -1 past the valid ones; ids from `experts` on are dropped."""
    order = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=experts)[:experts]
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(counts, 0)
    valid = torch.arange(ids.shape[0], device=ids.device) < offsets[-1]
    return offsets, torch.where(valid, order, -1).to(torch.int32), counts


def prepare(case, seed):
    s = {"case": case}
    op = case["op"]
    if op == "quantize":
        s["x"] = _x(case, case["groups"] * case["m"], case["k"], seed).view(case["groups"], case["m"], case["k"])
    elif op == "linear":
        cols = 2 * case["k"] if case["act"] in ("silu", "swiglu_oai") else case["k"]
        s["x"] = _x(case, case["m"], cols, seed)
        s["w"] = _weights(1, case["n"], case["k"], seed)
    elif op == "grouped":
        s["x"] = _x(case, case["m"], case["k"], seed)
        s["w"] = _weights(case["experts"], case["n"], case["k"], seed)
        logits = torch.randn(case["m"], case["experts"] + case["drop"], generator=_gen(seed, 3), device="cuda")
        if case["hot"]:
            logits[:, : case["hot"]] += 2.0
        ids = torch.topk(logits, case["top_k"], dim=-1).indices.reshape(-1)
        s["offsets"], s["routes"], counts = _pack(ids, case["experts"])
        s["most"], s["used"] = max(1, int(counts.max())), torch.nonzero(counts).flatten()
    else:
        s["logits"], s["bias"] = _logits(case, seed)
        if op == "moe":
            h, i = case["hidden"], case["inter"]
            s["x"] = _x(case, case["m"], h, seed)
            s["w13"] = _weights(case["experts"], i if case["act"] == "relu2" else 2 * i, h, seed)
            s["w2"] = _weights(case["experts"], h, i, seed, 6)
            if not own:  # the plain form pads the groups: to the longest, known here so that a pass need not wait
                ids, _ = _route_plain(s["logits"], s["bias"], case)
                counts = torch.bincount(ids.reshape(-1), minlength=case["experts"])
                s["most"], s["used"] = int(counts.max()), torch.nonzero(counts).flatten()
    return s


# ------------------------------------------------------------ plain forms


def _route_plain(z, bias, case):
    """ids [m, k] int64 and weights [m, k] f32; scores in 64 bits, since neighbours in the order may differ by less
    than 32 bits hold."""
    z = z.double()
    if case["score"] == "softmax":
        s = torch.exp(z - z.amax(-1, keepdim=True))
        s = s / s.sum(-1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-z))
    c = s if bias is None else s + bias.double()
    key = z if bias is None else c
    if case["groups"] > 1:
        per = c.view(*c.shape[:-1], case["groups"], -1)
        best = torch.sort(per, dim=-1, descending=True).values[..., : case["group_top"]].sum(-1)
        order = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, : case["top_groups"]]
        keep = torch.zeros_like(best, dtype=torch.bool)
        keep.scatter_(1, order, torch.ones_like(order, dtype=torch.bool))
        keep = keep[..., None].expand(per.shape).reshape(c.shape)
        key = torch.where(keep, key, -torch.inf)
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, : case["top_k"]]
    w = s.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids, (w * case["scale"]).float()


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


def _quantize_plain(h, block_rows, pow2):
    """h [G, m, K] f32 -> (E4M3 values, scales [G, m or ceil(m/128), ceil(K/128)], scales spread over the elements)."""
    g, m, k = h.shape
    pad = torch.zeros(g, _cdiv(m, block_rows) * block_rows, _cdiv(k, 128) * 128, device=h.device)
    pad[:, :m, :k] = h.abs()
    amax = pad.view(g, -1, block_rows, _cdiv(k, 128), 128).amax((2, 4))
    if pow2:
        f, ex = torch.frexp(amax)  # 448 = 0.875 2^9
        s = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), ex - 9 + (f > 0.875)), torch.ones_like(amax))
    else:
        s = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    spread = s.repeat_interleave(block_rows, 1)[:, :m].repeat_interleave(128, 2)[:, :, :k]
    return torch.clamp(h / spread, -448.0, 448.0).to(E4M3).float(), s, spread


def _dequant_plain(codes, scales):
    n, k = codes.shape[1:]
    w = codes.float()
    for b in range(scales.shape[1]):  # (a block of rows at a time: no second copy of the weights)
        rows = w[:, 128 * b : min(128 * b + 128, n)]
        rows *= scales[:, b, None, :].repeat_interleave(128, 2)[:, :, :k]
    return w


def _operand_plain(h, pow2=False):
    c, _, spread = _quantize_plain(h[None], 1, pow2)
    return (c * spread)[0]


def _grouped_plain(a, w, off, most, used, experts):
    """Rows of a grouped by expert (off) times w, the weights of the `used` experts -> [rows, n] f32, others zero."""
    rows = a.shape[0]
    pos = torch.arange(rows, device=a.device)
    live = pos < off[-1]
    e = torch.clamp(torch.searchsorted(off[1:], pos, right=True), max=experts - 1)
    groups = used.shape[0]
    slot = torch.where(live, torch.searchsorted(used, e) * most + (pos - off[e]), groups * most)
    pad = torch.zeros(groups * most + 1, a.shape[1], device=a.device)
    pad[slot] = a
    y = torch.bmm(pad[:-1].view(groups, most, -1), w.transpose(1, 2)).view(groups * most, -1)
    y = torch.cat((y, torch.zeros(1, y.shape[1], device=y.device)))[slot]
    return torch.where(live[:, None], y, 0.0)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "route":
        ids, w = _route_plain(s["logits"], s["bias"], case)
        return {"ids": ids.to(torch.int32), "weights": w}
    if op == "quantize":
        c, sc, spread = _quantize_plain(s["x"].float(), case["block_rows"], case["pow2"])
        return {"values": (c * spread).to(s["x"].dtype), "scales": sc}
    if op == "linear":
        a = _operand_plain(_act_plain(s["x"], case["act"]), case["pow2"])
        return (a @ _dequant_plain(*s["w"])[0].T).to(torch.bfloat16)
    if op == "grouped":
        codes, scales = s["w"]
        used = s["used"]
        token = torch.clamp(s["routes"], min=0).long() // case["top_k"]
        a = _operand_plain(s["x"].float())[token]
        w = _dequant_plain(codes[used], scales[used])
        return _grouped_plain(a, w, s["offsets"].long(), s["most"], used, case["experts"]).to(torch.bfloat16)
    ids, weights = _route_plain(s["logits"], s["bias"], case)
    off, routes, _ = _pack(ids.reshape(-1), case["experts"])
    off, routes, used = off.long(), routes.long(), s["used"]
    a = _operand_plain(s["x"].float())[routes // case["top_k"]]
    y = _grouped_plain(a, _dequant_plain(s["w13"][0][used], s["w13"][1][used]), off, s["most"], used, case["experts"])
    h = _operand_plain(_act_plain(y, case["act"]))
    y = _grouped_plain(h, _dequant_plain(s["w2"][0][used], s["w2"][1][used]), off, s["most"], used, case["experts"])
    back = torch.empty_like(y)
    back[routes] = y
    return (back.view(*ids.shape, -1) * weights[..., None]).sum(1).to(torch.bfloat16)


# ---------------------------------------------------- the framework's calls


def _router(b4, case, m, dtype):
    return b4.RouterConfig(m=m, num_experts=case["experts"], top_k=case["top_k"], score=b4.SCORES[case["score"]],
                           renormalize=case["renorm"], scale=case["scale"], num_groups=case["groups"],
                           top_groups=case["top_groups"], group_top=case["group_top"], dtype=dtype)


def _run_own(s):
    import w4a16_moe_gb300 as b4

    case = s["case"]
    op = case["op"]
    if "plan" not in s:  # what a program keeps: the call's shape, its output buffers and workspace
        if op in ("route", "moe"):
            m, k = case["m"], case["top_k"]
            plan = [_router(b4, case, m, s["logits"].dtype), torch.empty(m, k, dtype=torch.int32, device="cuda"),
                    torch.empty(m, k, dtype=torch.float32, device="cuda")]
            if op == "moe":
                act = b4.ACTIVATIONS[case["act"]]
                cfg = b4.MoEConfig(m, k, case["experts"], case["experts"], case["hidden"], case["inter"])
                ws = torch.empty(b4.fused_moe_fp8_workspace_bytes(cfg, act), dtype=torch.uint8, device="cuda")
                plan += [cfg, act, torch.empty_like(s["x"]), ws]
            s["plan"] = tuple(plan)
        else:
            mode = b4.FP8_SCALE_POW2 if case.get("pow2") else b4.FP8_SCALE_F32
            if op == "quantize":
                cfg = b4.Fp8Config(m=case["m"], k=case["k"], num_groups=case["groups"], x_dtype=s["x"].dtype,
                                   scale_mode=mode, block_rows=case["block_rows"])
                codes, scales = b4.fp8_empty(cfg, "cuda")
                s["plan"] = (cfg, codes, scales, torch.empty_like(s["x"]))
            else:
                grouped = op == "grouped"
                cfg = b4.Fp8Config(m=s["routes"].shape[0] if grouped else case["m"], n=case["n"], k=case["k"],
                                   num_groups=case["experts"] if grouped else 1, x_dtype=s["x"].dtype, scale_mode=mode,
                                   activation=b4.ACTIVATIONS.get(case.get("act")), row_div=case.get("top_k", 1))
                ws = torch.empty(b4.fp8_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
                s["plan"] = (cfg, torch.empty(cfg.m, cfg.n, dtype=torch.bfloat16, device="cuda"), ws)
    if op == "route":
        cfg, ids, weights = s["plan"]
        b4.route_topk(cfg, s["logits"], ids, weights, bias=s["bias"])
        return {"ids": ids, "weights": weights}
    if op == "quantize":
        cfg, codes, scales, values = s["plan"]
        b4.fp8_quantize(cfg, s["x"], codes, scales, values=values)
        return {"values": values, "scales": scales}
    if op == "moe":
        router, ids, weights, cfg, act, out, ws = s["plan"]
        b4.route_topk(router, s["logits"], ids, weights, bias=s["bias"])
        b4.fused_moe_fp8(cfg, s["x"], *s["w13"], *s["w2"], ids, weights, act, out, ws)
        return out
    cfg, out, ws = s["plan"]
    if op == "linear":
        b4.fp8_linear(cfg, s["x"], *s["w"], out, ws)
    else:
        b4.fp8_linear(cfg, s["x"], *s["w"], out, ws, rows=s["routes"], offsets=s["offsets"])
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------- accounting


def work(case):
    op = case["op"]
    fp8 = lambda rows, cols: rows * cols + 4 * _cdiv(rows, 128) * _cdiv(cols, 128)  # noqa: E731  weights and scales
    size = 4 if case.get("dtype") == "f32" else 2
    if op == "route":
        m, e = case["m"], case["experts"]
        return {"bytes": m * e * size + (4 * e if case["bias"] else 0) + 8 * m * case["top_k"], "flops": 8 * m * e}
    if op == "quantize":  # x in; values, codes and scales out
        rows, k = case["groups"] * case["m"], case["k"]
        blocks = case["groups"] * _cdiv(case["m"], case["block_rows"]) * _cdiv(k, 128)
        return {"bytes": 2 * rows * k * size + rows * k + 4 * blocks, "flops": 4 * rows * k}
    every = case["experts"] + case.get("drop", 0) if op != "linear" else 1
    used = 1 if op == "linear" else case["experts"] * (1 - (1 - case["top_k"] / every) ** case["m"])  # get a row, about
    if op == "moe":
        m, h, i = case["m"], case["hidden"], case["inter"]
        n1 = i if case["act"] == "relu2" else 2 * i
        return {"bytes": 4 * m * h + m * case["experts"] * size + used * (fp8(n1, h) + fp8(h, i)),
                "flops": 2 * m * case["top_k"] * h * (n1 + i)}
    n, k = case["n"], case["k"]
    if op == "linear":
        cols = 2 * k if case["act"] in ("silu", "swiglu_oai") else k
        return {"bytes": case["m"] * cols * size + fp8(n, k) + 2 * case["m"] * n, "flops": 2 * case["m"] * n * k}
    rows = case["m"] * case["top_k"]
    return {"bytes": 2 * case["m"] * k + used * fp8(n, k) + 2 * rows * n,
            "flops": 2 * rows * case["experts"] / every * n * k}


# ------------------------------------------------------- 64-bit definition


def _route64(z, bias, case):
    """By numpy on the host: scores, then whole orders by (value descending, index ascending)."""
    z = z.double().cpu().numpy()
    m, e = z.shape
    if case["score"] == "softmax":
        top = z.max(1, keepdims=True)
        s = np.exp(z - top) / np.exp(z - top).sum(1, keepdims=True)
    else:
        s = np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))
    b = None if bias is None else bias.double().cpu().numpy()
    c = s if b is None else s + b
    allowed = np.ones((m, e), bool)
    if case["groups"] > 1:
        per = np.sort(c.reshape(m, case["groups"], -1), -1)
        value = per[..., -1] + (per[..., -2] if case["group_top"] == 2 and per.shape[-1] > 1 else 0.0)
        rank = np.argsort(np.argsort(-value, 1, kind="stable"), 1, kind="stable")
        allowed = np.repeat(rank < case["top_groups"], e // case["groups"], 1)
    key = np.where(allowed, z if b is None else c, -np.inf)
    ids = np.argsort(-key, 1, kind="stable")[:, : case["top_k"]]
    w = np.take_along_axis(s, ids, 1)
    if case["renorm"]:
        w = w / w.sum(1, keepdims=True)
    return torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(w * case["scale"]).cuda()


def _blocks64(t, rows):
    """Block indices of every element of [.., m, k] for scales of `rows` rows x 128 columns."""
    return torch.arange(t.shape[-2], device=t.device)[:, None] // rows, torch.arange(t.shape[-1], device=t.device)[None] // 128


def _quant64(h, block_rows, pow2):
    """Dequantised h [G, m, K] and the scales, from the definition.  The scales are fp32 outputs of the operator: codes
    are chosen against the values they hold, by the quotient rounded to fp32."""
    g, m, k = h.shape
    br, bc = _blocks64(h, block_rows)
    nb = _cdiv(k, 128)
    at = (br * nb + bc).expand(g, m, k).reshape(g, -1)
    amax = torch.zeros(g, _cdiv(m, block_rows) * nb, dtype=torch.float64, device=h.device)
    amax.scatter_reduce_(1, at, h.abs().reshape(g, -1), "amax")
    if pow2:
        e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448.0))
        e = torch.where(torch.exp2(e - 1) * 448.0 >= amax, e - 1, e)  # the logarithm may be a rounding too high
        e = torch.where(torch.exp2(e) * 448.0 < amax, e + 1, e)
        s = torch.where(amax > 0, torch.exp2(e), 1.0)
    else:
        s = torch.where(amax > 0, (amax / 448.0).float().double(), 1.0)
    full = s.gather(1, at).view(g, m, k)
    q = (h / full).float().double()
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0**-6))) - 3)  # of E4M3: three bits, least exponent -6
    return torch.clamp(torch.round(q / step) * step, -448.0, 448.0) * full, s.view(g, -1, nb)


def _act64(x, act):
    if act == "none":
        return x
    if act == "relu2":
        return torch.where(x > 0, x * x, 0.0)
    g, u = x.chunk(2, -1)
    alpha, beta, limit = OAI if act == "swiglu_oai" else (1.0, 0.0, math.inf)
    g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    return g * torch.sigmoid(alpha * g) * (u + beta)


def _weights64(codes, scales):
    """One matrix [n, k] from its bits: sign, four exponent bits, three of mantissa."""
    b = codes.view(torch.uint8).long()
    e, f = b // 8 % 16, (b % 8).double() / 8.0
    v = torch.where(e > 0, (1.0 + f) * torch.exp2((e - 7).double()), f * 2.0**-6) * (1 - 2 * (b // 128)).double()
    return v * scales.double()[_blocks64(v, 128)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        ids, w = _route64(s["logits"], s["bias"], case)
        return {"ids": ids, "weights": w}
    if op == "quantize":
        v, sc = _quant64(s["x"].double(), case["block_rows"], case["pow2"])
        return {"values": v, "scales": sc}
    if op == "linear":
        a = _quant64(_act64(s["x"].double(), case["act"])[None], 1, case["pow2"])[0][0]
        return a @ _weights64(s["w"][0][0], s["w"][1][0]).T
    a = _quant64(s["x"].double()[None], 1, False)[0][0]
    if op == "grouped":
        off = s["offsets"].tolist()
        token = s["routes"].clamp(min=0).long() // case["top_k"]
        y = torch.zeros(s["routes"].shape[0], case["n"], dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                y[lo:hi] = a[token[lo:hi]] @ _weights64(s["w"][0][e], s["w"][1][e]).T
        return y
    ids, weights = _route64(s["logits"], s["bias"], case)
    out = torch.zeros(case["m"], case["hidden"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            y = a[t] @ _weights64(s["w13"][0][e], s["w13"][1][e]).T
            h = _quant64(_act64(y, case["act"])[None], 1, False)[0][0]
            out.index_add_(0, t, weights[t, j][:, None] * (h @ _weights64(s["w2"][0][e], s["w2"][1][e]).T))
    return out
