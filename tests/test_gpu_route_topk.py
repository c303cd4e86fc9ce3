"""GPU tests of the routing operator (b4_route_topk) against the float64 oracle.

Ids are equal, always.  Weights are fp32: an exponential of an argument off by 2^-24 |z - top| (here at most 2^5.5)
with one ulp of its own, sums of at most 1024 terms (32 in a lane, five shuffles: 37 roundings of 2^-24), a quotient
and the product with the scale: below 2^-18 + 2^-18.7 + 2^-22, so 2^-17 of the value.
"""

import numpy as np
import pytest
import torch

from gpu_util import dev
from oracle import router as R

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
TOL = 2.0**-17


@pytest.fixture(scope="module")
def b4():
    import w4a16_moe_gb300 as mod

    return mod


def _z(m, e, seed, dtype, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(m, e, generator=g) * spread).to(dtype)


def _run(b4, z, bias, top_k, score, renorm=True, scale=1.0, groups=1, top_groups=None, group_top=1, num_tokens=None):
    m, e = z.shape
    cfg = b4.RouterConfig(m, e, top_k, score=b4.SCORES[score], renormalize=renorm, scale=scale, num_groups=groups,
                          top_groups=top_groups, group_top=group_top, dtype=z.dtype, stride=z.stride(0) if m > 1 else 0)
    ids = torch.full((m + 1, top_k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((m + 1, top_k), 77.0, device="cuda")
    b4.route_topk(cfg, z, ids[:m], w[:m], bias=bias, num_tokens=num_tokens)
    torch.cuda.synchronize()
    assert torch.all(ids[m] == 77) and torch.all(w[m] == 77.0)
    return ids[:m].cpu().numpy(), w[:m].double().cpu().numpy()


def _compare(b4, z, bias, top_k, score, **kw):
    ids, w = _run(b4, z.cuda(), None if bias is None else bias.cuda(), top_k, score, **kw)
    want_ids, want_w = R.route(z.double().numpy(), None if bias is None else bias.double().numpy(), top_k, score, **kw)
    assert np.array_equal(ids, want_ids), np.argwhere(ids != want_ids)[:5]
    assert np.all(np.abs(w - want_w) <= TOL * np.abs(want_w))


SHAPES = [  # m, experts, top_k, groups, top_groups
    (1, 1, 1, 1, None), (3, 8, 2, 1, None), (5, 28, 4, 1, None), (33, 60, 6, 4, 2), (7, 64, 8, 8, 4), (130, 128, 8, 1, None),
    (64, 256, 8, 8, 4), (5, 160, 6, 5, 3), (9, 320, 8, 10, 4), (4, 384, 8, 3, 1), (2, 512, 32, 16, 7), (3, 1024, 32, 32, 3),
    (6, 33, 32, 1, None), (3, 1000, 9, 1, None), (5, 96, 3, 32, 5), (2, 31, 5, 31, 9),
]


@pytest.mark.parametrize("m,e,k,groups,top_groups", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_shapes(b4, m, e, k, groups, top_groups, score, bias, dtype):
    z = _z(m, e, e + k, dtype)
    b = torch.randn(e, generator=torch.Generator().manual_seed(9)) * 0.1 if bias else None
    for group_top in (1, 2) if groups > 1 else (1,):
        for renorm, scale in ((True, 2.5), (False, 1.0)):
            _compare(b4, z, b, k, score, renorm=renorm, scale=scale, groups=groups, top_groups=top_groups, group_top=group_top)


def test_many_tokens(b4):
    """Enough rows that scores closer than fp32 resolves occur, in both choices."""
    z = _z(3000, 256, 5, BF)
    b = torch.randn(256, generator=torch.Generator().manual_seed(6)) * 0.1
    _compare(b4, z, b, 8, "sigmoid", groups=8, top_groups=4, group_top=2, scale=2.5)
    _compare(b4, z, b, 8, "softmax")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k,groups,top_groups", [(64, 8, 1, None), (256, 32, 8, 4), (320, 8, 10, 4), (1024, 32, 1, None), (20, 3, 1, None)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_scores_that_fp32_does_not_separate(b4, score, e, k, groups, top_groups, group_top):
    """Biases that bring every c to one value but for their own rounding: the order is that of the 64-bit sums."""
    z = _z(1, e, 21, F32)
    b = torch.from_numpy((0.75 - R.scores(z.double().numpy()[0], score)).astype(np.float32))
    _compare(b4, z.repeat(5, 1), b, k, score, groups=groups, top_groups=top_groups, group_top=group_top)


def test_ties_go_to_the_lowest_index(b4):
    for dtype in (BF, F32):
        z = torch.zeros(4, 256, dtype=dtype)
        z[1, 100:] = 1.0
        z[2, ::3] = -0.0
        z[3] = torch.randint(0, 3, (256,), generator=torch.Generator().manual_seed(3)).to(dtype)
        for bias in (None, torch.zeros(256), torch.randint(0, 2, (256,), generator=torch.Generator().manual_seed(4)) * 0.5):
            for score in ("softmax", "sigmoid"):
                _compare(b4, z, bias, 8, score)
                _compare(b4, z, bias, 8, score, groups=8, top_groups=4, group_top=2)


def test_excluded_experts_and_infinities(b4):
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(BF).min
    z = _z(12, 64, 31, BF)
    z[0] = -inf
    z[1] = nan
    z[2, 3:] = -inf
    z[3, ::2] = nan
    z[4] = low
    z[5, 5:] = low
    z[6, 7] = inf
    z[7, [7, 30, 9]] = inf
    z[8] = inf
    z[9] = -200.0 - torch.arange(64)
    z[10, 16:32] = -inf
    z[11, 1:16] = nan
    bias = torch.randn(64, generator=torch.Generator().manual_seed(8)) * 0.1
    odd = bias.clone()
    odd[[1, 8, 40]] = torch.tensor([-inf, nan, inf])
    for b in (None, bias, odd):
        for score in ("softmax", "sigmoid"):
            for kw in (dict(), dict(groups=4, top_groups=2, group_top=2), dict(groups=4, top_groups=2, group_top=1)):
                rows = [i for i in range(12) if not (score == "sigmoid" and i in (4, 5, 9))]
                _compare(b4, z[rows], b, 6, score, **kw)
    # sigmoids that underflow keep their ratios
    ids, w = _run(b4, z[9:10].cuda(), None, 3, "sigmoid")
    want = np.exp(-np.arange(3)) / np.exp(-np.arange(3)).sum()
    assert ids.tolist() == [[0, 1, 2]] and np.all(np.abs(w[0] - want) <= TOL * want)


def test_rows_apart_and_unaligned(b4):
    base = _z(9, 300, 41, BF).cuda()
    for off in (0, 1, 8):
        view = base[:, off:off + 256]
        ids, w = _run(b4, view, None, 8, "softmax")
        want = R.route(view.double().cpu().numpy(), None, 8, "softmax")
        assert np.array_equal(ids, want[0]) and np.all(np.abs(w - want[1]) <= TOL * want[1])


def test_padded_batch(b4):
    z = _z(10, 64, 51, BF)
    z[7:] = float("nan")
    want = R.route(z.double().numpy()[:7], None, 4, "softmax")
    for n in (7, 0, 10, 100):
        ids, w = _run(b4, z.cuda(), None, 4, "softmax", num_tokens=dev(np.array([n], np.int32)))
        live = min(n, 7)
        assert np.array_equal(ids[:live], want[0][:live]) and np.all(ids[live:] == -1) and np.all(w[live:] == 0)


def test_no_tokens(b4):
    cfg = b4.RouterConfig(0, 8, 2)
    e = torch.empty(0, 2, device="cuda")
    b4.route_topk(cfg, torch.empty(0, 8, dtype=BF, device="cuda"), e.int(), e)


def test_graph_and_side_stream(b4):
    z, b = _z(70, 128, 61, F32).cuda(), torch.randn(128).cuda() * 0.1
    cfg = b4.RouterConfig(70, 128, 8, score=b4.SIGMOID, dtype=F32)
    ids, w = torch.empty(70, 8, dtype=torch.int32, device="cuda"), torch.empty(70, 8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b4.route_topk(cfg, z, ids, w, bias=b, stream=side)
    side.synchronize()
    first = ids.clone(), w.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b4.route_topk(cfg, z, ids, w, bias=b)
    z.copy_(_z(70, 128, 62, F32))
    graph.replay()
    torch.cuda.synchronize()
    want = R.route(z.double().cpu().numpy(), b.double().cpu().numpy(), 8, "sigmoid")
    assert np.array_equal(ids.cpu().numpy(), want[0]) and not torch.equal(ids, first[0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k,groups,top_groups", [(256, 8, 8, 4), (320, 6, 10, 3), (32, 4, 32, 7), (96, 5, 16, 2), (1024, 8, 4, 1)])
def test_groups_that_fp32_does_not_separate(b4, score, e, k, groups, top_groups):
    """Every group holds the same logits in another order, each a few ulps off: the groups' order is that of the 64-bit values;
    some rows have groups of excluded experts, of one that counts, or equal ones."""
    g = torch.Generator().manual_seed(31)
    per, m = e // groups, 40
    z = torch.randn(m, 1, per, generator=g).repeat(1, groups, 1)
    z = torch.gather(z, 2, torch.rand(m, groups, per, generator=g).argsort(-1))
    z = (z * (1 + torch.randint(-3, 4, z.shape, generator=g) * 2.0**-23)).to(F32)
    z[5, : groups // 2] = float("-inf")
    z[6, :, 1:] = float("nan")
    z[7] = z[7, :1]
    z[8, 1, 0] = float("inf")
    z = z.reshape(m, e)
    some = torch.full((e,), 0.25)
    some[e // 3] = float("-inf")
    first = some.clone()
    first[e // 2] = float("inf")
    for bias in (None, some, first):
        for group_top in (1, 2):
            _compare(b4, z, bias, k, score, groups=groups, top_groups=top_groups, group_top=group_top)
