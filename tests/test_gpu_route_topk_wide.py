"""GPU tests of the routing operator (b4_route_topk) where a lane holds many experts and where fp32 errs the most.

Against the float64 oracle, ids equal; weights within the tolerance that test_gpu_route_topk.py derives.
"""

import pytest
import torch

from oracle import router as R
from test_gpu_route_topk import BF, F32, HF, _compare, _z, b4  # noqa: F401

pytestmark = pytest.mark.gpu

# more than 32 experts a lane: a group has the power of two of lanes that fits (17 groups: one), and up to 60 experts
WIDE = [  # experts, groups, top_k, top_groups
    (561, 17, 8, 4), (645, 5, 6, 2), (771, 3, 8, 1), (720, 9, 8, 3), (960, 6, 32, 2), (1020, 17, 9, 17), (1023, 31, 8, 9),
    (720, 5, 4, 5), (960, 20, 8, 7), (1000, 10, 8, 3), (1023, 3, 8, 2), (1023, 11, 32, 1),
]


@pytest.mark.parametrize("e,groups,k,top_groups", WIDE)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_more_experts_than_32_a_lane(b4, e, groups, k, top_groups, score, bias):  # noqa: F811
    b = torch.randn(e, generator=torch.Generator().manual_seed(9)) * 0.1 if bias else None
    for dtype in (BF, HF, F32):
        z = _z(5, e, e + k, dtype)
        z[1, : e // 2] = float("-inf")
        z[2, e // 3:] = float("nan")
        for group_top in (1, 2):
            for renorm, scale in ((True, 2.5), (False, 1.0)):
                _compare(b4, z, b, k, score, renorm=renorm, scale=scale, groups=groups, top_groups=top_groups, group_top=group_top)


@pytest.mark.parametrize("e,groups,k,top_groups", WIDE)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_close_scores_of_more_experts_than_32_a_lane(b4, e, groups, k, top_groups, score):  # noqa: F811
    """Every c one value but for rounding, and groups of the same logits in another order, a few ulps off."""
    z = _z(1, e, 21, F32)
    b = torch.from_numpy((0.75 - R.scores(z.double().numpy()[0], score)).astype("float32"))
    g = torch.Generator().manual_seed(31)
    per = e // groups
    same = torch.randn(6, 1, per, generator=g).repeat(1, groups, 1)
    same = torch.gather(same, 2, torch.rand(6, groups, per, generator=g).argsort(-1))
    same = (same * (1 + torch.randint(-3, 4, same.shape, generator=g) * 2.0**-23)).to(F32).reshape(6, e)
    for group_top in (1, 2):
        _compare(b4, z.repeat(2, 1), b, k, score, groups=groups, top_groups=top_groups, group_top=group_top)
        for bias in (None, torch.full((e,), 0.25)):
            _compare(b4, same, bias, k, score, groups=groups, top_groups=top_groups, group_top=group_top)


def test_the_last_expert_of_a_lane(b4):  # noqa: F811
    """Each expert in turn is the only one that counts, or the largest."""
    for e, groups in ((561, 17), (720, 9), (1020, 17)):
        z = torch.full((e, e), -3.0)
        z.fill_diagonal_(3.0)
        for kw in (dict(groups=groups, top_groups=1), dict(groups=groups, top_groups=2, group_top=2)):
            _compare(b4, z[::7], None, 1, "softmax", **kw)
            _compare(b4, z[::7], torch.zeros(e), 1, "sigmoid", **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups,k,top_groups", [(64, 8, 8, 4), (256, 8, 8, 4), (160, 5, 6, 2), (720, 9, 8, 3)])
@pytest.mark.parametrize("size", [100.0, 3000.0])
def test_groups_whose_largest_cancel(b4, score, e, groups, k, top_groups, size):  # noqa: F811
    """A group's two largest far from zero and of opposite sign: their sum is small, the roundings of each are not.

    Sums of groups differ by some 1e-6, an fp32 of the size of 100 is rounded by up to 4e-6, of 3000 by 1.2e-4."""
    g = torch.Generator().manual_seed(41)
    per, m = e // groups, 60
    z = torch.randn(1, 1, per, generator=g) + torch.randn(m, groups, per, generator=g) * 1e-5
    bias = torch.full((groups, per), -4 * size)
    bias[:, 1], bias[:, 2] = size, -size
    _compare(b4, z.reshape(m, e), bias.reshape(e), k, score, groups=groups, top_groups=top_groups, group_top=2)
    # one group alone is far from zero: its sum's error counts against the others' small ones, above and below them
    for shift in (-1e-6, 0.0, 1e-6):
        bias = torch.full((groups, per), -4 * size)
        bias[:, 1], bias[:, 2] = 0.5, -0.5
        bias[1, 1], bias[1, 2] = size, -size
        zs = z.clone()
        zs[:, 1] += shift
        _compare(b4, zs.reshape(m, e), bias.reshape(e), k, score, groups=groups, top_groups=top_groups, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_of_the_largest_and_lowest_biases(b4, score):  # noqa: F811
    """Sums past fp32's range, groups masked by the type's lowest value or by -inf, infinite groups."""
    top, inf = torch.finfo(F32).max, float("inf")
    z = _z(9, 64, 43, F32)
    for case in range(6):
        bias = torch.randn(8, 8, generator=torch.Generator().manual_seed(44)) * 0.1
        if case == 0:
            bias[5] = bias[2] = top
            bias[5, 3:] = top / 2
            bias[2, 1:] = 0.75 * top
        elif case == 1:
            bias[:6] = -top
            bias[0] = -inf
            bias[3, 0] = -0.5 * top
        elif case == 2:
            bias[[1, 4, 6]] = inf
            bias[4, 1:] = -top
            bias[2, 2:4] = top
        elif case == 3:
            bias[:] = -top
            bias[::2] = -inf
        elif case == 4:
            bias[:, 1:] = -inf
            bias[3:, 0] = -top
        else:
            bias[:] = -inf
            bias[6, 1] = bias[7, 1] = -top
        for kw in (dict(groups=8, top_groups=2), dict(groups=8, top_groups=4), dict(groups=4, top_groups=3)):
            for group_top in (1, 2):
                _compare(b4, z, bias.reshape(64), 8, score, group_top=group_top, **kw)


@pytest.mark.parametrize("e,groups,v", [(1024, 1, 32), (960, 6, 40), (1020, 17, 60)])
def test_softmax_of_one_large_and_many_small(b4, e, groups, v):  # noqa: F811
    """Exponentials just over half a unit of the largest's last place: added one by one, each is rounded up to a whole one.

    The largest's score has the bias -1, so that c is what its score lacks of 1, some 2e-6; another expert's bias alone lies
    1e-8 below the exact c."""
    z = torch.full((1, e), -60.0, dtype=F32)
    step = e // groups if groups == 17 else -(-(e // groups) // (4 if groups == 6 else 32))  # experts of a lane
    z[0, :v] = -16.635  # e^z = 1.0005 2^-24
    z[0, 0] = 0.0
    for lane in (1, 2, 4, 8, 16):
        if lane * step < e:
            z[0, lane * step] = -16.635
    s = R.scores(z.double().numpy()[0], "softmax")
    bias = torch.full((e,), -2.0, dtype=F32)
    bias[0] = -1.0
    for shift in (-1e-8, 1e-8):
        bias[e - 1] = float(s[0] - 1.0 + shift)
        _compare(b4, z, bias, 2, "softmax", groups=groups, top_groups=groups)


def test_experts_out_by_their_bias_stay_in_the_softmax(b4):  # noqa: F811
    """Without renormalisation the weights show what the softmax's sum is made of."""
    z = _z(6, 64, 45, F32)
    z[1, 5] = z[2, 9] = float("-inf")
    z[3, 40:] = float("nan")
    bias = torch.randn(64, generator=torch.Generator().manual_seed(46)) * 0.1
    bias[[5, 30]] = float("-inf")
    bias[[7, 41]] = float("nan")
    for kw in (dict(), dict(groups=4, top_groups=2), dict(groups=4, top_groups=2, group_top=2)):
        _compare(b4, z, bias, 8, "softmax", renorm=False, scale=1.5, **kw)
