"""The router's choice by biased scores and by groups, where 32 bits cannot hold
or tell them: finite biases up to the type's largest, as masks and as
preferences, and values that are nearer to each other than the rounding of
values of that size, for each number of experts a lane has and for groups that
are not whole lanes.  The choice is equal to the definition's in 64 bits."""
import numpy as np
import pytest
import torch

import error_bounded_lossy_gb300 as ebc
from test_gpu_route import logits_of, scores

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

MOST = float(np.finfo(np.float32).max)
KINDS = ["softmax", "sigmoid"]
# experts, groups: 1 to 32 values a lane, groups of whole lanes and others
GROUPS = [(30, 3), (35, 5), (64, 8), (128, 8), (256, 8), (300, 6), (512, 4), (992, 31), (1024, 16)]


@pytest.fixture(scope="module")
def ex():
    e = ebc.Experts(0)
    yield e
    e.check()
    e.close()


def largest(v, n):
    """The places of the n largest in each row, the largest first, ties to the lower; -1 where only -inf is left."""
    at = np.argsort(-v, axis=1, kind="stable")[:, :n]
    return np.where(np.isneginf(np.take_along_axis(v, at, 1)), -1, at)


def check(ex, logits, top, bias, kind, groups=1, keep=1, group_top=1):
    """The ids, against the definition in 64 bits."""
    l = logits.cpu().numpy().astype(np.float64)
    b = 0.0 if bias is None else bias.cpu().numpy().astype(np.float64)
    c = np.where(np.isneginf(l + b), -np.inf, scores(l, kind) + b)
    v = l.copy() if bias is None else c.copy()
    if groups > 1:
        of = (c if bias is not None or group_top == 2 else l).reshape(len(l), groups, -1)
        two = -np.sort(-of, 2)[..., :group_top]
        total = np.where(np.isneginf(two[..., 0]), -np.inf, np.where(np.isneginf(two), 0.0, two).sum(2))
        kept = np.zeros((len(l), groups + 1), bool)
        np.put_along_axis(kept, largest(total, keep), True, 1)   # (-1: the column past the groups)
        v[~np.repeat(kept[:, :groups], l.shape[1] // groups, 1)] = -np.inf
    ids, _ = ex.route(logits, top, kind, bias, groups, keep, group_top)
    want = largest(v, top)
    assert want.shape[1] == top and np.array_equal(ids.cpu().numpy(), want)
    return ids


@pytest.mark.parametrize("kind", KINDS)
def test_sums_of_a_group_past_fp32(ex, kind):
    """The sum of two biased scores is past the largest number of fp32 on either side: the larger sum is kept, and a
    group masked with the type's lowest value is more than one that has no expert."""
    l = torch.zeros(7, 64, device="cuda")
    for low, high in ((3.0e38, 3.3e38), (1.8e38, 2.0e38), (-3.3e38, -3.0e38), (-MOST, 0.0), (-MOST, -3.3e38), (1.0, MOST)):
        b = torch.full((64,), low, device="cuda")
        b[32:] = high
        ids = check(ex, l, 4, kind=kind, bias=b, groups=2, keep=1, group_top=2)
        assert ids[0].tolist() == [32, 33, 34, 35]
    for low in (-MOST, -3.0e38, -1e9):
        b = torch.full((64,), -float("inf"), device="cuda")
        b[32:] = low
        ids = check(ex, l, 4, kind=kind, bias=b, groups=2, keep=1, group_top=2)
        assert ids[0].tolist() == [32, 33, 34, 35]
    b = torch.full((64,), -MOST, device="cuda")
    b[:16] = MOST            # the best two of the first group are more than what the second's cancel to
    b[32] = MOST
    ids = check(ex, l, 4, kind=kind, bias=b, groups=2, keep=1, group_top=2)
    assert ids[0].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [1e4, 1e9, 3e38, MOST])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("experts,groups", GROUPS)
def test_finite_biases_of_any_size(ex, experts, groups, sign, size, kind):
    inf = float("inf")
    l, b = logits_of(20, experts, torch.float32, experts)
    each, some = experts // groups, groups // 2 + 1
    one, third = b.clone(), b.clone()
    one[experts // 2] = sign * size
    third[::3] = sign * size
    whole = b.clone().view(groups, each)
    whole[:some] = sign * size * (1 - torch.arange(some, device="cuda").flip(0)[:, None] / 32)
    none = whole.clone()
    none[0] = -inf
    mixed = whole.clone()
    mixed[:, 0] = -sign * size
    for bias in (one, third, whole.reshape(-1), none.reshape(-1), mixed.reshape(-1)):
        check(ex, l, 8, kind=kind, bias=bias)
        for group_top in (1, 2):
            for keep in (1, some, groups - 1):
                check(ex, l, 8, kind=kind, bias=bias, groups=groups, keep=keep, group_top=group_top)


def near(rng, tokens, target, kind, size):
    """Logits [tokens, experts] and a bias with which every token's biased scores are at their targets but for the
    bias's rounding, and differ from token to token by a few units of it."""
    base = rng.standard_normal(target.size)
    s = scores(base[None].astype(np.float32).astype(np.float64), kind)[0]
    bias = (target - s).astype(np.float32)
    slope = s if kind == "softmax" else s * (1 - s)
    step = np.minimum(np.spacing(np.float32(size)) / slope, 0.05)
    l = (base + rng.uniform(-2, 2, (tokens, target.size)) * step).astype(np.float32)
    return l, bias, scores(l.astype(np.float64), kind) + bias


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [1, 10, 1000])
@pytest.mark.parametrize("experts", [30, 64, 100, 256, 300, 512, 1000, 1024])
def test_scores_of_any_size_that_32_bits_cannot_tell_apart(ex, experts, size, kind):
    """Pairs whose biased scores are within the bias's rounding, the pairs themselves apart."""
    rng = np.random.default_rng(experts)
    steps = np.repeat(np.arange(1, experts // 2 + 2) * (0.5 / experts), 2)[:experts]
    l, bias, c = near(rng, 20, size - rng.permutation(steps), kind, size)
    order = -np.sort(-c, 1)
    gaps = order[:, :8] - order[:, 1:9]
    assert (gaps < 2 * np.spacing(np.float32(size))).mean() > 0.2
    # (candidates: what may be among the best 8, with four times the rounding of such a value)
    assert ((c >= order[:, 7:8] - 4 * (80 + size) * 2.0 ** -23).sum(1) <= 32).all()
    lt, bt = torch.from_numpy(l).cuda(), torch.from_numpy(bias).cuda()
    for top in (1, 7, 8):
        check(ex, lt, top, kind=kind, bias=bt)
    check(ex, lt, 20, kind=kind, bias=bt)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [1, 10, 1000])
@pytest.mark.parametrize("experts,groups", GROUPS)
def test_groups_of_any_size_that_32_bits_cannot_tell_apart(ex, experts, groups, size, kind):
    """Up to twelve groups whose best two are within the bias's rounding, a few kept: the sums of their candidates
    (24 at most) decide in 64 bits, and then those candidates' order."""
    rng = np.random.default_rng(experts + groups)
    each, alike = experts // groups, min(groups, 12)
    keep = max(alike // 2, 1)
    target = np.full((groups, each), 0.0)
    for g, at in enumerate(rng.permutation(groups)):
        v = size - 1.5 - 0.01 * np.arange(each)
        v[:2] = (size, size - 0.5) if g < alike else (size - 0.7, size - 0.8)
        target[at] = rng.permutation(v)
    l, bias, c = near(rng, 20, target.reshape(-1), kind, size)
    two = -np.sort(-c.reshape(20, groups, each), 2)[..., :2]
    for best in (1, 2):
        order = -np.sort(-two[..., :best].sum(2), 1)
        assert ((order[:, keep - 1] - order[:, keep]) < 2 * np.spacing(np.float32(size))).mean() > 0.2
    lt, bt = torch.from_numpy(l).cuda(), torch.from_numpy(bias).cuda()
    for group_top in (1, 2):
        for top in (1, keep, 2 * keep):
            check(ex, lt, top, kind=kind, bias=bt, groups=groups, keep=keep, group_top=group_top)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("experts,groups", GROUPS)
def test_group_sums_of_the_same_scores(ex, experts, groups, kind):
    """Groups of the same logits in another order, a unit apart here and there, without a bias and with one of zeros."""
    rng = np.random.default_rng(groups)
    each = experts // groups
    base = rng.standard_normal((20, 1, each)).astype(np.float32)
    l = np.take_along_axis(np.repeat(base, groups, 1), rng.random((20, groups, each)).argsort(2), 2).reshape(20, experts)
    l += (rng.integers(-1, 2, l.shape) * np.spacing(np.abs(l))).astype(np.float32)
    lt = torch.from_numpy(l).cuda()
    for bias in (None, torch.zeros(experts, device="cuda")):
        for keep in (1, groups // 2, groups - 1):
            check(ex, lt, 8, kind=kind, bias=bias, groups=groups, keep=keep, group_top=2)
