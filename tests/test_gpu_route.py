"""The router against its definition in 64 bits: the choice is equal whatever
the scores, weights and gradients are near.

In units of 2^-24, relative: a score takes an exponential (4), a sum of the
exponentials (a lane's share of the experts and 5 joins, or the 5 joins of the
chosen ones), one more addition, a quotient (2 or, fast, 4) and a product;
before the exponential the difference of two logits was rounded, which is their
difference's size times one unit.  `lost` adds that up, with 4 units to spare.
A gradient is a sum of products of two such scores with the weights' gradients,
each within three times that of its magnitude."""
import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import error_bounded_lossy_gb300 as ebc

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

TYPES = [torch.float32, torch.bfloat16, torch.float16]
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ex():
    e = ebc.Experts(0)
    yield e
    e.check()
    e.close()


def scores(l, kind):
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return np.where(l > 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
        top = l.max(1, keepdims=True)
        p = np.exp(l - np.where(np.isneginf(top), 0, top))
        return p / np.where(np.isneginf(top), 1, p.sum(1, keepdims=True))


def best(v, n):
    """The places of the n largest of v, the largest first, ties to the lower; NaN is the largest, -inf is nothing."""
    key = np.where(np.isnan(v), np.inf, v)
    order = sorted(range(len(v)), key=lambda i: (not np.isnan(v[i]), -key[i], i))
    return [i for i in order if not np.isneginf(v[i])][:n]


def defined(l, top, kind="softmax", bias=None, groups=1, keep=None, group_top=1, renorm=True, scale=1.0):
    l = l.astype(np.float64)
    s = scores(l, kind)
    b = np.zeros(l.shape[1]) if bias is None else bias.astype(np.float64)
    dead = np.isneginf(l) | np.isneginf(b)
    with np.errstate(invalid="ignore"):
        c = np.where(dead, -np.inf, s + b)
    v = c if bias is not None else np.where(dead, -np.inf, l)      # what is compared
    g = c if bias is not None or group_top == 2 else v
    ids, w = np.full((len(l), top), -1), np.zeros((len(l), top))
    for t in range(len(l)):
        row = v[t].copy()
        if groups > 1:
            size = l.shape[1] // groups
            total = np.full(groups, -np.inf)
            for j in range(groups):
                part = g[t, j * size:(j + 1) * size]
                two = best(part, group_top)
                if two:
                    total[j] = part[two].sum()
            for j in set(range(groups)) - set(best(total, keep or groups)):
                row[j * size:(j + 1) * size] = -np.inf
        got = best(row, top)
        ids[t, :len(got)] = got
        w[t, :len(got)] = s[t, got]
        if renorm and got:
            # the shares of scores that may be far below the smallest number
            x = l[t, got]
            n = np.exp(x - x.max()) if kind == "softmax" else s[t, got] if s[t, got].max() > 1e-200 else np.exp(x - x.max())
            w[t, :len(got)] = n / n.sum()
    return ids, scale * w


def lost(l, ids, kind, renorm):
    """Units that a weight may be off, [tokens, 1]."""
    l = np.where(np.isfinite(l), l, np.nan).astype(np.float64)
    with np.errstate(all="ignore"):
        import warnings
        with warnings.catch_warnings():
            warnings.simplefilter("ignore")
            x = np.where(ids >= 0, np.take_along_axis(l, np.maximum(ids, 0), 1), np.nan)
            span = np.nanmax(x, 1) - np.nanmin(x, 1) if renorm else np.nanmax(l, 1) - np.nanmin(x, 1)
            if kind == "sigmoid":
                span = np.maximum(span, 0) if renorm else np.zeros(len(l))
    terms = 5 if renorm else l.shape[1] / 32 + 5
    return np.nan_to_num(4 + terms + 1 + 4 + 2 + span + 4)[:, None]


def check(ex, logits, top, ids=None, weights=None, **how):
    l = logits.float().cpu().numpy()
    bias = how.get("bias")
    named = {**how, "bias": None if bias is None else bias.cpu().numpy()}
    if ids is None:
        ids, weights = ex.route(logits, top, how.get("kind", "softmax"), bias, how.get("groups", 1), how.get("keep"),
                                how.get("group_top", 1), how.get("renorm", True), how.get("scale", 1.0))
    want, w = defined(l, top, **named)
    assert ids.dtype == torch.int32 and weights.dtype == torch.float32
    assert np.array_equal(ids.cpu().numpy(), want)
    off = np.abs(weights.double().cpu().numpy() - w)
    bound = lost(l, want, how.get("kind", "softmax"), how.get("renorm", True)) * U * np.abs(w) + 1e-37
    assert (off <= bound).all(), (off / np.maximum(bound, 1e-300)).max()
    return ids, weights


def logits_of(tokens, experts, dtype, seed, masked=0.0, spread=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    l = spread * torch.randn(tokens, experts, generator=g, device="cuda") + torch.randn(experts, generator=g, device="cuda")
    if masked:
        gone = torch.rand(tokens, experts, generator=g, device="cuda") < masked
        gone |= torch.rand(tokens, 1, generator=g, device="cuda") < masked / 2
        l = torch.where(gone, -torch.inf, l)
    b = 0.1 * torch.randn(experts, generator=g, device="cuda")
    return l.to(dtype), b


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,top,masked", [
    (1, 1, 1, 0.0), (1, 64, 8, 0.0), (5, 2, 2, 0.3), (33, 10, 3, 0.2), (7, 32, 32, 0.0), (40, 33, 7, 0.1), (100, 64, 6, 0.0), (20, 100, 32, 0.5),
    (50, 128, 8, 0.0), (300, 256, 8, 0.0), (30, 257, 16, 0.1), (9, 512, 1, 0.0), (6, 1000, 31, 0.0), (6, 1024, 32, 0.9), (40, 256, 24, 0.0), (40, 64, 31, 0.0), (3, 40, 9, 1.0)])
def test_without_groups(ex, tokens, experts, top, masked, kind, dtype):
    l, b = logits_of(tokens, experts, dtype, tokens + experts, masked)
    check(ex, l, top, kind=kind)
    check(ex, l, top, kind=kind, renorm=False, scale=2.5)
    check(ex, l, top, kind=kind, bias=b, scale=-0.5)
    check(ex, l, top, kind=kind, bias=b, renorm=False)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,groups,keep,top,masked", [
    (1, 256, 8, 4, 8, 0.0), (300, 256, 8, 4, 8, 0.0), (50, 256, 8, 1, 6, 0.1), (40, 64, 32, 5, 8, 0.2), (20, 32, 32, 7, 7, 0.0), (60, 30, 3, 2, 4, 0.2),
    (33, 35, 5, 2, 6, 0.1), (21, 1024, 16, 3, 20, 0.0), (60, 256, 8, 2, 8, 0.0), (60, 256, 8, 2, 24, 0.1), (30, 512, 4, 1, 32, 0.0), (15, 992, 31, 30, 32, 0.0), (10, 12, 2, 1, 9, 0.3), (10, 12, 2, 2, 9, 0.3), (8, 48, 24, 3, 2, 1.0)])
def test_groups(ex, tokens, experts, groups, keep, top, masked, kind):
    l, b = logits_of(tokens, experts, torch.float32, tokens + experts, masked)
    for group_top in (1, 2):
        for bias in (None, b):
            check(ex, l, top, kind=kind, bias=bias, groups=groups, keep=keep, group_top=group_top)
    check(ex, l.to(torch.bfloat16), top, kind=kind, bias=b, groups=groups, keep=keep, group_top=2, renorm=False)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_scores_that_32_bits_cannot_tell_apart(ex, kind, group_top):
    """Experts in pairs whose biased scores are a few units of 2^-26 apart, or a few parts of one: the bias makes up
    for the score's difference.  Which of the two is larger is asked in 64 bits."""
    rng = np.random.default_rng(0)
    tokens, experts = 200, 64
    l = rng.standard_normal((tokens, experts)).astype(np.float32)
    l[:] = l[0]                       # one row of scores, so that one bias suits it
    s = scores(l[:1].astype(np.float64), kind)[0]
    target = np.repeat(np.sort(s)[::-1][:experts // 2], 2)[rng.permutation(experts)]
    bias = (target - s).astype(np.float32)
    l += (rng.integers(-2, 3, l.shape) * np.spacing(np.abs(l))).astype(np.float32)
    lt, bt = torch.from_numpy(l).cuda(), torch.from_numpy(bias).cuda()
    c = scores(l.astype(np.float64), kind) + bias
    gaps = -np.diff(-np.sort(-c, 1), axis=1)
    assert (np.abs(gaps) < 2.0 ** -24).mean() > 0.2
    check(ex, lt, 8, kind=kind, bias=bt)
    check(ex, lt, 32, kind=kind, bias=bt, renorm=False)
    check(ex, lt, 6, kind=kind, bias=bt, groups=8, keep=3, group_top=group_top)
    check(ex, lt[:, :32].contiguous(), 32, kind=kind, bias=bt[:32].contiguous())


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_groups_that_32_bits_cannot_tell_apart(ex, kind):
    """Group sums of the same numbers in another order, a unit apart here and there."""
    rng = np.random.default_rng(1)
    base = rng.standard_normal((100, 1, 16)).astype(np.float32)
    l = np.take_along_axis(np.repeat(base, 8, 1), rng.random((100, 8, 16)).argsort(2), 2).reshape(100, 128)
    l += (rng.integers(-1, 2, l.shape) * np.spacing(np.abs(l))).astype(np.float32)
    for bias in (None, torch.zeros(128, device="cuda")):
        check(ex, torch.from_numpy(l).cuda(), 8, kind=kind, bias=bias, groups=8, keep=3, group_top=2)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_ties_go_to_the_lower_expert(ex, kind, bias):
    l = torch.randint(-1, 2, (64, 300), device="cuda").to(torch.bfloat16)
    l[1] = 0.0
    l[2, ::2] = -0.0
    b = torch.zeros(300, device="cuda") if bias else None
    for top in (1, 7, 32):
        ids, _ = check(ex, l, top, kind=kind, bias=b)
        assert ids[1].tolist() == list(range(top))
        check(ex, l, top, kind=kind, bias=b, groups=6, keep=2, group_top=2)
    same = torch.zeros(5, 1024, device="cuda")
    assert (ex.route(same, 32, kind, torch.full((1024,), 0.25, device="cuda"))[0].cpu() == torch.arange(32)).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_rows_of_one_score(ex, kind, group_top):
    """Every value ties, among them scores that are zero in 32 bits, rows but for one expert, and groups with one
    expert left: the lower expert and the lower group, and two scores of a group are more than one."""
    inf = float("inf")
    l = torch.zeros(10, 256, device="cuda")
    l[1] = -200.0
    l[2], l[2, 100] = -200.0, -199.0
    l[3, 200] = 1.0
    l[4, :31] = -inf
    l[5] = -200.0
    l[5, :31] = -inf
    l[6] = torch.finfo(torch.float32).min
    l[7, 1::2] = torch.tensor(1.0).nextafter(torch.tensor(0.0)) * 1e-30
    l[8, 3:] = -inf
    l[9] = 90.0
    for bias in (None, torch.zeros(256, device="cuda"), torch.full((256,), 0.25, device="cuda")):
        for top in (1, 8, 32):
            for dtype in (torch.float32, torch.bfloat16):
                check(ex, l[[0, 3, 4, 8, 9]].to(dtype), top, kind=kind, bias=bias)
                check(ex, l[[0, 3, 4, 8, 9]].to(dtype), top, kind=kind, bias=bias, groups=8, keep=4, group_top=group_top)
            named = dict(bias=None if bias is None else bias.cpu().numpy(), kind=kind)
            for how in (dict(), dict(groups=8, keep=4, group_top=group_top)):
                ids, _ = ex.route(l, top, kind, bias, how.get("groups", 1), how.get("keep"), how.get("group_top", 1))
                want = defined(l.cpu().numpy(), top, **named, **how)[0]
                assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_masks_that_leave_little_or_nothing(ex, kind):
    inf = float("inf")
    l = torch.full((6, 40), -inf, device="cuda")
    l[1, 39] = -5.0
    l[2, [3, 30]] = torch.tensor([1.0, 2.0], device="cuda")
    l[3] = torch.finfo(torch.float32).min      # a mask of the type's lowest value is a value
    l[4] = torch.finfo(torch.float32).min
    l[4, 7] = 3.0
    l[5] = torch.randn(40, device="cuda") - 1000.0   # scores that are zero in 32 bits
    for renorm in (True, False):
        for bias in (None, torch.zeros(40, device="cuda")):
            ids, w = ex.route(l, 3, kind, bias, renormalize=renorm)
            assert ids[:3].tolist() == [[-1, -1, -1], [39, -1, -1], [30, 3, -1]]
            assert not w[0].any() and not w[1, 1:].any() and not w[2, 2].any() and bool(torch.isfinite(w).all())
            if bias is None:
                assert ids[3].tolist() == [0, 1, 2] and ids[4].tolist() == [7, 0, 1]
                assert ids[5].tolist() == l[5].topk(3).indices.tolist()
        check(ex, l[:3], 3, kind=kind, renorm=renorm)
    ids, w = ex.route(l, 3, kind)
    assert bool(((w[1:].double().sum(1) - 1).abs() < 1e-6).all())   # (three roundings of 2^-24 and the quotients')
    check(ex, l[5:], 3, kind=kind)
    # ruled out by the bias
    b = torch.zeros(40, device="cuda")
    b[5:] = -inf
    ids, w = ex.route(torch.randn(9, 40, device="cuda"), 8, kind, b)
    assert bool((ids[:, 5:] == -1).all()) and bool((ids[:, :5].sort(1).values.cpu() == torch.arange(5)).all()) and not w[:, 5:].any()
    # groups that are masked out, and more choices than the kept groups have
    l = torch.randn(9, 40, device="cuda")
    l[:, :30] = -inf
    ids, _ = check(ex, l, 12, kind=kind, groups=4, keep=2, group_top=2)
    assert bool((ids[:, 10:] == -1).all())


@pytest.mark.parametrize("bias", [False, True])
def test_nan_and_infinity_stay_in_their_rows(ex, bias):
    l = torch.randn(4, 50, device="cuda")
    clean = l.clone()
    l[1, 20] = float("nan")
    l[2, 30] = float("inf")
    b = torch.zeros(50, device="cuda") if bias else None
    for kind in ("softmax", "sigmoid"):
        ids, w = ex.route(l, 4, kind, b)
        i0, w0 = ex.route(clean, 4, kind, b)
        assert torch.equal(ids[[0, 3]], i0[[0, 3]]) and torch.equal(w[[0, 3]], w0[[0, 3]])
        assert bool(w[1].isnan().any()) and bool(((ids >= 0) & (ids < 50)).all())
        if kind == "sigmoid":
            assert ids[1, 0] == 20 and ids[2, 0] == 30 and bool(torch.isfinite(w[2]).all())
        d = ex.route_grad(torch.randn(4, 4, device="cuda"), l, ids, kind)
        assert bool(torch.isfinite(d[[0, 3]]).all())


def grad_of(l, ids, dw, kind, renorm, scale):
    """The gradient in 64 bits, and the magnitudes that its error is relative to."""
    l, g = l.astype(np.float64), dw.astype(np.float64) * scale
    t = np.arange(len(l))[:, None]
    none = ids < 0
    at = np.maximum(ids, 0)
    s = scores(l, kind)
    u = np.where(none, 0.0, s[t, at])
    if renorm:
        x = np.where(none, -np.inf, l[t, at])
        m = np.where(none.all(1), 0.0, x.max(1))[:, None]
        n = np.exp(x - m) if kind == "softmax" else u
        u = np.where(none, 0.0, n / np.where(none.all(1), 1.0, n.sum(1))[:, None])
    g = np.where(none, 0.0, g)
    slope = scores(-l, "sigmoid")[t, at] if kind == "sigmoid" else 1.0
    out, size = np.zeros_like(l), np.zeros_like(l)
    d = u * slope * (g - ((u * g).sum(1, keepdims=True) if renorm else 0))
    e = u * slope * (np.abs(g) + ((u * np.abs(g)).sum(1, keepdims=True) if renorm else 0))
    for j in range(ids.shape[1]):
        live = ~none[:, j]
        out[t[live, 0], at[live, j]] += d[live, j]
        size[t[live, 0], at[live, j]] += e[live, j]
    if kind == "softmax" and not renorm:
        out -= s * (u * g).sum(1, keepdims=True)
        size += s * (u * np.abs(g)).sum(1, keepdims=True)
    return out, size


def check_grad(l, ids, dw, got, kind, renorm, scale):
    a = l.float().cpu().numpy()
    i = ids.cpu().numpy()
    want, size = grad_of(a, i, dw.cpu().numpy(), kind, renorm, scale)
    bound = 3 * lost(a, i, kind, renorm) * U * size
    if kind == "softmax" and not renorm:   # of every expert, so down to the smallest logit
        low = np.where(np.isfinite(a), a, a.max(1, keepdims=True))
        bound += U * size * np.nan_to_num(a.max(1, keepdims=True) - low.min(1, keepdims=True), nan=0.0)
    bound = bound + UNIT[l.dtype] * (np.abs(want) + bound) + (2.0 ** -25 if l.dtype == torch.float16 else 1e-37)
    off = np.abs(got.double().cpu().numpy() - want)
    assert got.dtype == l.dtype and got.shape == l.shape and (off <= bound).all(), (off / bound).max()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("tokens,experts,top,masked", [
    (1, 1, 1, 0.0), (1, 64, 8, 0.0), (5, 2, 2, 0.3), (33, 10, 3, 0.2), (7, 32, 32, 0.0), (40, 33, 7, 0.1), (20, 100, 32, 0.5), (300, 256, 8, 0.0),
    (30, 257, 16, 0.1), (9, 512, 1, 0.0), (6, 1023, 31, 0.0), (6, 1024, 32, 0.9), (40, 256, 24, 0.0), (40, 64, 31, 0.0), (3, 40, 9, 1.0)])
def test_the_gradient(ex, tokens, experts, top, masked, renorm, kind, dtype):
    l, b = logits_of(tokens, experts, dtype, tokens + experts, masked)
    dw = torch.randn(tokens, top, device="cuda")
    ids, _ = ex.route(l, top, kind, b, renormalize=renorm, scale=1.5)
    got = ex.route_grad(dw, l, ids, kind, renorm, 1.5)
    check_grad(l, ids, dw, got, kind, renorm, 1.5)
    assert torch.equal(got, ex.route_grad(dw, l, ids, kind, renorm, 1.5))


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_the_gradient_against_differences(ex, renorm, kind):
    """Central differences of the kernel's own weights where the choice stays the same: rounding leaves `lost` units of
    the weights over the step; the steps' error is a third of the difference to twice the step, to its leading order
    (doubled)."""
    l, _ = logits_of(50, 40, torch.float32, 2)
    l = l.double()
    v, g = torch.randn(50, 40, device="cuda").double(), torch.randn(50, 5, device="cuda").double()
    ids, w = ex.route(l.float(), 5, kind, renormalize=renorm)
    d = ex.route_grad(g.float(), l.float(), ids, kind, renorm)

    def slope(t):
        out = []
        for at in ((l + t * v).float(), (l - t * v).float()):
            chosen, got = ex.route(at, 5, kind, renormalize=renorm)
            back = torch.full((50, 40), float("nan"), device="cuda", dtype=torch.float64).scatter_(1, chosen.long(), got.double())
            out.append((back.gather(1, ids.long()) * g).sum(1))
        return (out[0] - out[1]) / (2 * t)

    fine, coarse = slope(2.0 ** -7), slope(2.0 ** -6)
    use = torch.isfinite(fine) & torch.isfinite(coarse)     # (tokens whose choice is another one on the way)
    assert int(use.sum()) > 25
    # the logits were rounded too: half a unit of at most 4, in the scores' own slope of at most 1
    rounding = (64 + 8) * U * (w.double() * g.abs()).sum(1) / 2.0 ** -7
    off = ((d.double() * v).sum(1) - fine).abs()
    assert bool((off <= 2 * (coarse - fine).abs() / 3 + rounding + 1e-6)[use].all())


def test_ids_of_any_kind_in_the_gradient():
    """The same index twice is the sum of both; dropped ones have none; those past the experts are recorded."""
    e = ebc.Experts(0)
    l = torch.randn(3, 20, device="cuda")
    dw = torch.randn(3, 4, device="cuda")
    ids = torch.tensor([[3, 3, 3, 5], [-1, 7, -9, 7], [-1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            check_grad(l, ids, dw, e.route_grad(dw, l, ids, kind, renorm, 1.0), kind, renorm, 1.0)
    e.check()
    ids[0, 0] = 20
    got = e.route_grad(dw, l, ids)
    with pytest.raises(ebc.EbcError):
        e.check()
    ids[0, 0] = -1
    assert torch.equal(got, e.route_grad(dw, l, ids))
    e.close()


def test_strides_streams_graphs_and_nothing(ex):
    l, b = logits_of(70, 100, torch.bfloat16, 4)
    wide = torch.zeros(70, 203, dtype=torch.bfloat16, device="cuda")
    want = ex.route(l, 6, "sigmoid", b, 10, 4, 2)
    dw = torch.randn(70, 6, device="cuda")
    dl = ex.route_grad(dw, l, want[0], "sigmoid")
    for at in (0, 1, 2, 4, 100):
        wide[:, at:at + 100] = l
        part = wide[:, at:at + 100]
        assert all(torch.equal(p, q) for p, q in zip(want, ex.route(part, 6, "sigmoid", b, 10, 4, 2)))
        assert torch.equal(dl, ex.route_grad(dw, part, want[0], "sigmoid"))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = ex.route(l, 6, "sigmoid", b, 10, 4, 2, stream=side)
    again = ex.route_grad(dw, l, got[0], "sigmoid", stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*want, dl), (*got, again)))
    graph, given = torch.cuda.CUDAGraph(), l.clone()
    with torch.cuda.graph(graph):
        ids, w = ex.route(given, 6, "sigmoid", b, 10, 4, 2)
        d = ex.route_grad(dw, given, ids, "sigmoid")
    given.copy_(l.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ids, want[0].flip(0)) and torch.equal(w, want[1].flip(0))
    assert torch.equal(d, ex.route_grad(dw, given, ids, "sigmoid"))
    ids, w = ex.route(l[:0], 6)
    assert ids.shape == w.shape == (0, 6) and ex.route_grad(dw[:0], l[:0], ids).shape == (0, 100)


def test_many_tokens(ex):
    """More than the machine has warps, and results past 2^31 bytes."""
    tokens, experts = 2_200_000, 256
    l = torch.randn(tokens, experts, device="cuda")
    ids, w = ex.route(l, 4)
    v, i = l.topk(4, 1)
    same = (i == ids).all(1)
    assert float(same.float().mean()) > 0.999          # (ties)
    off = (w[same] - v[same].softmax(1)).abs().max()
    assert float(off) < 1e-6
    d = ex.route_grad(w, l, ids)
    at = torch.tensor([0, 1, 2_097_151, 2_097_152, tokens - 1], device="cuda")
    check_grad(l[at], ids[at], w[at], d[at], "softmax", True, 1.0)


def test_recorded(ex):
    l0, b = logits_of(40, 64, torch.float32, 5)
    dw = torch.randn(40, 6, device="cuda")
    how = dict(score="sigmoid", bias=b, groups=8, keep_groups=3, group_top=2, scale=2.5)
    l = l0.clone().requires_grad_()
    ids, w = ex.route(l, 6, **how)
    assert w.requires_grad and not ids.requires_grad
    (w * dw).sum().backward()
    assert torch.equal(l.grad, ex.route_grad(dw, l0, ids, "sigmoid", True, 2.5))
    l.grad = None
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ids, w = ex.route(l, 6, renormalize=False, stream=side)
    torch.cuda.synchronize()
    w.sum().backward()       # one value, expanded
    torch.cuda.synchronize()
    assert torch.equal(l.grad, ex.route_grad(torch.ones_like(dw), l0, ids, "softmax", False))
    with torch.no_grad():
        assert not ex.route(l, 6)[1].requires_grad
    assert not ex.route(l0, 6, bias=b.clone().requires_grad_())[1].requires_grad   # the bias has none
    (d,) = torch.autograd.grad((ex.route(l, 6)[1] ** 2).sum(), l, create_graph=True)
    with pytest.raises(RuntimeError):
        d.sum().backward()
    with forward_ad.dual_level(), pytest.raises(ValueError, match="forward"):
        ex.route(forward_ad.make_dual(l0, l0), 6)


def test_refusals(ex):
    l, b = logits_of(8, 24, torch.float32, 6)
    ids, w = ex.route(l, 2)
    for call in (lambda: ex.route(l.double(), 2), lambda: ex.route(l.cpu(), 2), lambda: ex.route(l[0], 2), lambda: ex.route(l, 2, "tanh"),
                 lambda: ex.route(l, 2, bias=b[:23]), lambda: ex.route(l, 2, bias=b.half()), lambda: ex.route(l, 2, bias=b.cpu()),
                 lambda: ex.route(l.t(), 2), lambda: ex.route_grad(w.half(), l, ids), lambda: ex.route_grad(w, l, ids.long()),
                 lambda: ex.route_grad(w[:, :1], l, ids), lambda: ex.route_grad(w[:7], l, ids[:7]), lambda: ex.route_grad(w, l, ids, "tanh")):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ex.route(l, 0), lambda: ex.route(l, 33), lambda: ex.route(l, 2, groups=5), lambda: ex.route(l, 2, groups=0),
                 lambda: ex.route(l, 2, groups=4, keep_groups=5), lambda: ex.route(l, 2, groups=4, keep_groups=0),
                 lambda: ex.route(l, 2, groups=4, keep_groups=2, group_top=3), lambda: ex.route(l, 2, scale=float("nan")),
                 lambda: ex.route(l, 2, scale=float("inf")), lambda: ex.route(torch.zeros(2, 1025, device="cuda"), 2),
                 lambda: ex.route(torch.zeros(2, 1024, device="cuda"), 2, groups=64), lambda: ex.route(l, 2, groups=2 ** 40)):
        with pytest.raises(ebc.EbcError) as err:
            call()
        assert err.value.code == ebc.EBC_ERR_INVALID_ARG
    h, p, i, q = ex.handle, l.data_ptr(), ids.data_ptr(), w.data_ptr()
    inv = ebc.EBC_ERR_INVALID_ARG
    assert ebc.ebc_moe_route(h, None, 24, 0, 8, 24, 2, 0, None, 1, 1, 1, 1, 1.0, i, q, None) == inv
    assert ebc.ebc_moe_route(h, p, 23, 0, 8, 24, 2, 0, None, 1, 1, 1, 1, 1.0, i, q, None) == inv
    assert ebc.ebc_moe_route(h, p, 24, 3, 8, 24, 2, 0, None, 1, 1, 1, 1, 1.0, i, q, None) == inv
    assert ebc.ebc_moe_route(h, p, 24, 0, 8, 24, 2, 2, None, 1, 1, 1, 1, 1.0, i, q, None) == inv
    assert ebc.ebc_moe_route(h, p, 24, 0, -1, 24, 2, 0, None, 1, 1, 1, 1, 1.0, i, q, None) == inv
    assert ebc.ebc_moe_route(h, p, 24, 0, 8, 24, 2, 0, p + 2, 1, 1, 1, 1, 1.0, i, q, None) == inv
    assert ebc.ebc_moe_route(h, p, 24, 0, 8, 24, 2, 0, None, 1, 1, 1, 1, 1.0, i + 2, q, None) == inv
    assert ebc.ebc_moe_route_grad(h, q, p, 24, 0, 8, 24, 2, None, 0, 1, 1.0, p, None) == inv
    assert ebc.ebc_moe_route_grad(h, q, p, 24, 0, 8, 24, 2, i, 0, 1, 1.0, None, None) == inv
    ex.check()
