"""Tokens sorted by expert and back: plan, dispatch, combine and both gradients
against definitions in 64 bits.

Tolerances.  Copies and the plan are exact.  A sum of m products held in fp32
is within m * 2^-23 * (sum of the magnitudes) of the exact one (each product
and each addition rounds by at most 2^-24 of a partial sum that the magnitudes
bound), and its rounding to the output's type adds half a unit of its last
place: 2^-24 (fp32), 2^-8 (bf16), 2^-11 (fp16) of the value, and at most 2^-25
absolutely where fp16 runs out of exponents."""
import numpy as np
import pytest
import torch

import error_bounded_lossy_gb300 as ebc

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

TYPES = [torch.float32, torch.bfloat16, torch.float16]
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def ex():
    e = ebc.Experts(0)
    yield e
    e.check()
    e.close()


def route(tokens, top, experts, drop, seed, dtype=np.int32, repeat=False):
    rng = np.random.default_rng(seed)
    if repeat or top > experts:
        ids = rng.integers(0, experts, (tokens, top))
    else:
        ids = rng.random((tokens, experts)).argsort(1)[:, :top]
    ids = np.where(rng.random((tokens, top)) < drop, -1 - rng.integers(0, 5, (tokens, top)), ids)
    return ids.astype(dtype)


def plan_of(ids, experts):
    flat = ids.reshape(-1).astype(np.int64)
    live = np.flatnonzero((flat >= 0) & (flat < experts))
    order = live[np.argsort(flat[live], kind="stable")]
    rows = np.full(flat.size, -1)
    rows[:order.size] = order
    place = np.full(flat.size, -1)
    place[order] = np.arange(order.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[live], minlength=experts))])
    return rows, place.reshape(ids.shape), offsets


def near(got, want, size, terms, dtype):
    """|got - want| within the bound above; size: the sum of the magnitudes."""
    want, size = want.double().cpu(), size.double().cpu()
    bound = terms * 2.0 ** -23 * size + UNIT[dtype] * (want.abs() + terms * 2.0 ** -23 * size)
    bound += 2.0 ** -25 if dtype == torch.float16 else 1e-37
    off = (got.double().cpu() - want).abs()
    assert bool((off <= bound).all()), f"{(off - bound).max()} over the bound"


SHAPES = [(0, 1, 1, 0.0), (1, 1, 1, 0.0), (1, 8, 64, 0.0), (3, 2, 5, 1.0), (33, 3, 7, 0.3), (512, 40, 9, 0.1),
          (1000, 4, 1024, 0.0), (4097, 1, 2, 0.5), (20011, 8, 256, 0.05)]


@pytest.mark.parametrize("tokens,top,experts,drop", SHAPES)
@pytest.mark.parametrize("dtype", [np.int32, np.int64])
def test_plan(ex, tokens, top, experts, drop, dtype):
    ids = route(tokens, top, experts, drop, tokens + top, dtype)
    p = ex.plan(torch.from_numpy(ids).cuda(), experts)
    rows, place, offsets = plan_of(ids, experts)
    assert np.array_equal(p.rows.cpu().numpy(), rows)
    assert np.array_equal(p.place.cpu().numpy(), place)
    assert np.array_equal(p.offsets.cpu().numpy(), offsets)


def test_plan_where_one_expert_takes_all(ex):
    ids = np.full((70000, 2), 3, np.int32)
    p = ex.plan(torch.from_numpy(ids).cuda(), 5)
    assert torch.equal(p.rows.cpu(), torch.arange(140000, dtype=torch.int32))
    assert p.offsets.tolist() == [0, 0, 0, 0, 140000, 140000]


@pytest.mark.parametrize("dtype,big", [(torch.int32, 2 ** 31 - 1), (torch.int64, 2 ** 40)])
def test_an_id_past_the_experts_is_dropped_and_recorded(dtype, big):
    e = ebc.Experts(0)
    ids = torch.tensor([[0, 4], [big, 1], [-5, 3]], dtype=dtype, device="cuda")
    p = e.plan(ids, 4)
    assert p.place.tolist() == [[0, -1], [-1, 1], [-1, 2]] and p.offsets.tolist() == [0, 1, 2, 2, 3]
    with pytest.raises(ebc.EbcError) as err:
        e.check()
    assert err.value.code == ebc.EBC_ERR_INVALID_ARG
    e.check()   # recorded once
    e.close()


WIDTHS = [1, 7, 8, 64, 1001, 1024, 2056]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("tokens,top,experts,drop", [(1, 8, 64, 0.0), (33, 3, 7, 0.3), (5, 2, 4, 1.0), (130, 40, 9, 0.1)])
def test_dispatch_and_back(ex, tokens, top, experts, drop, width, dtype):
    ids = route(tokens, top, experts, drop, width)
    plan = ex.plan(torch.from_numpy(ids).cuda(), experts)
    rows, place, offsets = plan_of(ids, experts)
    g = torch.Generator("cuda").manual_seed(width)
    x = torch.randn(tokens, width, generator=g, device="cuda").to(dtype)
    # a token without any expert may hold anything
    lost = torch.from_numpy((place < 0).all(1)).cuda()
    x[lost] = float("nan")
    xs = ex.dispatch(x, plan)
    live = int(offsets[-1])
    assert torch.equal(xs[:live], x[torch.from_numpy(rows[:live] // top).cuda()])
    assert not xs[live:].any()
    # the rows past the last expert's may hold anything on the way back
    ys = torch.randn(tokens * top, width, generator=g, device="cuda").to(dtype)
    ys[live:] = float("nan")
    w = torch.rand(tokens, top, generator=g, device="cuda") - 0.3
    w[torch.from_numpy(place < 0).cuda()] = float("inf")
    kept = torch.from_numpy(place >= 0).cuda()
    picked = torch.where(kept[..., None], ys.double()[torch.from_numpy(place).cuda().clamp(min=0)], 0.0)
    w64 = torch.where(kept, w.double(), 0.0)[..., None]
    near(ex.combine(ys, w, plan), (w64 * picked).sum(1), (w64 * picked).abs().sum(1), top + 1, dtype)
    near(ex.dispatch_grad(ys, plan), picked.sum(1), picked.abs().sum(1), top, dtype)
    dy = torch.randn(tokens, width, generator=g, device="cuda").to(dtype)
    dy[lost] = float("nan")
    dys, dw = ex.combine_grad(dy, ys, w, plan)
    slot = torch.from_numpy(rows[:live]).cuda()
    assert torch.equal(dys[:live], (w.reshape(-1)[slot][:, None] * dy.float()[slot // top]).to(dtype))
    assert not dys[live:].any()
    part = torch.where(kept[..., None], dy.double()[:, None, :] * picked, 0.0)
    near(dw, part.sum(2), part.abs().sum(2), width + 1, torch.float32)
    assert not dw[~kept].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (8, 1), (0, 2)])
def test_strided_and_unaligned_rows(ex, dtype, pad, shift):
    """Rows with a stride, and rows that start off a vector's boundary."""
    tokens, top, experts, width = 37, 3, 6, 264
    ids = route(tokens, top, experts, 0.2, 5)
    plan = ex.plan(torch.from_numpy(ids).cuda(), experts)

    def held(n):
        flat = torch.randn(n * (width + pad) + shift, device="cuda").to(dtype)
        return flat[shift:].view(n, width + pad)[:, :width]

    x, ys, dy = held(tokens), held(tokens * top), held(tokens)
    w = torch.rand(tokens, top, device="cuda")
    assert torch.equal(ex.dispatch(x, plan), ex.dispatch(x.clone().contiguous(), plan))
    assert torch.equal(ex.combine(ys, w, plan), ex.combine(ys.clone().contiguous(), w, plan))
    a, b = ex.combine_grad(dy, ys, w, plan), ex.combine_grad(dy.clone().contiguous(), ys.clone().contiguous(), w, plan)
    assert torch.equal(a[0], b[0])
    part = dy.double()[:, None, :] * torch.where((plan.place >= 0)[..., None], ys.double()[plan.place.clamp(min=0).long()], 0.0)
    near(a[1], part.sum(2), part.abs().sum(2), width + 1, torch.float32)
    near(b[1], part.sum(2), part.abs().sum(2), width + 1, torch.float32)


def test_gradients_against_differences(ex):
    """combine is linear in ys and in the weights, so a difference over any step
    is the derivative: f(a + d) - f(a - d) = 2 <gradient, d>.  Each value of y
    is within (top + 1) 2^-23 of its magnitudes, which the sums below bound."""
    tokens, top, experts, width = 29, 4, 6, 515
    ids = route(tokens, top, experts, 0.25, 11)
    plan = ex.plan(torch.from_numpy(ids).cuda(), experts)
    g = torch.Generator("cuda").manual_seed(3)
    n = tokens * top

    def grid(*shape):   # multiples of 2^-7 below 4: sums and differences of them are exact in fp32
        return torch.randint(-511, 512, shape, generator=g, device="cuda").float() / 128

    ys, d_ys, w, d_w, dy = grid(n, width), grid(n, width), grid(tokens, top), grid(tokens, top), grid(tokens, width)
    dys, dw = ex.combine_grad(dy, ys, w, plan)
    f = lambda a, b: float((ex.combine(a, b, plan).double() * dy.double()).sum())  # noqa: E731
    kept = (plan.place >= 0)[..., None]
    big = lambda a, b: float(((torch.where(kept, a.abs().double()[plan.place.clamp(min=0).long()], 0.0)  # noqa: E731
                               * b.abs().double()[..., None]).sum(1) * dy.abs().double()).sum())
    slack = (top + 2) * 2.0 ** -23
    live = int(plan.offsets[-1])
    got = f(ys + d_ys, w) - f(ys - d_ys, w)
    want = 2 * float((dys[:live].double() * d_ys[:live].double()).sum())
    assert abs(got - want) <= slack * 2 * big(ys.abs() + d_ys.abs(), w)
    got = f(ys, w + d_w) - f(ys, w - d_w)
    want = 2 * float((dw.double() * d_w.double()).sum())
    assert abs(got - want) <= (slack + width * 2.0 ** -23) * 2 * big(ys, w.abs() + d_w.abs())
    # dispatch: <dispatch(x), g> = <x, dispatch_grad(g)>
    x = grid(tokens, width)
    left = float((ex.dispatch(x, plan)[:live].double() * ys[:live].double()).sum())
    right = float((x.double() * ex.dispatch_grad(ys, plan).double()).sum())
    assert abs(left - right) <= slack * float((x.abs().double()[:, None] * torch.where(
        kept, ys.abs().double()[plan.place.clamp(min=0).long()], 0.0)).sum())


def test_rows_past_32_bits_of_elements(ex):
    """2^31 elements and more in the sending buffer."""
    tokens, top, experts, width = 70001, 4, 16, 8192
    ids = torch.from_numpy(route(tokens, top, experts, 0.0, 2)).cuda()
    plan = ex.plan(ids, experts)
    x = torch.randn(tokens, width, device="cuda").to(torch.bfloat16)
    xs = ex.dispatch(x, plan)
    for lo in range(0, tokens * top, 40000):
        at = slice(lo, min(lo + 40000, tokens * top))
        assert torch.equal(xs[at], x[plan.rows[at].long() // top])
    # every weight a quarter: the sum of four equal values, exactly
    assert torch.equal(ex.combine(xs, torch.full((tokens, top), 0.25, device="cuda"), plan), x)
    dys, dw = ex.combine_grad(x, xs, torch.ones(tokens, top, device="cuda"), plan)
    assert torch.equal(dys, xs)
    want = x.float().square().sum(1).double()
    assert bool(((dw.double() - want[:, None]).abs() <= 2e-3 * want[:, None]).all())


def test_the_same_bits_in_every_run_and_on_another_stream(ex):
    ids = torch.from_numpy(route(3001, 6, 32, 0.1, 8)).cuda()
    x = torch.randn(3001, 520, device="cuda").to(torch.bfloat16)
    w = torch.rand(3001, 6, device="cuda")
    dy = torch.randn(3001, 520, device="cuda").to(torch.bfloat16)

    def go(stream=None):
        plan = ex.plan(ids, 32, stream=stream)
        xs = ex.dispatch(x, plan, stream=stream)
        return (plan.rows, plan.place, plan.offsets, xs, ex.combine(xs, w, plan, stream=stream),
                *ex.combine_grad(dy, xs, w, plan, stream=stream))

    first = go()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, None, side):
        again = go(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    with torch.cuda.stream(side):
        again = go()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_in_a_cuda_graph(ex):
    ids = torch.from_numpy(route(64, 4, 8, 0.1, 8)).cuda()
    x = torch.randn(64, 256, device="cuda")
    w = torch.rand(64, 4, device="cuda")
    for _ in range(2):
        plan = ex.plan(ids, 8)
        ex.combine(ex.dispatch(x, plan), w, plan)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = ex.plan(ids, 8)
        y = ex.combine(ex.dispatch(x, plan), w, plan)
    ids.copy_(torch.from_numpy(route(64, 4, 8, 0.4, 9)).cuda())
    x.copy_(torch.randn(64, 256, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    p2 = ex.plan(ids, 8)
    assert torch.equal(y, ex.combine(ex.dispatch(x, p2), w, p2))


def test_a_plan_that_points_outside_is_skipped_and_recorded():
    e = ebc.Experts(0)
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = ebc.Plan(i([0, 1, 2, 3]), i([[0, 1], [2, 9]]), i([0, 2, 4]))
    x = torch.randn(2, 16, device="cuda")
    xs = e.dispatch(x, plan)
    assert torch.equal(xs[:3], x[[0, 0, 1]])
    with pytest.raises(ebc.EbcError):
        e.check()
    y = e.combine(x[[0, 0, 1, 1]], torch.ones(2, 2, device="cuda"), plan)
    assert torch.equal(y, torch.stack([x[0] + x[0], x[1]]))
    with pytest.raises(ebc.EbcError):
        e.check()
    e.combine_grad(x, x[[0, 0, 1, 1]], torch.ones(2, 2, device="cuda"), plan)
    with pytest.raises(ebc.EbcError):
        e.check()
    e.close()


def test_refusals(ex):
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    plan = ex.plan(ids, 3)
    x = torch.zeros(4, 8, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    for bad in (0, -1, ebc.EBC_MAX_EXPERTS + 1):
        with pytest.raises(ebc.EbcError):
            ex.plan(ids, bad)
    for bad in (ids.float(), ids.view(-1), torch.zeros(2, 4, dtype=torch.int32, device="cuda").t(), ids.cpu()):
        with pytest.raises(ValueError):
            ex.plan(bad, 3)
    for bad in (x.double(), x[:3], x.cpu(), torch.zeros(8, 4, device="cuda").t()):
        with pytest.raises(ValueError):
            ex.dispatch(bad, plan)
        with pytest.raises(ValueError):
            ex.dispatch_mx4(bad, plan)
    with pytest.raises(ebc.EbcError):
        ex.dispatch(torch.zeros(4, 0, device="cuda"), plan)
    ys = torch.zeros(8, 8, device="cuda")
    for bad in (ys[:7], ys.double(), ys.cpu()):
        with pytest.raises(ValueError):
            ex.combine(bad, w, plan)
    for bad in (w.double(), w[:3], w.cpu(), torch.zeros(2, 4, device="cuda").t()):
        with pytest.raises(ValueError):
            ex.combine(ys, bad, plan)
        with pytest.raises(ValueError):
            ex.combine_grad(x, ys, bad, plan)
    for dy, y in ((x.half(), ys), (x[:3], ys), (x, ys[:7]), (x, ys[:, :7])):
        with pytest.raises(ValueError):
            ex.combine_grad(dy, y, w, plan)
    h, s = ex.handle, None
    a = plan.place.data_ptr()
    inv = ebc.EBC_ERR_INVALID_ARG
    assert ebc.ebc_moe_plan(h, a, 3, 4, 2, 3, a, a, a, s) == inv            # id size
    assert ebc.ebc_moe_plan(h, a, 4, -1, 2, 3, a, a, a, s) == inv           # tokens
    assert ebc.ebc_moe_plan(h, a, 4, 2 ** 30, 2, 3, a, a, a, s) == inv      # 2^31 slots
    assert ebc.ebc_moe_plan(h, a, 4, 4, 0, 3, a, a, a, s) == inv            # top
    assert ebc.ebc_moe_plan(h, None, 4, 4, 2, 3, a, a, a, s) == inv
    assert ebc.ebc_moe_plan(h, a, 4, 4, 2, 3, a, a, None, s) == inv
    assert ebc.ebc_moe_plan(h, a + 2, 4, 4, 2, 3, a, a, a, s) == inv        # alignment
    d = x.data_ptr()
    assert ebc.ebc_moe_dispatch(h, d, 8, 3, 4, 2, 8, a, a, 3, d, s) == inv  # type
    assert ebc.ebc_moe_dispatch(h, d, 7, 0, 4, 2, 8, a, a, 3, d, s) == inv  # row stride below the width
    assert ebc.ebc_moe_dispatch(h, d + 2, 8, 0, 4, 2, 8, a, a, 3, d, s) == inv
    assert ebc.ebc_moe_dispatch(h, d, 8, 0, 4, 2, 8, a, a, 3, None, s) == inv
    assert ebc.ebc_moe_combine(h, d, 8, 0, 4, 2, 0, a, None, d, s) == inv
    assert ebc.ebc_moe_combine(h, d, 8, 0, 4, 2, 8, a, d + 1, d, s) == inv
    assert ebc.ebc_moe_combine(h, d, 8, 0, 4, 2, 8, None, None, d, s) == inv
    assert ebc.ebc_moe_combine_grad(h, d, 8, d, 8, 0, 4, 2, 8, a, a, 3, None, d, d, s) == inv
    assert ebc.ebc_moe_combine_grad(h, d, 8, d, 8, 0, 4, 2, 8, a, None, 3, d, d, d, s) == inv
    ex.check()
