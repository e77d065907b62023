"""4-bit microscaled values: codes and scales against a search over the
sixteen values in 64 bits, the error bound, and the experts' products.

Codes, scales and read-back values are exact.  A product sums `width` exact
products in 32 bits: whatever the order, it is within width * 2^-23 of the sum
of the magnitudes (every partial sum is below that sum, and an addition loses
at most one unit in the last place, 2^-23, also where a matrix unit truncates
instead of rounding); rounding to the output's type adds 2^-24, 2^-8 or 2^-11
of the value, and at most 2^-25 absolutely where fp16 runs out of exponents."""
import numpy as np
import pytest
import torch

import error_bounded_lossy_gb300 as ebc

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

TYPES = [torch.float32, torch.bfloat16, torch.float16]
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


@pytest.fixture(scope="module")
def ex():
    e = ebc.Experts(0)
    yield e
    e.check()
    e.close()


def encode(x):
    """(codes [n, padded] one a byte, scales [n, blocks], values [n, padded]) of x [n, k] by search, in 64 bits."""
    n, k = x.shape
    full = np.zeros((n, -(-k // 32) * 32))
    full[:, :k] = x
    sign = np.zeros(full.shape, bool)
    sign[:, :k] = np.signbit(x)
    b = full.reshape(n, -1, 32)
    top = np.abs(b).max(2)
    scales = np.full(top.shape, 255)
    fine = np.isfinite(top)
    for e in range(126, -128, -1):   # the least e that holds the block
        scales[fine & (top <= 6.0 * 2.0 ** e)] = e + 127
    unit = np.where(fine, 2.0 ** (np.where(fine, scales, 127) - 127.0), np.nan)
    with np.errstate(invalid="ignore"):
        v = np.abs(b) / unit[..., None]
        d = np.abs(v[..., None] - VALUES)
        best = d.min(-1, keepdims=True)
        even = (d == best) & (np.arange(8) % 2 == 0)
        code = np.where(even.any(-1), even.argmax(-1), (d == best).argmax(-1))
    code = code + 8 * sign.reshape(b.shape)
    code[~fine] = 0
    values = np.where(code >= 8, -1.0, 1.0) * VALUES[code % 8] * unit[..., None]
    return code.reshape(n, -1), scales, values.reshape(n, -1)


def unpack(q):
    c = q.codes.cpu().numpy()
    return np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)


def special(width, seed, dtype):
    """Rows that reach every case of the rounding: plain values, every exponent, exact ties, blocks whose largest
    value sits at a scale's edge, zeros of both signs, subnormals, infinities and NaN."""
    rng = np.random.default_rng(seed)
    rows = [rng.standard_normal(width) for _ in range(6)]
    lo, hi = (-24, 15) if dtype == torch.float16 else (-140, 127)
    rows.append(np.ldexp(1 + rng.random(width), rng.integers(lo, hi, width)))
    ties = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, -0.0], width) * rng.choice([-1, 1], width)
    rows += [ties, ties * 2.0 ** -5, ties * (2.0 ** 3)]
    edge = rng.standard_normal(width) * 0.1
    edge[::32] = rng.choice([6.0, 6.0 + 2 ** -5, 8.0, 7.96875, 4.0, 3.0, 3.015625], edge[::32].shape)
    rows.append(edge)
    rows += [np.zeros(width), -np.zeros(width)]
    if dtype != torch.float16:
        rows += [rng.standard_normal(width) * 2.0 ** -135, rng.standard_normal(width) * 1e-45]
    big = rng.standard_normal(width)
    big[0] = 65504.0 if dtype == torch.float16 else 3e38
    rows.append(big)
    for bad in (np.inf, -np.inf, np.nan):
        r = rng.standard_normal(width)
        r[rng.integers(0, width)] = bad
        rows.append(r)
    with np.errstate(over="ignore"):
        return torch.from_numpy(np.array(rows)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [1, 31, 32, 40, 64, 100, 128, 129, 264, 301, 512, 1000, 1056])
def test_codes_scales_and_values(ex, width, dtype):
    x = special(width, width, dtype)
    code, scale, values = encode(x.double().cpu().numpy())
    q = ex.quantize(x)
    assert np.array_equal(unpack(q), code)
    got = q.scales.cpu().numpy()
    assert np.array_equal(got[:, :scale.shape[1]], scale) and not got[:, scale.shape[1]:].any()
    for out in TYPES:
        back = ex.dequantize(q, out)
        assert torch.equal(back.nan_to_num(nan=1234.0), torch.from_numpy(values[:, :width]).to(out).cuda().nan_to_num(nan=1234.0))


@pytest.mark.parametrize("dtype", TYPES)
def test_the_error_bound(ex, dtype):
    x = (torch.randn(300, 1000, device="cuda") * torch.exp2(torch.randint(-9, 9, (300, 1), device="cuda").float())).to(dtype)
    q = ex.quantize(x)
    unit = torch.exp2(q.scales[:, :32].double() - 127).repeat_interleave(32, 1)[:, :1000]
    off = (ex.dequantize(q).double() - x.double()).abs()
    v = x.double().abs() / unit
    assert bool((v <= 6).all())
    assert bool((off <= unit * torch.where(v <= 2, 0.25, torch.where(v <= 4, 0.5, 1.0))).all())


def test_the_top_of_the_range(ex):
    """The bound holds up to the value whose nearest is the first past fp32's range, and the products take that one as
    what it stands for."""
    edge = np.float32(3.5 * 2.0 ** 126)
    below = np.nextafter(edge, np.float32(0))
    x = torch.zeros(4, 32, device="cuda")
    x[:, 5] = torch.tensor([below, -below, edge, torch.finfo(torch.float32).max], device="cuda")
    q = ex.quantize(x)
    assert q.scales[:, 0].tolist() == [253] * 4
    for dtype in (torch.float32, torch.bfloat16):
        back = ex.dequantize(q, dtype)[:, 5].double().cpu()
        assert back.tolist() == [3 * 2.0 ** 126, -3 * 2.0 ** 126, np.inf, np.inf]
    assert abs(3 * 2.0 ** 126 - float(below)) <= 2.0 ** 126
    w = ex.quantize(torch.full((1, 32), 2.0 ** -8, device="cuda"))
    assert ex.product(q, w, dtype=torch.float32)[:, 0].tolist() == [3 * 2.0 ** 118, -3 * 2.0 ** 118, 2.0 ** 120, 2.0 ** 120]
    half = torch.tensor([[57312.0] + [0.0] * 31, [57344.0] + [0.0] * 31, [65504.0] + [0.0] * 31], device="cuda").half()
    assert ex.dequantize(ex.quantize(half), torch.float16)[:, 0].tolist() == [49152.0, np.inf, np.inf]
    assert ex.dequantize(ex.quantize(half))[:, 0].tolist() == [49152.0, 65536.0, 65536.0]


def test_leading_shapes_strides_and_nothing(ex):
    x = torch.randn(5, 6, 96, device="cuda").to(torch.bfloat16)
    q = ex.quantize(x)
    assert q.shape == (5, 6, 96) and torch.equal(ex.dequantize(q)[3], ex.dequantize(ex.quantize(x[3])))
    wide = torch.randn(9, 203, device="cuda")
    for at in (slice(0, 64), slice(1, 65), slice(4, 133)):
        assert torch.equal(ex.quantize(wide[:, at]).codes, ex.quantize(wide[:, at].clone().contiguous()).codes)
    assert ex.dequantize(ex.quantize(torch.zeros(0, 64, device="cuda"))).shape == (0, 64)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,top,experts,width,drop", [(1, 8, 64, 512, 0.0), (37, 3, 5, 1000, 0.3), (6, 2, 3, 40, 1.0), (500, 3, 7, 96, 0.2), (77, 2, 7, 31, 0.5), (300, 2, 4, 333, 0.1)])
def test_dispatch_in_4_bits(ex, tokens, top, experts, width, drop, dtype):
    rng = np.random.default_rng(1)
    ids = rng.integers(0, experts, (tokens, top))
    ids[rng.random(ids.shape) < drop] = -1
    plan = ex.plan(torch.from_numpy(ids).cuda(), experts)
    x = torch.randn(tokens, width, device="cuda").to(dtype)
    got, want = ex.dispatch_mx4(x, plan), ex.quantize(ex.dispatch(x, plan))
    assert torch.equal(got.codes, want.codes)
    live = int(plan.offsets[-1])
    assert torch.equal(got.scales[:live], want.scales[:live])
    assert not ex.dequantize(got)[live:].any()


def case(ex, rows, experts, outs, width, seed, cut=None):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(rows, width, generator=g, device="cuda")
    w = torch.randn(experts, outs, width, generator=g, device="cuda")
    if cut is None:
        rng = np.random.default_rng(seed)
        cut = np.concatenate([[0], np.sort(rng.integers(0, rows + 1, experts - 1)), [rows]])
    return ex.quantize(x), ex.quantize(w), torch.tensor(cut, dtype=torch.int32, device="cuda")


def check_product(ex, x, w, offsets, dtype, ys=None):
    ys = ex.product(x, w, offsets, dtype) if ys is None else ys
    xv, wv = ex.dequantize(x).double(), ex.dequantize(w).double()
    cut = offsets.tolist()
    assert not ys[:cut[0]].any() and not ys[cut[-1]:].any()
    for e in range(len(cut) - 1):
        at = slice(cut[e], cut[e + 1])
        want = xv[at] @ wv[e].T
        size = xv[at].abs() @ wv[e].abs().T
        lost = x.width * 2.0 ** -23 * size
        bound = lost + UNIT[dtype] * (want.abs() + lost) + (2.0 ** -25 if dtype == torch.float16 else 1e-37)
        off = (ys[at].double() - want).abs()
        assert bool((off <= bound).all()), (e, float((off - bound).max()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,experts,outs,width", [
    (1, 1, 1, 1), (1, 1, 128, 64), (1, 3, 200, 33), (7, 4, 129, 96), (16, 2, 256, 256), (33, 5, 8, 32),
    (65, 3, 127, 160), (128, 1, 128, 512), (130, 2, 300, 544), (257, 3, 513, 1056), (600, 9, 136, 2048),
    (1000, 2, 96, 4128)])
def test_product(ex, rows, experts, outs, width, dtype):
    x, w, offsets = case(ex, rows, experts, outs, width, rows + outs)
    check_product(ex, x, w, offsets, dtype)


@pytest.mark.parametrize("rows,experts,outs,width", [
    (4000, 3, 4000, 800), (5000, 7, 2056, 2592), (3001, 1, 3999, 4192), (2500, 2, 2500, 8480), (9000, 40, 1300, 1056)])
def test_product_of_many_tiles(ex, rows, experts, outs, width):
    """Large tiles, several of them one after the other, long sums of every number of stages."""
    x, w, offsets = case(ex, rows, experts, outs, width, rows + outs)
    for dtype in TYPES:
        check_product(ex, x, w, offsets, dtype)


@pytest.mark.parametrize("rows,experts,outs,width", [
    (1, 1, 1024, 16384), (3, 1, 130, 1024), (1, 2, 500, 2080), (17, 1, 1024, 4096), (40, 2, 300, 3104), (100, 1, 200, 1568),
    (5, 3, 128, 544), (128, 1, 64, 9000)])
def test_product_of_few_tiles(ex, rows, experts, outs, width):
    """Few tiles and long sums, which several CTAs share."""
    for cut in (None, [0] * experts + [rows], [0] * experts + [rows // 2]):
        x, w, offsets = case(ex, rows, experts, outs, width, rows + outs, cut)
        for dtype in TYPES:
            check_product(ex, x, w, offsets, dtype)
        assert torch.equal(ex.product(x, w, offsets), ex.product(x, w, offsets))


@pytest.mark.parametrize("rows,experts", [(5, 1024), (3000, 700), (40, 64)])
def test_product_of_many_experts(ex, rows, experts):
    x, w, offsets = case(ex, rows, experts, 40, 64, rows)
    check_product(ex, x, w, offsets, torch.float32)


@pytest.mark.parametrize("cut", [[0, 0, 0, 50], [0, 50, 50, 50], [0, 0, 0, 0], [0, 3, 3, 20], [0, 17, 34, 49]])
def test_product_of_empty_segments_and_rows_of_no_expert(ex, cut):
    x, w, offsets = case(ex, 50, 3, 70, 128, 4, cut)
    check_product(ex, x, w, offsets, torch.bfloat16)


def test_product_of_one_matrix(ex):
    x, w, _ = case(ex, 77, 1, 130, 320, 5)
    flat = ebc.Mx4(w.codes[0], w.scales[0], w.width)
    ys = ex.product(x, flat, dtype=torch.float32)
    check_product(ex, x, w, torch.tensor([0, 77], dtype=torch.int32), torch.float32, ys)
    assert ex.product(ex.quantize(torch.zeros(0, 320, device="cuda")), flat).shape == (0, 130)


@pytest.mark.parametrize("rows,outs,width", [(4, 130, 64), (200, 300, 1000)])
def test_a_nan_stays_in_its_row_and_in_its_output(ex, rows, outs, width):
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(rows, width, generator=g, device="cuda")
    w = torch.randn(2, outs, width, generator=g, device="cuda")
    x[rows // 2, width - 1] = float("inf")
    w[1, outs - 1, 0] = float("nan")
    cut = [0, rows // 4, rows]
    ys = ex.product(ex.quantize(x), ex.quantize(w), torch.tensor(cut, dtype=torch.int32, device="cuda"), torch.float32)
    want = torch.zeros(rows, outs, dtype=torch.bool)
    want[rows // 2] = True
    want[cut[1]:, outs - 1] = True
    assert torch.equal(ys.isnan().cpu(), want)


def test_scales_of_every_size(ex):
    """Blocks from the smallest scale to large ones: products are exact, so one block's product is exact too."""
    width, rows, outs = 64, 130, 140
    rng = np.random.default_rng(0)
    x = rng.choice([-6.0, -1.5, 0.5, 3.0], (rows, width)) * 2.0 ** rng.integers(-50, 50, (rows, 1))
    w = rng.choice([-6.0, -2.0, 1.0, 4.0], (1, outs, width)) * 2.0 ** rng.integers(-50, 50, (1, outs, 1))
    q = ex.quantize(torch.from_numpy(x).float().cuda())
    p = ex.quantize(torch.from_numpy(w).float().cuda())
    ys = ex.product(q, p, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), torch.float32)
    want = torch.from_numpy((ex.dequantize(q).double().cpu().numpy() @ ex.dequantize(p)[0].double().cpu().numpy().T)).float()
    assert torch.equal(ys.cpu(), want)


def test_padding_bytes_of_the_scales_are_not_read(ex):
    x, w, offsets = case(ex, 60, 2, 140, 96, 9)
    ys = ex.product(x, w, offsets)
    x.scales[..., 3:] = 255
    w.scales[..., 3:] = 255
    assert torch.equal(ex.product(x, w, offsets), ys)


def test_rows_past_32_bits_of_outputs(ex):
    rows, outs, width = 70000, 32768, 32
    x = ex.quantize(torch.randn(rows, width, device="cuda"))
    w = ex.quantize(torch.randn(1, outs, width, device="cuda"))
    ys = ex.product(x, w, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), torch.bfloat16)
    for at in (slice(0, 300), slice(65400, 65700), slice(rows - 300, rows)):
        part = ebc.Mx4(x.codes[at], x.scales[at], width)
        check_product(ex, part, w, torch.tensor([0, 300]), torch.bfloat16, ys[at])


def test_as_many_rows_as_a_product_takes(ex):
    """Segments that end at 2^31 - 256 rows: the first, the last and some in between."""
    rows, width = 2 ** 31 - 256, 32
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB")
    x = ebc.Mx4(*(torch.zeros(rows, 16, dtype=torch.uint8, device="cuda") for _ in range(2)), width)
    w = ex.quantize(torch.ones(2, 1, width, device="cuda") * torch.tensor([1.0, 2.0], device="cuda")[:, None, None])
    x.scales[:, 0] = 127
    at = torch.tensor([0, 1, 127, 255, 2 ** 30 - 1, 2 ** 30, 2 ** 31 - 513, 2 ** 31 - 512, 2 ** 31 - 258, 2 ** 31 - 257], device="cuda")
    x.codes[at, 0] = 0x62   # 1 and 4
    want = torch.zeros(rows, 1, dtype=torch.float16, device="cuda")
    for cut in ([0, 0, rows], [0, rows, rows], [0, 2 ** 30, rows]):
        offsets = torch.tensor(cut, dtype=torch.int32, device="cuda")
        ys = ex.product(x, w, offsets, torch.float16)
        ex.check()
        want[at] = torch.where(at < cut[1], 5.0, 10.0).half()[:, None]
        assert torch.equal(ys, want)
        del ys


def test_the_same_bits_in_every_run_and_on_another_stream(ex):
    x, w, offsets = case(ex, 700, 6, 520, 2080, 12)
    first = ex.product(x, w, offsets)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, None, side):
        again = ex.product(x, w, offsets, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(first, again)


@pytest.mark.parametrize("cut", [[1, 20, 50], [0, 30, 20], [0, 20, 51], [0, -1, 50], [-3, 5, 50]])
def test_offsets_that_do_not_ascend_inside_the_rows_are_recorded(cut):
    e = ebc.Experts(0)
    x, w, offsets = case(e, 50, 2, 70, 128, 4, cut)
    e.check()
    ys = e.product(x, w, offsets, torch.float32)
    with pytest.raises(ebc.EbcError) as err:
        e.check()
    assert err.value.code == ebc.EBC_ERR_INVALID_ARG
    at = np.maximum.accumulate(np.clip([0, *cut[1:]], 0, 50))
    check_product(e, x, w, torch.tensor(at), torch.float32, ys)
    e.close()


@pytest.mark.parametrize("rows,experts,outs,width", [(16, 8, 2000, 2048), (6000, 4, 4000, 1024), (2, 1, 600, 8192)])
def test_a_wait_that_runs_out_is_recorded_and_the_context_recovers(rows, experts, outs, width):
    """Single CTAs, pairs and clusters that share K: the first stage's wait gives up at once; every CTA ends, the
    status says so, and the next product is right."""
    e = ebc.Experts(0)
    x, w, offsets = case(e, rows, experts, outs, width, 3)
    assert ebc.ebc_set_first_wait_polls(e.handle, 0) == 0
    e.product(x, w, offsets)
    with pytest.raises(ebc.EbcError) as err:
        e.check()
    assert err.value.code == ebc.EBC_ERR_DEVICE_TIMEOUT
    assert ebc.ebc_set_first_wait_polls(e.handle, -1) == 0
    check_product(e, x, w, offsets, torch.bfloat16)
    e.check()
    e.close()


def test_refusals(ex):
    x, w, offsets = case(ex, 8, 2, 16, 64, 1)
    with pytest.raises(ValueError):
        ex.product(x, ex.quantize(torch.zeros(2, 16, 96, device="cuda")), offsets)
    with pytest.raises(ValueError):
        ex.product(x, w)
    with pytest.raises(ValueError):
        ex.product(x, w, offsets.long())
    with pytest.raises(ValueError):
        ex.product(x, w, offsets[:2])
    with pytest.raises(ValueError):
        ex.product(x, w, offsets, torch.float64)
    with pytest.raises(ValueError):
        ex.dequantize(x, torch.int32)
    with pytest.raises(ValueError):
        ex.quantize(torch.zeros(4, 64, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        ex.quantize(torch.zeros(4, 64))
    h = ex.handle
    c, s, o, y = (t.data_ptr() for t in (x.codes, x.scales, offsets, torch.empty(8, 16, device="cuda")))
    inv = ebc.EBC_ERR_INVALID_ARG
    assert ebc.ebc_mx4_product(h, c, s, -1, 64, c, s, 16, 2, o, 0, y, None) == inv
    assert ebc.ebc_mx4_product(h, c, s, 8, 0, c, s, 16, 2, o, 0, y, None) == inv
    assert ebc.ebc_mx4_product(h, c, s, 8, 64, c, s, 0, 2, o, 0, y, None) == inv
    assert ebc.ebc_mx4_product(h, c, s, 8, 64, c, s, 16, 0, o, 0, y, None) == inv
    assert ebc.ebc_mx4_product(h, c, s, 8, 64, c, s, 16, 1025, o, 0, y, None) == inv
    assert ebc.ebc_mx4_product(h, c, s, 8, 64, c, s, 2 ** 31 - 1, 2, o, 0, y, None) == inv
    assert ebc.ebc_mx4_product(h, c, s, 8, 64, c, s, 16, 2, None, 0, y, None) == inv
    assert ebc.ebc_mx4_product(h, c, s, 8, 64, c, s, 16, 2, o, 3, y, None) == inv
    assert ebc.ebc_mx4_product(h, c + 8, s, 8, 64, c, s, 16, 2, o, 0, y, None) == inv
    assert ebc.ebc_mx4_product(h, c, s, 8, 64, c, s, 16, 2, o, 0, y + 2, None) == inv
    assert ebc.ebc_mx4_quantize(h, y, 64, 0, 2, 0, c, s, None) == inv
    assert ebc.ebc_mx4_quantize(h, y, 63, 0, 2, 64, c, s, None) == inv
    assert ebc.ebc_mx4_quantize(h, y, 64, 9, 2, 64, c, s, None) == inv
    assert ebc.ebc_mx4_quantize(h, y, 64, 0, 2, 64, c + 4, s, None) == inv
    assert ebc.ebc_mx4_quantize(h, y, 2 ** 25, 0, 2, 2 ** 25, c, s, None) == inv
    assert ebc.ebc_mx4_dequantize(h, c, s, 2, 64, 7, y, None) == inv
    assert ebc.ebc_mx4_dequantize(h, None, s, 2, 64, 0, y, None) == inv
    assert ebc.ebc_moe_dispatch_mx4(h, y, 64, 0, 2, 0, 64, o, o, 2, c, s, None) == inv
    assert ebc.ebc_moe_dispatch_mx4(h, y, 64, 0, 2, 1, 64, None, o, 2, c, s, None) == inv
    ex.check()
