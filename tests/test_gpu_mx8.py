"""8-bit microscaled values: codes and scales against a search over the 256
codes in 64 bits, the error bound, dispatch of such rows, and the experts'
products.

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
# E4M3: sign, 4 exponent bits (bias 7, 0: subnormal), 3 fraction bits; 127 would be a NaN
FIELD, FRAC = np.arange(127) >> 3, np.arange(127) & 7
VALUES = np.where(FIELD == 0, FRAC * 2.0 ** -9, (8.0 + FRAC) * 2.0 ** (FIELD - 10.0))


@pytest.fixture(scope="module")
def ex():
    e = ebc.Experts(0)
    yield e
    e.check()
    e.close()


def encode(x):
    """(codes [n, padded], scales [n, blocks], values [n, padded]) of x [n, k] by search, in 64 bits."""
    n, k = x.shape
    full = np.zeros((n, -(-k // 32) * 32))
    full[:, :k] = x
    sign = np.zeros(full.shape, bool)
    sign[:, :k] = np.signbit(x)
    b = full.reshape(n, -1, 32)
    top = np.abs(b).max(2)
    scales = np.full(top.shape, 255)
    fine = np.isfinite(top)
    for e in range(120, -128, -1):   # the least e that holds the block
        scales[fine & (top <= 448.0 * 2.0 ** e)] = e + 127
    unit = np.where(fine, 2.0 ** (np.where(fine, scales, 127) - 127.0), np.nan)
    with np.errstate(invalid="ignore"):
        v = np.where(fine[..., None], np.abs(b) / unit[..., None], 0.0)
    above = np.minimum(np.searchsorted(VALUES, v), 126)
    below = np.maximum(above - 1, 0)
    to_above, to_below = VALUES[above] - v, v - VALUES[below]
    code = np.where((to_above < to_below) | ((to_above == to_below) & (above % 2 == 0)), above, below)
    code = code + 128 * sign.reshape(b.shape)
    code[~fine] = 0
    values = np.where(code >= 128, -1.0, 1.0) * VALUES[code % 128] * unit[..., None]
    return code.reshape(n, -1), scales, values.reshape(n, -1)


def special(width, seed, dtype):
    """Rows that reach every case of the rounding: plain values, every exponent, exact ties, blocks whose largest
    value sits at a scale's edge, zeros of both signs, subnormals, infinities and NaN."""
    rng = np.random.default_rng(seed)
    rows = [rng.standard_normal(width) for _ in range(6)]
    lo, hi = (-24, 15) if dtype == torch.float16 else (-140, 126)
    rows.append(np.ldexp(1 + rng.random(width), rng.integers(lo, hi, width)))
    middles = np.concatenate([(VALUES[1:] + VALUES[:-1]) / 2, [448.0, 0.0, -0.0]])
    ties = rng.choice(middles, width) * rng.choice([-1, 1], width)
    ties[::32] = 448.0
    rows += [ties, ties * 2.0 ** -5, ties * 2.0 ** 3]
    edge = rng.standard_normal(width) * 0.1
    edge[::32] = rng.choice([448.0, 449.0, 450.0, 512.0, 511.5, 256.0, 224.0, 224.25, 447.75], edge[::32].shape)
    rows.append(edge)
    rows += [np.zeros(width), -np.zeros(width)]
    if dtype != torch.float16:
        rows += [rng.standard_normal(width) * 2.0 ** -135, rng.standard_normal(width) * 1e-45,
                 rng.standard_normal(width) * 2.0 ** -119]
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
@pytest.mark.parametrize("width", [1, 2, 31, 32, 40, 64, 100, 128, 129, 264, 301, 512, 1000, 1056, 2050])
def test_codes_scales_and_values(ex, width, dtype):
    x = special(width, width, dtype)
    code, scale, values = encode(x.double().cpu().numpy())
    q = ex.quantize_mx8(x)
    assert np.array_equal(q.codes.cpu().numpy(), code)
    got = q.scales.cpu().numpy()
    assert np.array_equal(got[:, :scale.shape[1]], scale) and not got[:, scale.shape[1]:].any()
    for out in TYPES:
        back = ex.dequantize(q, out)
        assert torch.equal(back.nan_to_num(nan=1234.0), torch.from_numpy(values[:, :width]).to(out).cuda().nan_to_num(nan=1234.0))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", [(300, 1000), (20000, 64), (4000, 4096), (1, 100000), (3001, 1001)])
def test_the_error_bound(ex, rows, width, dtype):
    x = (torch.randn(rows, width, device="cuda") * torch.exp2(torch.randint(-9, 9, (rows, 1), device="cuda").float())).to(dtype)
    q = ex.quantize_mx8(x)
    blocks = -(-width // 32)
    unit = (q.scales[:, :blocks].int() << 23).view(torch.float32).double().repeat_interleave(32, 1)[:, :width]
    off = (ex.dequantize(q).double() - x.double()).abs()
    assert bool((x.double().abs() <= 448 * unit).all())
    assert bool((off <= torch.maximum(x.double().abs() / 16, unit / 1024)).all())
    top = torch.nn.functional.pad(x.double().abs(), (0, blocks * 32 - width)).view(rows, blocks, 32).amax(2)
    assert bool((top > 224 * unit[:, ::32]).all())   # the least such scale


def test_the_top_of_the_range(ex):
    """The nearest value of 1.9375 * 2^127 and more is 2^128: infinity where it is read back, itself in a product."""
    edge = np.float32(1.9375 * 2.0 ** 127)
    below = np.nextafter(edge, np.float32(0))
    x = torch.zeros(4, 32, device="cuda")
    x[:, 5] = torch.tensor([below, -below, edge, torch.finfo(torch.float32).max], device="cuda")
    q = ex.quantize_mx8(x)
    assert q.scales[:, 0].tolist() == [247] * 4
    for dtype in (torch.float32, torch.bfloat16):
        assert ex.dequantize(q, dtype)[:, 5].double().tolist() == [1.875 * 2.0 ** 127, -1.875 * 2.0 ** 127, np.inf, np.inf]
    w = ex.quantize_mx8(torch.full((1, 32), 2.0 ** -8, device="cuda"))
    assert ex.product(q, w, dtype=torch.float32)[:, 0].tolist() == [1.875 * 2.0 ** 119, -1.875 * 2.0 ** 119, 2.0 ** 120, 2.0 ** 120]


def test_leading_shapes_strides_and_nothing(ex):
    x = torch.randn(5, 6, 96, device="cuda").to(torch.bfloat16)
    q = ex.quantize_mx8(x)
    assert q.shape == (5, 6, 96) and torch.equal(ex.dequantize(q)[3], ex.dequantize(ex.quantize_mx8(x[3])))
    wide = torch.randn(9, 203, device="cuda")
    for at in (slice(0, 64), slice(1, 65), slice(2, 100), slice(4, 133), slice(8, 200)):
        a, b = ex.quantize_mx8(wide[:, at]), ex.quantize_mx8(wide[:, at].clone().contiguous())
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    assert ex.dequantize(ex.quantize_mx8(torch.zeros(0, 64, device="cuda"))).shape == (0, 64)


def test_more_values_than_31_bits(ex):
    rows, width = 66000, 32800
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, 65471, 65472, 65536, rows - 1]
    x[at] = torch.randn(len(at), width, device="cuda").to(torch.bfloat16)
    q, part = ex.quantize_mx8(x), ex.quantize_mx8(x[at])
    assert torch.equal(q.codes[at], part.codes) and torch.equal(q.scales[at], part.scales)
    back = ex.dequantize(q, torch.bfloat16)
    assert torch.equal(back[at], ex.dequantize(part, torch.bfloat16))
    back[at] = 0
    assert not back.any()
    odd = x.view(-1)[:65500 * 32797].view(65500, 32797)   # rows off any vector's boundary, a lane a value
    q = ex.quantize_mx8(odd)
    for i in (0, 65499):
        assert torch.equal(q.codes[i], ex.quantize_mx8(odd[i:i + 1].clone()).codes[0])


@pytest.mark.parametrize("quantize", ["quantize", "quantize_mx8"])
@pytest.mark.parametrize("tokens,top,experts,width,drop", [(1, 8, 64, 512, 0.0), (37, 3, 5, 1000, 0.3), (6, 2, 3, 40, 1.0), (500, 3, 7, 96, 0.2), (77, 2, 7, 31, 0.5), (300, 40, 60, 5000, 0.1)])
def test_dispatch_of_rows_in_few_bits(ex, tokens, top, experts, width, drop, quantize):
    rng = np.random.default_rng(1)
    ids = rng.integers(0, experts, (tokens, top))
    ids[rng.random(ids.shape) < drop] = -1
    plan = ex.plan(torch.from_numpy(ids).cuda(), experts)
    q = getattr(ex, quantize)(torch.randn(tokens, width, device="cuda"))
    got = ex.dispatch(q, plan)
    assert type(got) is type(q) and got.shape == (tokens * top, width)
    slot = plan.rows.long().clamp(min=0) // top
    live = (plan.rows >= 0)[:, None]
    assert torch.equal(got.codes, torch.where(live, q.codes[slot], 0)) and torch.equal(got.scales, torch.where(live, q.scales[slot], 0))
    again = ex.dispatch(q, plan, stream=torch.cuda.current_stream())
    assert torch.equal(again.codes, got.codes) and torch.equal(again.scales, got.scales)


def case(ex, rows, experts, outs, width, seed, cut=None):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(rows, width, generator=g, device="cuda")
    w = torch.randn(experts, outs, width, generator=g, device="cuda")
    if cut is None:
        rng = np.random.default_rng(seed)
        cut = np.concatenate([[0], np.sort(rng.integers(0, rows + 1, experts - 1)), [rows]])
    return ex.quantize_mx8(x), ex.quantize_mx8(w), torch.tensor(cut, dtype=torch.int32, device="cuda")


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
    (1000, 2, 96, 4128), (50, 2, 70, 1001)])
def test_product(ex, rows, experts, outs, width, dtype):
    x, w, offsets = case(ex, rows, experts, outs, width, rows + outs)
    check_product(ex, x, w, offsets, dtype)


@pytest.mark.parametrize("rows,experts,outs,width", [
    (4000, 3, 4000, 800), (5000, 7, 2056, 2592), (3001, 1, 3999, 4192), (2500, 2, 2500, 8480), (9000, 40, 1300, 1056),
    (6000, 2, 4096, 32), (6000, 2, 4096, 160)])
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


@pytest.mark.parametrize("tiles", [39, 75, 76, 77, 151, 152, 153, 170, 227, 228, 229, 303, 304, 305, 380, 381, 456, 500])
@pytest.mark.parametrize("width", [544, 1056])
def test_product_of_a_few_rows_of_one_of_some_experts(ex, tiles, width):
    """Counts of small tiles around whole and half turns of 152 CTAs; the host is told of four experts, any of which may
    have rows."""
    for cut in ([0, 0, 8, 8, 8], [0, 0, 0, 3, 3]):
        x, w, offsets = case(ex, 8, 4, 128 * tiles - 60, width, tiles, cut)
        check_product(ex, x, w, offsets, torch.float32)
        check_product(ex, x, w, offsets, torch.bfloat16)
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
    flat = ebc.Mx8(w.codes[0], w.scales[0], w.width)
    ys = ex.product(x, flat, dtype=torch.float32)
    check_product(ex, x, w, torch.tensor([0, 77], dtype=torch.int32), torch.float32, ys)
    assert ex.product(ex.quantize_mx8(torch.zeros(0, 320, device="cuda")), flat).shape == (0, 130)


@pytest.mark.parametrize("rows,outs,width", [(4, 130, 64), (200, 300, 1000)])
def test_a_nan_stays_in_its_row_and_in_its_output(ex, rows, outs, width):
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(rows, width, generator=g, device="cuda")
    w = torch.randn(2, outs, width, generator=g, device="cuda")
    x[rows // 2, width - 1] = float("inf")
    w[1, outs - 1, 0] = float("nan")
    cut = [0, rows // 4, rows]
    ys = ex.product(ex.quantize_mx8(x), ex.quantize_mx8(w), torch.tensor(cut, dtype=torch.int32, device="cuda"), torch.float32)
    want = torch.zeros(rows, outs, dtype=torch.bool)
    want[rows // 2] = True
    want[cut[1]:, outs - 1] = True
    assert torch.equal(ys.isnan().cpu(), want)


def test_scales_of_every_size(ex):
    """A scale for each row and block: values of four bits' fraction and few terms a sum, which is then exact."""
    width, rows, outs = 96, 130, 140
    rng = np.random.default_rng(0)
    x, w = np.zeros((rows, width)), np.zeros((outs, width))
    x[:, ::32] = rng.choice([-448.0, -1.5, 0.5, 3.0, 13.0], (rows, 3))
    w[:, ::32] = rng.choice([-6.0, -2.0, 1.0, 4.0, 240.0], (outs, 3))
    x *= (2.0 ** rng.integers(-50, 50, (rows, 1)))
    w *= 2.0 ** rng.integers(-50, 50, (outs, 1))
    q, p = (ex.quantize_mx8(torch.from_numpy(v).float().cuda()) for v in (x, w))
    assert torch.equal(ex.dequantize(q).cpu().double(), torch.from_numpy(x)) and torch.equal(ex.dequantize(p).cpu().double(), torch.from_numpy(w))
    ys = ex.product(q, p, dtype=torch.float32)
    assert torch.equal(ys.cpu(), torch.from_numpy(x @ w.T).float())


def test_padding_bytes_of_the_scales_are_not_read(ex):
    x, w, offsets = case(ex, 60, 2, 140, 96, 9)
    ys = ex.product(x, w, offsets)
    x.scales[..., 3:] = 255
    w.scales[..., 3:] = 255
    assert torch.equal(ex.product(x, w, offsets), ys)


def test_rows_past_32_bits_of_outputs(ex):
    rows, outs, width = 70000, 32768, 32
    x = ex.quantize_mx8(torch.randn(rows, width, device="cuda"))
    w = ex.quantize_mx8(torch.randn(1, outs, width, device="cuda"))
    ys = ex.product(x, w, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), torch.bfloat16)
    for at in (slice(0, 300), slice(65400, 65700), slice(rows - 300, rows)):
        part = ebc.Mx8(x.codes[at], x.scales[at], width)
        check_product(ex, part, w, torch.tensor([0, 300]), torch.bfloat16, ys[at])


def test_the_same_bits_in_every_run_and_on_another_stream(ex):
    x, w, offsets = case(ex, 700, 6, 520, 2080, 12)
    first = ex.product(x, w, offsets)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, None, side):
        again = ex.product(x, w, offsets, stream=stream)
        back = ex.dequantize(ex.quantize_mx8(first, stream=stream), torch.bfloat16, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(first, again) and torch.equal(back, ex.dequantize(ex.quantize_mx8(first), torch.bfloat16))


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


@pytest.mark.parametrize("rows,experts,outs,width", [(16, 8, 2000, 2048), (6000, 4, 4000, 1024), (2, 1, 600, 8192), (16384, 3, 4096, 4000), (16, 32, 4096, 2048), (13, 32, 4000, 1000)])
def test_a_wait_that_runs_out_is_recorded_and_the_context_recovers(rows, experts, outs, width):
    """Single CTAs, pairs and clusters that share K: the first stage's wait gives up at once; every CTA ends, the
    status says so, and the next product is right."""
    e = ebc.Experts(0)
    x, w, offsets = case(e, rows, experts, outs, width, 3)
    want = e.product(x, w, offsets)
    for _ in range(2):
        assert ebc.ebc_set_first_wait_polls(e.handle, 0) == 0
        e.product(x, w, offsets)
        assert ebc.ebc_set_first_wait_polls(e.handle, -1) == 0
        again = e.product(x, w, offsets)
        with pytest.raises(ebc.EbcError) as err:
            e.check()
        assert err.value.code == ebc.EBC_ERR_DEVICE_TIMEOUT
        assert torch.equal(again, want)
    check_product(e, x, w, offsets, torch.bfloat16)
    e.check()
    e.close()


def test_refusals(ex):
    x, w, offsets = case(ex, 8, 2, 16, 64, 1)
    with pytest.raises(ValueError):
        ex.product(x, ex.quantize_mx8(torch.zeros(2, 16, 96, device="cuda")), offsets)
    with pytest.raises(ValueError, match="same kind"):
        ex.product(x, ex.quantize(torch.zeros(2, 16, 64, device="cuda")), offsets)
    with pytest.raises(ValueError, match="same kind"):
        ex.product(ex.quantize(torch.zeros(8, 64, device="cuda")), w, offsets)
    with pytest.raises(ValueError):
        ex.product(x, w)
    with pytest.raises(ValueError):
        ex.product(x, w, offsets.long())
    with pytest.raises(ValueError):
        ex.quantize_mx8(torch.zeros(4, 64, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        ex.quantize_mx8(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        ex.dispatch(x, ex.plan(torch.zeros(9, 1, dtype=torch.int32, device="cuda"), 2))
    h = ex.handle
    c, s, o, y = (t.data_ptr() for t in (x.codes, x.scales, offsets, torch.empty(8, 16, device="cuda")))
    inv = ebc.EBC_ERR_INVALID_ARG
    assert ebc.ebc_mx8_product(h, c, s, -1, 64, c, s, 16, 2, o, 0, y, None) == inv
    assert ebc.ebc_mx8_product(h, c, s, 8, 0, c, s, 16, 2, o, 0, y, None) == inv
    assert ebc.ebc_mx8_product(h, c, s, 8, 64, c, s, 16, 1025, o, 0, y, None) == inv
    assert ebc.ebc_mx8_product(h, c, s, 8, 64, c, s, 16, 2, None, 0, y, None) == inv
    assert ebc.ebc_mx8_product(h, c + 8, s, 8, 64, c, s, 16, 2, o, 0, y, None) == inv
    assert ebc.ebc_mx8_quantize(h, y, 64, 0, 2, 0, c, s, None) == inv
    assert ebc.ebc_mx8_quantize(h, y, 63, 0, 2, 64, c, s, None) == inv
    assert ebc.ebc_mx8_quantize(h, y, 64, 9, 2, 64, c, s, None) == inv
    assert ebc.ebc_mx8_quantize(h, y, 64, 0, 2, 64, c + 4, s, None) == inv
    assert ebc.ebc_mx8_quantize(h, y, 2 ** 25, 0, 2, 2 ** 25, c, s, None) == inv
    assert ebc.ebc_mx8_dequantize(h, c, s, 2, 64, 7, y, None) == inv
    assert ebc.ebc_mx8_dequantize(h, None, s, 2, 64, 0, y, None) == inv
    assert ebc.ebc_moe_dispatch_mx(h, c, 60, s, 16, 2, 1, o, o, 2, c, s, None) == inv
    assert ebc.ebc_moe_dispatch_mx(h, c, 64, s, 16, 2, 1, None, o, 2, c, s, None) == inv
    assert ebc.ebc_moe_dispatch_mx(h, c + 4, 64, s, 16, 2, 1, o, o, 2, c, s, None) == inv
    ex.check()
