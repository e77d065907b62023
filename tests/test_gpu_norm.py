"""The norm with the residual's addition against its definition in 64 bits, its
8-bit output, and its gradients against the formulas and against differences.

In units of 2^-24: a row's sum of squares takes at most 32 additions in a
thread, 9 joins, a rounding a square, and 3 more to mean + eps; the inverse
root halves their 45 and adds 4 of its own, and the sum x + residual and two
products add 3.  So y is within 30 (rounded up: 32) of its magnitude before it
is rounded to its type.  The gradients of a row are a sum of two products with
those, each within 80 of its magnitude."""
import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import error_bounded_lossy_gb300 as ebc

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

TYPES = [torch.float32, torch.bfloat16, torch.float16]
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
U = 2.0 ** -24
EPS = 1e-6
SIZES = [(1, 1), (3, 2), (1, 8), (5, 31), (40, 33), (9, 64), (1000, 64), (70, 65), (300, 128), (13, 136), (257, 256), (7, 258),
         (3, 301), (600, 512), (5, 520), (2, 1000), (3, 1001), (4, 1002), (400, 1024), (1, 2048), (3, 2050), (650, 4096), (3, 4098),
         (2, 5001), (700, 7168), (3, 8192), (2, 8200), (2, 12289), (2, 16384), (2, 16383), (2, 16382),
         (300, 8199), (200, 12289), (97, 16377), (400, 16383), (400, 16382),
         (1100, 4099), (5000, 1001)]


@pytest.fixture(scope="module")
def ex():
    e = ebc.Experts(0)
    yield e
    e.check()
    e.close()


def tiny(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 1e-37


def batch(rows, width, dtype, seed, wtype=None):
    g = torch.Generator("cuda").manual_seed(seed)
    make = lambda: (torch.randn(rows, width, generator=g, device="cuda")  # noqa: E731
                    * torch.exp2(torch.randint(-4, 5, (rows, 1), generator=g, device="cuda").float())).to(dtype)
    w = (1 + 0.5 * torch.randn(width, generator=g, device="cuda")).to(wtype or dtype)
    return make(), make(), w, make(), make()


def defined(x, r, w, eps=EPS):
    h = x.double() if r is None else x.double() + r.double()
    return h / ((h * h).mean(1, keepdim=True) + eps).sqrt() * w.double(), h


def check_forward(x, r, w, y, h, eps=EPS):
    want, sum_ = defined(x, r, w, eps)
    dtype = x.dtype
    off = (y.double() - want).abs()
    bound = (32 * U + UNIT[dtype] * (1 + 32 * U)) * want.abs() + tiny(dtype)
    assert bool((off <= bound).all()), float((off - bound).max())
    if r is None:
        assert h is x
    else:
        assert bool(((h.double() - sum_).abs() <= (UNIT[dtype] * (1 + U) + U) * sum_.abs() + tiny(dtype)).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", SIZES)
def test_norm(ex, rows, width, dtype):
    x, r, w, _, _ = batch(rows, width, dtype, rows + width)
    check_forward(x, None, w, *ex.norm(x, w))
    check_forward(x, r, w, *ex.norm(x, w, r))
    check_forward(x, r, w, *ex.norm(x, w, r, eps=0.25), eps=0.25)


def check_8_bit(ex, q, x, r, w):
    want, _ = defined(x, r, w)
    unit = (q.scales[:, :-(-q.width // 32)].int() << 23).view(torch.float32).double().repeat_interleave(32, 1)[:, :q.width]
    near = want.abs() * (1 + 32 * U)
    off = (ex.dequantize(q).double() - want).abs()
    assert bool((off <= torch.maximum(near / 16, unit / 1024) + 32 * U * want.abs()).all())
    assert bool((near * (1 + 32 * U) <= 448 * unit * (1 + 128 * U)).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", SIZES)
def test_the_8_bit_output(ex, rows, width, dtype):
    x, r, w, _, _ = batch(rows, width, dtype, rows + width + 1)
    y, h = ex.norm(x, w, r)
    q, y2, h2 = ex.norm_mx8(x, w, r, wide=True)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    q1, none, h3 = ex.norm_mx8(x, w, r)
    assert none is None and torch.equal(h, h3) and torch.equal(q.codes, q1.codes) and torch.equal(q.scales, q1.scales)
    blocks = -(-width // 32)
    assert q.shape == (rows, width) and not q.scales[:, blocks:].any() and not q.codes[:, width:].any()
    if dtype == torch.float32:   # then y is what was rounded
        p = ex.quantize_mx8(y)
        assert torch.equal(q.codes, p.codes) and torch.equal(q.scales, p.scales)
    check_8_bit(ex, q, x, r, w)
    q, _, h = ex.norm_mx8(x, w)
    assert h is x
    if dtype == torch.float32:
        assert torch.equal(q.codes, ex.quantize_mx8(ex.norm(x, w)[0]).codes)


def formulas(dy, h, w, dh, eps=EPS):
    """dx and dweight at h, and the magnitudes that their errors are relative to."""
    h, dy, w = h.double(), dy.double(), w.double()
    s = 1 / ((h * h).mean(1, keepdim=True) + eps).sqrt()
    u, q = h * s, dy * w
    dx = s * (q - u * (q * u).mean(1, keepdim=True)) + (0 if dh is None else dh.double())
    size = s * (q.abs() + u.abs() * (q * u).abs().mean(1, keepdim=True))
    return dx, (dy * u).sum(0), size, (dy * u).abs().sum(0)


def check_backward(dy, h, w, dh, dx, dw, eps=EPS):
    want, wantw, size, sizew = formulas(dy, h, w, dh, eps)
    dtype = dy.dtype
    off = (dx.double() - want).abs()
    lost = 80 * U * size + U * want.abs()
    bound = lost + UNIT[dtype] * (want.abs() + lost) + tiny(dtype)
    assert dx.dtype == dtype and dw.dtype == w.dtype
    assert bool((off <= bound).all()), float((off - bound).max())
    off = (dw.double() - wantw).abs()
    lost = (dy.shape[0] + 80) * U * sizew
    bound = lost + UNIT[w.dtype] * (wantw.abs() + lost) + tiny(w.dtype)
    assert bool((off <= bound).all()), float((off - bound).max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width,pad", [(511, 1), (1, 7), (7, 1), (30, 2), (33, 7), (509, 3), (1001, 7), (1001, 1), (4095, 1), (8191, 1), (8195, 5), (16383, 1)])
def test_what_is_beside_the_rows_takes_no_part(ex, width, pad, dtype):
    """Aligned rows of a wider buffer whose other values are NaN, of a width that is no multiple of a vector."""
    rows = 20
    t = list(batch(rows, width, dtype, width))
    w = t.pop(2)
    wide = [torch.full((rows, width + pad), float("nan"), device="cuda", dtype=dtype) for _ in t]
    for a, b in zip(wide, t):
        a[:, :width] = b
    x, r, dy, dh = (a[:, :width] for a in wide)
    check_forward(x, None, w, *ex.norm(x, w))
    check_forward(x, r, w, *ex.norm(x, w, r))
    for residual in (None, r):
        check_8_bit(ex, ex.norm_mx8(x, w, residual)[0], x, residual, w)
        check_8_bit(ex, ex.norm_mx8(x, w, residual, wide=True)[0], x, residual, w)
    check_backward(dy, x, w, None, *ex.norm_grad(dy, x, w))
    check_backward(dy, x, w, dh, *ex.norm_grad(dy, x, w, dh))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", SIZES)
def test_the_gradients(ex, rows, width, dtype):
    h, _, w, dy, dh = batch(rows, width, dtype, rows + width + 2)
    check_backward(dy, h, w, dh, *ex.norm_grad(dy, h, w, dh))
    first = ex.norm_grad(dy, h, w)
    check_backward(dy, h, w, None, *first)
    assert all(torch.equal(a, b) for a, b in zip(first, ex.norm_grad(dy, h, w)))
    check_backward(dy, h, w, dh, *ex.norm_grad(dy, h, w, dh, eps=0.25), eps=0.25)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("wtype", TYPES)
def test_a_weight_of_another_type(ex, dtype, wtype):
    x, r, w, dy, dh = batch(50, 520, dtype, 3, wtype)
    y, h = ex.norm(x, w, r)
    check_forward(x, r, w, y, h)
    check_backward(dy, h, w, dh, *ex.norm_grad(dy, h, w, dh))


@pytest.mark.parametrize("at", [slice(0, 64), slice(1, 65), slice(2, 100), slice(4, 133), slice(8, 1000)])
def test_rows_with_strides(ex, at):
    for dtype in TYPES:
        x, r, w, dy, dh = batch(9, 1203, dtype, 4)
        a = [t[:, at] for t in (x, r, dy, dh)]
        b = [t.contiguous() for t in a]
        w = w[at].clone()
        # (a row's sum has another order where its vectors are of another size, so not the same bits)
        for p, q in ((a[0], a[1]), (a[0], b[1]), (b[0], a[1])):
            check_forward(b[0], b[1], w, *ex.norm(p, w, q))
            check_8_bit(ex, ex.norm_mx8(p, w, q)[0], b[0], b[1], w)
        check_backward(a[2], a[0], w, a[3], *ex.norm_grad(a[2], a[0], w, a[3]))
        check_backward(a[2], b[0], w, None, *ex.norm_grad(a[2], b[0], w))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", [(1, 9), (2, 9), (20, 9), (5, 57), (40, 63), (9, 121), (21, 203), (3, 249), (50, 505), (17, 1001), (33, 2047), (9, 5003), (12, 8185), (3, 8187), (700, 999)])
def test_what_is_beside_a_row_stays_out_of_it(ex, rows, width, dtype):
    """Rows off a vector's boundary are read in whole vectors: what stands between them, and NaN in the rows before
    and after, do not get in, and nothing is written beside the results."""
    g = torch.Generator("cuda").manual_seed(rows + width)
    pitch = width + 8
    x, r, dy, dh = (torch.full((rows * pitch,), float("nan"), dtype=dtype, device="cuda").as_strided((rows, width), (pitch, 1)) for _ in range(4))
    for t in (x, r, dy, dh):
        t.copy_(torch.randn(rows, width, generator=g, device="cuda"))
    w = torch.randn(width, generator=g, device="cuda").to(dtype)
    check_forward(x, r, w, *ex.norm(x, w, r))
    check_forward(x, None, w, *ex.norm(x, w))
    check_backward(dy, x, w, dh, *ex.norm_grad(dy, x, w, dh))
    check_backward(dy, x, w, None, *ex.norm_grad(dy, x, w))
    check_8_bit(ex, ex.norm_mx8(x, w, r)[0], x, r, w)
    dense = [t.clone(memory_format=torch.contiguous_format) for t in (x, r, dy, dh)]
    dense[0][::2] = float("nan")
    y, h = ex.norm(dense[0], w, dense[1])
    good = torch.arange(rows, device="cuda") % 2 == 1
    assert bool(y[~good].isnan().all()) and bool(h[~good].isnan().all())
    check_forward(x[good], r[good], w, y[good], h[good])
    dx, dw = ex.norm_grad(dense[2], dense[0], w, dense[3])
    assert bool(dx[~good].isnan().all()) and bool(dw.isnan().all())
    if rows > 1:
        check_backward(dy[good], x[good], w, dh[good], dx[good], ex.norm_grad(dy[good], x[good], w, dh[good])[1])
    # through the C calls, into buffers with something behind their ends
    out = torch.full((rows * width + 64,), 7.0, dtype=dtype, device="cuda")
    type_ = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[dtype]
    d = [t.contiguous() for t in (x, r, dy)]
    st = torch.cuda.current_stream().cuda_stream
    for shift in (0, 32):
        at = out.data_ptr() + shift * out.element_size()
        assert ebc.ebc_norm(ex.handle, d[0].data_ptr(), width, None, 0, type_, w.data_ptr(), type_, rows, width, EPS, at, None, None, None, st) == 0
        check_forward(d[0], None, w, out[shift:shift + rows * width].view(rows, width).clone(), d[0])
        assert bool((out[:shift] == 7).all()) and bool((out[shift + rows * width:] == 7).all())
        out.fill_(7.0)


def test_leading_shapes_one_row_and_nothing(ex):
    x, r, w, _, _ = batch(30, 96, torch.bfloat16, 5)
    y, h = ex.norm(x, w, r)
    shaped = ex.norm(x.view(5, 6, 96), w, r.view(5, 6, 96))
    assert shaped[0].shape == (5, 6, 96) and torch.equal(shaped[0].view(30, 96), y) and torch.equal(shaped[1].view(30, 96), h)
    q, _, h3 = ex.norm_mx8(x.view(5, 6, 96), w, r.view(5, 6, 96))
    assert q.shape == (5, 6, 96) and q.codes.shape == (5, 6, 96) and q.scales.shape == (5, 6, 16) and torch.equal(h3.view(30, 96), h)
    x3 = x.view(5, 6, 96)
    assert ex.norm(x3, w)[1] is x3
    t = torch.randn(96, 40, device="cuda").t()    # rows that are not contiguous have to be laid out first
    one = ex.norm(x[0], w, r[0])
    assert one[0].shape == (96,) and torch.equal(one[0], y[0])
    with pytest.raises(ValueError):
        ex.norm(t, torch.ones(96, device="cuda"))
    none = ex.norm(x[:0], w, r[:0])
    assert none[0].shape == none[1].shape == (0, 96) and ex.norm_mx8(x[:0], w)[0].codes.shape == (0, 96)
    dx, dw = ex.norm_grad(x[:0], x[:0], w)
    assert dx.shape == (0, 96) and dw.shape == (96,) and not dw.any()


def test_zeros_infinities_and_nan(ex):
    """A row of zeros is zero (and with eps = 0 NaN, as 0 / 0 is); what is not finite stays in its row."""
    x = torch.randn(6, 200, device="cuda")
    x[1] = 0
    x[2, 7] = float("inf")
    x[3, 8] = float("nan")
    x[4, 9] = 1e30            # its square is past fp32
    w = torch.ones(200, device="cuda")
    y, _ = ex.norm(x, w)
    assert not y[1].any()
    assert bool(y[2, 7].isnan()) and not y[2, :7].any() and not y[2, 8:].any()
    assert bool(y[3].isnan().all()) and not y[4].any()
    clean = ex.norm(x[[0, 5]].contiguous(), w)[0]
    assert torch.equal(y[[0, 5]], clean)
    q, _, _ = ex.norm_mx8(x, w)
    assert torch.equal(q.scales[[0, 5]], ex.quantize_mx8(clean).scales) and (q.scales[3, :7] == 255).all() and not q.codes[1].any()
    assert bool(ex.norm(x[1:2], w, eps=0.0)[0].isnan().all())
    dx, dw = ex.norm_grad(torch.ones_like(x), x, w)
    assert bool(dx[3].isnan().all()) and bool(torch.isfinite(dx[[0, 1, 5]]).all()) and bool(dw.isnan().all())


def test_rows_past_31_bits(ex):
    rows, width = 66000, 32800 // 4
    x = torch.zeros(rows * 4, width, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, 261888, 262143, 262144, rows * 4 - 1]
    x[at] = torch.randn(len(at), width, device="cuda").to(torch.bfloat16)
    w = torch.ones(width, dtype=torch.bfloat16, device="cuda")
    q, y, _ = ex.norm_mx8(x, w, wide=True)
    p, z, _ = ex.norm_mx8(x[at], w, wide=True)
    assert torch.equal(y[at], z) and torch.equal(q.codes[at], p.codes) and torch.equal(q.scales[at], p.scales)
    del q
    dx, dw = ex.norm_grad(x, x, w)
    check_backward(x[at], x[at], w, None, dx[at], dw)


def test_the_gradients_against_differences(ex):
    """The directional derivative of sum(y * dy) + sum(h * dh) by central differences of the kernel's own fp32
    results: rounding leaves 33 U of the outputs' magnitudes over the step, and the steps' error is a quarter of the
    difference between a step and twice it, to its leading order (doubled)."""
    g = torch.Generator("cuda").manual_seed(0)
    x, r, dy, dh, v = (torch.randn(20, 600, generator=g, device="cuda").double() for _ in range(5))
    w, vw = (torch.randn(600, generator=g, device="cuda").double() for _ in range(2))

    def value(t):
        xs, ws = (x + t * v).float(), (w + t * vw).float()
        y, h = ex.norm(xs, ws, r.float())
        # (the inputs were rounded: what they are is what counts)
        return (y.double() * dy).sum() + (h.double() * dh).sum(), (y.double() * dy).abs().sum() + (h.double() * dh).abs().sum()

    def slope(t):
        (a, size), (b, _) = value(t), value(-t)
        return float((a - b) / (2 * t)), float(33 * U * size / t)

    h = ex.norm(x.float(), w.float(), r.float())[1]
    dx, dw = ex.norm_grad(dy.float(), h, w.float(), dh.float())
    got = float((dx.double() * v).sum() + (dw.double() * vw).sum())
    (fine, lost), (coarse, _) = slope(2.0 ** -6), slope(2.0 ** -5)
    assert abs(got - fine) <= 2 * abs(coarse - fine) / 3 + 2 * lost + 1e-3 * abs(got)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("use", ["y", "h", "both"])
def test_recorded(ex, dtype, use):
    x0, r0, w0, dy, dh = batch(33, 264, dtype, 6)
    x, r, w = (t.clone().requires_grad_() for t in (x0, r0, w0))
    y, h = ex.norm(x, w, r)
    outs, grads = zip(*[p for p, u in (((y, dy), "y"), ((h, dh), "h")) if use in (u, "both")])
    torch.autograd.backward(outs, grads)
    if use == "h":
        assert torch.equal(x.grad, dh) and torch.equal(r.grad, dh) and w.grad is None
        return
    dx, dw = ex.norm_grad(dy, h.detach(), w0, dh if use == "both" else None)
    assert torch.equal(x.grad, dx) and torch.equal(r.grad, dx) and torch.equal(w.grad, dw)


def test_recorded_forms(ex):
    x0, r0, w0, dy, dh = batch(24, 96, torch.float32, 7)
    x = x0.clone().requires_grad_()
    y, h = ex.norm(x.view(4, 6, 96), w0)         # no residual, other shapes, a weight that needs none
    y.backward(dy.view(4, 6, 96))
    assert torch.equal(x.grad, ex.norm_grad(dy, x0, w0)[0])
    # the 8-bit form: y and h carry gradients, the codes none
    x.grad = None
    q, y, h = ex.norm_mx8(x, w0, r0, wide=True)
    assert y.requires_grad and h.requires_grad and not q.codes.requires_grad and not q.scales.requires_grad
    (y * dy + h * dh).sum().backward()
    assert torch.equal(x.grad, ex.norm_grad(dy, h.detach(), w0, dh)[0])
    x.grad = None
    q, y, h = ex.norm_mx8(x, w0, r0)
    assert y is None
    h.backward(dh)
    assert torch.equal(x.grad, dh)
    # expanded gradients, no_grad, once
    x.grad = None
    ex.norm(x, w0)[0].sum().backward()
    assert torch.equal(x.grad, ex.norm_grad(torch.ones_like(x0), x0, w0)[0])
    with torch.no_grad():
        assert not ex.norm(x, w0)[0].requires_grad
    (dx,) = torch.autograd.grad((ex.norm(x, w0)[0] ** 2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()
    with forward_ad.dual_level(), pytest.raises(ValueError, match="forward"):
        ex.norm(forward_ad.make_dual(x0, x0), w0)


def test_streams_and_graphs(ex):
    x, r, w, dy, dh = batch(70, 4096, torch.bfloat16, 8)
    want = (*ex.norm(x, w, r), *ex.norm_grad(dy, x, w, dh))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = (*ex.norm(x, w, r, stream=side), *ex.norm_grad(dy, x, w, dh, stream=side))
    shaped = ex.norm(x.view(7, 10, 4096), w, r.view(7, 10, 4096), stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(shaped[0].view(70, 4096), want[0])
    graphs = []
    for k in range(2):   # two graphs, replayed at the same time
        graph, inputs = torch.cuda.CUDAGraph(), [t.clone() for t in (x, r, w, dy, dh)]
        with torch.cuda.graph(graph):
            a, b, c, d, e = inputs
            outs = (*ex.norm(a, c, b), *ex.norm_grad(d, a, c, e))
        graphs.append((graph, inputs, outs))
    graphs[1][1][0].neg_()
    torch.cuda.synchronize()
    for graph, _, _ in graphs:
        with torch.cuda.stream(torch.cuda.Stream()):
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, graphs[0][2]))
    other = (*ex.norm(-x, w, r), *ex.norm_grad(dy, -x, w, dh))
    assert all(torch.equal(a, b) for a, b in zip(other, graphs[1][2]))


def test_refusals(ex):
    x, r, w, dy, dh = batch(8, 64, torch.float32, 9)
    wide = torch.zeros(2, ebc.EBC_MAX_NORM_WIDTH + 8, device="cuda")
    for call in (lambda: ex.norm(x.double(), w), lambda: ex.norm(x.cpu(), w), lambda: ex.norm(x, w.cpu()), lambda: ex.norm(x, w[:63]),
                 lambda: ex.norm(x, w[None]), lambda: ex.norm(x, w, r[:7]), lambda: ex.norm(x, w, r.half()), lambda: ex.norm(x, w.double()),
                 lambda: ex.norm(x, w.repeat(2)[::2]), lambda: ex.norm_grad(dy, x[:, :32], w), lambda: ex.norm_grad(dy, x, w, dh.half())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ex.norm(wide, wide[0]), lambda: ex.norm(x, w, eps=-1.0), lambda: ex.norm(x, w, eps=float("nan")),
                 lambda: ex.norm_grad(wide, wide, wide[0])):
        with pytest.raises(ebc.EbcError) as err:
            call()
        assert err.value.code == ebc.EBC_ERR_INVALID_ARG
    h, p, q = ex.handle, x.data_ptr(), w.data_ptr()
    o = torch.empty(8, 64, device="cuda").data_ptr()
    inv = ebc.EBC_ERR_INVALID_ARG
    assert ebc.ebc_norm(h, p, 64, None, 0, 0, q, 0, 8, 64, 1e-6, None, None, None, None, None) == inv
    assert ebc.ebc_norm(h, p, 64, None, 0, 0, q, 0, 8, 64, 1e-6, o, None, o, None, None) == inv
    assert ebc.ebc_norm(h, p, 63, None, 0, 0, q, 0, 8, 64, 1e-6, o, None, None, None, None) == inv
    assert ebc.ebc_norm(h, p, 64, p, 63, 0, q, 0, 8, 64, 1e-6, o, o, None, None, None) == inv
    assert ebc.ebc_norm(h, p, 64, None, 0, 3, q, 0, 8, 64, 1e-6, o, None, None, None, None) == inv
    assert ebc.ebc_norm(h, p, 64, None, 0, 0, None, 0, 8, 64, 1e-6, o, None, None, None, None) == inv
    assert ebc.ebc_norm(h, p + 2, 64, None, 0, 0, q, 0, 8, 64, 1e-6, o, None, None, None, None) == inv
    assert ebc.ebc_norm_grad(h, p, 64, p, 64, None, 0, 0, q, 0, 8, 64, 1e-6, o, q, None, None) == inv
    assert ebc.ebc_norm_grad(h, p, 64, p, 64, None, 0, 0, q, 0, 8, 64, 1e-6, o, None, o, None) == inv
    ex.check()
