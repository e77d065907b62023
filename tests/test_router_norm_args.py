"""The router, norm and 8-bit calls on a machine without a GPU: refusing what is
wrong before any device work, and what they do on the host (the library's
objects linked with a CUDA runtime without a device)."""
import ctypes
import os
import random
import re
import subprocess

import pytest
import torch

import error_bounded_lossy_gb300 as ebc
from error_bounded_lossy_gb300 import build as ebc_build

HERE = os.path.dirname(os.path.abspath(__file__))
A = 1 << 20   # an address that is aligned to anything; nothing reads it
BAD = ebc.EBC_ERR_INVALID_ARG


@pytest.fixture(scope="module", autouse=True)
def lib():
    ebc_build.build()
    return ebc.lib()


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    """The library on the runtime without a device."""
    out = str(tmp_path_factory.mktemp("fake") / "libebc_fake2.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(ebc_build.nvcc())), "include")
    objs = [os.path.join(ebc_build.BUILD, s.replace(".cu", ".o")) for s in ebc_build.SOURCES]
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wl,-Bsymbolic", f"-I{cuda}", "-o", out,
                    os.path.join(HERE, "fake_cudart.cpp"), *objs], check=True)
    L = ctypes.CDLL(out)
    real = ebc.lib()
    for name in ebc.EXPORTED_SYMBOLS:
        getattr(L, name).argtypes, getattr(L, name).restype = getattr(real, name).argtypes, getattr(real, name).restype
    L.cudaSetDevice.argtypes, L.cudaGetDevice.argtypes, L.fake_static_shared.argtypes = [ctypes.c_int], [ctypes.c_void_p], [ctypes.c_int]
    L.fake_log.restype = ctypes.c_char_p
    L.cudaSetDevice(0)
    return L


def context(fake, device=0):
    h = ctypes.c_void_p()
    assert fake.ebc_create(ctypes.byref(h), None, device) == 0
    fake.fake_clear()
    return h


def launches(fake):
    found = re.findall(r"launch (\S+) grid (\d+) cluster (\d+) shared (\d+) stream (\S+) device (\d+)", fake.fake_log().decode())
    fake.fake_clear()
    return found


def calls(lib, ctx, tokens=4, stream=None):
    """Every call with arguments that are in order: name -> (call, launches)."""
    return {
        "quantize_mx8": (lambda: lib.ebc_mx8_quantize(ctx, A, 64, 0, tokens, 64, A, A, stream), 1),
        "dequantize_mx8": (lambda: lib.ebc_mx8_dequantize(ctx, A, A, tokens, 64, 0, A, stream), 1),
        "product_mx8": (lambda: lib.ebc_mx8_product(ctx, A, A, tokens, 64, A, A, 16, 2, A, 0, A, stream), 1),
        "dispatch_mx": (lambda: lib.ebc_moe_dispatch_mx(ctx, A, 64, A, 16, tokens, 2, A, A, 3, A, A, stream), 1),
        "route": (lambda: lib.ebc_moe_route(ctx, A, 8, 0, tokens, 8, 2, 1, A, 4, 2, 2, 1, 1.0, A, A, stream), 1),
        "route_grad": (lambda: lib.ebc_moe_route_grad(ctx, A, A, 8, 0, tokens, 8, 2, A, 1, 1, 1.0, A, stream), 1),
        "norm": (lambda: lib.ebc_norm(ctx, A, 64, A, 64, 1, A, 0, tokens, 64, 1e-6, A, A, A, A, stream), 1),
        "norm_grad": (lambda: lib.ebc_norm_grad(ctx, A, 4096, A, 4096, A, 4096, 1, A, 0, tokens, 4096, 1e-6, A, A, A, stream), 2),
    }


def test_a_null_context_is_refused(lib):
    for name, (call, _) in calls(lib, None).items():
        assert call() == BAD, name


def test_no_rows_is_no_launch_and_the_callers_device_stays(fake):
    now = ctypes.c_int(-1)
    ctx = context(fake, 1)
    for device in (0, 1):
        fake.cudaSetDevice(device)
        for name, (call, n) in calls(fake, ctx).items():
            assert call() == 0, name
            assert fake.cudaGetDevice(ctypes.byref(now)) == 0 and now.value == device, name
            assert [x[5] for x in launches(fake)] == ["1"] * n, name
    fake.cudaSetDevice(0)
    for name, (call, n) in calls(fake, ctx, 0).items():
        assert call() == 0, name
        assert len(launches(fake)) == (name == "norm_grad"), name     # (the weight's gradient is zero)
    for name, (call, n) in calls(fake, ctx, 4, 0x70).items():
        assert call() == 0, name
        assert {x[4] for x in launches(fake)} == {"0x70"}, name
    fake.fake_static_shared(1 << 20)   # no launch fits
    for name, (call, _) in calls(fake, ctx).items():
        assert call() == ebc.EBC_ERR_CUDA, name
        assert fake.cudaGetDevice(ctypes.byref(now)) == 0 and now.value == 0, name
    fake.fake_static_shared(256)
    fake.ebc_destroy(ctx)


def test_what_is_out_of_range_is_refused(fake):
    ctx = context(fake)

    def route(tokens=4, ld=8, type=0, experts=8, top=2, score=0, bias=None, groups=1, keep=1, best=1, renorm=1, scale=1.0, logits=A, ids=A, w=A):
        return fake.ebc_moe_route(ctx, logits, ld, type, tokens, experts, top, score, bias, groups, keep, best, renorm, scale, ids, w, None)

    assert route() == 0 and route(tokens=(2 ** 31 - 1) // 2) == 0 and route(experts=1024, ld=1024, top=32, groups=32, keep=32, best=2) == 0
    for wrong in (dict(tokens=-1), dict(tokens=2 ** 30), dict(ld=7), dict(ld=2 ** 41), dict(type=3), dict(experts=0), dict(experts=1025, ld=1025),
                  dict(top=0), dict(top=33), dict(score=2), dict(bias=A + 2), dict(groups=3), dict(groups=0), dict(groups=64, experts=64, ld=64),
                  dict(keep=0), dict(keep=2), dict(groups=4, keep=5), dict(best=0), dict(best=3), dict(scale=float("nan")),
                  dict(scale=float("inf")), dict(logits=None), dict(logits=A + 2), dict(ids=None), dict(ids=A + 1), dict(w=None)):
        assert route(**wrong) == BAD, wrong

    def norm(ld=64, r=None, ld_r=64, type=1, w=A, wt=0, rows=4, width=64, eps=1e-6, y=A, h=None, c=None, s=None, x=A):
        return fake.ebc_norm(ctx, x, ld, r, ld_r, type, w, wt, rows, width, eps, y, h, c, s, None)

    most = ebc.EBC_MAX_NORM_WIDTH
    assert norm() == 0 and norm(y=None, c=A, s=A) == 0 and norm(ld=most, width=most) == 0 and norm(rows=2 ** 31 - 1) == 0 and norm(eps=0.0) == 0
    for wrong in (dict(ld=63), dict(r=A, ld_r=63), dict(r=A + 1), dict(type=4), dict(wt=-1), dict(w=None), dict(w=A + 2), dict(rows=-1), dict(rows=2 ** 31),
                  dict(width=0), dict(width=most + 1, ld=most + 1), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")), dict(y=None),
                  dict(c=A), dict(s=A), dict(c=A + 8, s=A), dict(h=A + 1), dict(x=None)):
        assert norm(**wrong) == BAD, wrong

    def grad(ld=64, dh=None, type=1, rows=4, width=64, eps=1e-6, dx=A, dw=A, scratch=A, w=A):
        return fake.ebc_norm_grad(ctx, A, ld, A, 64, dh, 64, type, w, 0, rows, width, eps, dx, dw, scratch, None)

    assert grad() == 0 and grad(dh=A) == 0
    for wrong in (dict(ld=8), dict(dh=A + 1), dict(type=9), dict(rows=-5), dict(width=0), dict(dx=None), dict(dw=None), dict(scratch=None),
                  dict(scratch=A + 4), dict(dw=A + 1), dict(w=None), dict(eps=-1.0)):
        assert grad(**wrong) == BAD, wrong

    def dispatch(cb=64, sb=16, tokens=4, top=2, experts=3, codes=A, place=A, offsets=A):
        return fake.ebc_moe_dispatch_mx(ctx, codes, cb, A, sb, tokens, top, place, offsets, experts, A, A, None)

    assert dispatch() == 0
    for wrong in (dict(cb=0), dict(cb=24), dict(cb=2 ** 24 + 16), dict(sb=8), dict(sb=0), dict(tokens=-1), dict(tokens=2 ** 30), dict(top=0),
                  dict(experts=0), dict(codes=None), dict(codes=A + 8), dict(place=None), dict(offsets=None), dict(offsets=A + 2)):
        assert dispatch(**wrong) == BAD, wrong
    fake.ebc_destroy(ctx)


def test_the_norms_gradient_stays_inside_its_scratch(fake):
    """A partial row a CTA, and no more CTAs than the scratch has rows for."""
    ctx = context(fake)
    rng = random.Random(0)
    for _ in range(500):
        rows, width = int(2 ** rng.uniform(0, 20)), int(2 ** rng.uniform(0, 14))
        for shift in (0, 2, 4, 8, 16):
            assert fake.ebc_norm_grad(ctx, A + shift, width, A, width, None, 0, 1, A, 0, rows, width, 1e-6, A, A, A + 16, None) == 0
            first, *second = launches(fake)
            assert 1 <= int(first[1]) <= min(rows, 608)
            assert [int(x[1]) for x in second] == ([-(-width // 32)] if int(first[1]) > 1 else [])   # one has nothing to add up
    fake.ebc_destroy(ctx)


def test_a_kernel_is_allowed_the_same_shared_memory_by_every_call(fake):
    """Contexts of two host threads then do not take it from each other; and every launch stays within it."""
    ctx = context(fake)
    rng = random.Random(1)
    allowed = {}
    fake.fake_static_shared(1024)
    for i in range(600):
        rows, width, kind = int(2 ** rng.uniform(0, 16)), int(2 ** rng.uniform(0, 14)) if i else 16377, rng.randrange(3)
        for shift in (0, 4):
            assert fake.ebc_norm(ctx, A + shift, width, None, 0, kind, A, 0, rows, width, 1e-6, A + shift, None, A, A, None) == 0, (rows, width)
            assert fake.ebc_norm_grad(ctx, A + shift, width, A + shift, width, A + shift, width, kind, A, 0, rows, width, 1e-6,
                                      A + shift, A, A, None) == 0, (rows, width)
        log = fake.fake_log().decode()
        fake.fake_clear()
        assert "refused" not in log
        for name, most in re.findall(r"shared (\S+) (\d+)", re.sub(r"launch.*", "", log)):
            allowed.setdefault(name, set()).add(int(most))
    fake.fake_static_shared(256)
    fake.ebc_destroy(ctx)
    assert len(allowed) > 10 and all(len(v) == 1 and max(v) <= 226 * 1024 for v in allowed.values()), allowed


def test_an_8_bit_product_takes_no_more_rows_than_its_tiles_can_count(fake):
    ctx = context(fake)
    most = 2 ** 31 - 256
    call = lambda rows, outs, experts: fake.ebc_mx8_product(ctx, A, A, rows, 32, A, A, outs, experts, A, ebc.EBC_BF16, A, None)  # noqa: E731
    for rows, outs, experts in [(most, 1, 1), (most, 4096, 32), (1, most, 1), (5, most // 2, 2), (5, most // 1024, 1024)]:
        assert call(rows, outs, experts) == 0
    for rows, outs, experts in [(most + 1, 1, 1), (2 ** 31 - 1, 1, 1), (1, most + 1, 1), (5, most // 2 + 1, 2)]:
        assert call(rows, outs, experts) == BAD
    fake.ebc_destroy(ctx)


def test_the_launches_of_8_bit_products(fake):
    """Single CTAs, pairs and clusters that share K as those of 4 bits, by the sizes; only the smallest tiles share."""
    ctx = context(fake)

    def product(rows, experts, outs, width):
        assert fake.ebc_mx8_product(ctx, A, A, rows, width, A, A, outs, experts, A, ebc.EBC_BF16, A, None) == 0
        (found,) = launches(fake)
        tile, ctas = re.search(r"k_mx8_productILi(\d+)ELi(\d)E", found[0]).groups()
        return int(tile), int(ctas), int(found[1]), int(found[2])

    assert product(16, 8, 2000, 2048) == (16, 1, 144, 1)
    assert product(2, 1, 600, 8192) == (16, 1, 40, 8)
    assert product(2048, 8, 1024, 1024)[:2] == (64, 1)
    assert product(16384, 4, 4096, 4096) == (256, 2, 152, 2)
    rng, seen = random.Random(0), set()
    for _ in range(2000):
        rows, experts = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 8))
        outs, width = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 15))
        tile, ctas, grid, cluster = product(rows, experts, outs, width)
        assert grid % cluster == 0 and grid <= 152 and (cluster == ctas or tile == 16), (rows, experts, outs, width)
        seen.add((tile, cluster))
    assert {(16, 1), (16, 8), (64, 1), (256, 2)} <= seen
    fake.ebc_destroy(ctx)


def test_the_torch_types_refuse_other_tensors():
    b, s = torch.zeros(3, 64, dtype=torch.uint8), torch.zeros(3, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        ebc.Mx8(b, s, 64)
    with pytest.raises(ValueError, match="do not hold"):
        ebc.Mx8(b, s, 65)
    with pytest.raises(ValueError, match="do not hold"):
        ebc.Mx8(b, torch.zeros(4, 16, dtype=torch.uint8), 64)


@pytest.mark.parametrize("name", ["ebc_route.cu", "ebc_norm.cu", "ebc_mx8.cu", "ebc_mx8_product.cu", "ebc_mx8.cuh", "ebc_mx_product.cuh"])
def test_kernels_that_start_early_read_with_ordinary_loads(name):
    text = open(os.path.join(ebc_build.CSRC, name)).read()
    assert name.endswith(".cuh") or "pdl_enter();" in text
    assert not re.findall(r"const\s+\w+\s*\*\s*__restrict__|__ldg|ld\.global\.nc", text)
