"""What the expert-parallel and 4-bit calls do on the host: the library's
objects linked with a CUDA runtime without a device (fake_cudart.cpp), which
writes down the calls that reach it."""
import ctypes
import os
import random
import re
import shutil
import subprocess
import threading

import pytest

import error_bounded_lossy_gb300 as ebc
from error_bounded_lossy_gb300 import build as ebc_build

HERE = os.path.dirname(os.path.abspath(__file__))
A = 1 << 20   # an address that is aligned to anything; nothing reads it


class Fake:
    """The library on the runtime without a device."""

    def __init__(self, path):
        self.lib = L = ctypes.CDLL(path)
        P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        for name, args in {
            "ebc_create": [P, P, I], "ebc_last_device_error": [P],
            "ebc_moe_plan": [P, P, I, I64, I, I, P, P, P, P],
            "ebc_moe_dispatch": [P, P, I64, I, I64, I, I64, P, P, I, P, P],
            "ebc_moe_combine": [P, P, I64, I, I64, I, I64, P, P, P, P],
            "ebc_moe_combine_grad": [P, P, I64, P, I64, I, I64, I, I64, P, P, I, P, P, P, P],
            "ebc_mx4_quantize": [P, P, I64, I, I64, I64, P, P, P],
            "ebc_mx4_dequantize": [P, P, P, I64, I64, I, P, P],
            "ebc_moe_dispatch_mx4": [P, P, I64, I, I64, I, I64, P, P, I, P, P, P],
            "ebc_mx4_product": [P, P, P, I64, I64, P, P, I64, I, P, I, P, P],
            "ebc_compress": [P, P, I64, I, I, P, P, ctypes.c_uint64, P, P],
            "cudaSetDevice": [I], "cudaGetDevice": [P], "fake_max_clusters": [I], "fake_static_shared": [I],
        }.items():
            getattr(L, name).argtypes = args
        L.ebc_destroy.argtypes = [P]
        L.ebc_destroy.restype = None
        L.fake_log.restype = ctypes.c_char_p

    def context(self, device=0):
        h = ctypes.c_void_p()
        assert self.lib.ebc_create(ctypes.byref(h), None, device) == 0
        self.log()
        return h

    def log(self):
        """The calls since the last look."""
        lines = self.lib.fake_log().decode().splitlines()
        self.lib.fake_clear()
        return lines

    def launches(self):
        return [m.groupdict() for m in (re.match(
            r"launch (?P<name>\S+) grid (?P<grid>\d+) cluster (?P<cluster>\d+) shared (?P<shared>\d+) "
            r"stream (?P<stream>\S+) device (?P<device>\d+)(?P<refused> refused)?", s) for s in self.log()) if m]

    def product(self, ctx, rows, experts, outs, width, out_type=ebc.EBC_BF16, stream=None):
        rc = self.lib.ebc_mx4_product(ctx, A, A, rows, width, A, A, outs, experts, A, out_type, A, stream)
        assert rc == 0
        (launch,) = self.launches()
        tile, ctas = re.search(r"k_mx4_productILi(\d+)ELi(\d)E", launch["name"]).groups()
        return int(tile), int(ctas), int(launch["cluster"])

    def plan(self, ctx, experts, tokens=64, top=2, id_bytes=4, stream=None):
        return self.lib.ebc_moe_plan(ctx, A, id_bytes, tokens, top, experts, A, A, A, stream)


@pytest.fixture(scope="module")
def path(tmp_path_factory):
    ebc_build.build()
    d = tmp_path_factory.mktemp("fake")
    out = str(d / "libebc_fake.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(ebc_build.nvcc())), "include")
    objs = [os.path.join(ebc_build.BUILD, s.replace(".cu", ".o")) for s in ebc_build.SOURCES]
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wl,-Bsymbolic", f"-I{cuda}", "-o", out,
                    os.path.join(HERE, "fake_cudart.cpp"), *objs], check=True)
    return out


@pytest.fixture
def fake(path):
    f = Fake(path)
    f.lib.cudaSetDevice(0)
    f.log()
    return f


def test_a_plan_fits_its_shared_memory_whatever_was_planned_before(fake):
    """The counts of 360 experts leave no room in 48 KB for the kernel's own variables; and what a plan of fewer
    experts allows itself must not take from one of more that another thread is about to launch."""
    ctx = fake.context()
    for experts in (1, 359, 360, 361, 362, 400, ebc.EBC_MAX_EXPERTS, 400, ebc.EBC_MAX_EXPERTS):
        for id_bytes in (4, 8):
            assert fake.plan(ctx, experts, id_bytes=id_bytes) == 0, experts
    most = 4 * (32 * (ebc.EBC_MAX_EXPERTS | 1) + 2 * ebc.EBC_MAX_EXPERTS)
    allowed = [int(s.split()[-1]) for s in fake.log() if s.startswith("shared") and "plan" in s]
    assert allowed and set(allowed) == {most}
    fake.lib.ebc_destroy(ctx)


def test_the_sizes_of_the_time_out_tests_reach_single_ctas_pairs_and_clusters(fake):
    ctx = fake.context()
    assert fake.product(ctx, 16, 8, 2000, 2048) == (16, 1, 1)
    assert fake.product(ctx, 2, 1, 600, 8192)[1:] == (1, 8)
    for rows, experts, outs, width in [(6000, 4, 4000, 1024), (16384, 4, 4096, 32), (16384, 4, 4096, 288), (16384, 3, 4096, 4000)]:
        assert fake.product(ctx, rows, experts, outs, width) == (256, 2, 2)
    fake.lib.ebc_destroy(ctx)


def test_a_product_takes_no_more_rows_than_its_tiles_can_count(fake):
    """A tile of 256 that starts at the last row or output must end inside 31 bits."""
    ctx = fake.context()
    most = 2 ** 31 - 256
    call = lambda rows, outs, experts: fake.lib.ebc_mx4_product(  # noqa: E731
        ctx, A, A, rows, 32, A, A, outs, experts, A, ebc.EBC_BF16, A, None)
    for rows, outs, experts in [(most, 1, 1), (most, 4096, 32), (1, most, 1), (5, most // 2, 2), (5, most // 1024, 1024)]:
        assert call(rows, outs, experts) == 0
    for rows, outs, experts in [(most + 1, 1, 1), (2 ** 31 - 1, 1, 1), (1, most + 1, 1), (5, most // 2 + 1, 2)]:
        assert call(rows, outs, experts) == ebc.EBC_ERR_INVALID_ARG
    fake.lib.ebc_destroy(ctx)


def test_a_check_waits_for_every_stream_of_the_experts_calls(fake):
    """An error may come from any of the streams, or from a graph's replay."""
    ctx = fake.context()
    # the codec's calls share a scratch, so they are ordered: the last stream is enough
    assert fake.lib.ebc_compress(ctx, A, 0, 1, 16, (ctypes.c_float * 1)(0.1), A, 1 << 20, A, 0x70) == 0
    fake.log()
    assert fake.lib.ebc_last_device_error(ctx) == 0
    assert [s for s in fake.log() if s.startswith("sync")] == ["sync stream 0x70"]
    for stream in (0x10, 0x20):
        assert fake.plan(ctx, 4, stream=stream) == 0
    for _ in range(2):   # a graph may be replayed after a check, too
        fake.log()
        assert fake.lib.ebc_last_device_error(ctx) == 0
        assert "sync device 0" in fake.log()
    fake.lib.ebc_destroy(ctx)


def test_the_callers_device_stays_current(fake):
    """A context of another device than the thread's current one: kernels are launched there, and the thread's device
    is what it was, also where a launch fails."""
    lib, now = fake.lib, ctypes.c_int(-1)
    ctx = fake.context(1)
    calls = {
        "plan": lambda: fake.plan(ctx, 4),
        "dispatch": lambda: lib.ebc_moe_dispatch(ctx, A, 8, 0, 4, 2, 8, A, A, 3, A, None),
        "combine": lambda: lib.ebc_moe_combine(ctx, A, 8, 0, 4, 2, 8, A, A, A, None),
        "combine_grad": lambda: lib.ebc_moe_combine_grad(ctx, A, 8, A, 8, 0, 4, 2, 8, A, A, 3, A, A, A, None),
        "quantize": lambda: lib.ebc_mx4_quantize(ctx, A, 64, 0, 4, 64, A, A, None),
        "dequantize": lambda: lib.ebc_mx4_dequantize(ctx, A, A, 4, 64, 0, A, None),
        "dispatch_mx4": lambda: lib.ebc_moe_dispatch_mx4(ctx, A, 64, 0, 4, 2, 64, A, A, 3, A, A, None),
        "product": lambda: lib.ebc_mx4_product(ctx, A, A, 4, 64, A, A, 16, 2, A, 0, A, None),
    }
    for device in (0, 1):
        lib.cudaSetDevice(device)
        for name, call in calls.items():
            assert call() == 0, name
            assert lib.cudaGetDevice(ctypes.byref(now)) == 0 and now.value == device, name
            assert [x["device"] for x in fake.launches()] == ["1"], name
    lib.cudaSetDevice(0)
    lib.fake_static_shared(1 << 20)   # no launch fits
    for name, call in calls.items():
        assert call() == ebc.EBC_ERR_CUDA, name
        assert lib.cudaGetDevice(ctypes.byref(now)) == 0 and now.value == 0, name
    lib.fake_static_shared(256)
    lib.ebc_destroy(ctx)


def test_the_torch_class_makes_its_contexts_own_calls_under_its_device(monkeypatch):
    """Creating, checking and closing a context leave its device current; the class puts the caller's back."""
    import contextlib
    import torch
    from error_bounded_lossy_gb300 import experts
    inside, seen = [], []

    @contextlib.contextmanager
    def device(d):
        inside.append(d)
        yield
        inside.pop()

    def call(result):
        return lambda *a: (seen.append(list(inside)), result)[1]

    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(experts, "ebc_create", call(ctypes.c_void_p(8)))
    for name in ("ebc_last_device_error", "ebc_set_profiling", "ebc_destroy"):
        monkeypatch.setattr(experts, name, call(0))
    ex = experts.Experts(1)
    ex.check()
    ex.set_profiling(False)
    ex.close()
    assert seen == [[torch.device("cuda", 1)]] * 4


def test_the_first_products_of_several_threads(path, tmp_path):
    """The driver's entry point is looked up once, by one of them."""
    fake = Fake(shutil.copy(path, tmp_path / "libebc_first.so"))   # (nothing has been looked up in this copy)
    ctxs = [fake.context() for _ in range(4)]
    rcs = []
    threads = [threading.Thread(target=lambda c=c: rcs.append(
        fake.lib.ebc_mx4_product(c, A, A, 4, 64, A, A, 16, 2, A, 0, A, None))) for c in ctxs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert rcs == [0] * 4
    assert sum(s.startswith("entry point") for s in fake.log()) == 1
    for c in ctxs:
        fake.lib.ebc_destroy(c)


def test_a_large_plans_cluster_is_one_that_fits(fake):
    """Sixteen CTAs are more than a cluster has everywhere: where none fits, eight."""
    for fits, cluster in ((8, "16"), (0, "8")):
        fake.lib.fake_max_clusters(fits)
        ctx = fake.context()
        for tokens in (8192, 100000):
            for id_bytes in (4, 8):
                assert fake.plan(ctx, 64, tokens=tokens, id_bytes=id_bytes) == 0
                assert [x["cluster"] for x in fake.launches()] == [cluster]
        assert fake.plan(ctx, 64, tokens=512) == 0
        assert [x["cluster"] for x in fake.launches()] == ["1"]
        fake.lib.ebc_destroy(ctx)
    fake.lib.fake_max_clusters(8)


def test_only_the_smallest_tiles_share_their_sums(fake):
    """The kernels of larger tiles have no code for it."""
    ctx = fake.context()
    rng = random.Random(0)
    shared = 0
    for _ in range(4000):
        rows, experts = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 8))
        outs, width = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 15))
        tile, ctas, cluster = fake.product(ctx, rows, experts, outs, width)
        assert cluster == ctas or tile == 16, (rows, experts, outs, width)
        shared += cluster > ctas
    assert shared > 200
    fake.lib.ebc_destroy(ctx)
