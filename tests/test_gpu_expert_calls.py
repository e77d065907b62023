"""The expert-parallel and 4-bit calls where what matters is not a kernel's
arithmetic but how a program makes them: processes, threads, streams, graphs."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import error_bounded_lossy_gb300 as ebc

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(program):
    """A program in a process of its own, from the repository's root."""
    r = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("experts", [359, 360, 361, 362])
def test_a_plan_whose_counts_just_fill_48_kb_in_a_fresh_process(experts):
    run(f"""
import torch
import error_bounded_lossy_gb300 as ebc
for kind in (torch.int32, torch.int64):
    ex = ebc.Experts(0)
    ids = torch.arange({experts}, device="cuda", dtype=kind)[:, None]
    plan = ex.plan(ids.flip(0).contiguous(), {experts})
    ex.check()
    assert torch.equal(plan.rows.cpu(), torch.arange({experts}, dtype=torch.int32).flip(0))
    assert torch.equal(plan.offsets.cpu(), torch.arange({experts} + 1, dtype=torch.int32))
    ex.close()
""")


def test_plans_of_different_sizes_in_two_threads():
    """Each thread has a context of its own; the C calls run without the interpreter's lock."""
    ids = torch.from_numpy(np.random.default_rng(0).integers(0, 400, (512, 2)).astype(np.int32)).cuda()
    torch.cuda.synchronize()
    failed = []

    def plans(experts):
        h = ebc.ebc_create(0)
        out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (1024, 1024, experts + 1)]
        stream = torch.cuda.Stream()
        for _ in range(3000):
            rc = ebc.ebc_moe_plan(h, ids.data_ptr(), 4, 512, 2, experts, *(t.data_ptr() for t in out), stream.cuda_stream)
            if rc:
                failed.append((experts, rc))
                break
        stream.synchronize()
        ebc.ebc_destroy(h)

    threads = [threading.Thread(target=plans, args=(e,)) for e in (400, ebc.EBC_MAX_EXPERTS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


@pytest.mark.parametrize("rows,experts,outs,width", [(6000, 4, 4000, 1024), (16384, 4, 4096, 32), (16384, 4, 4096, 288), (16384, 3, 4096, 4000)])
def test_a_pair_that_gives_up_with_one_of_its_ctas_ahead(rows, experts, outs, width):
    """The first CTA of each pair gives up before it has asked for anything, the second has asked for as many stages
    as fit: both wait for what is in flight, the status says so, and what comes after on the stream is right."""
    e = ebc.Experts(0)
    g = torch.Generator("cuda").manual_seed(rows)
    x = e.quantize(torch.randn(rows, width, generator=g, device="cuda"))
    w = e.quantize(torch.randn(experts, outs, width, generator=g, device="cuda"))
    cut = torch.tensor([rows * i // experts for i in range(experts + 1)], dtype=torch.int32, device="cuda")
    want = e.product(x, w, cut)
    e.check()
    for _ in range(3):
        assert ebc.ebc_set_first_wait_polls(e.handle, 0) == 0
        e.product(x, w, cut)
        assert ebc.ebc_set_first_wait_polls(e.handle, -1) == 0
        again = e.product(x, w, cut)   # starts as soon as the CTAs that gave up have gone
        with pytest.raises(ebc.EbcError) as err:
            e.check()
        assert err.value.code == ebc.EBC_ERR_DEVICE_TIMEOUT
        assert torch.equal(again, want)
    e.close()


def test_a_check_finds_an_error_of_an_earlier_stream_and_of_a_replay():
    e = ebc.Experts(0)
    ids = {k: torch.full((4, 2), v, dtype=torch.int32, device="cuda") for k, v in (("good", 0), ("bad", 99))}
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        torch.cuda._sleep(100_000_000)   # about 50 ms
    e.plan(ids["bad"], 4, stream=a)
    e.plan(ids["good"], 4, stream=b)
    with pytest.raises(ebc.EbcError):
        e.check()
    e.check()
    given = ids["good"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e.plan(given, 4)
    given.copy_(ids["bad"])
    torch.cuda.synchronize()
    for _ in range(2):
        with torch.cuda.stream(a):
            torch.cuda._sleep(100_000_000)
            graph.replay()
        with pytest.raises(ebc.EbcError):
            e.check()
    e.check()
    e.close()


@pytest.mark.parametrize("width", [96, 1000])
def test_4_bit_rows_of_several_ranks_to_one_product(width):
    """What a rank receives is one piece a sender, each sorted by expert: a plan of one choice a row sorts the pieces
    together (dispatch copies bits, so codes and scales go through it as fp32 rows), and combine without weights
    brings the results back into the order of arrival."""
    ex = ebc.Experts(0)
    ranks, experts, outs, top = 3, 8, 70, 2
    g = torch.Generator("cuda").manual_seed(width)
    w = ex.quantize(torch.randn(experts, outs, width, generator=g, device="cuda"))
    pieces, ids, values = [], [], []
    for r in range(ranks):
        x = torch.randn(50 + r, width, generator=g, device="cuda")
        x[3, 5] = float("inf")   # a block of NaN: the byte 255
        plan = ex.plan(torch.randint(0, experts, (50 + r, top), generator=g, device="cuda"), experts)
        pieces.append(ex.dispatch_mx4(x, plan))
        ids.append(torch.repeat_interleave(torch.arange(experts, device="cuda"), plan.offsets.diff()))
    codes, scales, e = torch.cat([q.codes for q in pieces]), torch.cat([q.scales for q in pieces]), torch.cat(ids)
    # the receiving rank
    plan = ex.plan(e[:, None], experts)
    rows = lambda t: ex.dispatch(t.view(torch.float32), plan).view(torch.uint8)  # noqa: E731
    q = ebc.Mx4(rows(codes), rows(scales), width)
    order = torch.sort(e, stable=True).indices
    assert torch.equal(q.codes, codes[order]) and torch.equal(q.scales, scales[order])
    back = ex.combine(ex.product(q, w, plan.offsets, torch.float32), None, plan)
    ex.check()
    x64 = ex.dequantize(ebc.Mx4(codes, scales, width)).double()
    w64 = ex.dequantize(w).double()
    want = torch.einsum("rk,rok->ro", x64, w64[e])
    size = torch.einsum("rk,rok->ro", x64.abs(), w64[e].abs())
    assert torch.equal(back.isnan(), want.isnan()) and want.isnan().any()
    off = (back.double() - want).abs().nan_to_num(nan=0.0)
    # width exact products summed in 32 bits, one unit in the last place an addition
    assert bool((off <= (width + 1) * 2.0 ** -23 * size.nan_to_num(nan=1.0)).all())
    ex.close()
