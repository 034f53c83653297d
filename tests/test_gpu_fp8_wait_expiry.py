"""Failure detection of the e4m3 products without a fault: their tensor-core kernels bound every wait.  With
the roles' waits cut to a few polls (bnn_probe_wait_limit) they run out before the first copies land, or
somewhere on the way.  The kernel must count the run-outs, wait for its own copies and MMAs, free its tensor
memory and return normally, and with the first waits run out it must have stored nothing.  The next normal
call gives the bits of the call before."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import fp8
from ternary_neural_net_b200 import synth

pytestmark = pytest.mark.gpu

# (m, n, k, groups): each kernel and shape with waits (test_fp8_plan.py has the kernel of each size)
CASES = [
    (16, 300, 640, 0),        # weights on the lanes, 16 rows, split over 2 CTAs
    (12, 400, 1024, 0),       # 4 CTAs
    (16, 1000, 8192, 0),      # 8 CTAs
    (16, 40000, 300, 0),      # no split, several tiles a CTA
    (24, 300, 640, 0),        # 32 rows, 2 CTAs
    (24, 400, 1024, 0),       # 4 CTAs
    (20, 500, 8192, 0),       # 8 CTAs
    (30, 40000, 300, 0),      # no split
    (64, 1000, 8192, 0),      # 128 x 32 tiles
    (300, 2000, 4100, 0),     # 128 x 64
    (3000, 9100, 1100, 0),    # 128 x 128, several tiles each
    (1101, 2304, 2000, 0),    # CTA pairs, 256 x 256
    (2048, 4600, 2000, 0),    # pairs, several tiles each
    (200, 300, 2000, 20),     # groups, 16 rows
    (200, 300, 2000, 8),      # 32 rows
    (900, 700, 2000, 4),      # 128 x 128
    (4000, 4100, 2000, 4),    # 128 x 256
]


@pytest.fixture(scope="module")
def bnn(cuda_device):
    from ternary_neural_net_b200 import bnn as mod
    return mod


def _limit(bnn, polls):
    f = bnn.lib().bnn_probe_wait_limit
    f.argtypes = [C.c_uint32]
    f.restype = C.c_int
    assert f(polls) == bnn.BNN_OK


def _case(bnn, m, n, k, groups):
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n + k)
    x = torch.randn((m, k), device="cuda", generator=g)
    w = torch.randn((groups, n, k) if groups else (n, k), device="cuda", generator=g) * 0.05
    ops = (*bnn.bnn_fp8_pack_rows(x), *bnn.bnn_fp8_pack_weight(w))
    if not groups:
        return lambda out: bnn.bnn_fp8_gemm(*ops, out=out)
    offsets = torch.tensor([m * i // groups for i in range(groups + 1)], device="cuda")
    return lambda out: bnn.bnn_fp8_grouped_gemm(*ops, offsets, out=out)


@pytest.mark.parametrize("m,n,k,groups", CASES)
def test_waits_run_out_then_a_normal_call_is_the_same(bnn, m, n, k, groups):
    call = _case(bnn, m, n, k, groups)
    want = call(torch.empty((m, n), device="cuda"))
    torch.cuda.synchronize()
    assert bnn.device_error_count(reset=True) == 0
    out = torch.full((m, n), float("nan"), device="cuda")
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for polls in (1, 2, 4, 8, 16, 32, 64, 128, 256, 512):
        _limit(bnn, polls)
        try:
            out.fill_(float("nan"))
            begin.record()
            call(out)
            end.record()
            torch.cuda.synchronize()
        finally:
            _limit(bnn, 0)
        # the final waits keep their bound of 2^20 polls, 30 ms at the least: none of them ran out
        assert begin.elapsed_time(end) < 20.0, polls
        count = bnn.device_error_count(reset=True)
        if polls == 1:
            assert count > 0, "no wait ran out"
            assert bool(torch.isnan(out).all()), "a CTA stored without its sums"
        elif count == 0:
            assert torch.equal(out, want)
        # what is stored is right: a role that gave up stores nothing
        stored = ~torch.isnan(out)
        assert torch.equal(out[stored], want[stored]), polls
        # and nothing of it is left for the next call
        assert torch.equal(call(torch.empty((m, n), device="cuda")), want), polls
        torch.cuda.synchronize()
        assert bnn.device_error_count(reset=True) == 0


def test_a_limited_call_between_others(bnn):
    """Calls enqueued right before and behind one whose waits run out, which start while it still runs, are exact."""
    calls = [_case(bnn, *c) for c in ((16, 4000, 4096, 0), (1101, 2304, 2000, 0), (300, 2000, 4100, 0))]
    shapes = [(16, 4000), (1101, 2304), (300, 2000)]
    want = [c(torch.empty(s, device="cuda")) for c, s in zip(calls, shapes)]
    torch.cuda.synchronize()
    bnn.device_error_count(reset=True)
    for bad in range(3):
        got = [c(torch.empty(s, device="cuda")) for c, s in zip(calls, shapes)]
        _limit(bnn, 1)
        try:
            calls[bad](torch.empty(shapes[bad], device="cuda"))
        finally:
            _limit(bnn, 0)
        got += [c(torch.empty(s, device="cuda")) for c, s in zip(calls, shapes)]
        torch.cuda.synchronize()
        assert bnn.device_error_count(reset=True) > 0
        for y, w in zip(got, want * 2):
            assert torch.equal(y, w)


def test_products_agree_with_the_oracle_after_a_run_out(bnn):
    m, n, k = 16, 300, 640
    xq, xs = fp8.pack_rows(synth.normal_f32(1, 1, (m, k)))
    wq, ws = fp8.pack_weight(synth.normal_f32(1, 2, (1, n, k)))
    d = [torch.from_numpy(a).cuda() for a in (xq, xs, wq[0], ws[0])]
    d[0], d[2] = d[0].view(torch.float8_e4m3fn), d[2].view(torch.float8_e4m3fn)
    _limit(bnn, 1)
    try:
        bnn.bnn_fp8_gemm(*d)
        torch.cuda.synchronize()
    finally:
        _limit(bnn, 0)
    assert bnn.device_error_count(reset=True) > 0
    y, mag = fp8.gemm(xq, xs, wq[0], ws[0])
    # 128 steps of a block's float32 sum, and a rounding each for the scale product, its use, the kb additions and the output
    lim = (128 * 2.0 ** -23 + (fp8.blocks(k) + 4) * 2.0 ** -24) * mag
    assert np.all(np.abs(bnn.bnn_fp8_gemm(*d).double().cpu().numpy() - y) <= lim)
    assert bnn.device_error_count() == 0
