"""Refusals of the 8-bit block-scaled calls: every call here fails its host checks or is empty, so none
reaches a kernel (no GPU needed)."""
import ctypes as C

import pytest
import torch

P = C.c_void_p
G = P(0x1000)
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def bnn():
    from ternary_neural_net_b200 import bnn as mod
    return mod


def test_pack_rows_refusals(bnn):
    f = bnn.lib().bnn_fp8_pack_rows
    bad, mis = bnn.BNN_ERR_INVALID_ARG, bnn.BNN_ERR_MISALIGNED
    assert f(G, 3, 1, None, 1, 8, G, G, None) == bad                     # unknown type
    assert f(G, -1, 1, None, 1, 8, G, G, None) == bad
    assert f(G, F32, -1, G, 1, 8, G, G, None) == bad                     # negative sizes
    assert f(G, F32, 1, None, -1, 8, G, G, None) == bad
    assert f(G, F32, 1, None, 1, -8, G, G, None) == bad
    assert f(G, F32, 1, None, 2, 8, G, G, None) == bad                   # fewer rows of x than asked for
    assert f(G, F32, 1 << 31, G, 1, 8, G, G, None) == bad                # too large
    assert f(G, F32, 1, G, 1 << 31, 8, G, G, None) == bad
    assert f(G, F32, 1, None, 1, bnn.MAX_K_FP8 + 1, G, G, None) == bad
    assert f(None, F32, 1, None, 1, 8, G, G, None) == bad                # missing pointers
    assert f(G, F32, 1, None, 1, 8, None, G, None) == bad
    assert f(G, F32, 1, None, 1, 8, G, None, None) == bad
    assert f(P(0x1002), F32, 1, None, 1, 8, G, G, None) == mis           # misaligned
    assert f(P(0x1001), BF16, 1, None, 1, 8, G, G, None) == mis
    assert f(G, F16, 1, P(0x1002), 1, 8, G, G, None) == mis
    assert f(G, F32, 1, None, 1, 8, P(0x1008), G, None) == mis
    assert f(G, F32, 1, None, 1, 8, G, P(0x1002), None) == mis
    assert f(None, F32, 0, None, 0, 8, None, None, None) == bnn.BNN_OK   # empty
    assert f(G, BF16, 5, None, 5, 0, None, None, None) == bnn.BNN_OK


def test_pack_weight_refusals(bnn):
    f = bnn.lib().bnn_fp8_pack_weight
    bad, mis = bnn.BNN_ERR_INVALID_ARG, bnn.BNN_ERR_MISALIGNED
    assert f(G, 7, 1, 4, 8, G, G, None) == bad
    assert f(G, F32, -1, 4, 8, G, G, None) == bad
    assert f(G, F32, 1, -4, 8, G, G, None) == bad
    assert f(G, F32, 1, 4, -8, G, G, None) == bad
    assert f(G, F32, bnn.MAX_GROUPS + 1, 4, 8, G, G, None) == bad
    assert f(G, F32, 1, 1 << 31, 8, G, G, None) == bad
    assert f(G, F32, 1024, 1 << 21, 8, G, G, None) == bad                # groups * n
    assert f(G, F32, 1, 4, bnn.MAX_K_FP8 + 1, G, G, None) == bad
    assert f(None, F32, 1, 4, 8, G, G, None) == bad
    assert f(G, F32, 1, 4, 8, None, G, None) == bad
    assert f(G, F32, 1, 4, 8, G, None, None) == bad
    assert f(P(0x1002), F32, 1, 4, 8, G, G, None) == mis
    assert f(G, BF16, 1, 4, 8, P(0x1004), G, None) == mis
    assert f(G, BF16, 1, 4, 8, G, P(0x1001), None) == mis
    for g, n, k in ((0, 4, 8), (1, 0, 8), (1, 4, 0)):
        assert f(None, F32, g, n, k, None, None, None) == bnn.BNN_OK


def test_gemm_refusals(bnn):
    f = bnn.lib().bnn_fp8_gemm
    bad, mis = bnn.BNN_ERR_INVALID_ARG, bnn.BNN_ERR_MISALIGNED

    def call(xq=G, xs=G, wq=G, ws=G, bias=None, m=1, n=1, k=8, out=G, ot=F32):
        return f(xq, xs, wq, ws, bias, m, n, k, out, ot, None)
    for kw in (dict(m=-1), dict(n=-1), dict(k=-1), dict(m=1 << 31), dict(n=1 << 31), dict(k=bnn.MAX_K_FP8 + 1),
               dict(ot=3), dict(ot=-1), dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None), dict(out=None),
               dict(out=None, k=0)):
        assert call(**kw) == bad, kw
    for kw in (dict(xq=P(0x1008)), dict(wq=P(0x1008)), dict(xs=P(0x1002)), dict(ws=P(0x1001)), dict(bias=P(0x1002)),
               dict(out=P(0x1002)), dict(out=P(0x1001), ot=BF16), dict(out=P(0x1001), ot=F16)):
        assert call(**kw) == mis, kw
    assert call(None, None, None, None, m=0, out=None) == bnn.BNN_OK
    assert call(None, None, None, None, n=0, out=None) == bnn.BNN_OK


def test_grouped_refusals(bnn):
    f = bnn.lib().bnn_fp8_grouped_gemm
    bad, mis = bnn.BNN_ERR_INVALID_ARG, bnn.BNN_ERR_MISALIGNED

    def call(xq=G, xs=G, wq=G, ws=G, off=G, g=2, rows=1, n=1, k=8, out=G, ot=F32):
        return f(xq, xs, wq, ws, off, g, rows, n, k, out, ot, None)
    for kw in (dict(g=-1), dict(g=bnn.MAX_GROUPS + 1), dict(rows=-1), dict(n=-1), dict(k=-1), dict(rows=1 << 31),
               dict(g=1024, n=1 << 21), dict(k=bnn.MAX_K_FP8 + 1), dict(ot=5), dict(xq=None), dict(xs=None),
               dict(wq=None), dict(ws=None), dict(off=None), dict(out=None), dict(off=None, k=0)):
        assert call(**kw) == bad, kw
    for kw in (dict(xq=P(0x1004)), dict(wq=P(0x1004)), dict(xs=P(0x1002)), dict(ws=P(0x1002)), dict(off=P(0x1004)),
               dict(out=P(0x1002)), dict(out=P(0x1001), ot=BF16)):
        assert call(**kw) == mis, kw
    for kw in (dict(g=0), dict(rows=0), dict(n=0)):
        assert call(None, None, None, None, None, out=None, **kw) == bnn.BNN_OK


def test_binding_rejects_host_tensors(bnn):
    q = torch.zeros(2, 128).to(torch.float8_e4m3fn)
    s = torch.zeros(1, 2)
    with pytest.raises(ValueError):
        bnn.bnn_fp8_pack_rows(torch.zeros(2, 3))
    with pytest.raises(ValueError):
        bnn.bnn_fp8_pack_weight(torch.zeros(2, 3))
    with pytest.raises(ValueError):
        bnn.bnn_fp8_gemm(q, s, q, torch.zeros(1, 1))
    with pytest.raises(ValueError):
        bnn.bnn_fp8_grouped_gemm(q, s, q[None], torch.zeros(1, 1, 1), torch.zeros(2, dtype=torch.int64))
