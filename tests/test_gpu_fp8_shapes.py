"""The 8-bit calls at sizes that take the kernels and tile shapes which small sizes do not reach (test_fp8_plan.py
has the kernel of each): CTA pairs, groups in 128 x 256 tiles, and the weights on the tensor-memory lanes with
a bias, in every output type, and with more tiles than CTAs.  Tolerances as derived in test_gpu_fp8.py."""
import functools

import numpy as np
import pytest
import torch

from gpu_util import to_dev_f32
from oracle import fp8
from ternary_neural_net_b200 import synth
from test_gpu_fp8 import OUTS, activations, assert_close, codes_of, offsets_of, on_dev, packed_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bnn(cuda_device):
    from ternary_neural_net_b200 import bnn as mod
    return mod


LANES = [(9, 131, 260), (16, 300, 640), (12, 400, 1024), (16, 1000, 8192), (16, 40000, 300), (1, 28672, 1280),
         (5, 28672, 1200), (24, 300, 640), (24, 400, 1024), (24, 700, 4100), (32, 129, 4100), (30, 40000, 300)]
PAIRS = [(1101, 2304, 2000), (1101, 2307, 2000), (2048, 4600, 2000)]


@functools.lru_cache(maxsize=2)
def _dense(m, n, k, with_bias):
    ops = packed_case(m + n + k, m, n, k)
    bias = synth.normal_f32(m, 9, (n,)) * np.float32(3.0) if with_bias else None
    return ops, bias, *fp8.gemm(*ops, bias)


@pytest.mark.parametrize("out", list(OUTS))
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("m,n,k", LANES + PAIRS)
def test_types_bias_and_bases(bnn, m, n, k, with_bias, out):
    ops, bias, y, mag = _dense(m, n, k, with_bias)
    d, b = on_dev(*ops), to_dev_f32(bias) if with_bias else None
    got = bnn.bnn_fp8_gemm(*d, b, out_dtype=OUTS[out][0])
    assert_close(got, y, mag, fp8.blocks(k), out, f"{m}x{n}x{k} {out}")
    # the same bits into a base that only the element's alignment holds, and into an aligned one; around it nothing
    buf = torch.empty((m * n + 40,), dtype=OUTS[out][0], device="cuda")
    for off in (1, 8):
        buf.fill_(3.0)
        bnn.bnn_fp8_gemm(*d, b, out=buf[off:off + m * n].view(m, n))
        assert torch.equal(buf[off:off + m * n].view(m, n), got)
        assert bool((buf[:off] == 3).all()) and bool((buf[off + m * n:] == 3).all())
    assert bnn.device_error_count() == 0


@pytest.mark.parametrize("m,n,k", [(1101, 2307, 2000), (16, 40000, 300), (24, 700, 4100), (16, 1000, 8192)])
def test_nan_stays_in_its_row_and_column(bnn, m, n, k):
    xq, xs, wq, ws = packed_case(3, m, n, k)
    xs, wq = xs.copy(), wq.copy()
    xs[1, m // 2] = np.nan
    wq[n - 2, 77] = 0x7f  # e4m3 NaN
    y = bnn.bnn_fp8_gemm(*on_dev(xq, xs, wq, ws)).cpu().numpy()
    nan = np.zeros((m, n), bool)
    nan[m // 2], nan[:, n - 2] = True, True
    assert np.array_equal(np.isnan(y), nan)


def test_same_bits_again_on_streams_and_in_a_graph(bnn):
    """Calls that take the pair, the split cluster and the persistent lanes kernel, at once on two streams, and
    replayed from a graph that has them back to back."""
    cases = [on_dev(*packed_case(s, m, n, k)) for s, (m, n, k) in
             enumerate([(1101, 2307, 2000), (24, 700, 4100), (16, 40000, 300), (2048, 4600, 2000)])]
    torch.cuda.synchronize()
    first = [bnn.bnn_fp8_gemm(*c) for c in cases]
    torch.cuda.synchronize()
    streams, again = [torch.cuda.Stream() for _ in range(2)], []
    for rep in range(3):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[(i + rep) % 2]):
                again.append((i, bnn.bnn_fp8_gemm(*c)))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [bnn.bnn_fp8_gemm(*c) for c in cases]
    for rep in range(3):
        for y in outs:
            y.fill_(float("nan"))
        graph.replay()
        again += [(i, y.clone()) for i, y in enumerate(outs)]
    torch.cuda.synchronize()
    for i, y in again:
        assert torch.equal(y, first[i]), i
    assert bnn.device_error_count() == 0


@pytest.mark.parametrize("m,n,k,g", [(3, 1000, 2000, 0), (16, 300, 640, 0), (24, 700, 4100, 0), (16, 40000, 300, 0),
                                     (64, 1000, 8192, 0), (300, 2000, 4100, 0), (600, 3000, 760, 0), (1101, 2307, 2000, 0),
                                     (200, 300, 2000, 20), (200, 300, 2000, 8), (900, 700, 2000, 4), (300, 2707, 2000, 8)])
def test_operands_packed_right_before(bnn, m, n, k, g):
    """Rows and weights packed right before the product that reads them, over and over with other values in the same
    buffers and nothing in between: the product starts early and must wait for each of them."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(m + n)
    xs = [torch.randn((m, k), device="cuda", generator=gen) for _ in range(4)]
    ws = [torch.randn((g, n, k) if g else (n, k), device="cuda", generator=gen) for _ in range(4)]
    off = torch.tensor([m * i // g for i in range(g + 1)], device="cuda") if g else None
    ops = (*bnn.bnn_fp8_pack_rows(xs[0]), *bnn.bnn_fp8_pack_weight(ws[0]))

    def product():
        return bnn.bnn_fp8_grouped_gemm(*ops, off) if g else bnn.bnn_fp8_gemm(*ops)

    def both(i, wait):
        bnn.bnn_fp8_pack_rows(xs[i], q=ops[0], scale=ops[1])
        bnn.bnn_fp8_pack_weight(ws[i], q=ops[2], scale=ops[3])
        if wait:
            torch.cuda.synchronize()
        first = product()
        bnn.bnn_fp8_pack_rows(xs[(i + 1) % 4], q=ops[0], scale=ops[1])
        if wait:
            torch.cuda.synchronize()
        return first, product()
    want = [both(i, True) for i in range(4)]
    torch.cuda.synchronize()
    got = [(i, *both(i, False)) for _ in range(4) for i in range(4)]
    torch.cuda.synchronize()
    for i, a, b in got:
        assert torch.equal(a, want[i][0]) and torch.equal(b, want[i][1]), i
    assert bnn.device_error_count() == 0


# groups in 128 x 256 tiles: ragged, empty ones, rows before and behind
WIDE_SIZES, WIDE_N, WIDE_K = [0, 7, 129, 0, 1, 100, 43, 5], 2707, 2000


@functools.lru_cache(maxsize=1)
def _wide():
    offsets = offsets_of(WIDE_SIZES, 3)
    rows = int(offsets[-1]) + 12
    ops = packed_case(rows, rows, WIDE_N, WIDE_K, len(WIDE_SIZES))
    return offsets, ops, *fp8.grouped_gemm(*ops, offsets)


@pytest.mark.parametrize("out", list(OUTS))
@pytest.mark.parametrize("base", [0, 1])
def test_grouped_wide_tiles(bnn, out, base):
    offsets, ops, y, mag, live = _wide()
    rows = len(live)
    assert rows == 300  # (as in test_fp8_plan.py)
    buf = torch.full((rows * WIDE_N + 8,), 7.0, dtype=OUTS[out][0], device="cuda")
    got = buf[base:base + rows * WIDE_N].view(rows, WIDE_N)
    bnn.bnn_fp8_grouped_gemm(*on_dev(*ops), torch.from_numpy(offsets).cuda(), out=got)
    lt = torch.from_numpy(live).cuda()
    assert_close(got[lt], y[live], mag[live], fp8.blocks(WIDE_K), out, "grouped")
    assert bool((got[~lt] == 7).all()) and bool((buf[:base] == 7).all()) and bool((buf[base + rows * WIDE_N:] == 7).all())
    assert bnn.device_error_count() == 0


def test_grouped_wide_tiles_keep_nan_out(bnn):
    """NaN in the rows around a group, and in the other experts' weights, reaches nothing of it."""
    offsets, (xq, xs, wq, ws), y, mag, _ = _wide()
    a, b = int(offsets[2]), int(offsets[3])
    other = np.arange(len(xq))
    other = (other < a) | (other >= b)
    experts = [g for g in range(len(WIDE_SIZES)) if g != 2]
    xq, xs, wq, ws = xq.copy(), xs.copy(), wq.copy(), ws.copy()
    xq[other], wq[experts] = 0x7f, 0xff
    xs[:, other], ws[experts] = np.nan, np.inf
    got = bnn.bnn_fp8_grouped_gemm(*on_dev(xq, xs, wq, ws), torch.from_numpy(offsets).cuda())
    assert_close(got[a:b], y[a:b], mag[a:b], fp8.blocks(WIDE_K), "f32", "clean group")


# ------------------------------------------------------------------------------------------ packs
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_pack_weight_one_bad_block_among_good_ones(bnn, dtype):
    """An infinity or a NaN takes its own 128 x 128 block and none beside, below or in the next expert."""
    w = torch.from_numpy(synth.normal_f32(5, 4, (2, 300, 520))).to(dtype)
    w[0, 130, 140], w[0, 299, 519], w[1, 5, 300] = float("nan"), float("inf"), -float("inf")
    want_q, want_s = fp8.pack_weight(w.float().numpy())
    bad = np.zeros((2, 3, 5), bool)
    bad[0, 1, 1] = bad[0, 2, 4] = bad[1, 0, 2] = True
    assert np.array_equal(np.isnan(want_s), bad)
    q, s = bnn.bnn_fp8_pack_weight(w.cuda())
    assert np.array_equal(np.isnan(s.cpu().numpy()), bad)
    assert np.array_equal(np.nan_to_num(s.cpu().numpy()), np.nan_to_num(want_s))
    assert np.array_equal(codes_of(q), want_q)


@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("k", [264, 260, 258, 257])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_pack_weight_unaligned_base(bnn, dtype, k, offset):
    """A base that only element (or a few elements') alignment holds."""
    g, n = 2, 150
    w = torch.from_numpy(synth.normal_f32(k, 4, (g, n, k))).to(dtype)
    buf = torch.zeros(g * n * k + 16, dtype=dtype, device="cuda")
    view = buf[offset:offset + g * n * k].view(g, n, k)
    view.copy_(w)
    want_q, want_s = fp8.pack_weight(w.float().numpy())
    q, s = bnn.bnn_fp8_pack_weight(view)
    assert np.array_equal(codes_of(q), want_q) and np.array_equal(s.cpu().numpy(), want_s)


def test_pack_weight_into_given_buffers_stays_inside(bnn):
    g, n, k = 3, 130, 520
    kb, nb = fp8.blocks(k), fp8.blocks(n)
    qbuf = torch.full((g * n * kb * 128 + 256,), 7, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((g * nb * kb + 16,), -5.0, device="cuda")
    q = qbuf[128:-128].view(torch.float8_e4m3fn).view(g, n, kb * 128)
    s = sbuf[8:-8].view(g, nb, kb)
    w = synth.normal_f32(2, 4, (g, n, k))
    bnn.bnn_fp8_pack_weight(to_dev_f32(w), q=q, scale=s)
    want_q, want_s = fp8.pack_weight(w)
    assert np.array_equal(codes_of(q), want_q) and np.array_equal(s.cpu().numpy(), want_s)
    assert bool((qbuf[:128] == 7).all()) and bool((qbuf[-128:] == 7).all())
    assert bool((sbuf[:8] == -5).all()) and bool((sbuf[-8:] == -5).all())


# ------------------------------------------------------------------------------------------ memory
def test_calls_take_no_device_memory(bnn):
    """With outputs given, no call takes memory from the device: after one call of each kernel (whose code the
    driver loads then), larger calls leave the free memory as it was, while they run and behind them."""
    def make(m, n, k, g):
        x = torch.randn((m, k), device="cuda")
        w = torch.randn((g, n, k) if g else (n, k), device="cuda")
        ops = (*bnn.bnn_fp8_pack_rows(x), *bnn.bnn_fp8_pack_weight(w))
        out = torch.empty((m, n), device="cuda")
        off = torch.tensor([m * i // g for i in range(g + 1)], device="cuda") if g else None

        def call():
            bnn.bnn_fp8_pack_rows(x, q=ops[0], scale=ops[1])
            bnn.bnn_fp8_pack_weight(w, q=ops[2], scale=ops[3])
            if g:
                bnn.bnn_fp8_grouped_gemm(*ops, off, out=out)
            else:
                bnn.bnn_fp8_gemm(*ops, out=out)
        return call
    small = [(4, 300, 640, 0), (16, 1000, 8192, 0), (600, 3000, 760, 0), (20, 500, 8192, 0), (64, 1000, 8192, 0), (300, 2000, 4100, 0),
             (1101, 2304, 2000, 0), (200, 300, 2000, 20), (200, 300, 2000, 8), (900, 700, 2000, 4), (300, 2707, 2000, 8)]
    large = [(8, 2000, 4096, 0), (16, 900, 8192, 0), (32, 2000, 8192, 0), (100, 1000, 16384, 0), (700, 3000, 4100, 0),
             (4096, 4600, 2000, 0), (900, 500, 2000, 64), (1200, 300, 2000, 40), (5000, 700, 2000, 4), (4000, 4100, 2000, 4)]
    calls = [make(*c) for c in small + large]
    for c in calls[:len(small)]:
        c()
    torch.cuda.synchronize()
    before, held = torch.cuda.mem_get_info()[0], torch.cuda.memory_reserved()
    for _ in range(3):
        for c in calls[len(small):]:
            c()
    during = torch.cuda.mem_get_info()[0]
    torch.cuda.synchronize()
    assert torch.cuda.memory_reserved() == held
    assert during >= before and torch.cuda.mem_get_info()[0] >= before
