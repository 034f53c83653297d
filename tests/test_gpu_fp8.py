"""GPU parity of the 8-bit block-scaled calls against the numpy oracle (float64).

Tolerance of a product, derived: the tensor cores' products are exact and a block's 128 are added in
float32 (in any order and with truncation: at most 128 errors of one float32 step, 2^-23, of the block's
sum of absolute products); the scale product, its product with the block's sum and the kb additions round
once each (2^-24 of the running absolute sum).  So before the last rounding the error is at most
(128 * 2^-23 + (kb + 3) * 2^-24) * mag with mag = sum |x w| + |bias|, and the output type adds half a
step of |y| (2^-8 bfloat16, 2^-11 float16, 2^-24 float32; float16 below 2^-14 in steps of 2^-24)."""
import numpy as np
import pytest
import torch

from gpu_util import to_dev_f32
from oracle import fp8
from ternary_neural_net_b200 import synth

pytestmark = pytest.mark.gpu

OUTS = {"f32": (torch.float32, 2.0 ** -24), "bf16": (torch.bfloat16, 2.0 ** -8), "f16": (torch.float16, 2.0 ** -11)}


@pytest.fixture(scope="module")
def bnn(cuda_device):
    from ternary_neural_net_b200 import bnn as mod
    return mod


def dev_fp8(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).cuda().view(torch.float8_e4m3fn)


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def tolerance(y, mag, kb, out):
    half = OUTS[out][1]
    lim = (128 * 2.0 ** -23 + (kb + 3) * 2.0 ** -24) * mag * (1 + half) + half * np.abs(y)
    return lim + (2.0 ** -25 if out == "f16" else 0.0)


def assert_close(got, y, mag, kb, out, what):
    got = got.double().cpu().numpy()
    assert got.shape == y.shape, what
    bad = np.argwhere(~(np.abs(got - y) <= tolerance(y, mag, kb, out)))
    assert bad.size == 0, f"{what}: {len(bad)} of {y.size} outside, first {bad[:4].tolist()}: " \
                          f"{got[tuple(bad[0])]} for {y[tuple(bad[0])]} (mag {mag[tuple(bad[0])]})"


def activations(seed, m, k):
    return (synth.normal_f32(seed, 1, (m, k)) * np.exp(synth.normal_f32(seed, 2, (k,)))).astype(np.float32)


def packed_case(seed, m, n, k, groups=None):
    """Operands as the packs make them, from normal values."""
    xq, xs = fp8.pack_rows(activations(seed, m, k))
    g = groups or 1
    wq, ws = fp8.pack_weight(synth.normal_f32(seed, 3, (g, n, k)) * np.float32(0.05))
    return (xq, xs, wq, ws) if groups else (xq, xs, wq[0], ws[0])


def raw_case(seed, m, n, k, groups=None):
    """Operands as another packer may make them: any finite codes, scales of both signs over six decades."""
    rng = np.random.default_rng(seed)
    kb, g = fp8.blocks(k), groups or 1

    def codes(*shape):
        c = rng.integers(0, 127, (*shape, 128 * kb)).astype(np.uint8) | (rng.integers(0, 2, (*shape, 128 * kb)) << 7).astype(np.uint8)
        c[..., k:] = 0
        return c

    def scales(*shape):
        return (np.exp(rng.uniform(-7, 7, shape)) * rng.choice([-1.0, 1.0], shape)).astype(np.float32)
    xq, xs, wq, ws = codes(m), scales(kb, m), codes(g, n), scales(g, fp8.blocks(n), kb)
    return (xq, xs, wq, ws) if groups else (xq, xs, wq[0], ws[0])


def on_dev(xq, xs, wq, ws):
    return dev_fp8(xq), to_dev_f32(xs), dev_fp8(wq), to_dev_f32(ws)


# ------------------------------------------------------------------------------------------ packing
PACK_TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", PACK_TYPES)
@pytest.mark.parametrize("m,k", [(1, 1), (1, 8192), (3, 127), (5, 129), (33, 250), (31, 252), (64, 1000), (100, 4100),
                                 (257, 384), (2, 128), (1000, 136)])
def test_pack_rows_matches_oracle(bnn, dtype, m, k):
    x = torch.from_numpy(activations(m + k, m, k)).to(dtype)
    want_q, want_s = fp8.pack_rows(x.float().numpy())
    q, s = bnn.bnn_fp8_pack_rows(x.cuda())
    assert q.dtype == torch.float8_e4m3fn and s.dtype == torch.float32
    assert np.array_equal(s.cpu().numpy().view(np.uint32), want_s.view(np.uint32))
    assert np.array_equal(codes_of(q), want_q)


@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("dtype", PACK_TYPES)
def test_pack_rows_unaligned_base(bnn, dtype, offset):
    """A base that only element (or a few elements') alignment holds."""
    m, k = 9, 264
    x = torch.from_numpy(activations(5, m, k)).to(dtype)
    buf = torch.zeros(m * k + 16, dtype=dtype, device="cuda")
    view = buf[offset:offset + m * k].view(m, k)
    view.copy_(x)
    want_q, want_s = fp8.pack_rows(x.float().numpy())
    q, s = bnn.bnn_fp8_pack_rows(view)
    assert np.array_equal(codes_of(q), want_q) and np.array_equal(s.cpu().numpy(), want_s)


def test_pack_rows_every_rounding(bnn):
    """Every e4m3 value, every midpoint and its float32 neighbours, with the block's maximum at 448."""
    pts = np.concatenate([fp8._POS, fp8._MID]).astype(np.float32)
    pts = np.concatenate([pts, np.nextafter(pts, np.float32(0)), np.nextafter(pts, np.float32(448))])
    pts = np.concatenate([pts, -pts])
    rows = -(-len(pts) // 127)
    x = np.zeros((rows, 128), np.float32)
    x[:, :127].reshape(-1)[:] = 0
    flat = np.zeros(rows * 127, np.float32)
    flat[:len(pts)] = pts
    x[:, :127] = flat.reshape(rows, 127)
    x[:, 127] = 448.0
    want_q, want_s = fp8.pack_rows(x)
    q, s = bnn.bnn_fp8_pack_rows(to_dev_f32(x))
    assert np.array_equal(codes_of(q), want_q) and np.all(s.cpu().numpy() == 1.0) and np.all(want_s == 1.0)


@pytest.mark.parametrize("dtype", PACK_TYPES)
def test_pack_special_values(bnn, dtype):
    x = np.zeros((8, 300), np.float32)
    x[1, 5] = np.inf
    x[2, 200] = np.nan
    x[3, 299] = -np.inf
    x[4, 0], x[4, 1] = 2.0 ** -120, -(2.0 ** -133)
    x[5, 0], x[5, 130] = 6e4, -6e4
    x[6] = 1e-7
    x[7, ::2] = -0.0
    t = torch.from_numpy(x).to(dtype)
    x = t.float().numpy()
    want_q, want_s = fp8.pack_rows(x)
    q, s = bnn.bnn_fp8_pack_rows(t.cuda())
    assert np.array_equal(np.isnan(s.cpu().numpy()), np.isnan(want_s))
    assert np.array_equal(np.nan_to_num(s.cpu().numpy()), np.nan_to_num(want_s))
    assert np.array_equal(codes_of(q), want_q)
    wq, ws = bnn.bnn_fp8_pack_weight(t.cuda())
    ow, os_ = fp8.pack_weight(x[None])
    assert np.isnan(ws.cpu().numpy()).all() and np.isnan(os_).all() and not codes_of(wq).any() and not ow.any()


def test_pack_rows_index(bnn):
    m, k = 40, 300
    x = activations(8, m, k)
    rng = np.random.default_rng(8)
    index = rng.integers(0, m, 133).astype(np.int32)
    index[[0, 50, 132]] = [-1, m, np.iinfo(np.int32).max]
    index[[1, 2]] = index[3]  # the same row more than once
    want_q, want_s = fp8.pack_rows(x, index)
    q, s = bnn.bnn_fp8_pack_rows(to_dev_f32(x), torch.from_numpy(index).cuda())
    assert np.array_equal(codes_of(q), want_q) and np.array_equal(s.cpu().numpy(), want_s)
    q, s = bnn.bnn_fp8_pack_rows(torch.empty((0, k), device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert not codes_of(q).any()


@pytest.mark.parametrize("dtype", PACK_TYPES)
@pytest.mark.parametrize("g,n,k", [(1, 1, 1), (1, 128, 128), (3, 130, 200), (2, 300, 260), (1, 70, 4100), (5, 127, 385)])
def test_pack_weight_matches_oracle(bnn, dtype, g, n, k):
    w = torch.from_numpy(synth.normal_f32(g + n + k, 4, (g, n, k))).to(dtype)
    want_q, want_s = fp8.pack_weight(w.float().numpy())
    q, s = bnn.bnn_fp8_pack_weight(w.cuda())
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(codes_of(q), want_q)
    q2, s2 = bnn.bnn_fp8_pack_weight(w[0].contiguous().cuda())
    assert torch.equal(q2.view(torch.uint8), q[0].view(torch.uint8)) and torch.equal(s2, s[0])


def test_pack_into_given_buffers_stays_inside(bnn):
    """Packs into the middle of larger buffers: nothing around them changes."""
    m, k = 37, 520
    kb = fp8.blocks(k)
    qbuf = torch.full((m * kb * 128 + 256,), 7, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((kb * m + 16,), -5.0, device="cuda")
    q, s = qbuf[128:128 + m * kb * 128].view(torch.float8_e4m3fn).view(m, kb * 128), sbuf[8:8 + kb * m].view(kb, m)
    x = activations(9, m, k)
    bnn.bnn_fp8_pack_rows(to_dev_f32(x), q=q, scale=s)
    want_q, want_s = fp8.pack_rows(x)
    assert np.array_equal(codes_of(q), want_q) and np.array_equal(s.cpu().numpy(), want_s)
    assert bool((qbuf[:128] == 7).all()) and bool((qbuf[-128:] == 7).all())
    assert bool((sbuf[:8] == -5).all()) and bool((sbuf[-8:] == -5).all())


# ------------------------------------------------------------------------------------------ products
# one row to many, every edge of a 128-block, of 16/32/64/128/256-row tiles, k from one element to long
GEMM_SHAPES = [(1, 1, 1), (1, 1024, 1000), (1, 5, 20000), (2, 129, 130), (3, 4096, 512), (7, 300, 4100), (8, 128, 128),
               (9, 257, 640), (15, 1100, 8192), (16, 1000, 8192), (17, 200, 256), (32, 129, 900), (33, 640, 1280),
               (64, 1108, 512), (65, 130, 1001), (100, 5000, 640), (127, 130, 384), (128, 256, 384), (129, 513, 2000),
               (200, 64, 16384), (255, 257, 383), (256, 512, 4096), (300, 700, 2000), (513, 1025, 260),
               (777, 1100, 300), (2304, 1219, 130), (600, 3000, 760), (1500, 300, 128), (1024, 4096, 256)]


@pytest.mark.parametrize("m,n,k", GEMM_SHAPES)
@pytest.mark.parametrize("make", [packed_case, raw_case])
def test_gemm_matches_oracle(bnn, m, n, k, make):
    xq, xs, wq, ws = make(m * 5 + n + k, m, n, k)
    y, mag = fp8.gemm(xq, xs, wq, ws)
    got = bnn.bnn_fp8_gemm(*on_dev(xq, xs, wq, ws))
    assert_close(got, y, mag, fp8.blocks(k), "f32", f"{m}x{n}x{k}")
    assert bnn.device_error_count() == 0


@pytest.mark.parametrize("out", list(OUTS))
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("m,n,k", [(1, 300, 700), (6, 131, 260), (50, 259, 640), (64, 256, 512), (130, 1000, 384),
                                   (700, 1027, 256), (1100, 2048, 128)])
def test_gemm_types_and_bias(bnn, out, with_bias, m, n, k):
    xq, xs, wq, ws = packed_case(m + n + k, m, n, k)
    bias = synth.normal_f32(m, 9, (n,)) * np.float32(3.0) if with_bias else None
    y, mag = fp8.gemm(xq, xs, wq, ws, bias)
    d = on_dev(xq, xs, wq, ws)
    b = to_dev_f32(bias) if with_bias else None
    got = bnn.bnn_fp8_gemm(*d, b, out_dtype=OUTS[out][0])
    assert got.dtype == OUTS[out][0]
    assert_close(got, y, mag, fp8.blocks(k), out, f"{m}x{n}x{k} {out}")
    # into a buffer whose base holds the element's alignment only; what lies around stays
    buf = torch.full((m * n + 40,), 3.0, dtype=OUTS[out][0], device="cuda")
    for off in (1, 8):
        buf.fill_(3.0)
        bnn.bnn_fp8_gemm(*d, b, out=buf[off:off + m * n].view(m, n))
        assert torch.equal(buf[off:off + m * n].view(m, n), got)
        assert bool((buf[:off] == 3).all()) and bool((buf[off + m * n:] == 3).all())


def test_gemm_large_sampled(bnn):
    """Many tiles of the largest kind: whole rows and columns sampled, and every row against a checksum of
    the weights' columns."""
    m, n, k = 3000, 9100, 1100
    xq, xs, wq, ws = packed_case(12, m, n, k)
    got = bnn.bnn_fp8_gemm(*on_dev(xq, xs, wq, ws))
    rows = np.array([0, 1, 127, 128, 255, 256, 1499, 2815, 2816, 2999])
    y, mag = fp8.gemm(xq[rows], xs[:, rows], wq, ws)
    assert_close(got[torch.from_numpy(rows).cuda()], y, mag, fp8.blocks(k), "f32", "rows")
    cols = np.concatenate([np.arange(0, 128, 37), [127, 128, 255, 256, 4999, 8959, 8960, 9099]])
    x, w = fp8.row_values(xq, xs), fp8.weight_values(wq, ws)
    assert_close(got[:, torch.from_numpy(cols).cuda()], x @ w[cols].T, np.abs(x) @ np.abs(w[cols]).T, fp8.blocks(k),
                 "f32", "columns")
    total, mag = x @ w.sum(axis=0), np.abs(x) @ np.abs(w).sum(axis=0)
    err = np.abs(got.double().sum(dim=1).cpu().numpy() - total)
    assert np.all(err <= tolerance(total, mag, fp8.blocks(k), "f32"))


@pytest.mark.parametrize("m", [1, 12, 90, 600])
def test_gemm_k_zero_and_empty(bnn, m):
    n = 131
    e = lambda *shape: torch.empty(shape, device="cuda")
    q = lambda *shape: torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    bias = to_dev_f32(synth.normal_f32(1, 1, (n,)))
    assert torch.equal(bnn.bnn_fp8_gemm(q(m, 0), e(0, m), q(n, 0), e(2, 0), bias), bias.expand(m, n))
    assert not bnn.bnn_fp8_gemm(q(m, 0), e(0, m), q(n, 0), e(2, 0), out_dtype=torch.bfloat16).any()
    assert bnn.bnn_fp8_gemm(q(0, 128), e(1, 0), q(n, 128), e(2, 1)).shape == (0, n)
    assert bnn.bnn_fp8_gemm(q(m, 128), e(1, m), q(0, 128), e(0, 1)).shape == (m, 0)
    off = torch.tensor([1, m], device="cuda")
    y = torch.full((m, n), 5.0, device="cuda")
    bnn.bnn_fp8_grouped_gemm(q(m, 0), e(0, m), q(1, n, 0), e(1, 2, 0), off, out=y)
    assert bool((y[:1] == 5).all()) and not y[1:].any()


@pytest.mark.parametrize("m", [1, 3, 20, 100, 300, 800])
def test_gemm_nan_stays_in_its_row_and_column(bnn, m):
    """A NaN or infinity in one row of x, or in one weight row, reaches that output row or column alone."""
    n, k = 400, 520
    x = activations(3, m, k)
    x[m // 2, 200] = np.inf
    w = synth.normal_f32(4, 3, (n, k))
    wq, ws = fp8.pack_weight(w[None])
    xq, xs = fp8.pack_rows(x)
    wq = wq[0].copy()
    wq[301, 77] = 0x7f  # e4m3 NaN
    y = bnn.bnn_fp8_gemm(*on_dev(xq, xs, wq, ws[0])).cpu().numpy()
    nan = np.zeros((m, n), bool)
    nan[m // 2], nan[:, 301] = True, True
    assert np.array_equal(np.isnan(y), nan)


def test_gemm_is_reproducible_and_streams_are_independent(bnn):
    """The same call twice, and calls on two streams at once, give the same bits."""
    cases = [on_dev(*packed_case(s, m, n, k)) for s, (m, n, k) in
             enumerate([(1, 4096, 2048), (16, 2000, 4096), (100, 1000, 2048), (256, 1024, 2048), (1300, 1500, 640)])]
    torch.cuda.synchronize()
    first = [bnn.bnn_fp8_gemm(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    again = []
    for rep in range(4):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[(i + rep) % 2]):
                again.append((i, bnn.bnn_fp8_gemm(*c)))
    torch.cuda.synchronize()
    for i, y in again:
        assert torch.equal(y, first[i])


@pytest.mark.parametrize("m", [1, 40, 500])
def test_pack_then_gemm_back_to_back(bnn, m):
    """Weights and activations packed right before the products that read them, with nothing in between, over
    and over with other values: no product reads an earlier pack."""
    n, k = 1000, 1920
    ws_, xs_ = [], []
    for i in range(4):
        ws_.append(to_dev_f32(synth.normal_f32(i, 5, (n, k))))
        xs_.append(to_dev_f32(activations(i, m, k)))
    q = torch.empty((n, k), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((8, 15), device="cuda")
    xq = torch.empty((m, k), dtype=torch.float8_e4m3fn, device="cuda")
    xs = torch.empty((15, m), device="cuda")

    def one(i, sync):
        bnn.bnn_fp8_pack_rows(xs_[i], q=xq, scale=xs)
        bnn.bnn_fp8_pack_weight(ws_[i], q=q, scale=s)
        if sync:
            torch.cuda.synchronize()
        y = bnn.bnn_fp8_gemm(xq, xs, q, s)
        bnn.bnn_fp8_pack_rows(xs_[(i + 1) % 4], q=xq, scale=xs)
        return y, bnn.bnn_fp8_gemm(xq, xs, q, s)
    want = [one(i, True) for i in range(4)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [one(i, False) for i in range(4)]
        for (a, b), (c, d) in zip(got, want):
            assert torch.equal(a, c) and torch.equal(b, d)


# ------------------------------------------------------------------------------------------ grouped
def offsets_of(sizes, start=0):
    return np.concatenate([[start], start + np.cumsum(sizes)]).astype(np.int64)


GROUPED = [  # sizes, rows before the first group, rows behind the last, n, k
    ([1], 0, 0, 128, 128), ([0], 0, 3, 100, 200), ([5], 2, 1, 131, 300), ([3, 0, 0, 1], 0, 0, 257, 640),
    ([1] * 20, 0, 5, 300, 1000), ([0, 17, 0, 64, 1, 128, 0], 3, 9, 260, 390), ([129, 127, 128, 255, 257], 0, 0, 384, 256),
    ([0] * 30 + [2] + [0] * 33, 0, 0, 200, 512), ([300, 0, 700, 5], 0, 11, 520, 384), ([1, 600], 1, 0, 1000, 260),
    ([16, 16, 16, 16, 15, 17, 33, 31], 0, 0, 512, 1152), ([2] * 64, 0, 0, 140, 260), ([40] * 16, 0, 64, 129, 128),
    ([7] * 130, 0, 2, 33, 130), ([260, 3, 0, 513, 90, 1], 4, 4, 1300, 1000)]


@pytest.mark.parametrize("sizes,before,behind,n,k", GROUPED)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_grouped_matches_oracle(bnn, sizes, before, behind, n, k, out):
    offsets = offsets_of(sizes, before)
    rows = int(offsets[-1]) + behind
    xq, xs, wq, ws = (packed_case if out == "bf16" else raw_case)(rows + n, rows, n, k, len(sizes))
    y, mag, live = fp8.grouped_gemm(xq, xs, wq, ws, offsets)
    buf = torch.full((rows, n), 7.0, dtype=OUTS[out][0], device="cuda")
    got = bnn.bnn_fp8_grouped_gemm(*on_dev(xq, xs, wq, ws), torch.from_numpy(offsets).cuda(), out=buf)
    assert got.data_ptr() == buf.data_ptr()
    lt = torch.from_numpy(live).cuda()
    assert_close(got[lt], y[live], mag[live], fp8.blocks(k), out, str(sizes))
    assert bool((got[~lt] == 7).all())
    assert bnn.device_error_count() == 0


@pytest.mark.parametrize("offsets", [[5, 3, 20, 10, 60], [-7, 10, 10, 200, 30], [0, 1 << 40, 0, 0, 1 << 62],
                                     [-(1 << 62), -5, -1, 0, 0], [100, 90, 80, 70, 60]])
@pytest.mark.parametrize("rows", [50, 400])
def test_grouped_any_offsets_stay_inside(bnn, offsets, rows):
    n, k = 150, 256
    xq, xs, wq, ws = packed_case(6, rows, n, k, 4)
    y, mag, live = fp8.grouped_gemm(xq, xs, wq, ws, offsets)
    buf = torch.full((rows * n + 64,), 7.0, device="cuda")
    got = buf[32:32 + rows * n].view(rows, n)
    bnn.bnn_fp8_grouped_gemm(*on_dev(xq, xs, wq, ws), torch.tensor(offsets, device="cuda"), out=got)
    lt = torch.from_numpy(live).cuda()
    assert_close(got[lt], y[live], mag[live], 2, "f32", str(offsets))
    assert bool((got[~lt] == 7).all()) and bool((buf[:32] == 7).all()) and bool((buf[-32:] == 7).all())


def test_grouped_many_experts(bnn):
    """As many groups as a call takes, most of them empty, and one more is refused."""
    g, n, k = bnn.MAX_GROUPS, 20, 128
    rng = np.random.default_rng(2)
    sizes = rng.integers(0, 4, g) * (rng.random(g) < 0.3)
    offsets = offsets_of(sizes)
    rows = int(offsets[-1])
    xq, xs, wq, ws = packed_case(3, rows, n, k, g)
    y, mag, _ = fp8.grouped_gemm(xq, xs, wq, ws, offsets)
    d = on_dev(xq, xs, wq, ws)
    got = bnn.bnn_fp8_grouped_gemm(*d, torch.from_numpy(offsets).cuda())
    assert_close(got, y, mag, 1, "f32", "1024 groups")
    with pytest.raises(bnn.BnnError):
        bnn.bnn_fp8_grouped_gemm(d[0], d[1], torch.zeros((g + 1, 1, 128), device="cuda").to(torch.float8_e4m3fn),
                                 torch.zeros((g + 1, 1, 1), device="cuda"),
                                 torch.zeros(g + 2, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("per", [2, 30, 200])
def test_grouped_nan_stays_in_its_group(bnn, per):
    """NaN bytes and scales in the rows around a group, and in the other experts' weights, reach nothing of it."""
    n, k, g = 300, 384, 4
    offsets = offsets_of([per, per + 1, 0, per], 3)
    rows = int(offsets[-1]) + 5
    xq, xs, wq, ws = packed_case(7, rows, n, k, g)
    y, mag, _ = fp8.grouped_gemm(xq, xs, wq, ws, offsets)
    a, b = int(offsets[1]), int(offsets[2])
    bad = np.ones(rows, bool)
    bad[a:b] = False
    xq, xs, wq, ws = xq.copy(), xs.copy(), wq.copy(), ws.copy()
    xq[bad], wq[[0, 2, 3]] = 0x7f, 0xff
    xs[:, bad], ws[[0, 2, 3]] = np.nan, np.inf
    got = bnn.bnn_fp8_grouped_gemm(*on_dev(xq, xs, wq, ws), torch.from_numpy(offsets).cuda())
    assert_close(got[a:b], y[a:b], mag[a:b], 3, "f32", "clean group")


def test_grouped_equals_gemm_of_each_group(bnn):
    sizes = [70, 0, 200, 33]
    offsets = offsets_of(sizes)
    n, k = 500, 700
    xq, xs, wq, ws = packed_case(9, int(offsets[-1]), n, k, 4)
    dx, dxs, dw, dws = on_dev(xq, xs, wq, ws)
    got = bnn.bnn_fp8_grouped_gemm(dx, dxs, dw, dws, torch.from_numpy(offsets).cuda())
    for g, (a, b) in enumerate(zip(offsets, offsets[1:])):
        if b > a:
            one = bnn.bnn_fp8_gemm(dx[a:b], dxs[:, a:b].contiguous(), dw[g], dws[g])
            _, mag = fp8.gemm(xq[a:b], xs[:, a:b], wq[g], ws[g])
            err = (one - got[a:b]).abs().double().cpu().numpy()
            assert np.all(err <= 2 * tolerance(0 * mag, mag, fp8.blocks(k), "f32"))


def test_graphs_follow_their_inputs(bnn):
    """Two captured graphs (pack with index, grouped product; pack, product) replayed in turn on two streams with
    other values, indexes and offsets: each replay answers for what its buffers hold."""
    n, k, g, tokens, rows = 260, 512, 6, 30, 75
    xq0, xs0, wq, ws = packed_case(13, 1, n, k, g)
    dw, dws = dev_fp8(wq), to_dev_f32(ws)
    x = torch.empty((tokens, k), device="cuda")
    index = torch.zeros(rows, dtype=torch.int32, device="cuda")
    off = torch.zeros(g + 1, dtype=torch.int64, device="cuda")
    y1, x2 = torch.zeros((rows, n), device="cuda"), torch.empty((3, k), device="cuda")
    graphs, outs = [], []

    def first():
        q, s = bnn.bnn_fp8_pack_rows(x, index)
        return bnn.bnn_fp8_grouped_gemm(q, s, dw, dws, off, out=y1)

    def second():
        q, s = bnn.bnn_fp8_pack_rows(x2)
        return bnn.bnn_fp8_gemm(q, s, dw[2], dws[2])
    x.zero_(), x2.zero_()
    first(), second()
    torch.cuda.synchronize()
    for f in (first, second):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(f())
        graphs.append(graph)
    rng = np.random.default_rng(4)
    side = torch.cuda.Stream()
    for rep in range(4):
        hx, hx2 = activations(rep, tokens, k), activations(rep + 50, 3, k)
        hi = rng.integers(0, tokens, rows).astype(np.int32)
        ho = np.sort(rng.integers(0, rows + 1, g + 1)).astype(np.int64)
        x.copy_(torch.from_numpy(hx)), x2.copy_(torch.from_numpy(hx2))
        index.copy_(torch.from_numpy(hi)), off.copy_(torch.from_numpy(ho))
        y1.fill_(7.0)
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        y, mag, live = fp8.grouped_gemm(*fp8.pack_rows(hx, hi), wq, ws, ho)
        lt = torch.from_numpy(live).cuda()
        assert_close(outs[0][lt], y[live], mag[live], 4, "f32", "grouped replay")
        assert bool((outs[0][~lt] == 7).all())
        y, mag = fp8.gemm(*fp8.pack_rows(hx2), wq[2], ws[2])
        assert_close(outs[1], y, mag, 4, "f32", "gemm replay")


# ------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("tokens,top", [(1, 2), (9, 2), (150, 4)])
def test_expert_layer(bnn, tokens, top):
    """A layer of experts as it is used: route, dispatch and pack, up product, gate, pack, down product, combine;
    each step's output checked against the oracle on that step's own inputs."""
    g, d, h = 8, 384, 520
    x = torch.from_numpy(activations(tokens, tokens, d)).to(torch.bfloat16)
    up = synth.normal_f32(1, 7, (g, 2 * h, d)) * np.float32(0.05)
    down = synth.normal_f32(2, 7, (g, d, h)) * np.float32(0.05)
    logits = torch.from_numpy(synth.normal_f32(tokens, 8, (tokens, g))).cuda()
    uq, us = bnn.bnn_fp8_pack_weight(to_dev_f32(up))
    dq, ds = bnn.bnn_fp8_pack_weight(to_dev_f32(down))
    gate, expert = torch.topk(logits.softmax(dim=1), top, dim=1)
    order = torch.argsort(expert.reshape(-1), stable=True)
    token = (order // top).to(torch.int32)
    offsets = torch.zeros(g + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(expert.reshape(-1), minlength=g), 0)
    xq, xs = bnn.bnn_fp8_pack_rows(x.cuda(), token)
    hid = bnn.bnn_fp8_grouped_gemm(xq, xs, uq, us, offsets, out_dtype=torch.bfloat16)
    act = (torch.nn.functional.silu(hid[:, :h].float()) * hid[:, h:].float()).to(torch.bfloat16)
    aq, as_ = bnn.bnn_fp8_pack_rows(act)
    res = bnn.bnn_fp8_grouped_gemm(aq, as_, dq, ds, offsets)
    y = torch.zeros((tokens, d), device="cuda").index_add_(0, token.long(), res * gate.reshape(-1)[order][:, None])
    # step by step
    ho = offsets.cpu().numpy()
    wantq = fp8.pack_rows(x.float().numpy(), token.cpu().numpy())
    assert np.array_equal(codes_of(xq), wantq[0]) and np.array_equal(xs.cpu().numpy(), wantq[1])
    ouq, ods = fp8.pack_weight(up), fp8.pack_weight(down)
    h64, hm, _ = fp8.grouped_gemm(*wantq, *ouq, ho)
    assert_close(hid, h64, hm, 3, "bf16", "up")
    r64, rm, _ = fp8.grouped_gemm(*fp8.pack_rows(act.float().cpu().numpy()), *ods, ho)
    assert_close(res, r64, rm, 5, "f32", "down")
    # and the whole against the unquantised layer.  A rounding to e4m3 is off by at most 2^-4 of the value, 2^-4 /
    # sqrt(3) in the mean square; a product has two (its operands), the gated activation is a product of two
    # products' outputs, and the second product adds its two: sqrt(2 * 2 + 2) * 2^-4 / sqrt(3) = 0.088 of the norm
    # for errors that are independent.  A wrong expert, row or scale is off by about 1; 0.25 tells the two apart.
    xf = x.double().numpy()
    ref = np.zeros((tokens, d))
    ge, ex = gate.double().cpu().numpy(), expert.cpu().numpy()
    for t in range(tokens):
        for j in range(top):
            v = up[ex[t, j]].astype(np.float64) @ xf[t]
            a = v[:h] / (1 + np.exp(-v[:h])) * v[h:]
            ref[t] += ge[t, j] * (down[ex[t, j]].astype(np.float64) @ a)
    rel = np.linalg.norm(y.double().cpu().numpy() - ref) / np.linalg.norm(ref)
    assert rel < 0.25


def test_raw_tbin_layer_through_fp8(bnn):
    """A .tbin raw record (a layer kept out of the ternary form) loaded, packed to e4m3 and applied."""
    from oracle import tbin
    n, k, m = 70, 200, 5
    w = (synth.normal_f32(3, 1, (n, k)) * np.float32(0.1)).astype(np.float16)
    data = tbin.write([dict(kind="raw", name="head", dims=[n, k], data=w.reshape(-1))])
    _, _, recs = bnn.bnn_tbin_parse(data)
    file_dev = torch.frombuffer(bytearray(data), dtype=torch.uint8).cuda()
    wd = bnn.bnn_tbin_load_raw(file_dev, recs[0])
    wq, ws = bnn.bnn_fp8_pack_weight(wd)
    x = activations(2, m, k)
    xq, xs = bnn.bnn_fp8_pack_rows(to_dev_f32(x))
    y, mag = fp8.gemm(*fp8.pack_rows(x), *[a[0] for a in fp8.pack_weight(w.astype(np.float32)[None])])
    assert_close(bnn.bnn_fp8_gemm(xq, xs, wq, ws), y, mag, 2, "f32", "raw layer")


# ------------------------------------------------------------------------------------------ the binding's refusals
def test_binding_refusals(bnn):
    q = lambda *s: torch.zeros(s, device="cuda").to(torch.float8_e4m3fn)
    f = lambda *s: torch.zeros(s, device="cuda")
    xq, xs, wq, ws = q(4, 256), f(2, 4), q(130, 256), f(2, 2)
    bad = [dict(xq=f(4, 256)), dict(xq=q(4, 200)), dict(xq=q(512, 8).t()), dict(xs=f(4, 2)), dict(xs=f(2, 4).double()),
           dict(xs=f(4, 2).t()), dict(wq=q(130, 128)), dict(wq=q(1, 130, 256)), dict(ws=f(1, 2)), dict(ws=f(2, 2).cpu()),
           dict(bias=f(129)), dict(bias=f(130).half()), dict(out_dtype=torch.float64), dict(out=f(4, 131)),
           dict(out=f(4, 130).double()), dict(out=f(130, 4).t()), dict(out=torch.zeros(4, 130))]
    for kw in bad:
        with pytest.raises((TypeError, ValueError)):
            bnn.bnn_fp8_gemm(**{**dict(xq=xq, xs=xs, wq=wq, ws=ws), **kw})
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    wq3, ws3 = q(3, 130, 256), f(3, 2, 2)
    for kw in (dict(offsets=off[:3]), dict(offsets=off.int()), dict(offsets=off.cpu()), dict(wq=wq), dict(ws=ws),
               dict(out=f(5, 130)), dict(offsets=off[None])):
        with pytest.raises((TypeError, ValueError)):
            bnn.bnn_fp8_grouped_gemm(**{**dict(xq=xq, xs=xs, wq=wq3, ws=ws3, offsets=off), **kw})
    x = f(4, 200)
    for kw in (dict(x=x.double()), dict(x=x[0]), dict(x=x.t()), dict(index=off), dict(index=off.int().cpu()),
               dict(index=off.int()[None]), dict(q=q(4, 128)), dict(q=f(4, 256)), dict(scale=f(4, 2))):
        with pytest.raises((TypeError, ValueError)):
            bnn.bnn_fp8_pack_rows(**{**dict(x=x), **kw})
    for kw in (dict(w=x.int()), dict(w=x[0]), dict(w=x[None, None]), dict(w=x.t()), dict(q=q(4, 128)),
               dict(scale=f(2, 1))):
        with pytest.raises((TypeError, ValueError)):
            bnn.bnn_fp8_pack_weight(**{**dict(w=x), **kw})
    assert bnn.bnn_fp8_gemm(xq, xs, wq, ws).shape == (4, 130)


# ------------------------------------------------------------------------------------------ calls in other orders
@pytest.mark.parametrize("m", [1, 20, 300])
def test_weights_packed_inside_a_graph(bnn, m):
    """A captured graph that packs weights and rows and multiplies them, replayed right behind the copies of its
    next inputs: every replay's products are those of its own weights."""
    n, k, g = 700, 1300, 3
    ws_ = [to_dev_f32(synth.normal_f32(i, 6, (g, n, k))) for i in range(4)]
    xs_ = [to_dev_f32(activations(i + 9, m, k)) for i in range(4)]
    w, x = torch.empty((g, n, k), device="cuda"), torch.empty((m, k), device="cuda")
    off = torch.tensor([0, m // 3, m // 3, m], device="cuda")

    def call():
        q, s = bnn.bnn_fp8_pack_weight(w)
        xq, xs = bnn.bnn_fp8_pack_rows(x)
        q2, s2 = bnn.bnn_fp8_pack_weight(w[1])
        return bnn.bnn_fp8_gemm(xq, xs, q2, s2), bnn.bnn_fp8_grouped_gemm(xq, xs, q, s, off)
    want = []
    for i in range(4):
        w.copy_(ws_[i]), x.copy_(xs_[i])
        torch.cuda.synchronize()
        want.append(call())
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    got = []
    for rep in range(3):
        for i in range(4):
            w.copy_(ws_[i]), x.copy_(xs_[i])
            graph.replay()
            got.append((i, outs[0].clone(), outs[1].clone()))
    torch.cuda.synchronize()
    for i, y, z in got:
        assert torch.equal(y, want[i][0]) and torch.equal(z, want[i][1])
    assert bnn.device_error_count() == 0


@pytest.mark.parametrize("groups,rows", [(64, 900), (64, 2500), (8, 1500)])
@pytest.mark.parametrize("place", [0, -1])
def test_grouped_all_rows_in_one_group(bnn, groups, rows, place):
    """The kernel is chosen by the mean size; here one group has every row and the others none."""
    n, k = 300, 520
    sizes = [0] * groups
    sizes[place] = rows
    xq, xs, wq, ws = packed_case(rows + groups, rows, n, k, groups)
    offsets = offsets_of(sizes)
    y, mag, live = fp8.grouped_gemm(xq, xs, wq, ws, offsets)
    assert live.all()
    got = bnn.bnn_fp8_grouped_gemm(*on_dev(xq, xs, wq, ws), torch.from_numpy(offsets).cuda())
    assert_close(got, y, mag, fp8.blocks(k), "f32", f"{groups} {rows} {place}")


def test_calls_from_several_threads(bnn):
    """Host threads that pack and multiply at the same time, each on a stream of its own."""
    import threading
    shapes = [(1, 1000, 2000), (24, 700, 1100), (300, 900, 1000), (900, 1500, 640)]
    data = [(to_dev_f32(activations(i, m, k)), to_dev_f32(synth.normal_f32(i, 7, (n, k))))
            for i, (m, n, k) in enumerate(shapes)]

    def call(x, w):
        return bnn.bnn_fp8_gemm(*bnn.bnn_fp8_pack_rows(x), *bnn.bnn_fp8_pack_weight(w))
    want = [call(*d) for d in data]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                ys = [call(*data[i]) for _ in range(20)]
                torch.cuda.current_stream().synchronize()
                wrong.extend(i for y in ys if not torch.equal(y, want[i]))
        except Exception as e:  # noqa: BLE001 (reported by the main thread)
            wrong.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(data))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("m", [1, 9, 40, 300])
def test_scales_far_apart(bnn, m):
    """Scales near both ends of float32 whose products are ordinary numbers."""
    n, k = 260, 900
    xq, xs, wq, ws = packed_case(m, m, n, k)
    xs = (xs * np.float32(2.0 ** -100)).astype(np.float32)
    ws = (ws * np.float32(2.0 ** 110)).astype(np.float32)
    y, mag = fp8.gemm(xq, xs, wq, ws)
    assert_close(bnn.bnn_fp8_gemm(*on_dev(xq, xs, wq, ws)), y, mag, fp8.blocks(k), "f32", f"{m}")
