"""Pins of the 8-bit block-scaled oracle: the e4m3 table and rounding against torch's float8_e4m3fn, the
packing rule on hand-made blocks, the rounding bound of include/bnn.h, and the products against loops."""
import numpy as np
import pytest
import torch

from oracle import fp8


def test_table_is_e4m3():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(fp8.VALUES))
    assert np.array_equal(t[~np.isnan(t)], fp8.VALUES[~np.isnan(t)])
    assert fp8.VALUES[0x7e] == 448.0 and fp8.VALUES[1] == 2.0 ** -9


def test_encode_is_nearest_even():
    rng = np.random.default_rng(1)
    v = np.concatenate([rng.normal(size=20000) * np.exp2(rng.uniform(-12, 8, 20000)), fp8._MID, -fp8._MID, fp8._POS,
                        np.nextafter(fp8._MID, 0), np.nextafter(fp8._MID, 1e9), [0.0, -0.0]]).clip(-448, 448)
    v = v.astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.encode(v), want)
    assert np.array_equal(fp8.encode(np.array([460.0, 1e30, -1e30])), [0x7e, 0x7e, 0xfe])
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    assert np.array_equal(fp8.encode(fp8.decode(codes)), codes)


@pytest.mark.parametrize("k", [1, 127, 128, 129, 300])
def test_pack_rows_bound_and_layout(k):
    rng = np.random.default_rng(k)
    x = (rng.normal(size=(7, k)) * np.exp2(rng.uniform(-20, 20, (7, k)))).astype(np.float32)
    q, s = fp8.pack_rows(x)
    kb = fp8.blocks(k)
    assert q.shape == (7, 128 * kb) and s.shape == (kb, 7)
    assert not q[:, k:].any()
    v = fp8.row_values(q, s)[:, :k]
    a = np.repeat(s.T.astype(np.float64) * 448.0, 128, axis=1)[:, :k]
    assert np.all(np.abs(v - x) <= (2.0 ** -4 * np.abs(x) + a * 2.0 ** -18) * (1 + 2.0 ** -21))
    for b in range(kb):  # the block's largest element lands on 448
        part = np.abs(x[:, 128 * b:128 * b + 128])
        i = part.argmax(axis=1)
        assert np.all(np.abs(fp8.decode(q[np.arange(7), 128 * b + i])) == 448.0)


def test_pack_special_blocks():
    x = np.zeros((5, 256), np.float32)
    x[1, 5] = np.inf
    x[2, 200] = np.nan
    x[3, 0], x[3, 1] = 2.0 ** -120, -(2.0 ** -149)
    x[4, 0], x[4, 130] = 3.4e38, -3.4e38
    q, s = fp8.pack_rows(x)
    floor = np.float32(2.0 ** -100) / np.float32(448)
    assert np.array_equal(s[:, 0], [floor, floor]) and not q[0].any()
    assert np.isnan(s[0, 1]) and s[1, 1] == floor and not q[1].any()
    assert s[0, 2] == floor and np.isnan(s[1, 2]) and not q[2].any()
    assert s[0, 3] == floor and q[3, 0] == 0 and q[3, 1] == 0x80
    assert q[4, 0] == 0x7e and q[4, 130] == 0xfe


def test_pack_rows_index():
    x = np.arange(6 * 130, dtype=np.float32).reshape(6, 130) + 1
    q, s = fp8.pack_rows(x)
    qi, si = fp8.pack_rows(x, [3, 3, 0, -1, 6, 5])
    assert np.array_equal(qi[[0, 1, 2, 5]], q[[3, 3, 0, 5]]) and np.array_equal(si[:, [0, 1, 2, 5]], s[:, [3, 3, 0, 5]])
    assert not qi[[3, 4]].any()


def test_pack_weight_blocks():
    rng = np.random.default_rng(3)
    w = rng.normal(size=(2, 130, 200)).astype(np.float32)
    q, s = fp8.pack_weight(w)
    assert q.shape == (2, 130, 256) and s.shape == (2, 2, 2)
    for g in range(2):
        for t in range(2):
            for b in range(2):
                part = w[g, 128 * t:128 * t + 128, 128 * b:128 * b + 128]
                assert s[g, t, b] == np.abs(part).max() / np.float32(448)
        v = fp8.weight_values(q[g], s[g])[:, :200]
        assert np.all(np.abs(v - w[g]) <= 2.0 ** -4 * np.abs(w[g]) + 448 * s[g].max() * 2.0 ** -18 * 1.001)


def test_products_against_loops():
    rng = np.random.default_rng(4)
    m, n, kb = 5, 131, 2
    xq, wq = rng.integers(0, 127, (m, 256)).astype(np.uint8), rng.integers(128, 255, (3, n, 256)).astype(np.uint8)
    xs, ws = rng.uniform(0.5, 2, (kb, m)).astype(np.float32), rng.uniform(-2, 2, (3, 2, kb)).astype(np.float32)
    bias = rng.normal(size=n).astype(np.float32)
    y, mag = fp8.gemm(xq, xs, wq[0], ws[0], bias)
    offsets = [1, 3, 2, 9]  # as read: 1, 3, 3, 5
    yg, _, live = fp8.grouped_gemm(xq, xs, wq, ws, offsets)
    assert fp8.clamped_offsets(offsets, m) == [1, 3, 3, 5] and fp8.clamped_offsets([-4, 2, 2, 2], m) == [0, 2, 2, 2]
    assert live.tolist() == [False, True, True, True, True]
    for i in range(m):
        g = {1: 0, 2: 0, 3: 2, 4: 2}.get(i)
        for j in (0, 1, 127, 128, 130):
            terms = lambda e: [fp8.VALUES[xq[i, t]] * float(xs[t // 128, i]) * fp8.VALUES[wq[e, j, t]] *
                               float(ws[e, j // 128, t // 128]) for t in range(256)]
            assert y[i, j] == pytest.approx(sum(terms(0)) + float(bias[j]), rel=1e-12, abs=1e-9 * mag[i, j])
            assert mag[i, j] == pytest.approx(sum(map(abs, terms(0))) + abs(float(bias[j])), rel=1e-12)
            if g is not None:
                assert yg[i, j] == pytest.approx(sum(terms(g)), rel=1e-10, abs=1e-9 * mag[i, j])
