"""The 8-bit block-scaled form restated in numpy: e4m3 codes from their definition (a table of the 256
values, nearest by comparison with the midpoints), scales of blocks of 128, and the matrix products in
float64.  Test infrastructure only; shares nothing with the library."""
from __future__ import annotations

import numpy as np

TOP = np.float32(448.0)
FLOOR = np.float32(2.0 ** -100)


def _table() -> np.ndarray:
    """e4m3: sign, 4 exponent bits (bias 7), 3 fraction bits; exponent 0 is subnormal, S.1111.111 is NaN."""
    t = np.empty(256, np.float64)
    for code in range(256):
        e, f = (code >> 3) & 15, code & 7
        v = np.nan if (e, f) == (15, 7) else (f / 8.0) * 2.0 ** -6 if e == 0 else (1.0 + f / 8.0) * 2.0 ** (e - 7)
        t[code] = -v if code & 128 else v
    return t


VALUES = _table()
_POS = VALUES[:127]                      # codes 0x00..0x7e, increasing
_MID = (_POS[1:] + _POS[:-1]) / 2.0      # exact in float64


def decode(q: np.ndarray) -> np.ndarray:
    return VALUES[np.asarray(q, np.uint8)]


def encode(v: np.ndarray) -> np.ndarray:
    """Nearest code of finite float64 values, ties to the even code, saturated at 448."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    lo = np.searchsorted(_MID, a, side="left")    # a tie stays below
    hi = np.searchsorted(_MID, a, side="right")   # a tie goes above
    code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi)).astype(np.uint8)
    return code | (np.signbit(v).astype(np.uint8) << 7)


def blocks(k: int) -> int:
    return -(-k // 128)


def _scales(top: np.ndarray):
    """float32 block maxima (NaN or inf where the block is not finite) -> scale, factor, fine."""
    fine = np.isfinite(top)
    a = np.maximum(np.where(fine, top, np.float32(1.0)), FLOOR).astype(np.float32)
    scale = np.where(fine, a / TOP, np.float32(np.nan)).astype(np.float32)
    return scale, (TOP / a).astype(np.float32), fine


def pack_rows(x: np.ndarray, index=None):
    """float32 [m, k] -> (codes uint8 [rows, 128 kb], scale float32 [kb, rows])."""
    x = np.asarray(x, np.float32)
    m, k = x.shape
    if index is not None:
        index = np.asarray(index)
        ok = (index >= 0) & (index < m)
        x = np.where(ok[:, None], x[np.where(ok, index, 0)], np.float32(0.0)) if m else np.zeros((len(index), k), np.float32)
    rows, kb = x.shape[0], blocks(k)
    v = np.zeros((rows, 128 * kb), np.float32)
    v[:, :k] = x
    v = v.reshape(rows, kb, 128)
    scale, factor, fine = _scales(np.abs(v).max(axis=2) if kb else np.zeros((rows, 0), np.float32))
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.where(fine[:, :, None], v * factor[:, :, None], np.float32(0.0))
    return encode(p).reshape(rows, 128 * kb), np.ascontiguousarray(scale.T)


def pack_weight(w: np.ndarray):
    """float32 [g, n, k] -> (codes uint8 [g, n, 128 kb], scale float32 [g, ceil(n/128), kb])."""
    w = np.asarray(w, np.float32)
    g, n, k = w.shape
    kb, nb = blocks(k), blocks(n)
    v = np.zeros((g, 128 * nb, 128 * kb), np.float32)
    v[:, :n, :k] = w
    v = v.reshape(g, nb, 128, kb, 128)
    scale, factor, fine = _scales(np.abs(v).max(axis=(2, 4)))
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.where(fine[:, :, None, :, None], v * factor[:, :, None, :, None], np.float32(0.0))
    return encode(p).reshape(g, 128 * nb, 128 * kb)[:, :n].copy(), scale


def row_values(xq, xs) -> np.ndarray:
    return decode(xq) * np.repeat(np.asarray(xs, np.float64).T, 128, axis=1)


def weight_values(wq, ws) -> np.ndarray:
    n = wq.shape[0]
    s = np.repeat(np.repeat(np.asarray(ws, np.float64), 128, axis=0)[:n], 128, axis=1)
    return decode(wq) * s


def gemm(xq, xs, wq, ws, bias=None):
    """(y float64 [m, n], sum of the absolute products and the bias, [m, n])."""
    x, w = row_values(xq, xs), weight_values(wq, ws)
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        y, mag = y + np.asarray(bias, np.float64), mag + np.abs(np.asarray(bias, np.float64))
    return y, mag


def clamped_offsets(offsets, rows: int) -> list[int]:
    """Offsets as the grouped product reads them: inside [0, rows] and never decreasing."""
    out, top = [], 0
    for o in offsets:
        top = max(top, min(rows, int(o)))
        out.append(top)
    return out


def grouped_gemm(xq, xs, wq, ws, offsets):
    """(y float64 [rows, n], mag, live bool [rows]); rows outside every group are not live."""
    rows, n = xq.shape[0], wq.shape[1]
    y, mag, live = np.zeros((rows, n)), np.zeros((rows, n)), np.zeros(rows, bool)
    o = clamped_offsets(offsets, rows)
    for g in range(wq.shape[0]):
        a, b = o[g], o[g + 1]
        if b > a:
            y[a:b], mag[a:b] = gemm(xq[a:b], xs[:, a:b], wq[g], ws[g])
            live[a:b] = True
    return y, mag, live
