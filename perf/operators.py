"""The 8-bit block-scaled operators as they are measured: packing of activations and weights into e4m3 with a
scale for each block of 128, the matrix product on them, and the products grouped by expert.

`run` computes an operator in its plain form (elementary torch operations in 32 bits), or, where `own` is true,
through the library's own calls.  Layouts (kb = ceil(k / 128), pad elements 0):

  activations  e4m3 [rows, 128 kb], scales float32 [kb, rows]
  weights      e4m3 [n, 128 kb] or [groups, n, 128 kb], scales float32 [ceil(n/128), kb] or [groups, ceil(n/128), kb]
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}
SIZES = {"bf16": 2, "f32": 4, "f16": 2}
TINY = 2.0 ** -100  # the least block maximum: blocks of zeros get a scale too
TOP = 448.0         # the largest e4m3 value


def blocks(k):
    return -(-k // 128)


# ------------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # one token's activations before a projection: a launch, little else
        dict(name="pack-token", op="pack_rows", m=1, k=8192, x="bf16"),
        # the activations of a large prefill
        dict(name="pack-prefill", op="pack_rows", m=8192, k=8192, x="bf16"),
        # one float32 layer packed at load time
        dict(name="pack-layer", op="pack_weight", g=1, n=11008, k=4096, x="f32"),
        # a layer of experts with sizes off every block boundary, bfloat16
        dict(name="pack-experts", op="pack_weight", g=8, n=2050, k=4100, x="bf16"),
        # the smallest product: one token, a short row that ends inside a block, a bias
        dict(name="gemm-small", op="gemm", m=1, n=1024, k=1000, out="f32", bias=True),
        # decoding one token through a wide projection: the weights' bytes
        dict(name="linear-token", op="linear", m=1, n=28672, k=8192, x="bf16", out="bf16", bias=False),
        # decoding a batch of 64
        dict(name="gemm-64", op="gemm", m=64, n=11008, k=4096, out="f32", bias=False),
        # a short prompt
        dict(name="gemm-256", op="gemm", m=256, n=4096, k=4096, out="bf16", bias=False),
        # nothing a multiple of a tile, float32 out, a bias
        dict(name="gemm-odd", op="gemm", m=777, n=11007, k=4100, out="f32", bias=True),
        # a long prefill: the tensor cores
        dict(name="gemm-8192", op="gemm", m=8192, n=8192, k=8192, out="bf16", bias=False),
        # eight tokens decoded through 64 experts, eight experts a token: dispatch, pack, product
        dict(name="experts-token", op="experts", g=64, tokens=8, top=8, n=2048, k=4096, x="bf16", out="bf16"),
        # prefill through the same number of experts, ragged groups, some empty, room behind the last row
        dict(name="experts-prefill", op="grouped", g=64, rows=16384, tail=100, n=4096, k=4096, out="bf16"),
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))

    op = rng.choice(["pack_rows", "pack_weight", "gemm", "gemm", "gemm", "linear", "grouped", "grouped", "experts"])
    x, out = rng.choice(["bf16", "bf16", "f32", "f16"]), rng.choice(["bf16", "bf16", "f32", "f16"])
    while True:
        n, k = size(16, 28672), size(64, 16384)
        if rng.random() < 0.5:
            n, k = max(64, n // 64 * 64), max(128, k // 128 * 128)
        if op == "pack_rows":
            m = size(1, 16384)
            if m * k <= 2 ** 26:
                return dict(op=op, m=m, k=k, x=x)
        elif op == "pack_weight":
            g = rng.choice([1, 1, 4, 16])
            if g * n * k <= 2 ** 26:
                return dict(op=op, g=g, n=n, k=k, x=x)
        elif op in ("gemm", "linear"):
            m = size(1, 8192)
            if n * k <= 2 ** 28 and m * n * k <= 2 ** 38:
                case = dict(op=op, m=m, n=n, k=k, out=out, bias=rng.random() < 0.4)
                return dict(case, x=x) if op == "linear" else case
        elif op == "grouped":
            g, rows = rng.choice([4, 8, 16, 32, 64, 128]), size(16, 16384)
            if g * n * k <= 2 ** 30 and rows * n * k <= 2 ** 37 and rows * (n + k) <= 2 ** 28:
                return dict(op=op, g=g, rows=rows, tail=rng.choice([0, rng.randint(1, 200)]), n=n, k=k, out=out)
        else:
            g, tokens = rng.choice([8, 16, 64, 128]), size(1, 1024)
            top = rng.choice([1, 2, 4, 8])
            if g * n * k <= 2 ** 30 and tokens * top * n * k <= 2 ** 37:
                return dict(op=op, g=g, tokens=tokens, top=top, n=n, k=k, x=x, out=out)


def work(case):
    op, k, kb = case["op"], case["k"], blocks(case["k"])
    if op == "pack_rows":
        m = case["m"]
        return dict(bytes=m * k * SIZES[case["x"]] + m * 128 * kb + 4 * m * kb, flops=0)
    n = case["n"]
    nb = blocks(n)
    if op == "pack_weight":
        g = case["g"]
        return dict(bytes=g * (n * k * SIZES[case["x"]] + n * 128 * kb + 4 * nb * kb), flops=0)
    if op in ("gemm", "linear"):
        m = case["m"]
        into = m * k * SIZES[case["x"]] if op == "linear" else m * k + 4 * m * kb
        bias = 4 * n if case["bias"] else 0
        return dict(bytes=into + n * k + 4 * nb * kb + bias + m * n * SIZES[case["out"]], flops=2 * m * n * k)
    g = case["g"]
    if op == "experts":
        rows = case["tokens"] * case["top"]
        into = case["tokens"] * k * SIZES[case["x"]] + 4 * rows
    else:
        rows = case["rows"]
        into = rows * k + 4 * rows * kb
    busy = min(rows, g * (1.0 - (1.0 - 1.0 / g) ** rows))  # the experts that get rows, in the mean
    return dict(bytes=into + 8 * (g + 1) + busy * (n * k + 4 * nb * kb) + rows * n * SIZES[case["out"]], flops=2 * rows * n * k)


# ------------------------------------------------------------------------------------------------ inputs


def activations(gen, m, k, dtype):
    """Normal values, columns of differing size and a few that stand out, as hidden states have them."""
    x = torch.randn((m, k), generator=gen, device=DEV)
    col = torch.exp(0.5 * torch.randn((k,), generator=gen, device=DEV))
    col = torch.where(torch.rand((k,), generator=gen, device=DEV) < 0.004, col * 20.0, col)
    return (x * col).to(dtype)


def weights(gen, g, n, k, dtype):
    w = torch.randn((g, n, k), generator=gen, device=DEV)
    return (w * (0.02 * torch.exp(0.3 * torch.randn((g, n, 1), generator=gen, device=DEV)))).to(dtype)


def spread(rng, rows, g):
    """Offsets of ragged groups that add up to `rows`: the shares differ and one group in eight is empty."""
    share = [rng.gammavariate(4.0, 1.0) for _ in range(g)]
    for i in rng.sample(range(g), g // 8):
        share[i] = 0.0
    total, offsets, acc = sum(share), [0], 0.0
    for s in share:
        acc += s
        offsets.append(round(rows * acc / total))
    offsets[-1] = rows
    return offsets


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1000003 * int(seed) + 17)
    rng = random.Random(7919 * int(seed) + 5)
    op, k = case["op"], case["k"]
    s = dict(op=op, k=k)
    if op in ("pack_rows", "linear"):
        s["x"] = activations(gen, case["m"], k, DTYPES[case["x"]])
    if op == "pack_weight":
        w = weights(gen, case["g"], case["n"], k, DTYPES[case["x"]])
        s["w"] = w if case["g"] > 1 else w[0]
        return s
    if op == "pack_rows":
        return s
    n, s["n"], s["out"] = case["n"], case["n"], DTYPES[case["out"]]
    if op in ("gemm", "linear"):
        wq, ws = pack_weight(weights(gen, 1, n, k, torch.float32))
        s["wq"], s["ws"] = wq[0], ws[0]
        s["bias"] = torch.randn((n,), generator=gen, device=DEV) if case["bias"] else None
        if op == "gemm":
            s["xq"], s["xs"] = pack_rows(activations(gen, case["m"], k, torch.float32), None)
        return s
    g = case["g"]
    packed = [pack_weight(weights(gen, 1, n, k, torch.float32)) for _ in range(g)]
    s["wq"], s["ws"] = torch.cat([p[0] for p in packed]), torch.cat([p[1] for p in packed])
    del packed
    if op == "experts":
        # each token goes to `top` distinct experts; the rows of an expert are in token order
        top = min(case["top"], g)
        pairs = sorted((e, t) for t in range(case["tokens"]) for e in rng.sample(range(g), top))
        count = [0] * g
        for e, _ in pairs:
            count[e] += 1
        offsets = [0]
        for c in count:
            offsets.append(offsets[-1] + c)
        s["x"] = activations(gen, case["tokens"], k, DTYPES[case["x"]])
        s["index"] = torch.tensor([t for _, t in pairs], dtype=torch.int32, device=DEV)
        room = len(pairs)
    else:
        offsets = spread(rng, case["rows"], g)
        room = case["rows"] + case["tail"]
        s["xq"], s["xs"] = pack_rows(activations(gen, room, k, torch.float32), None)
    s["offsets"] = torch.tensor(offsets, dtype=torch.int64, device=DEV)
    s["longest"] = max(b - a for a, b in zip(offsets, offsets[1:]))
    s["y"] = torch.zeros((room, n), dtype=s["out"], device=DEV)
    return s


# ------------------------------------------------------------------------------------------------ plain forms


def scale_of(top):
    """Block maxima -> (scale, factor): NaN and 0 where a block holds an infinity or a NaN."""
    fine = torch.isfinite(top)
    a = torch.clamp(torch.where(fine, top, torch.ones_like(top)), min=TINY)
    c = torch.full_like(a, TOP)  # a tensor: division by a number may become a product with its reciprocal
    return torch.where(fine, a / c, torch.full_like(a, math.nan)), c / a, fine


def e4m3(v):
    return torch.clamp(v, -TOP, TOP).to(torch.float8_e4m3fn)


def pack_rows(x, index):
    """[m, k] -> e4m3 [rows, 128 kb], scales [kb, rows]."""
    if index is not None:
        x = x[index.long()]
    m, k = x.shape
    kb = blocks(k)
    v = torch.nn.functional.pad(x.float(), (0, 128 * kb - k)).view(m, kb, 128)
    scale, factor, fine = scale_of(v.abs().amax(dim=2))
    q = torch.where(fine[:, :, None], v * factor[:, :, None], torch.zeros_like(v))
    return e4m3(q).view(m, 128 * kb), scale.t().contiguous()


def pack_weight(w):
    """[g, n, k] -> e4m3 [g, n, 128 kb], scales [g, ceil(n/128), kb]."""
    g, n, k = w.shape
    kb, nb = blocks(k), blocks(n)
    v = torch.nn.functional.pad(w.float(), (0, 128 * kb - k, 0, 128 * nb - n)).view(g, nb, 128, kb, 128)
    scale, factor, fine = scale_of(v.abs().amax(dim=4).amax(dim=2))
    q = torch.where(fine[:, :, None, :, None], v * factor[:, :, None, :, None], torch.zeros_like(v))
    return e4m3(q).view(g, 128 * nb, 128 * kb)[:, :n].contiguous(), scale


def rows_of(xq, xs):
    m, kp = xq.shape
    return (xq.float().view(m, kp // 128, 128) * xs.t()[:, :, None]).view(m, kp)


def weights_of(wq, ws):
    g, n, kp = wq.shape
    each = ws.repeat_interleave(128, dim=1)[:, :n]
    return (wq.float().view(g, n, kp // 128, 128) * each[:, :, :, None]).view(g, n, kp)


def gemm(xq, xs, wq, ws, bias, out):
    y = rows_of(xq, xs) @ weights_of(wq[None], ws[None])[0].t()
    return (y if bias is None else y + bias).to(out)


def grouped(xq, xs, wq, ws, offsets, longest, y):
    """The groups padded to the longest, one batched product, and the rows picked out of it."""
    room, n = y.shape
    x = rows_of(xq, xs)
    at = offsets[:-1, None] + torch.arange(longest, device=x.device)[None, :]
    z = torch.bmm(x[at.clamp(max=room - 1)], weights_of(wq, ws).transpose(1, 2))
    row = torch.arange(room, device=x.device)
    live = row < offsets[-1]
    group = (torch.searchsorted(offsets, row, right=True) - 1).clamp(max=offsets.numel() - 2)
    pick = (row - offsets[group]).clamp(max=longest - 1)
    y.copy_(torch.where(live[:, None], z[group, pick].to(y.dtype), y))
    return y


def run(s):
    op = s["op"]
    if own:
        from ternary_neural_net_b200 import bnn

        if op == "pack_rows":
            return bnn.bnn_fp8_pack_rows(s["x"])
        if op == "pack_weight":
            return bnn.bnn_fp8_pack_weight(s["w"])
        if op == "gemm":
            return bnn.bnn_fp8_gemm(s["xq"], s["xs"], s["wq"], s["ws"], s["bias"], out_dtype=s["out"])
        if op == "linear":
            xq, xs = bnn.bnn_fp8_pack_rows(s["x"])
            return bnn.bnn_fp8_gemm(xq, xs, s["wq"], s["ws"], s["bias"], out_dtype=s["out"])
        xq, xs = bnn.bnn_fp8_pack_rows(s["x"], s["index"]) if op == "experts" else (s["xq"], s["xs"])
        return bnn.bnn_fp8_grouped_gemm(xq, xs, s["wq"], s["ws"], s["offsets"], out=s["y"])
    if op == "pack_rows":
        return pack_rows(s["x"], None)
    if op == "pack_weight":
        w = s["w"]
        q, scale = pack_weight(w if w.dim() == 3 else w[None])
        return (q, scale) if w.dim() == 3 else (q[0], scale[0])
    if op == "gemm":
        return gemm(s["xq"], s["xs"], s["wq"], s["ws"], s["bias"], s["out"])
    if op == "linear":
        xq, xs = pack_rows(s["x"], None)
        return gemm(xq, xs, s["wq"], s["ws"], s["bias"], s["out"])
    xq, xs = pack_rows(s["x"], s["index"]) if op == "experts" else (s["xq"], s["xs"])
    return grouped(xq, xs, s["wq"], s["ws"], s["offsets"], s["longest"], s["y"])


# ------------------------------------------------------------------------------------------------ in 64 bits


def nearest_e4m3(v):
    """float64 values to the nearest of e4m3's, ties to the even one: 3 fraction bits, exponents from -6, 448 the largest."""
    e = torch.floor(torch.log2(torch.clamp(v.abs(), min=2.0 ** -20))).clamp(min=-6.0)
    e = e + (v.abs() >= torch.exp2(e + 1.0)).double() - ((v.abs() < torch.exp2(e)) & (e > -6.0)).double()
    step = torch.exp2(e - 3.0)
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def exact_pack(x, rows_per_scale):
    """[n, k] -> (values of q [n, 128 kb], scales [n / rows_per_scale rounded up, kb]); the scale and the factor 448 / a are
    float32 numbers by the operator's definition, and so is the product that is rounded to e4m3."""
    n, k = x.shape
    kb, nr = -(-k // 128), -(-n // rows_per_scale)
    v = torch.zeros((nr * rows_per_scale, 128 * kb), dtype=torch.float64, device=x.device)
    v[:n, :k] = x.double()
    v = v.reshape(nr, rows_per_scale, kb, 128).transpose(1, 2)
    a = torch.maximum(v.abs().reshape(nr, kb, -1).max(dim=2).values, torch.tensor(2.0 ** -100, dtype=torch.float64, device=x.device))
    scale = (a / 448.0).float().double()
    factor = (448.0 / a).float().double()
    q = nearest_e4m3((v * factor[:, :, None, None]).float().double())
    return q.transpose(1, 2).reshape(nr * rows_per_scale, 128 * kb)[:n], scale


def exact_values(q, scale, rows_per_scale):
    n = q.shape[0]
    return q.double() * scale.double().repeat_interleave(rows_per_scale, 0)[:n].repeat_interleave(128, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "pack_rows":
        q, scale = exact_pack(s["x"], 1)
        return q, scale.t().contiguous()
    if op == "pack_weight":
        w = s["w"] if s["w"].dim() == 3 else s["w"][None]
        parts = [exact_pack(w[i], 128) for i in range(w.shape[0])]
        q, scale = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
        return (q, scale) if s["w"].dim() == 3 else (q[0], scale[0])
    if op in ("gemm", "linear"):
        if op == "linear":
            x = exact_values(*exact_pack(s["x"], 1), 1)
        else:
            x = exact_values(s["xq"], s["xs"].t(), 1)
        y = torch.matmul(x, exact_values(s["wq"], s["ws"], 128).t())
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "experts":
        x = exact_values(*exact_pack(s["x"], 1), 1)[s["index"].long()]
    else:
        x = exact_values(s["xq"], s["xs"].t(), 1)
    offsets = s["offsets"].tolist()
    y = s["y"].double()
    for g in range(case["g"]):
        a, b = offsets[g], offsets[g + 1]
        if b > a:
            y[a:b] = torch.matmul(x[a:b], exact_values(s["wq"][g], s["ws"][g], 128).t())
    return y
