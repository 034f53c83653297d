"""The 8-bit block-scaled calls where offsets pass 32 bits (operands and outputs of more than 2^32 bytes or
elements), and as the very first calls of a process inside a graph capture."""
import os
import subprocess
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bnn(cuda_device):
    if torch.cuda.get_device_properties(0).total_memory < 60e9:
        pytest.skip("needs 60 GB")
    from ternary_neural_net_b200 import bnn as mod
    yield mod
    torch.cuda.empty_cache()


def _values(q, s):
    """Packed rows as float64 [rows, 128 kb]."""
    return q.double() * s.t().double().repeat_interleave(128, dim=1)


def _weights(q, s):
    return q.double() * s.double().repeat_interleave(128, dim=0)[:q.shape[0]].repeat_interleave(128, dim=1)


def _tolerance(y, mag, kb, half):
    # as derived in test_gpu_fp8.py: 128 steps of a block's sum, kb + 3 roundings, the output type's half step
    return (128 * 2.0 ** -23 + (kb + 3) * 2.0 ** -24) * mag * (1 + half) + half * y.abs()


def _random_rows(rows, kb, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = torch.randint(0, 120, (rows, 128 * kb), dtype=torch.uint8, device="cuda", generator=g)
    q |= torch.randint(0, 2, (rows, 128 * kb), dtype=torch.uint8, device="cuda", generator=g) << 7
    return q.view(torch.float8_e4m3fn), torch.rand((kb, rows), device="cuda", generator=g) + 0.5


@pytest.mark.parametrize("rows,kb,n,out", [(540_000, 64, 130, torch.bfloat16),    # 4.4e9 operand bytes
                                           (70_000, 1, 65_600, torch.bfloat16)])  # 4.6e9 outputs
def test_gemm_past_32_bits(bnn, rows, kb, n, out):
    xq, xs = _random_rows(rows, kb, 1)
    wq, _ = _random_rows(n, kb, 2)
    ws = torch.rand((-(-n // 128), kb), device="cuda") + 0.5
    torch.cuda.synchronize()
    y = bnn.bnn_fp8_gemm(xq, xs, wq, ws, out_dtype=out)
    at = torch.tensor([0, 1, 255, rows // 2, rows - 257, rows - 2, rows - 1], device="cuda")
    x, w = _values(xq[at], xs[:, at]), _weights(wq, ws)
    want, mag = x @ w.t(), x.abs() @ w.abs().t()
    assert bool(((y[at].double() - want).abs() <= _tolerance(want, mag, kb, 2.0 ** -8)).all())
    assert bnn.device_error_count() == 0


@pytest.mark.parametrize("per", [3, 100])
def test_grouped_weights_past_32_bits(bnn, per):
    g, n, kb = 300, 4100, 32  # 5.0e9 bytes of weights
    wq, _ = _random_rows(g * n, kb, 3)
    wq = wq.view(g, n, 128 * kb)
    ws = torch.rand((g, -(-n // 128), kb), device="cuda") + 0.5
    rows = g * per
    xq, xs = _random_rows(rows, kb, 4)
    offsets = torch.arange(0, rows + 1, per, device="cuda")
    torch.cuda.synchronize()
    y = bnn.bnn_fp8_grouped_gemm(xq, xs, wq, ws, offsets)
    for e in (0, 1, 254, 255, 256, 298, 299):
        a, b = e * per, (e + 1) * per
        x, w = _values(xq[a:b], xs[:, a:b]), _weights(wq[e], ws[e])
        want, mag = x @ w.t(), x.abs() @ w.abs().t()
        assert bool(((y[a:b].double() - want).abs() <= _tolerance(want, mag, kb, 2.0 ** -24)).all()), e


def test_packs_past_32_bits(bnn):
    rows, k = 270_000, 8192  # 2.2e9 elements, 4.4e9 bytes of input
    x = torch.empty((rows, k), dtype=torch.bfloat16, device="cuda")
    for a in range(0, rows, 30_000):
        x[a:a + 30_000].normal_()
    at = torch.tensor([0, 7, 8, 131_071, 131_072, 262_143, 262_144, rows - 1], device="cuda")
    q, s = bnn.bnn_fp8_pack_rows(x)
    q1, s1 = bnn.bnn_fp8_pack_rows(x[at])
    assert torch.equal(q[at].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[:, at], s1)
    index = torch.cat([at, at.flip(0)]).int()
    q2, s2 = bnn.bnn_fp8_pack_rows(x, index)
    assert torch.equal(q2[:8].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s2[:, :8], s1)
    assert torch.equal(q2[8:].view(torch.uint8), q1.flip(0).view(torch.uint8))
    del q, s
    w = x[:266_240].view(65, 4096, k)
    q, s = bnn.bnn_fp8_pack_weight(w)
    for g in (0, 64):
        q1, s1 = bnn.bnn_fp8_pack_weight(w[g])
        assert torch.equal(q[g].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[g], s1)


FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
from ternary_neural_net_b200 import bnn
m, n, k, g = {m}, 1000, 1024, 4
x = torch.randn(m, k, device="cuda")
w = torch.randn(g, n, k, device="cuda")
off = torch.tensor([0, m // 3, m // 3, m, m], device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    wq, ws = bnn.bnn_fp8_pack_weight(w)
    xq, xs = bnn.bnn_fp8_pack_rows(x)
    y = bnn.bnn_fp8_gemm(xq, xs, wq[1], ws[1], out_dtype=torch.bfloat16)
    z = bnn.bnn_fp8_grouped_gemm(xq, xs, wq, ws, off)
graph.replay()
torch.cuda.synchronize()
a, b = bnn.bnn_fp8_pack_weight(w)
c, d = bnn.bnn_fp8_pack_rows(x)
assert torch.equal(bnn.bnn_fp8_gemm(c, d, a[1], b[1], out_dtype=torch.bfloat16), y)
assert torch.equal(bnn.bnn_fp8_grouped_gemm(c, d, a, b, off), z)
torch.cuda.synchronize()
assert bnn.device_error_count() == 0
print("same")
"""


@pytest.mark.parametrize("m", [1, 30, 300])
def test_first_calls_inside_a_capture(cuda_device, m):
    """A process whose first calls of the library are captured: nothing of their set-up breaks the capture."""
    env = dict(os.environ)
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, m=m)], capture_output=True, text=True, timeout=300,
                       env=env)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
