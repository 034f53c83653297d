"""Device times of the 8-bit operators: each listed case of perf/operators.py, and some more sizes, as calls back
to back in a CUDA graph.

    python perf/device_times.py [--only TEXT] [--csv]

The calls of a graph take their inputs in turn from copies of more than twice the L2 size in all (24 copies at
most, so that operands of up to 10 MB stay in L2), with events around a replay: the median of nine replays, after
three. Beside it the SM clock sampled meanwhile and the reasons that the driver gave for lowering it. The first
figure of a case is a short burst; "held" is the same graph replayed for half a second, where the power cap
settles.
"""
import argparse
import os
import statistics
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

from bench import L2_BYTES, ClockSampler  # noqa: E402
from perf import operators  # noqa: E402
from ternary_neural_net_b200 import bnn  # noqa: E402


def bytes_of(state):
    return sum(v.numel() * v.element_size() for v in state.values() if torch.is_tensor(v))


def operator_case(case):
    """Copies of a listed case's state, as calls."""
    first = operators.prepare(case, 1)
    copies = max(1, min(24, int(2.2 * L2_BYTES / bytes_of(first)) + 1))
    states = [first] + [operators.prepare(case, s) for s in range(2, copies + 1)]
    return [lambda s=s: operators.run(s) for s in states]


def codes(*shape):
    q = torch.randint(0, 120, shape, dtype=torch.uint8, device="cuda")
    return (q | torch.randint(0, 2, shape, dtype=torch.uint8, device="cuda") << 7).view(torch.float8_e4m3fn)


def product(m, n, k, out, sizes=None):
    """Copies of one product, as calls; with `sizes` grouped, its rows in a buffer of m."""
    kb, nb = -(-k // 128), -(-n // 128)
    lead = (len(sizes),) if sizes else ()
    copies = max(1, min(24, int(2.2 * L2_BYTES / ((len(sizes) if sizes else 1) * n * k + m * k)) + 1))
    off = torch.tensor([sum(sizes[:i]) for i in range(len(sizes) + 1)], device="cuda") if sizes else None
    calls = []
    for _ in range(copies):
        ops = (codes(m, 128 * kb), torch.rand(kb, m, device="cuda"), codes(*lead, n, 128 * kb),
               torch.rand(*lead, nb, kb, device="cuda"))
        y = torch.empty((m, n), dtype=out, device="cuda")
        calls.append((lambda o=ops, y=y: bnn.bnn_fp8_grouped_gemm(*o, off, out=y)) if sizes else
                     (lambda o=ops, y=y: bnn.bnn_fp8_gemm(*o, out=y)))
    return calls


F32, BF16 = torch.float32, torch.bfloat16
MORE = {
    "product 16x28672x8192 bf16": lambda: product(16, 28672, 8192, BF16),
    "product 1x28672x8192 bf16": lambda: product(1, 28672, 8192, BF16),
    "product 1x4096x4096 bf16": lambda: product(1, 4096, 4096, BF16),
    "product 32x4096x4096 f32": lambda: product(32, 4096, 4096, F32),
    "product 64x11008x4096 bf16": lambda: product(64, 11008, 4096, BF16),
    "product 256x4096x4096 f32": lambda: product(256, 4096, 4096, F32),
    "product 1024x11008x4096 bf16": lambda: product(1024, 11008, 4096, BF16),
    "product 2048x4096x4096 bf16": lambda: product(2048, 4096, 4096, BF16),
    # a long k and few tiles
    "product 32x512x16384 f32": lambda: product(32, 512, 16384, F32),
    "product 33x512x16384 f32": lambda: product(33, 512, 16384, F32),
    "product 64x1024x16384 f32": lambda: product(64, 1024, 16384, F32),
    "product 128x256x16384 f32": lambda: product(128, 256, 16384, F32),
    # groups as decoding has them, even, all rows in a few, and in a buffer of fixed capacity
    "64 experts, 512 rows even, 2048x4096 bf16": lambda: product(512, 2048, 4096, BF16, [8] * 64),
    "64 experts, 512 rows in one, 2048x4096 bf16": lambda: product(512, 2048, 4096, BF16, [0] * 9 + [512] + [0] * 54),
    "64 experts, 4096 rows even, 2048x4096 bf16": lambda: product(4096, 2048, 4096, BF16, [64] * 64),
    "64 experts, 4096 rows in 4, 2048x4096 bf16": lambda: product(4096, 2048, 4096, BF16, [1024] * 4 + [0] * 60),
    "64 experts, 64 rows, 2048x4096 bf16": lambda: product(64, 2048, 4096, BF16, [1] * 64),
    "64 experts, 64 rows in a buffer of 4096, 2048x4096 bf16": lambda: product(4096, 2048, 4096, BF16, [1] * 64),
}


def measure(calls):
    """(us a call in a short burst, us a call held for half a second, clocks of the burst, clocks of the hold)."""
    for c in calls:
        c()
    torch.cuda.synchronize()
    graph, per = torch.cuda.CUDAGraph(), len(calls) * -(-24 // len(calls))
    with torch.cuda.graph(graph):
        for i in range(per):
            calls[i % len(calls)]()

    def replay(n):
        marks = [torch.cuda.Event(enable_timing=True) for _ in range(n + 1)]
        marks[0].record()
        for m in marks[1:]:
            graph.replay()
            m.record()
        torch.cuda.synchronize()
        return [a.elapsed_time(b) * 1000 / per for a, b in zip(marks, marks[1:])]
    replay(3)
    with ClockSampler(0, 0.0005) as burst:
        times = replay(9)
    us = statistics.median(times)
    n = max(9, int(0.5e6 / (us * per)))
    with ClockSampler(0, 0.002) as hold:
        held = replay(n)
    return us, statistics.median(held[n // 2:]), burst.summary(), hold.summary()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--only", default="")
    ap.add_argument("--csv", action="store_true")
    args = ap.parse_args()
    operators.own = True
    cases = {c["name"]: (lambda c=c: operator_case(c)) for c in operators.listed()}
    cases.update(MORE)
    if args.csv:
        print("case,us,held_us,sm_mhz,held_sm_mhz,held_reasons")
    for name, make in cases.items():
        if args.only not in name:
            continue
        calls = make()
        us, held, a, b = measure(calls)
        del calls
        torch.cuda.empty_cache()
        why = "+".join(b["reasons"]) or "none"
        if args.csv:
            print(f'"{name}",{us:.2f},{held:.2f},{a["sm_mhz"]},{b["sm_mhz"]},{why}', flush=True)
        else:
            print(f"{name:58s} {us:8.2f} us at {a['sm_mhz']} MHz   held {held:8.2f} us at {b['sm_mhz']} MHz ({why})",
                  flush=True)


if __name__ == "__main__":
    main()
