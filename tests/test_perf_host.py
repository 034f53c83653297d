"""perf/: the listed cases and the device-time program load without a GPU, and their names are their own."""
import random
import subprocess
import sys

from conftest import ROOT


def test_cases_and_draws():
    from perf import operators
    cases = operators.listed()
    names = [c["name"] for c in cases]
    assert len(set(names)) == len(names) and operators.own is False
    rng = random.Random(1)
    for c in cases + [operators.draw(rng) for _ in range(20)]:
        w = operators.work(c)
        assert w["bytes"] > 0 and w["flops"] >= 0


def test_device_times_loads():
    from perf import device_times, operators
    assert not set(device_times.MORE) & {c["name"] for c in operators.listed()}
    r = subprocess.run([sys.executable, "perf/device_times.py", "--help"], cwd=ROOT, capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0 and "--only" in r.stdout
