"""How a product is laid out on a device, from that device's own cluster counts: compiled from
csrc/train_plan.h alone, for devices that are not here (a part of a GPU, one with fewer SMs together)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "decoupled_momentum_optimizer_gb300", "csrc")
SIZES = [(m, n, kb) for m in (1, 8, 57, 128, 129, 200, 768, 2100, 8192) for n in (1, 33, 300, 768, 2048, 8192, 32128)
         for kb in (0, 1, 5, 16, 64, 128)]
# pairs, then clusters of 1 .. 8
WHOLE = [76, 152, 76, 48, 36, 28, 24, 20, 16]
DEVICES = {"whole": WHOLE, "no eights": WHOLE[:8] + [0], "pairs alone": [4, 8, 4, 0, 0, 0, 0, 0, 0],
           "no pairs": [0, 6, 0, 0, 0, 0, 0, 0, 0], "one": [0, 1, 0, 0, 0, 0, 0, 0, 0]}


@pytest.fixture(scope="module")
def plans():
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    out_dir = os.path.join(ROOT, "_build")
    os.makedirs(out_dir, exist_ok=True)
    exe = os.path.join(out_dir, "plan_client")
    r = subprocess.run([cxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC,
                        os.path.join(ROOT, "tests", "plan_client.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(clusters):
        text = " ".join(map(str, clusters)) + "\n" + "\n".join(" ".join(map(str, s)) for s in SIZES)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
        assert r.returncode == 0
        keys = ("group", "bn", "split", "stages", "rows_a", "rows_b", "chain", "grid")
        return [dict(zip(keys, map(int, line.split()))) for line in r.stdout.splitlines()]

    return run


@pytest.mark.parametrize("device", DEVICES)
def test_plans_fit_their_device(plans, device):
    """Whole clusters that the device can run, every tile covered, stages and boxes within their limits."""
    of = DEVICES[device]
    got = plans(of)
    assert len(got) == len(SIZES)
    for (m, n, kb), p in zip(SIZES, got):
        tiles = -(-m // (128 * p["group"])) * -(-n // p["bn"])
        assert p["bn"] % 32 == 0 and 64 <= p["bn"] <= 224 and p["rows_b"] * p["group"] == p["bn"]
        assert p["rows_a"] % 8 == 0 and min(m, 128) <= p["rows_a"] <= 128 and p["chain"] == 4
        if p["group"] == 2:
            assert of[0] > 0 and p["grid"] == 2 * min(tiles, of[0]) and p["split"] == 1 and p["stages"] == 5
        else:
            assert p["grid"] == tiles * p["split"] and 1 <= p["split"] <= max(1, -(-kb // 4))
            assert p["split"] == 1 or tiles <= of[p["split"]]
            assert 3 <= p["stages"] <= 8 and p["stages"] * (p["rows_a"] + p["bn"]) * 128 <= 3 * 352 * 128


def test_a_missing_cluster_size_takes_only_itself_away(plans):
    """Where no cluster of eight fits, everything that does not cut k into eight stays as it was."""
    for a, b in zip(plans(WHOLE), plans(DEVICES["no eights"])):
        assert a == b or a["split"] == 8
    assert {2, 4, 8} <= {p["split"] for p in plans(WHOLE)} and {1, 2} == {p["group"] for p in plans(WHOLE)}


def test_a_device_without_place_for_the_kernel(plans):
    assert all(p["grid"] == 0 for p in plans([0] * 9))
