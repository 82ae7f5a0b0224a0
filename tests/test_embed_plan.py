"""How the gradient of a token table is cut, from its sizes alone: compiled from csrc/train_embed_plan.h."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "decoupled_momentum_optimizer_gb300", "csrc")


@pytest.fixture(scope="module")
def plan():
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    out_dir = os.path.join(ROOT, "_build")
    os.makedirs(out_dir, exist_ok=True)
    exe = os.path.join(out_dir, "embed_plan_client")
    r = subprocess.run([cxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC,
                        os.path.join(ROOT, "tests", "embed_plan_client.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(sizes):
        r = subprocess.run([exe], input="\n".join(" ".join(map(str, s)) for s in sizes), capture_output=True, text=True, timeout=60)
        assert r.returncode == 0
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]

    return run


def test_rows_behind_the_filled_ones_start_on_16_bytes(plan):
    """Runs of rows that a warp zeroes start a multiple of four rows behind the filled ones."""
    vocab = 2 ** 31 - 512
    sizes = [(n, vocab, cols) for n in (33, 40, 3000, 4096, 9000, 65536) for cols in [*range(1, 1100), 1033, 2051, 8193, 32768, 2 ** 31 - 512]]
    for (n, _, cols), (rows, _) in zip(sizes, plan(sizes)):
        want = (44 * 2 ** 20 + 1536 * n) * (2 if cols < 128 else 1)  # bytes that the sort takes time for
        assert rows % 4 == 0 and want <= rows * cols * 4 < want + 5 * cols * 4


def test_no_more_rows_are_filled_than_there_are(plan):
    sizes = [(4096, vocab, cols) for vocab in (1, 2, 3, 5, 1001, 32128) for cols in (1, 3, 64, 765)]
    assert all(rows <= vocab for (_, vocab, _), (rows, _) in zip(sizes, plan(sizes)))
    assert plan([(4096, 1001, 3)])[0][0] == 1001


def test_pieces_follow_from_the_positions_and_the_columns(plan):
    """The order of the sums is decided by both: columns of a table need not be summed as the whole table is."""
    sizes = [(n, vocab, cols) for n in (33, 128, 4096, 65536) for vocab in (5, 32128, 2 ** 31 - 512) for cols in (1, 256, 768, 1024, 2048)]
    pieces = {}
    for (n, _, cols), (_, piece) in zip(sizes, plan(sizes)):
        assert piece in (8, 16, 32) and pieces.setdefault((n, cols), piece) == piece
    assert [pieces[4096, cols] for cols in (256, 768, 1024)] == [8, 16, 32]
