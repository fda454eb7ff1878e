"""How a prompt attention's key tiles are shared out over the CTAs, checked on the CPU with the kernel's own arithmetic."""
import os
import random
import subprocess

import pytest

from skinny_gemm_bit_gb300 import build as tfq_build

SMS = 2 * 152  # two groups a CTA, each with a share


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = tmp_path_factory.mktemp("shares") / "prompt_shares"
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "prompt_shares.cu")
    subprocess.run([tfq_build.nvcc(), *tfq_build.ARCH, "-O1", "-std=c++17", "--expt-relaxed-constexpr", "-I", tfq_build.INCLUDE, "-I",
                    tfq_build.CSRC, src, "-o", str(exe)], check=True, capture_output=True)
    return exe


def run(program, calls):
    lines = [f"{SMS} {n_kv} {group} {over} {len(seqs)} " + " ".join(f"{r} {n}" for r, n in seqs) for n_kv, group, over, seqs in calls]
    r = subprocess.run([str(program)], input="\n".join(lines), capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == f"{len(calls)} calls\n", r.stdout + r.stderr


def test_every_tile_once(program):
    rng = random.Random(2)
    calls = []
    for _ in range(1500):
        B = rng.choice([1, 1, 2, 3, 8, 32, 152, 300])
        most, ctx = int(2 ** rng.uniform(0, 13 if B < 10 else 9)), rng.choice([0, 0, int(2 ** rng.uniform(0, 17))])
        seqs = []
        for _ in range(B):
            rows = rng.randint(0, most)
            seqs.append((rows, rows + rng.randint(0, ctx)))
        calls.append((rng.choice([1, 2, 4, 8, 19]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 63, 64]), rng.choice([2, 4, 8, 20]), seqs))
    run(program, calls)


@pytest.mark.parametrize("n_kv,group,seqs", [(1, 1, [(1, 1)]), (1, 64, [(1, 1)]), (8, 2, [(100_000, 1_000_000)]), (256, 1, [(700, 70_000)]),
                                             (2, 63, [(30_000, 30_000), (0, 5), (1, 900_000)])])
def test_the_smallest_and_the_largest(program, n_kv, group, seqs):
    run(program, [(n_kv, group, 8, seqs)])
