"""How an attention call's key tiles are shared out over the CTAs, checked on the CPU with the arithmetic that the
kernels themselves compile: every tile once, and every part that a join waits for written."""
import os
import random
import subprocess

import pytest

from skinny_gemm_bit_gb300 import build as tfq_build

SMS = 152


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = tmp_path_factory.mktemp("shares") / "attn_shares"
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "attn_shares.cu")
    subprocess.run([tfq_build.nvcc(), *tfq_build.ARCH, "-O1", "-std=c++17", "--expt-relaxed-constexpr", "-I", tfq_build.INCLUDE, "-I",
                    tfq_build.CSRC, src, "-o", str(exe)], check=True, capture_output=True)
    return exe


def call(kernel, n_kv, group, seqs, max_rows):
    """A call as tf_tree_attn_run describes it to the kernel of `kernel` rows (1616: 16 rows, 16-key tiles)."""
    rows = 16 if kernel == 1616 else kernel
    items = len(seqs) * n_kv * -(-max_rows * group // rows)
    few = items <= SMS and len(seqs) <= 256
    over = 20 if rows > 32 else 28 if items > SMS else 16
    return f"{kernel} {SMS} {n_kv} {group} {int(few)} {over} {len(seqs)} " + " ".join(f"{r} {n}" for r, n in seqs)


def run(program, calls):
    r = subprocess.run([str(program)], input="\n".join(calls), capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == f"{len(calls)} calls\n", r.stdout + r.stderr


def test_every_tile_once(program):
    rng = random.Random(1)
    calls = []
    for _ in range(3000):
        kernel = rng.choice([16, 1616, 32, 128, 256])
        n_kv, group, max_rows = rng.choice([1, 2, 4, 8, 19]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 8, 33, 64])
        B = rng.choice([1, 1, 2, 3, 8, 19, 64, 152, 300])
        most = int(2 ** rng.uniform(0, 17))
        seqs = []
        for _ in range(B):
            rows = rng.randint(0, max_rows)
            seqs.append((rows, rows + rng.randint(0, most)))
        calls.append(call(kernel, n_kv, group, seqs, max_rows))
    run(program, calls)


@pytest.mark.parametrize("kernel,n_kv,B,tokens", [(16, 8, 19, 40_000_000), (16, 1, 152, 33_600_000), (32, 4, 38, 60_000_000),
                                                   (1616, 8, 19, 20_000_000), (16, 152, 1, 300_000_000), (16, 76, 2, 33_554_432)])
def test_very_long_sequences_with_an_item_for_each_cta(program, kernel, n_kv, B, tokens):
    run(program, [call(kernel, n_kv, 1, [(1, tokens)] * B, 1), call(kernel, n_kv, 1, [(1, tokens - 7 * b) for b in range(B)], 1)])
