"""How key tiles are shared out over an 8-bit cache, checked on the CPU with the kernels' own arithmetic: few rows, which two
CTAs an SM take, and prompts in row tiles of 256."""
import os
import random
import subprocess

import pytest

from skinny_gemm_bit_gb300 import build as tfq_build

SMS = 152


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = tmp_path_factory.mktemp("shares") / "shares_8bit"
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "shares_8bit.cu")
    subprocess.run([tfq_build.nvcc(), *tfq_build.ARCH, "-O1", "-std=c++17", "--expt-relaxed-constexpr", "-I", tfq_build.INCLUDE, "-I",
                    tfq_build.CSRC, src, "-o", str(exe)], check=True, capture_output=True)
    return exe


def drafts(n_kv, group, seqs, max_rows):
    """A call of at most 16 query rows to an item, as tf_tree_attn_run describes it to the kernel with two CTAs an SM."""
    items = len(seqs) * n_kv * -(-max_rows * group // 16)
    few = items <= SMS and len(seqs) <= 192
    return f"A 16 {2 * SMS} {n_kv} {group} {int(few)} {28 if items > SMS else 16} {len(seqs)} " + " ".join(f"{r} {n}" for r, n in seqs)


def prompts(n_kv, group, seqs, over=4):
    return f"P {SMS} {n_kv} {group} {over} {len(seqs)} " + " ".join(f"{r} {n}" for r, n in seqs)


def run(program, calls):
    r = subprocess.run([str(program)], input="\n".join(calls), capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == f"{len(calls)} calls\n", r.stdout + r.stderr


def test_every_tile_of_drafts_once(program):
    rng = random.Random(3)
    calls = []
    for _ in range(2500):
        n_kv, group = rng.choice([1, 2, 4, 8, 19]), rng.choice([1, 2, 4, 8])
        max_rows = rng.choice([1, 2, 8, 16 // group])
        B, most, seqs = rng.choice([1, 1, 2, 3, 8, 19, 38, 64, 152, 192, 300]), int(2 ** rng.uniform(0, 17)), []
        for _ in range(B):
            rows = rng.randint(0, max_rows)
            seqs.append((rows, rows + rng.randint(0, most)))
        calls.append(drafts(n_kv, group, seqs, max_rows))
    run(program, calls)


@pytest.mark.parametrize("n_kv,B", [(8, 32), (8, 19), (8, 20), (8, 38), (1, 152), (1, 304), (2, 304)])
def test_sequences_of_one_length_to_about_as_many_items_as_ctas(program, n_kv, B):
    run(program, [drafts(n_kv, 2, [(1, tokens)] * B, 1) for tokens in (1, 31, 32, 33, 200, 500, 768, 1000, 1800, 3000, 20000)])


@pytest.mark.parametrize("n_kv,B,tokens", [(8, 19, 40_000_000), (1, 152, 33_600_000), (152, 1, 300_000_000), (76, 2, 33_554_432)])
def test_very_long_sequences(program, n_kv, B, tokens):
    run(program, [drafts(n_kv, 1, [(1, tokens)] * B, 1), drafts(n_kv, 1, [(1, tokens - 7 * b) for b in range(B)], 1)])


def test_every_tile_of_prompts_once(program):
    rng = random.Random(4)
    calls = []
    for _ in range(1500):
        B = rng.choice([1, 1, 2, 3, 8, 32, 152, 300])
        most, ctx = int(2 ** rng.uniform(0, 13 if B < 10 else 9)), rng.choice([0, 0, int(2 ** rng.uniform(0, 17))])
        seqs = []
        for _ in range(B):
            rows = rng.randint(0, most)
            seqs.append((rows, rows + rng.randint(0, ctx)))
        calls.append(prompts(rng.choice([1, 2, 4, 8, 19]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 63, 64]), seqs, rng.choice([2, 4, 8, 20])))
    run(program, calls)


@pytest.mark.parametrize("n_kv,group,seqs", [(1, 1, [(1, 1)]), (1, 64, [(1, 1)]), (4, 1, [(255, 255)]), (4, 1, [(256, 256)]), (4, 1, [(257, 257)]),
                                             (8, 2, [(100_000, 1_000_000)]), (256, 1, [(700, 70_000)]),
                                             (2, 63, [(30_000, 30_000), (0, 5), (1, 900_000)])])
def test_the_smallest_and_the_largest_prompts(program, n_kv, group, seqs):
    run(program, [prompts(n_kv, group, seqs)])
