"""Attention over many key tiles, where what counts is that each tile takes part once: values that mark their tile, the
counters after a call, and a wait that runs out."""
import numpy as np
import pytest
import torch

import cached_ref as R
import test_gpu_cached_decode as D
from test_gpu_cached_decode import check_attn, filled_cache, i32, rand, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    from skinny_gemm_bit_gb300 import build
    build.build()
    from skinny_gemm_bit_gb300 import tfq
    return tfq


def counters(ws):
    """The part of an attention workspace that its CTAs count in (two words an SM), behind the status word's 256 bytes."""
    return ws[256:256 + 8 * torch.cuda.get_device_properties(0).multi_processor_count]


def marked_values(c, layer, n):
    """Slot 0's token r gets the value 1 in column r // 16 % head_dim and 0 elsewhere."""
    r = torch.arange(n, device="cuda")
    v = torch.zeros((n, c.n_kv, c.head_dim), dtype=torch.bfloat16, device="cuda")
    v[r, :, r // 16 % c.head_dim] = 1
    c.data[layer, 1, c.table[0].long()[r // c.page_size], :, r % c.page_size] = v


# query rows to a key/value head: 2 and 16 (16-row warp kernel), 32 (32-row), 64 and 128 (128 rows in tensor memory),
# 136 and 512 (256); head dim 256 is always the 16-row kernel's, with 16-key tiles
@pytest.mark.parametrize("n,rows,n_q,n_kv,hd,page", [
    (40000, 1, 4, 2, 128, 16), (40001, 8, 4, 2, 128, 32), (39999, 8, 8, 2, 128, 64), (20017, 5, 12, 2, 128, 16),
    (40000, 32, 2, 2, 64, 128), (40003, 8, 1, 1, 64, 16), (30011, 16, 8, 4, 64, 32), (40000, 64, 1, 1, 128, 32),
    (30000, 32, 8, 2, 128, 32), (24001, 17, 16, 2, 128, 32), (20000, 64, 8, 1, 128, 16), (30013, 64, 2, 1, 64, 32),
    (25000, 40, 8, 1, 64, 32), (30001, 3, 4, 2, 256, 32), (12345, 9, 8, 2, 256, 64),
])
def test_every_tile_takes_part_once(T, n, rows, n_q, n_kv, hd, page):
    """Weights near one another, so that a column's value is some tens of 16-token stretches' share each: leaving one out,
    or taking it twice, is 16 hd / n of the column (2 % and more), against a tolerance of 0.8 % of it."""
    assert 16 * hd / n > 2.5 * 2.0 ** -7
    c = filled_cache(T, [n, 3, 777], n_kv, hd, page, n, layers=1)
    marked_values(c, 0, n)
    M = rows + 2
    q, out = rand((M, n_q * hd), 5, 2.0), torch.full((M, n_q * hd), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = T.workspace(T.tf_tree_attn_workspace_bytes(c, n_q, 3, rows))
    for _ in range(2):
        T.tf_tree_attn_run(q, c, 0, i32([1, 0, 2]), i32([0, 1, 1 + rows, 2 + rows]), max_rows=rows, scale=0.01, out=out, ws=ws)
        assert int(torch.count_nonzero(counters(ws))) == 0
    assert T.tf_workspace_status(ws) == T.TF_OK
    qq = R.f64(q[1:1 + rows]).reshape(rows, n_q, hd)
    k = D.tokens(c, 0, 0, 0)
    group = n_q // n_kv
    ref = np.zeros((rows, n_q, hd))
    column = np.arange(n) // 16 % hd
    see = np.arange(n)[None] < n - rows + 1 + np.arange(rows)[:, None]
    for h in range(n_q):
        s = qq[:, h] @ k[:, h // group].T * 0.01
        p = np.where(see, np.exp(s - s.max(1, keepdims=True)), 0.0)
        p /= p.sum(1, keepdims=True)
        for t in range(rows):
            ref[t, h] = np.bincount(column, p[t], hd)
    within(R.f64(out[1:1 + rows]).reshape(rows, n_q, hd), ref, R.attn_tol(ref, ref))


@pytest.mark.parametrize("lens,rows,n_q,n_kv,hd,page", [
    ([9001, 2500, 40, 700], [8, 4, 8, 6], 16, 4, 128, 16),      # 17 to 32 query rows to a key/value head
    ([20000], [8], 8, 2, 128, 64),
    ([6000, 6100], [16, 15], 4, 2, 64, 128),
    ([9000, 300], [40, 33], 6, 2, 128, 32),                     # tensor memory, pages of 32
    ([5000, 60], [64, 17], 16, 2, 64, 32),
    ([3000, 900, 31], [64, 9, 20], 8, 1, 128, 32),
    ([7000, 33, 2100], [2, 1, 4], 4, 2, 128, 128),              # pages of 128
    ([8000], [3], 2, 1, 256, 128),
])
def test_many_tiles_to_a_warp(T, lens, rows, n_q, n_kv, hd, page):
    rng = np.random.default_rng(sum(lens))
    c = filled_cache(T, lens, n_kv, hd, page, 17 + sum(lens))
    seqs = list(range(len(lens)))
    check_attn(T, c, 1, seqs, rows, None, n_q, 3)
    check_attn(T, c, 0, seqs, rows, [D.tree(r, rng) for r in rows], n_q, 4, scale=0.2)


@pytest.mark.parametrize("hd,rows,n_q", [(128, 8, 8), (64, 16, 4), (128, 12, 4)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_in_items_of_32_rows(T, hd, rows, n_q, what):
    D.test_tree_attn_what_a_row_does_not_see_takes_no_part(T, hd, rows, n_q, what)


@pytest.mark.parametrize("rows,n_q", [(1, 4), (8, 16), (64, 4), (64, 16)])
def test_a_wait_that_runs_out_is_reported(T, rows, n_q):
    """Counters that start one below zero: every CTA of the split item writes its part and waits, within its limit, for
    one more than there are. The call ends with its status; the workspace zeroed, it is as good as new."""
    n = 30000
    c = filled_cache(T, [n], 2, 128, 64, 9, layers=1)
    q, seqs, start = rand((rows, n_q * 128), 5, 2.0), i32([0]), i32([0, rows])
    need = T.tf_tree_attn_workspace_bytes(c, n_q, 1, rows)
    want = T.tf_tree_attn_run(q, c, 0, seqs, start, max_rows=rows)
    ws, out = T.workspace(need), torch.empty_like(q)
    counters(ws).fill_(255)
    T.tf_tree_attn_run(q, c, 0, seqs, start, max_rows=rows, out=out, ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_E_TIMEOUT
    ws.zero_()
    T.tf_tree_attn_run(q, c, 0, seqs, start, max_rows=rows, out=out, ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_OK and torch.equal(out, want)
