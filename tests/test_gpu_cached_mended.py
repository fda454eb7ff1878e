"""Cached decoding where it once went wrong, or was compared with nothing."""
import numpy as np
import pytest
import torch

import cached_ref as R
from test_gpu_cached_decode import check_attn, filled_cache, i32, rand, tokens, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    from skinny_gemm_bit_gb300 import build
    build.build()
    from skinny_gemm_bit_gb300 import tfq
    return tfq


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("n_q,hd,good", [(16, 128, 8), (64, 128, 8), (4, 256, 3)])
def test_refused_rows_do_not_hold_up_the_others(T, n_q, hd, good):
    """60,000 rows of a refused sequence become zeros while the other sequence is worked on: within 10 ms, where
    a single thread takes 45 ms for 16 heads of 128."""
    many = 60000
    c = filled_cache(T, [2000, 30], 4, hd, 32, 5, layers=1)
    q = rand((good + many + 2, n_q * hd), 6, 2.0)
    out = torch.full_like(q, 5.0)
    ws = T.workspace(T.tf_tree_attn_workspace_bytes(c, n_q, 2, good))
    seqs, start = i32([0, 1]), i32([0, good, good + many])
    ms = []
    for _ in range(3):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        T.tf_tree_attn_run(q, c, 0, seqs, start, max_rows=good, out=out, ws=ws)
        b.record()
        torch.cuda.synchronize()
        ms.append(a.elapsed_time(b))
        assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG
    assert int(torch.count_nonzero(out[good:good + many])) == 0 and (out[good + many:] == 5).all()
    ref, spread = R.tree_attn(R.f64(q[:good]).reshape(good, n_q, hd), tokens(c, 0, 0, 0), tokens(c, 0, 1, 0),
                              [(1 << (i + 1)) - 1 for i in range(good)], hd ** -0.5)
    within(R.f64(out[:good]).reshape(good, n_q, hd), ref, R.attn_tol(ref, spread))
    assert min(ms) < 10, ms
