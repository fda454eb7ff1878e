"""Attention over the 8-bit cache and of prompts: a wait that runs out in each form of the kernels, the borders of their row
tiles, and outputs on a 16-byte boundary."""
import numpy as np
import pytest
import torch

import cache8_ref as Q
import cached_ref as R
from test_gpu_cache8 import E4M3, T, i32, paged, rand, tokens, within  # noqa: F401
from test_gpu_prompt_attn import held, run

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def counters(ws):
    """What an attention's CTAs (or groups) count in, behind the status word's 256 bytes: two words each, two of them an SM."""
    return ws[256:256 + 16 * torch.cuda.get_device_properties(0).multi_processor_count]


# trees over 8 bits: 2 and 32 query rows to a key/value head (warp MMAs: two CTAs an SM, one), 64 and 512 (tcgen05, both
# groups with the same rows and with their own), head dim 256; prompts of both kinds, a group's rows apart and a pair's
@pytest.mark.parametrize("prompt,dtype,rows,n_q,hd", [
    (False, E4M3, 1, 4, 128), (False, E4M3, 8, 8, 128), (False, E4M3, 64, 2, 64), (False, E4M3, 64, 16, 128), (False, E4M3, 3, 4, 256),
    (True, BF16, 300, 4, 128), (True, BF16, 90, 16, 64), (True, E4M3, 300, 4, 128), (True, E4M3, 90, 16, 64), (True, BF16, 50, 10, 128),
])
def test_a_wait_that_runs_out_is_reported(T, prompt, dtype, rows, n_q, hd):  # noqa: F811
    """Counters that start one below zero: whoever has a part of a split item writes it and waits, within the limit, for one
    more than there are. The call ends with its status; the workspace zeroed, it is as good as new."""
    c = paged(T, [30000], 2, hd, 64, 9, layers=1, dtype=dtype)
    q, seqs, start = rand((rows, n_q * hd), 5, 2.0), i32([0]), i32([0, rows])
    need = T.tf_prompt_attn_workspace_bytes(c, n_q, 1) if prompt else T.tf_tree_attn_workspace_bytes(c, n_q, 1, rows)
    ws, out = T.workspace(need), torch.empty_like(q)

    def call(**kw):
        return T.tf_prompt_attn_run(q, c, 0, seqs, start, **kw) if prompt else T.tf_tree_attn_run(q, c, 0, seqs, start, max_rows=rows, **kw)

    want = call()
    counters(ws).fill_(255)
    call(out=out, ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_E_TIMEOUT
    ws.zero_()
    call(out=out, ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_OK and torch.equal(out, want)
    assert int(torch.count_nonzero(counters(ws))) == 0


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("rows,context,n_q,n_kv,hd", [(700, 0, 2, 2, 128), (700, 90, 4, 2, 64), (600, 1, 3, 1, 128), (330, 500, 16, 2, 128),
                                                     (70, 3, 63, 1, 64)])
def test_borders_of_row_tiles(T, dtype, rows, context, n_q, n_kv, hd):  # noqa: F811
    """The rows beside each border of 128 and of 256 query rows, whose tiles end with different key tiles."""
    c = paged(T, [context + rows], n_kv, hd, 16, rows, dtype=dtype)
    q, out, _ = run(T, c, 1, [0], [rows], n_q, 3)
    group = n_q // n_kv
    picked = np.unique([min(max(k // group + d, 0), rows - 1) for k in range(0, rows * group + 128, 128) for d in (-1, 0, 1)])
    vals = held(c)
    see = np.arange(context + rows)[None, :] <= context + picked[:, None]
    ref, spread, more = Q.attn(R.f64(q[:rows]).reshape(rows, n_q, hd)[picked], tokens(c, vals, 1, 0, 0), tokens(c, vals, 1, 1, 0), see, hd ** -0.5,
                               Q.scales_of(c, 1, 0))
    within(R.f64(out[:rows]).reshape(rows, n_q, hd)[picked], ref, Q.attn_tol(ref, spread, more, dtype == E4M3))


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("prompt,rows,n_q,hd", [(True, 300, 8, 128), (True, 70, 16, 64), (False, 16, 16, 128), (False, 64, 16, 64), (False, 2, 4, 128)])
def test_outputs_on_a_16_byte_boundary(T, dtype, prompt, rows, n_q, hd):  # noqa: F811
    c = paged(T, [900, 333], 2, hd, 32, 7, dtype=dtype)
    q, seqs, start = rand((2 * rows, n_q * hd), 5, 2.0), i32([1, 0]), i32([0, rows, 2 * rows])

    def call(**kw):
        return T.tf_prompt_attn_run(q, c, 1, seqs, start, **kw) if prompt else T.tf_tree_attn_run(q, c, 1, seqs, start, max_rows=rows, **kw)

    want = call()
    wide = torch.full((want.numel() + 16,), 5.0, dtype=BF16, device="cuda")
    at = next(i for i in range(0, 16, 8) if (wide.data_ptr() + 2 * i) % 32 == 16)
    out = wide[at:at + want.numel()].view(want.shape)
    call(out=out)
    assert torch.equal(out, want) and (wide[:at] == 5).all() and (wide[at + want.numel():] == 5).all()
