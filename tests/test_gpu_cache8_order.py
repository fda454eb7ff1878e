"""Rows that come to a block of the 8-bit cache behind others of it, out of order or not beside them: not stored, with a
status, and everything else as if they had named no slot."""
import numpy as np
import pytest
import torch

from test_gpu_cache8 import T, i32, paged, rand, slots_of  # noqa: F401

pytestmark = pytest.mark.gpu


def refused(slots):
    """The rows whose run (neighbours of one block, in order) has a row of its block among the 32 before its first."""
    out, first = [], 0
    for m, s in enumerate(slots):
        if m == 0 or s < 0 or slots[m - 1] < 0 or slots[m - 1] // 16 != s // 16 or slots[m - 1] >= s:
            first = m
        if s >= 0 and any(o >= 0 and o // 16 == s // 16 for o in slots[max(first - 32, 0):first]):
            out.append(m)
    return out


def check(T, c, slots, seed, expect=None):
    n_q, hd, n_kv = 2 * c.n_kv, c.head_dim, c.n_kv
    no = refused(slots)
    assert expect is None or no == expect
    qkv = rand((len(slots), (n_q + 2 * n_kv) * hd), seed, 3.0)
    pos, rope, ws = i32(list(range(len(slots)))), T.RopeTable(1e4 ** (-np.arange(hd // 2) / (hd // 2))), T.workspace(256)
    raw, scales = c.data.clone(), c.scales.clone()
    q = T.tf_qk_norm_rope_run(qkv, c, 1, pos, i32(slots), rope, ws=ws, n_q=n_q)
    assert T.tf_workspace_status(ws) == (T.TF_E_INVALID_ARG if no else T.TF_OK)
    got = c.data.view(torch.uint8).clone(), c.scales.view(torch.uint8).clone()
    c.data.copy_(raw)
    c.scales.copy_(scales)
    kept = [-1 if m in set(no) else s for m, s in enumerate(slots)]
    want_q = T.tf_qk_norm_rope_run(qkv, c, 1, pos, i32(kept), rope, ws=ws, n_q=n_q)
    assert T.tf_workspace_status(ws) == T.TF_OK
    assert torch.equal(q, want_q) and torch.equal(got[0], c.data.view(torch.uint8)) and torch.equal(got[1], c.scales.view(torch.uint8))


# places in one sequence, and the rows that are not stored
@pytest.mark.parametrize("at,no", [
    ([5, 5], [1]),                                   # the same slot twice
    ([7, 6, 5], [1, 2]),                             # backwards
    ([0, 2, 1, 3], [2, 3]),
    ([3, 20, 4], [2]),                               # another block between
    ([3, -1, 4], [2]),                               # a row of no slot between
    ([14, 15, 16, 17, 2], [4]),
    ([0] + list(range(32, 63)) + [1, 2], [32, 33]),  # 32 rows apart
    (list(range(16, 32)) + list(range(16)) + [31], [32]),
    ([40, 41, 3, 42, 4, 5], [3, 4, 5]),
    (list(range(9, 60)), []),                        # as extend gives them
    ([0, 3, 9, 15, 16, 40], []),                     # gaps are in order
    ([-1, 4, 5, -1, 20, -1], []),
])
@pytest.mark.parametrize("hd,n_kv,page", [(64, 1, 64), (128, 8, 16), (256, 2, 32)])
def test_rows_behind_others_of_their_block(T, at, no, hd, n_kv, page):  # noqa: F811
    c = paged(T, [64, 5], n_kv, hd, page, 3 + len(at))
    own = slots_of(c, 0, 0, 64).tolist()
    check(T, c, [own[i] if i >= 0 else -1 for i in at], 2, no)


@pytest.mark.parametrize("rows", [700, 6000])
def test_among_many_rows(T, rows):  # noqa: F811
    """A prompt's rows with some of them moved or named again, at every place of the 32 rows that a block of threads looks at."""
    c = paged(T, [rows + 40], 4, 128, 64, rows)
    slots = slots_of(c, 0, 9, rows).tolist()
    rng = np.random.default_rng(rows)
    for m in range(40, rows, 61):  # again within 32 rows, so that no two runs of a block are farther apart
        slots[m] = slots[m - int(rng.integers(1, 9))]
    no = refused(slots)
    # every run of a block but its first is among the refused
    seen = {}
    for m, s in enumerate(slots):
        if m not in set(no):
            seen.setdefault(s // 16, []).append(m)
    assert no and all(b - a == 1 for ms in seen.values() for a, b in zip(ms, ms[1:]))
    check(T, c, slots, 4)
