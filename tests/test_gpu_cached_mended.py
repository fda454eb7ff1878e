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


# ---------------------------------------------------------------- norm + rotation

@pytest.mark.parametrize("hd,pairs", [(64, False), (128, False), (128, True), (256, True)])
def test_small_angles_keep_their_digits(T, hd, pairs):
    """Pairs (1, 0) become (cos, sin): each within a rounding of itself, not of the pair's length, so also the sine
    of a slow pair's small angle. The fraction of a turn is within 2^-22 of itself (conversions, a sum, a product),
    the polynomials within 2^-21, and an angle's own error does not grow in the result (x cot x and x tan x are at
    most 1 up to pi / 4): 2^-20. The reference's angle is within 2^-52 of itself, 40 radians at most: where a cosine is
    below 2^-30 that counts, and none of these is."""
    M, n = 40, hd // 2
    inv = 1e6 ** (-np.arange(n) / n)
    first = slice(0, hd, 2) if pairs else slice(0, n)
    second = slice(1, hd, 2) if pairs else slice(n, hd)
    x = torch.zeros((M, 3, hd), device="cuda", dtype=torch.bfloat16)
    x[:, 0, first] = 1
    c = T.KVCache.create(1, 1, hd, 16, 4, 1, 4)
    pos = np.concatenate([np.arange(-20, 0), np.arange(1, 21)])
    q = T.tf_qk_norm_rope_run(x.view(M, -1), c, 0, i32(pos.tolist()), i32([-1] * M), T.RopeTable(inv, pairs=pairs), n_q=1)
    angle = pos[:, None] * inv[None]
    assert (np.abs(angle) < 1e-4).any(0).sum() > n // 8
    for part, ref in ((first, np.cos(angle)), (second, np.sin(angle))):
        assert np.abs(ref).min() > 2.0 ** -30
        within(R.f64(q)[:, part], ref, (2.0 ** -8 + 2.0 ** -20) * np.abs(ref))


# ---------------------------------------------------------------- page operations

@pytest.mark.parametrize("entry", [-1, -7, 99, "n_pages", 2 ** 31 - 1])
@pytest.mark.parametrize("col,parent", [
    (0, [0, 0, 0, 3]),    # a full page of a slot that stays and is taken
    (1, [0, 0, 2, 3]),
    (2, [0, 0, 2, 3]),    # its unfilled page, which is copied
    (2, [-1, 0, 2, 3]),   # its unfilled page, which the taker keeps
    (1, [3, 2, 0, 3]),    # a full page that changes hands
])
def test_a_fork_over_an_entry_that_is_no_page_does_nothing(T, entry, col, parent):
    c = filled_cache(T, [40, 33, 5, 7], 1, 64, 16, 94, spare=4)
    c.table[0, col] = c.n_pages if entry == "n_pages" else entry
    ws = T.workspace(T.tf_kvcache_workspace_bytes(c))
    book, data = c.book.clone(), c.data.clone()
    T.tf_kvcache_fork(c, i32(parent), ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG
    assert torch.equal(c.book, book) and torch.equal(c.data, data)
    # nobody takes it: the others may be forked, and the slot emptied
    T.tf_kvcache_fork(c, i32([0, 1, 1, 3]), ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_OK and c.len.tolist() == [40, 33, 33, 7]
    T.tf_kvcache_fork(c, i32([-1, 1, 2, 3]), ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_OK and c.len.tolist() == [0, 33, 33, 7] and (c.table[0] == -1).all()


def test_a_fork_of_many_slots_finds_the_one_entry_that_is_no_page(T):
    c = filled_cache(T, [16 * (1 + s % 90) + s % 16 for s in range(1024)], 1, 64, 16, 95, layers=1, spare=2000)
    ws = T.workspace(T.tf_kvcache_workspace_bytes(c))
    rng = np.random.default_rng(1)
    parent = i32([s if s == 700 else int(rng.integers(1024)) for s in range(1023)] + [700])
    book = c.book.clone()
    for col in (0, 33, 69, 70):
        c.table[700, col] = c.n_pages + 5
        T.tf_kvcache_fork(c, parent, ws=ws)
        assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG
        c.table[700, col] = book[1024 + c.n_pages + 700 * c.max_pages + col]
        assert torch.equal(c.book, book)
    T.tf_kvcache_fork(c, parent, ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_OK


# ---------------------------------------------------------------- decoder step over a cache

@pytest.mark.parametrize("rows,n_q,n_kv,hd", [([1] * 8, 16, 2, 64), ([1] * 8, 8, 1, 128), ([2, 1, 2, 3], 12, 2, 64), ([4, 0, 4], 5, 1, 64)])
def test_the_step_takes_the_longest_block_for_its_attention(T, rows, n_q, n_kv, hd):
    """Several short blocks: bit for bit the separate calls that name the longest block, not the step's rows."""
    from test_gpu_cached_step import Model
    m = Model(T, seed=31 + n_q, n_layers=2, d_model=256, d_ff=384, n_q=n_q, n_kv=n_kv, hd=hd, vocab=500)
    B, M, most = len(rows), sum(rows), max(rows)
    caches = [m.cache(T, 16, 60, B, 9) for _ in range(2)]
    seqs, start = i32(list(range(B))), i32(np.cumsum([0] + rows).tolist())
    lens = [5 + 13 * b for b in range(B)]
    kv = rand((sum(lens), 2 * n_kv * hd), 3)
    x, got, ws = m.x[:M].contiguous(), [], None
    for i, c in enumerate(caches):
        at, _ = T.tf_kvcache_extend(c, seqs, i32(np.cumsum([0] + lens).tolist()), sum(lens))
        for l in range(2):
            c.data[l, 0, (at // 16).long(), :, (at % 16).long()] = kv[:, :n_kv * hd].view(-1, n_kv, hd)
            c.data[l, 1, (at // 16).long(), :, (at % 16).long()] = kv[:, n_kv * hd:].view(-1, n_kv, hd)
        slots, pos = T.tf_kvcache_extend(c, seqs, start, M)
        if i == 0:
            ws = T.workspace(T.tf_decode_step_attn_workspace_bytes(m.dec, c, m.attn))
            got.append(T.tf_decode_step_attn_run(m.dec, c, m.attn, x, seqs, start, slots, pos, ws=ws, max_rows=most))
            again = T.tf_decode_step_attn_run(m.dec, c, m.attn, x, seqs, start, slots, pos, ws=ws, max_rows=8 if M < 8 else None)
            assert T.tf_workspace_status(ws) == T.TF_OK and again.shape == got[0].shape
            T.tf_decode_step_attn_run(m.dec, c, m.attn, x, seqs, start, slots, pos, ws=ws, max_rows=most)
            # a block longer than that is refused by the attention, and said so
            if most > 1:
                T.tf_decode_step_attn_run(m.dec, c, m.attn, x, seqs, start, slots, pos, ws=ws, max_rows=most - 1)
                assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG
                T.tf_decode_step_attn_run(m.dec, c, m.attn, x, seqs, start, slots, pos, ws=ws, max_rows=most)
            continue
        h, a = x, m.attn
        for l, L in enumerate(m.dec.layers):
            qkv = T.tf_qlinear_run(L["qkv"], h, gamma=L["attn_norm"], eps=m.dec.desc.eps)
            q = T.tf_qk_norm_rope_run(qkv, c, l, pos, slots, m.rope, q_gamma=a.norms[l][0], k_gamma=a.norms[l][1], eps=a.desc.eps)
            o = T.tf_tree_attn_run(q, c, l, seqs, start, max_rows=most)
            h1 = T.tf_qlinear_run(L["o"], o, residual=h)
            h = T.tf_qlinear_run(L["down"], T.tf_qmlp_gateup_run(L["gate"], L["up"], h1, gamma=L["mlp_norm"], eps=m.dec.desc.eps),
                                 residual=h1)
        got.append(T.tf_qlinear_run(m.dec.readout, h, gamma=m.dec.final_norm, eps=m.dec.desc.eps))
    assert torch.equal(got[0], got[1]) and bool(torch.isfinite(got[0]).all())
    assert torch.equal(caches[0].data, caches[1].data)


# ---------------------------------------------------------------- log probabilities

def test_targets_of_no_dimension_are_refused(T):
    v = rand((1, 100), 1)
    for bad in (torch.tensor(3, dtype=torch.int32, device="cuda"), i32([1, 2]), i32([[[1]]])):
        with pytest.raises(ValueError):
            T.tf_logprobs_rows(v, bad)
