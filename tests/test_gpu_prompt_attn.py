"""Causal attention of whole prompts over the paged cache, bf16 and 8 bits, against a 64-bit reference."""
import numpy as np
import pytest
import torch

import cache8_ref as Q
import cached_ref as R
from test_gpu_cache8 import E4M3, i32, paged, rand, slots_of, tokens, within

pytestmark = pytest.mark.gpu
BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])


@pytest.fixture(scope="module")
def T():
    from skinny_gemm_bit_gb300 import build
    build.build()
    from skinny_gemm_bit_gb300 import tfq
    return tfq


def held(c):
    return Q.values(c) if c.data.dtype == E4M3 else R.f64(c.data)


def run(T, c, layer, seqs, rows, n_q, seed, scale=None, lead=0):
    """(q, o, q_start) of one call; rows before and behind the sequences' stay as they were."""
    start = np.cumsum([lead] + rows)
    M = int(start[-1]) + 3
    q = rand((M, n_q * c.head_dim), seed, 2.0)
    out = torch.full((M, n_q * c.head_dim), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = T.workspace(T.tf_prompt_attn_workspace_bytes(c, n_q, len(seqs)))
    for _ in range(2):  # the second call finds the workspace as the first left it
        T.tf_prompt_attn_run(q, c, layer, i32(seqs), i32(start.tolist()), scale=scale, out=out, ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_OK
    assert (out[:lead] == 5).all() and (out[int(start[-1]):] == 5).all()
    return q, out, start


def check(T, c, layer, seqs, rows, n_q, seed, scale=None, lead=0, which=None):
    q, out, start = run(T, c, layer, seqs, rows, n_q, seed, scale, lead)
    hd, vals = c.head_dim, held(c)
    for b in range(len(seqs)) if which is None else which:
        n = int(c.len[seqs[b]])
        base = n - rows[b]
        picked = np.arange(rows[b])
        if rows[b] > 200:  # the reference is slow: some rows at tiles' borders and anywhere
            rng = np.random.default_rng(b)
            picked = np.unique(np.concatenate([[0, 1, 63, 64, 127, 128, rows[b] - 1], rng.integers(0, rows[b], 60)]))
        qq = R.f64(q[start[b]:start[b + 1]]).reshape(rows[b], n_q, hd)[picked]
        see = np.arange(n)[None, :] <= base + picked[:, None]
        k, v = tokens(c, vals, layer, 0, seqs[b]), tokens(c, vals, layer, 1, seqs[b])
        ref, spread, size = Q.attn(qq, k, v, see, hd ** -0.5 if scale is None else scale, Q.scales_of(c, layer, seqs[b]))
        got = R.f64(out[start[b]:start[b + 1]]).reshape(rows[b], n_q, hd)[picked]
        within(got, ref, Q.attn_tol(ref, spread, size, c.data.dtype == E4M3))


@BOTH
@pytest.mark.parametrize("seqs,n_q,n_kv,hd,page", [
    ([(0, 1)], 1, 1, 128, 16),                         # one token
    ([(0, 2)], 16, 8, 128, 16),
    ([(0, 64), (0, 65)], 4, 4, 64, 16),
    ([(0, 333)], 16, 8, 128, 16),
    ([(700, 1), (63, 1), (64, 1)], 16, 2, 128, 64),    # single tokens behind contexts
    ([(0, 129), (5, 1), (200, 0), (17, 300), (0, 256)], 6, 2, 128, 32),  # a sequence without rows
    ([(1000, 257)], 8, 1, 64, 64),
    ([(31, 500), (0, 70)], 64, 1, 128, 128),           # 64 query heads to one key/value head
    ([(129, 140)], 5, 1, 128, 16),                     # a group that does not divide a tile's rows
    ([(0, 1025)], 3, 3, 128, 64),
])
def test_prompts(T, dtype, seqs, n_q, n_kv, hd, page):
    rng = np.random.default_rng(len(seqs))
    c = paged(T, [a + r for a, r in seqs], n_kv, hd, page, 11 + sum(r for _, r in seqs), dtype=dtype)
    order = rng.permutation(len(seqs)).tolist()
    check(T, c, 1, order, [seqs[s][1] for s in order], n_q, 21)
    check(T, c, 0, order, [seqs[s][1] for s in order], n_q, 22, scale=-0.05, lead=2)


@BOTH
def test_long_prompts(T, dtype):
    c = paged(T, [5000, 12000, 3], 2, 128, 64, 5, dtype=dtype)
    check(T, c, 1, [0, 1, 2], [5000, 777, 3], 4, 5)


@BOTH
def test_many_prompts(T, dtype):
    rng = np.random.default_rng(3)
    lens = rng.integers(1, 120, 300).tolist()
    rows = [int(rng.integers(0, n + 1)) for n in lens]
    c = paged(T, lens, 1, 64, 16, 9, dtype=dtype)
    check(T, c, 0, list(range(300)), rows, 2, 6, which=rng.permutation(300)[:60].tolist())


@BOTH
def test_the_most_prompts(T, dtype):
    lens = [1 + 7 * i % 90 for i in range(40)]
    c = paged(T, lens, 1, 128, 16, 101, dtype=dtype)
    rng = np.random.default_rng(1)
    seqs = rng.integers(0, 40, 1024).tolist()
    rr = [int(rng.integers(0, lens[s] + 1)) for s in seqs]
    check(T, c, 1, seqs, rr, 4, 6, which=rng.permutation(1024)[:40].tolist() + [0, 1023])


@BOTH
@pytest.mark.parametrize("rows,n_q", [(9, 4), (64, 16), (40, 2)])
def test_a_prompt_is_a_chain_of_drafts(T, dtype, rows, n_q):
    """Up to 64 rows the two attentions answer the same question."""
    c = paged(T, [500], 2, 128, 16, 17, dtype=dtype)
    q, out, _ = run(T, c, 0, [0], [rows], n_q, 2)
    other = T.tf_tree_attn_run(q[:rows], c, 0, i32([0]), i32([0, rows]), max_rows=rows)
    assert float((out[:rows].double() - other.double()).norm() / other.double().norm()) < 2.0 ** -7


@BOTH
@pytest.mark.parametrize("rows,n_q,hd", [(300, 4, 128), (520, 2, 64), (300, 16, 64), (100, 10, 128)])
def test_tokens_that_a_row_does_not_see_take_no_part(T, dtype, rows, n_q, hd):
    n = 90 + rows
    c = paged(T, [n], 2, hd, 16, 41, dtype=dtype)
    clean = run(T, c, 1, [0], [rows], n_q, 9)[1]
    for t in (90, 90 + rows // 3, 90 + rows // 2 + 1, n - 2):
        raw = c.data.clone()
        page, off = int(c.table[0, t // 16]), t % 16
        if dtype == E4M3:
            c.data.view(torch.uint8)[1, 1, page, 0, off, 3:] = 0x7F
            c.data.view(torch.uint8)[1, :, c.refs == 0] = 0xFF
            c.scales.view(torch.uint8)[1, :, c.refs == 0] = 255
        else:
            c.data[1, 1, page, 0, off, 3:] = float("inf")
            c.data[1, :, c.refs == 0] = float("nan")
        last = int(c.table[0, (n - 1) // 16])
        if n % 16:
            c.data.view(torch.uint8)[1, :, last, :, n % 16:] = 0x7F if dtype == E4M3 else 0xFF
        dirty = run(T, c, 1, [0], [rows], n_q, 9)[1]
        c.data.copy_(raw)
        i = t - 90
        a, b = clean[:rows].view(rows, 2, n_q // 2, hd), dirty[:rows].view(rows, 2, n_q // 2, hd)
        assert torch.equal(a[:i], b[:i]) and torch.equal(a[:, 1], b[:, 1]) and torch.equal(a[..., :3], b[..., :3])
        assert not torch.isfinite(b[i:, 0, :, 3:]).any()


@BOTH
def test_prompts_that_do_not_hold(T, dtype):
    c = paged(T, [40, 5], 2, 128, 16, 51, dtype=dtype)
    q = rand((200, 512), 1)
    for seqs, start, zero, same in [([2], [0, 3], range(0, 3), range(3, 8)), ([-1], [0, 3], range(0, 3), range(3, 8)),
                                    ([1], [0, 6], range(0, 6), range(6, 8)), ([0], [5, 3], [], range(8)), ([0], [2, 201], [], range(8))]:
        ws = T.workspace(T.tf_prompt_attn_workspace_bytes(c, 4, 1))
        out = torch.full((200, 512), 5.0, dtype=torch.bfloat16, device="cuda")
        T.tf_prompt_attn_run(q, c, 0, i32(seqs), i32(start), out=out, ws=ws)
        assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG, (seqs, start)
        assert (out[list(zero)] == 0).all() and (out[list(same)] == 5).all(), (seqs, start)
    # one that does not hold beside one that does
    ws = T.workspace(T.tf_prompt_attn_workspace_bytes(c, 4, 2))
    out = torch.full((200, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    T.tf_prompt_attn_run(q, c, 0, i32([1, 0]), i32([0, 100, 140]), out=out, ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG
    good = T.tf_prompt_attn_run(q[100:140], c, 0, i32([0]), i32([0, 40]))
    assert (out[:100] == 0).all() and torch.equal(out[100:140], good) and (out[140:] == 5).all()
    c.table[0, 1] = 99  # a page out of range counts as zeros
    vals = held(c)
    k, v = np.zeros((40, 2, 128)), np.zeros((40, 2, 128))
    for r in [*range(16), *range(32, 40)]:
        p = int(c.table[0, r // 16])
        k[r], v[r] = vals[0, 0, p, :, r % 16], vals[0, 1, p, :, r % 16]
    ws = T.workspace(T.tf_prompt_attn_workspace_bytes(c, 4, 1))
    out = T.tf_prompt_attn_run(q[:40], c, 0, i32([0]), i32([0, 40]), ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG
    ref, spread, size = Q.attn(R.f64(q[:40]).reshape(40, 4, 128), k, v, np.tril(np.ones((40, 40), bool)), 128 ** -0.5,
                                  np.full((40, 2), 2.0 ** Q.exponents(c)[0, 1].max()) if dtype == E4M3 else None)
    within(R.f64(out).reshape(40, 4, 128), ref, Q.attn_tol(ref, spread, size, dtype == E4M3))


@BOTH
def test_the_same_bits_in_a_graph_on_streams_and_from_strided_rows(T, dtype):
    c = paged(T, [1500, 70, 901], 2, 128, 16, 71, dtype=dtype)
    wide = rand((900, 4 * 128 + 40), 3, 2.0)
    q, seqs, start = wide[:, 16:16 + 512], i32([0, 1, 2]), i32([0, 600, 660, 900])
    want = T.tf_prompt_attn_run(q.contiguous(), c, 1, seqs, start)
    assert torch.equal(want, T.tf_prompt_attn_run(q, c, 1, seqs, start))
    need = T.tf_prompt_attn_workspace_bytes(c, 4, 3)
    streams, wss = [torch.cuda.Stream() for _ in range(2)], [T.workspace(need) for _ in range(2)]
    outs = [[torch.empty_like(want) for _ in range(6)] for _ in range(2)]
    torch.cuda.synchronize()
    for n in range(6):
        for i in (0, 1):
            T.tf_prompt_attn_run(q, c, 1, seqs, start, out=outs[i][n], ws=wss[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for x in outs for o in x)
    ws, out, g = wss[0], torch.empty_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        T.tf_prompt_attn_run(q, c, 1, seqs, start, out=out, ws=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    c.len[0] = 640  # the captured call reads lengths anew
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, T.tf_prompt_attn_run(q, c, 1, seqs, start))


def test_a_wait_that_runs_out_is_not_left_behind(T):
    """The workspace's counters are zero after calls of every size, whichever CTAs split which items."""
    c = paged(T, [4000, 10], 1, 64, 16, 8)
    for rows, n_q in [(1, 1), (300, 1), (4000, 2), (2000, 8), (65, 64)]:
        ws = T.workspace(T.tf_prompt_attn_workspace_bytes(c, n_q, 1))
        q = rand((rows, n_q * 64), 2)
        for _ in range(3):
            T.tf_prompt_attn_run(q, c, 0, i32([0]), i32([0, rows]), ws=ws)
        assert T.tf_workspace_status(ws) == T.TF_OK
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert int(torch.count_nonzero(ws[:256 + (sms * 8 + 255) // 256 * 256])) == 0


@BOTH
def test_a_prompt_served_from_its_first_token_to_its_drafts(T, dtype):
    """Prompt in chunks -> store -> prompt attention -> tokens and drafts -> keep, on one cache, each answer against the
    attention of the values that the cache then holds."""
    n_q, n_kv, hd = 8, 2, 128
    c = T.KVCache.create(1, n_kv, hd, 32, 40, 2, 16, dtype=dtype)
    rope, at = T.RopeTable(1e4 ** (-np.arange(64) / 64)), 0
    wsc = T.workspace(T.tf_kvcache_workspace_bytes(c))
    said = [[], []]

    def step(seqs, rows, prompt):
        nonlocal at
        start, M = i32(np.cumsum([0] + rows).tolist()), sum(rows)
        slots, pos = T.tf_kvcache_extend(c, i32(seqs), start, M, ws=wsc)
        qkv = rand((M, (n_q + 2 * n_kv) * hd), 100 + at)
        at += 1
        q = T.tf_qk_norm_rope_run(qkv, c, 0, pos, slots, rope, n_q=n_q)
        o = T.tf_prompt_attn_run(q, c, 0, i32(seqs), start) if prompt else T.tf_tree_attn_run(q, c, 0, i32(seqs), start, max_rows=max(rows))
        assert T.tf_workspace_status(wsc) == T.TF_OK
        vals, a = held(c), 0
        for s, r in zip(seqs, rows):
            n = int(c.len[s])
            see = np.arange(n)[None, :] <= n - r + np.arange(r)[:, None]
            ref, spread, size = Q.attn(R.f64(q[a:a + r]).reshape(r, n_q, hd), tokens(c, vals, 0, 0, s), tokens(c, vals, 0, 1, s), see, hd ** -0.5, Q.scales_of(c, 0, s))
            within(R.f64(o[a:a + r]).reshape(r, n_q, hd), ref, Q.attn_tol(ref, spread, size, dtype == E4M3))
            a += r

    step([0, 1], [150, 37], True)
    step([1, 0], [64, 101], True)
    for _ in range(3):
        step([0, 1], [1, 1], False)
    step([0, 1], [8, 5], False)
    T.tf_kvcache_keep(c, i32([0, 1]), i32([0, 8, 13]), i32([0, 1, 4, 6, 0, 0, 0, 0, 2, 4, 0, 0, 0]), i32([4, 2]), ws=wsc)
    step([0, 1], [1, 1], False)
    step([0], [90], True)
    assert c.len.tolist() == [150 + 101 + 3 + 4 + 1 + 90, 37 + 64 + 3 + 2 + 1]


def test_refusals(T):
    c = paged(T, [40], 2, 128, 16, 51)
    big = paged(T, [40], 1, 256, 16, 51)
    q = rand((4, 512), 1)
    with pytest.raises(T.TfqError):
        T.tf_prompt_attn_run(q, big, 0, i32([0]), i32([0, 4]))
    with pytest.raises(T.TfqError):
        T.tf_prompt_attn_run(rand((4, 384), 1), c, 0, i32([0]), i32([0, 4]))  # three heads over two
    for kw in (dict(layer=2), dict(scale=float("nan")), dict(out=q)):
        with pytest.raises(T.TfqError):
            T.tf_prompt_attn_run(q, c, kw.pop("layer", 0), i32([0]), i32([0, 4]), **kw)
    for bad in (q.float(), q.cpu(), q[:, :100], q.t()):
        with pytest.raises(ValueError):
            T.tf_prompt_attn_run(bad, c, 0, i32([0]), i32([0, 4]))
    with pytest.raises(ValueError):
        T.tf_prompt_attn_run(q, c, 0, i32([0]), i32([0]))
    with pytest.raises(T.TfqError):
        T.tf_prompt_attn_run(q, c, 0, i32([0]), i32([0, 4]), ws=T.workspace(256))
    assert T.tf_prompt_attn_workspace_bytes(big, 1, 1) == 0 and T.tf_prompt_attn_workspace_bytes(c, 4, 1025) == 0
