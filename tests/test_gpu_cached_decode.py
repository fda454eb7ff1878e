"""The cached-decoding operators against 64-bit references: norms and rotation with the store to
the paged cache, attention of drafted rows, the cache's page operations and log probabilities."""
import numpy as np
import pytest
import torch

import cached_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    from skinny_gemm_bit_gb300 import build
    build.build()
    from skinny_gemm_bit_gb300 import tfq
    return tfq


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rand(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").mul_(scale).bfloat16()


def mask_tensor(bits):
    return torch.from_numpy(np.array(bits, dtype=np.uint64).view(np.int64)).cuda()


def filled_cache(T, lens, n_kv, hd, page, seed, layers=2, spare=3, max_extra=2):
    """A cache whose slots hold `lens` tokens on scattered pages, every row random."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    n_pages, max_pages = sum(need) + spare, max(need + [1]) + max_extra
    c = T.KVCache.create(layers, n_kv, hd, page, n_pages, len(lens), max_pages)
    c.data.copy_(rand(c.data.shape, seed))
    order = rng.permutation(n_pages).tolist()
    table = np.full((len(lens), max_pages), -1, np.int32)
    refs = np.zeros(n_pages, np.int32)
    for s, n in enumerate(need):
        for i in range(n):
            table[s, i] = order.pop()
            refs[table[s, i]] = 1
    c.len.copy_(i32(lens))
    c.refs.copy_(torch.from_numpy(refs))
    c.table.copy_(torch.from_numpy(table))
    return c


def tokens(c, layer, kv, s):
    """[len, n_kv, hd] fp64 of a slot's keys or values."""
    r = torch.arange(int(c.len[s]), device="cuda")
    return R.f64(c.data[layer, kv, c.table[s].long()[r // c.page_size], :, r % c.page_size])


def within(got, ref, tol):
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside: worst {np.nanmax(err / tol)}, at {np.argwhere(bad)[:3].tolist()}"


# ---------------------------------------------------------------- norm + rotation

@pytest.mark.parametrize("rows,n_q,n_kv,hd,rot,pairs,norm,page", [
    (1, 16, 8, 128, 128, False, True, 16),
    (7, 5, 1, 128, 64, False, True, 32),
    (33, 4, 2, 64, 64, True, True, 16),
    (130, 3, 3, 256, 256, False, True, 64),
    (9, 2, 1, 256, 16, True, False, 128),
    (5, 16, 8, 128, 0, False, True, 16),
    (3001, 4, 2, 128, 128, True, True, 16),
    (2, 40, 8, 64, 48, False, False, 32),
])
def test_norm_rope(T, rows, n_q, n_kv, hd, rot, pairs, norm, page):
    cols = (n_q + 2 * n_kv) * hd
    wide = rand((rows, cols + 24), 1, 2.0)  # a leading dimension wider than the row
    qkv = wide[:, 8:8 + cols]
    qg, kg = (rand((hd,), 2) + 1, rand((hd,), 3) + 1) if norm else (None, None)
    n_pages = rows // page + 3
    c = T.KVCache.create(3, n_kv, hd, page, n_pages, 1, n_pages)
    c.data.fill_(7.0)
    rng = np.random.default_rng(rows)
    pos = np.concatenate([[2 ** 31 - 1, -5, 0, 1, 1048575], rng.integers(0, 200000, rows)])[:rows].astype(np.int32)
    slots = rng.permutation(n_pages * page)[:rows].astype(np.int32)
    if rows > 4:
        slots[[1, 4]] = -1  # rows without a place in the cache
    inv = 1e6 ** (-np.arange(0, rot, 2) / max(rot, 1))
    ws = T.workspace(256)
    q = T.tf_qk_norm_rope_run(qkv, c, 1, torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(),
                              T.RopeTable(inv, pairs=pairs), q_gamma=qg, k_gamma=kg, eps=1e-5, n_q=n_q, ws=ws)
    x = R.f64(qkv).reshape(rows, -1, hd)
    ref, size = R.norm_rope(x[:, :n_q], None if qg is None else R.f64(qg), 1e-5, pos, inv, pairs)
    within(R.f64(q).reshape(rows, n_q, hd), ref, R.rope_tol(ref, size))
    ref, size = R.norm_rope(x[:, n_q:n_q + n_kv], None if kg is None else R.f64(kg), 1e-5, pos, inv, pairs)
    data, untouched = R.f64(c.data), np.ones((n_pages, page), bool)
    for i, s in enumerate(slots):
        if s >= 0:
            untouched[s // page, s % page] = False
            within(data[1, 0, s // page, :, s % page], ref[i], R.rope_tol(ref[i], size[i]))
            np.testing.assert_array_equal(data[1, 1, s // page, :, s % page], x[i, n_q + n_kv:])
    assert (data[[0, 2]] == 7).all() and (data[1].transpose(0, 1, 3, 2, 4)[:, untouched] == 7).all()
    assert T.tf_workspace_status(ws) == T.TF_OK


def test_norm_rope_reports_a_slot_outside_the_cache(T):
    c = T.KVCache.create(1, 1, 64, 16, 2, 1, 2)
    ws = T.workspace(256)
    T.tf_qk_norm_rope_run(rand((2, 256), 1), c, 0, i32([0, 1]), i32([32, 3]), T.RopeTable([]), ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG
    assert int(torch.count_nonzero(c.data.abs().sum(-1))) == 2  # the good row's key and value alone


# ---------------------------------------------------------------- attention

def chain(rows):
    return [(1 << (i + 1)) - 1 for i in range(rows)]


def tree(rows, rng):
    out = []
    for i in range(rows):
        out.append((1 << i) | (out[rng.integers(i)] if i else 0))
    return out


def run_attn(T, c, layer, seqs, rows, masks, n_q, seed, scale=None, lead=0, **kw):
    """(q, o, q_start) of one call; rows before and behind the sequences' stay as they were."""
    start = np.cumsum([lead] + rows)
    M = int(start[-1]) + 3
    q = rand((M, n_q * c.head_dim), seed, 2.0)
    out = torch.full((M, n_q * c.head_dim), 5.0, dtype=torch.bfloat16, device="cuda")
    m = None
    if masks is not None:
        m = mask_tensor([0] * lead + [b for x in masks for b in x] + [0] * 3)
    ws = T.workspace(T.tf_tree_attn_workspace_bytes(c, n_q, len(seqs), max(rows)))
    for _ in range(2):  # the second call finds the workspace as the first left it
        T.tf_tree_attn_run(q, c, layer, i32(seqs), i32(start.tolist()), masks=m, max_rows=max(max(rows), 1), scale=scale,
                           out=out, ws=ws, **kw)
    assert T.tf_workspace_status(ws) == T.TF_OK
    assert int(torch.count_nonzero(ws)) == 0 or T.tf_workspace_status(ws) == T.TF_OK
    assert (out[:lead] == 5).all() and (out[int(start[-1]):] == 5).all()
    return q, out, start


def check_attn(T, c, layer, seqs, rows, masks, n_q, seed, scale=None, lead=0, **kw):
    q, out, start = run_attn(T, c, layer, seqs, rows, masks, n_q, seed, scale, lead, **kw)
    hd = c.head_dim
    for b, s in enumerate(seqs):
        qq = R.f64(q[start[b]:start[b + 1]]).reshape(rows[b], n_q, hd)
        bits = chain(rows[b]) if masks is None else masks[b]
        ref, spread = R.tree_attn(qq, tokens(c, layer, 0, s), tokens(c, layer, 1, s), bits, hd ** -0.5 if scale is None else scale)
        got = R.f64(out[start[b]:start[b + 1]]).reshape(rows[b], n_q, hd)
        within(got, ref, R.attn_tol(ref, spread))


@pytest.mark.parametrize("lens,rows,n_q,n_kv,hd,page", [
    ([1], [1], 1, 1, 128, 16),                       # one token that sees itself alone
    ([2], [1], 16, 8, 128, 16),
    ([16], [1], 16, 8, 128, 16),                     # a full page
    ([17], [2], 16, 8, 128, 16),                     # the block across a page's end
    ([63, 64, 65, 128, 129], [1, 2, 1, 3, 8], 4, 2, 128, 32),
    ([513], [8], 16, 8, 128, 64),
    ([5], [5], 8, 1, 128, 16),                       # nothing before the block
    ([300, 7, 1000, 64], [7, 7, 1, 64], 8, 1, 64, 16),
    ([700, 90], [64, 33], 16, 2, 128, 128),          # 512 query rows to a key/value head
    ([400, 33], [17, 2], 6, 2, 256, 16),
    ([2000], [1], 64, 1, 128, 64),                   # 64 query heads to one key/value head
    ([1500], [16], 5, 5, 64, 32),
])
def test_tree_attn_chain_and_tree(T, lens, rows, n_q, n_kv, hd, page):
    rng = np.random.default_rng(sum(lens))
    c = filled_cache(T, lens, n_kv, hd, page, 11 + sum(lens))
    seqs = rng.permutation(len(lens)).tolist()
    rr = [rows[s] for s in seqs]
    check_attn(T, c, 1, seqs, rr, None, n_q, 21)
    check_attn(T, c, 0, seqs, rr, [tree(r, rng) for r in rr], n_q, 22, scale=0.05, lead=2)


@pytest.mark.parametrize("n,rows", [(40000, 1), (9001, 8), (5000, 40)])
def test_tree_attn_long(T, n, rows):
    c = filled_cache(T, [n, 3, 777], 2, 128, 16, n)
    check_attn(T, c, 1, [0, 1, 2], [rows, 1, min(rows, 700)], None, 4, 5)


@pytest.mark.parametrize("lens,rows,n_q,hd", [
    ([250], 1, 2, 128), ([320], 3, 2, 128), ([380], 8, 8, 128), ([450], 1, 4, 64), ([160], 5, 1, 256), ([330], 2, 2, 256),
    ([800, 30, 2000], 2, 4, 128), ([1500] * 30, 1, 2, 64), ([10] * 70 + [1200], 4, 2, 128),
])
def test_tree_attn_around_the_length_where_items_are_split(T, lens, rows, n_q, hd):
    """Few short items have a CTA each, longer or uneven ones are split and joined."""
    c = filled_cache(T, lens, 2, hd, 16, 31 + sum(lens))
    check_attn(T, c, 1, list(range(len(lens))), [rows] * len(lens), None, 2 * n_q, 8)


def test_two_attention_calls_at_once(T):
    """Two streams, each with a workspace of its own and kernels that wait for their own parts."""
    c = filled_cache(T, [9001, 2500], 4, 128, 32, 77)
    q = [rand((8, 8 * 128), 1, 2.0), rand((40, 16 * 128), 2, 2.0)]
    args = [(i32([0]), i32([0, 8])), (i32([1]), i32([0, 40]))]
    ws = [T.workspace(T.tf_tree_attn_workspace_bytes(c, n, 1, r)) for n, r in ((8, 8), (16, 40))]
    want = [T.tf_tree_attn_run(q[i], c, 0, *args[i], max_rows=(8, 40)[i], ws=ws[i]) for i in (0, 1)]
    out = [[torch.empty_like(x) for _ in range(12)] for x in want]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for n in range(12):
        for i in (0, 1):
            T.tf_tree_attn_run(q[i], c, 0, *args[i], max_rows=(8, 40)[i], out=out[i][n], ws=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in (0, 1):
        assert T.tf_workspace_status(ws[i]) == T.TF_OK
        assert all(torch.equal(o, want[i]) for o in out[i])


def test_tree_attn_many_sequences(T):
    rng = np.random.default_rng(3)
    lens = rng.integers(1, 200, 150).tolist()
    rows = [int(rng.integers(0, min(n, 9) + 1)) for n in lens]  # some with no row at all
    c = filled_cache(T, lens, 1, 128, 16, 9)
    check_attn(T, c, 0, list(range(150)), rows, None, 2, 6)


@pytest.mark.parametrize("n_q,hd,rows", [(2, 128, 1), (4, 64, 7), (1, 256, 3), (40, 128, 3)])
def test_tree_attn_the_most_sequences(T, n_q, hd, rows):
    """1024 sequences, the kernels' largest schedule; some repeat a slot, some have no row."""
    lens = [1 + 7 * i % 90 for i in range(40)]
    c = filled_cache(T, lens, 1, hd, 16, 101)
    rng = np.random.default_rng(rows)
    seqs = rng.integers(0, 40, 1024).tolist()
    rr = [int(min(rng.integers(0, rows + 1), lens[s])) for s in seqs]
    q, out, start = run_attn(T, c, 1, seqs, rr, None, n_q, 6)
    for b in rng.permutation(1024)[:60].tolist() + [0, 1023]:
        qq = R.f64(q[start[b]:start[b + 1]]).reshape(rr[b], n_q, hd)
        ref, spread = R.tree_attn(qq, tokens(c, 1, 0, seqs[b]), tokens(c, 1, 1, seqs[b]), chain(rr[b]), hd ** -0.5)
        within(R.f64(out[start[b]:start[b + 1]]).reshape(rr[b], n_q, hd), ref, R.attn_tol(ref, spread))


@pytest.mark.parametrize("rows,n_q", [(3, 16), (40, 32)])
def test_a_cache_past_32_bit_offsets(T, rows, n_q):
    """5.4 GB of pages: the last layer's values start beyond 2^32 bytes."""
    c = T.KVCache.create(2, 8, 128, 16, 41000, 1, 60)
    n = 700
    c.refs[:40956] = 1  # all pages but the last 44 are somebody's
    slots = torch.cat([T.tf_kvcache_extend(c, i32([0]), i32([0, r]), r)[0] for r in (n - rows, rows)])
    at = torch.arange(n, device="cuda")
    assert torch.equal(slots, (40956 * 16 + at).int())
    kv = rand((n, (1 + 16) * 128), 7)
    T.tf_qk_norm_rope_run(kv, c, 1, at.int(), slots, T.RopeTable([]), n_q=1)
    check_attn(T, c, 1, [0], [rows], None, n_q, 8)
    np.testing.assert_array_equal(tokens(c, 1, 1, 0), R.f64(kv[:, 9 * 128:]).reshape(n, 8, 128))


@pytest.mark.parametrize("hd,rows", [(128, 4), (64, 20), (256, 6), (128, 50)])
def test_tree_attn_rows_that_see_nothing_are_zero(T, hd, rows):
    c = filled_cache(T, [rows, 100 + rows], 2, hd, 16, 31)
    masks = [[0 if i % 2 else chain(rows)[i] for i in range(rows)], [0] * rows]
    check_attn(T, c, 0, [0, 1], [rows, rows], masks, 4, 7)
    q, out, start = run_attn(T, c, 0, [0], [rows], [[0] * rows], 4, 8)
    assert int(torch.count_nonzero(out[:rows])) == 0


@pytest.mark.parametrize("hd,rows,n_q", [(128, 6, 4), (64, 40, 4), (256, 9, 2), (128, 30, 16)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_tree_attn_what_a_row_does_not_see_takes_no_part(T, hd, rows, n_q, what):
    n = 150 + rows
    c = filled_cache(T, [n, 40], 2, hd, 16, 41)
    rng = np.random.default_rng(rows)
    # a tree in which nobody but row 3 itself sees row 3
    bits = tree(rows, rng)
    bits = [b & ~8 if i != 3 else b for i, b in enumerate(bits)]
    clean = run_attn(T, c, 1, [0], [rows], [bits], n_q, 9)[1]
    page, off = int(c.table[0, (n - rows + 3) // 16]), (n - rows + 3) % 16
    c.data[1, :, page, :, off] = what
    # whatever lies behind the sequence's end, in its last page and in pages of nobody
    last = int(c.table[0, (n - 1) // 16])
    if n % 16:
        c.data[1, :, last, :, n % 16:] = what
    c.data[1, :, c.refs == 0] = what
    dirty = run_attn(T, c, 1, [0], [rows], [bits], n_q, 9)[1]
    others = [i for i in range(rows) if i != 3]
    assert torch.equal(clean[others], dirty[others])
    assert not torch.isfinite(dirty[3]).all()


def test_tree_attn_reports_what_does_not_hold(T):
    c = filled_cache(T, [40, 5], 2, 128, 16, 51)
    q = rand((8, 512), 1)
    for seqs, start, rows, zero, same in [
            ([2], [0, 3], 4, range(0, 3), range(3, 8)),      # a slot out of range
            ([-1], [0, 3], 4, range(0, 3), range(3, 8)),
            ([1], [0, 6], 8, range(0, 6), range(6, 8)),      # more rows than tokens
            ([0], [0, 6], 4, range(0, 6), range(6, 8)),      # more rows than max_rows
            ([0], [5, 3], 4, [], range(8)),                  # rows out of order
            ([0], [2, 9], 8, [], range(8)),                  # rows beyond M
    ]:
        ws = T.workspace(T.tf_tree_attn_workspace_bytes(c, 4, 1, rows))
        out = torch.full((8, 512), 5.0, dtype=torch.bfloat16, device="cuda")
        T.tf_tree_attn_run(q, c, 0, i32(seqs), i32(start), max_rows=rows, out=out, ws=ws)
        assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG, (seqs, start)
        assert (out[list(zero)] == 0).all() and (out[list(same)] == 5).all(), (seqs, start)
    # a page out of range counts as zeros
    c.table[0, 1] = 99
    ws = T.workspace(T.tf_tree_attn_workspace_bytes(c, 4, 1, 1))
    out = T.tf_tree_attn_run(q[:1], c, 0, i32([0]), i32([0, 1]), max_rows=1, ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG
    k, v = np.zeros((40, 2, 128)), np.zeros((40, 2, 128))
    for r in [*range(16), *range(32, 40)]:
        p = int(c.table[0, r // 16])
        k[r], v[r] = R.f64(c.data[0, 0, p, :, r % 16]), R.f64(c.data[0, 1, p, :, r % 16])
    ref, spread = R.tree_attn(R.f64(q[:1]).reshape(1, 4, 128), k, v, [1], 128 ** -0.5)
    within(R.f64(out).reshape(1, 4, 128), ref, R.attn_tol(ref, spread))


def test_tree_attn_strided_rows_and_a_repeated_slot(T):
    c = filled_cache(T, [90], 2, 128, 32, 61)
    wide = rand((6, 4 * 128 + 40), 2, 2.0)
    q = wide[:, 16:16 + 512]
    out = T.tf_tree_attn_run(q, c, 1, i32([0, 0]), i32([0, 2, 6]), max_rows=4)
    for lo, hi in [(0, 2), (2, 6)]:
        ref, spread = R.tree_attn(R.f64(q[lo:hi]).reshape(hi - lo, 4, 128), tokens(c, 1, 0, 0), tokens(c, 1, 1, 0),
                                  chain(hi - lo), 128 ** -0.5)
        within(R.f64(out[lo:hi]).reshape(hi - lo, 4, 128), ref, R.attn_tol(ref, spread))


def test_tree_attn_same_bits_every_time_in_a_graph_and_on_another_stream(T):
    c = filled_cache(T, [3000, 70, 901], 2, 128, 16, 71)
    q, seqs, start = rand((14, 512), 3, 2.0), i32([0, 1, 2]), i32([0, 8, 9, 14])
    want = T.tf_tree_attn_run(q, c, 1, seqs, start, max_rows=8)
    need = T.tf_tree_attn_workspace_bytes(c, 4, 3, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = T.tf_tree_attn_run(q, c, 1, seqs, start, max_rows=8, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    ws, out = T.workspace(need), torch.empty_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        T.tf_tree_attn_run(q, c, 1, seqs, start, max_rows=8, out=out, ws=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # the captured call reads lengths and pages anew: a shorter sequence, other queries
    c.len[0] = 100
    q.copy_(rand((14, 512), 4, 2.0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, T.tf_tree_attn_run(q, c, 1, seqs, start, max_rows=8))


# ---------------------------------------------------------------- page operations

def book_of(c):
    return c.book.tolist()


@pytest.mark.parametrize("page,n_seqs,n_pages,seed", [(16, 9, 60, 1), (32, 5, 20, 2), (64, 17, 40, 3), (128, 3, 9, 4)])
def test_page_operations_follow_the_model(T, page, n_seqs, n_pages, seed):
    """A long run of extend, fork and keep: after each the book is the model's, and every token
    of every slot is the one that was written for it."""
    rng = np.random.default_rng(seed)
    max_pages, layers, n_kv, hd = 7, 2, 3, 64
    c = T.KVCache.create(layers, n_kv, hd, page, n_pages, n_seqs, max_pages)
    m = R.Book(n_seqs, n_pages, max_pages, page)
    said = [[] for _ in range(n_seqs)]  # each slot's tokens
    ws = T.workspace(T.tf_kvcache_workspace_bytes(c))
    head = torch.arange(layers * 2 * n_kv * hd, device="cuda").view(layers, 2, n_kv, hd) % 7
    token = 0
    for step in range(60):
        seqs = rng.permutation(n_seqs)[:rng.integers(1, n_seqs + 1)].tolist()
        rows = [int(rng.choice([0, 1, 2, 9, 40, 64])) for _ in seqs]
        start = np.cumsum([1] + rows).tolist()
        M = start[-1] + 2
        slots, pos = T.tf_kvcache_extend(c, i32(seqs), i32(start), M, ws=ws)
        old = [m.len[s] for s in seqs]
        want = m.extend(seqs, rows)
        assert book_of(c) == m.flat(), step
        if want is None:
            code = T.tf_workspace_status(ws)
            assert code in (T.TF_E_CACHE_FULL, T.TF_E_INVALID_ARG) and (slots == -1).all()
            parent = [-1 if rng.random() < 0.4 else s for s in range(n_seqs)]  # make room
        else:
            assert slots.tolist() == [-1] + want + [-1, -1]
            assert pos.tolist() == [0] + [o + j for o, r in zip(old, rows) for j in range(r)] + [0, 0]
            for s, r in zip(seqs, rows):
                said[s] += list(range(token, token + r))
                token += r
            at = torch.tensor(want, dtype=torch.long, device="cuda")
            val = (torch.arange(token - len(want), token, device="cuda")[:, None, None, None, None] % 120 + head[None]).bfloat16()
            for l in range(layers):
                for kv in range(2):
                    c.data[l, kv, at // page, :, at % page] = val[:, l, kv]
            # keep some of the rows
            which = [i for i, r in enumerate(rows) if r > 0 and rng.random() < 0.6]
            kept, n_keep = [0] * M, []
            for i in range(len(seqs)):
                k = sorted(rng.permutation(rows[i])[:rng.integers(0, rows[i] + 1)].tolist()) if i in which else list(range(rows[i]))
                kept[start[i]:start[i] + len(k)] = k
                n_keep.append(len(k))
                m.keep(seqs[i], rows[i], k)
                s = said[seqs[i]]
                said[seqs[i]] = s[:len(s) - rows[i]] + [s[len(s) - rows[i] + j] for j in k]
            T.tf_kvcache_keep(c, i32(seqs), i32(start), i32(kept), i32(n_keep), ws=ws)
            assert T.tf_workspace_status(ws) == T.TF_OK
            assert book_of(c) == m.flat(), step
            parent = [int(rng.choice([-1, s, s, s, rng.integers(n_seqs)])) for s in range(n_seqs)]
        T.tf_kvcache_fork(c, i32(parent), ws=ws)
        if m.fork(parent) is None:
            assert T.tf_workspace_status(ws) == T.TF_E_CACHE_FULL
        else:
            assert T.tf_workspace_status(ws) == T.TF_OK
            said = [[] if p < 0 else list(said[p]) for p in parent]
        assert book_of(c) == m.flat(), step
        assert [len(x) for x in said] == m.len
        for s in range(n_seqs):
            if said[s]:
                at = torch.tensor([m.slot(s, r) for r in range(m.len[s])], device="cuda")
                want_rows = (torch.tensor(said[s], device="cuda")[:, None, None, None, None] % 120 + head[None]).bfloat16()
                got = torch.stack([torch.stack([c.data[l, kv, at // page, :, at % page] for kv in range(2)], 1)
                                   for l in range(layers)], 1)
                assert torch.equal(got, want_rows), (step, s)


def test_a_fork_without_enough_free_pages_does_nothing(T):
    c = filled_cache(T, [20, 33, 5, 7], 1, 64, 16, 94, spare=2)
    ws = T.workspace(T.tf_kvcache_workspace_bytes(c))
    before, data = book_of(c), c.data.clone()
    T.tf_kvcache_fork(c, i32([0, 0, 0, 0]), ws=ws)  # three copies, two free pages
    assert T.tf_workspace_status(ws) == T.TF_E_CACHE_FULL
    assert book_of(c) == before and torch.equal(c.data, data)
    T.tf_kvcache_fork(c, i32([0, 0, 0, 3]), ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_OK and c.len.tolist() == [20, 20, 20, 7]


def test_page_operations_of_the_most_slots(T):
    """1024 slots, all named in one call: extend, a reordering fork, keep."""
    c = T.KVCache.create(1, 1, 64, 16, 6000, 1024, 9)
    m = R.Book(1024, 6000, 9, 16)
    rng = np.random.default_rng(5)
    for step in range(3):
        seqs, rows = rng.permutation(1024).tolist(), rng.integers(0, 30, 1024).tolist()
        start = np.cumsum([0] + rows).tolist()
        slots, _ = T.tf_kvcache_extend(c, i32(seqs), i32(start), start[-1])
        assert slots.tolist() == m.extend(seqs, rows)
        parent = rng.integers(-1, 1024, 1024).tolist()
        T.tf_kvcache_fork(c, i32(parent))
        assert m.fork(parent) is not None
        assert book_of(c) == m.flat()
    seqs = [s for s in range(1024) if m.len[s] % 16 >= 3]
    T.tf_kvcache_keep(c, i32(seqs), i32(list(range(0, 3 * len(seqs) + 1, 3))), i32([0, 2, 0] * len(seqs)), i32([2] * len(seqs)))
    for s in seqs:
        m.keep(s, 3, [0, 2])
    assert book_of(c) == m.flat()


def test_extend_of_a_tree_gives_the_depths(T):
    c = filled_cache(T, [20, 0], 1, 64, 16, 81)
    masks = [0b1, 0b11, 0b101, 0b1011]  # root, two children, a grandchild of the first
    slots, pos = T.tf_kvcache_extend(c, i32([1, 0]), i32([0, 1, 5]), 5, masks=mask_tensor([1] + masks))
    assert pos.tolist() == [0, 20, 21, 21, 22]
    assert slots.tolist()[1:] == [int(c.table[0, 1]) * 16 + 4 + j for j in range(4)]


def test_a_prompt_longer_than_the_free_list(T):
    c = T.KVCache.create(1, 1, 64, 16, 9000, 2, 6000)
    m = R.Book(2, 9000, 6000, 16)
    c.refs[::3] = 1  # every third page taken
    m.refs = [1 if i % 3 == 0 else 0 for i in range(9000)]
    slots, _ = T.tf_kvcache_extend(c, i32([1, 0]), i32([0, 5, 80005]), 80005)
    assert slots.tolist() == m.extend([1, 0], [5, 80000])
    assert book_of(c) == m.flat()
    ws = T.workspace(T.tf_kvcache_workspace_bytes(c))
    T.tf_kvcache_extend(c, i32([1]), i32([0, 80000]), 80000, ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_E_CACHE_FULL and book_of(c) == m.flat()


def test_page_operations_refuse_on_the_device(T):
    c = filled_cache(T, [20, 33, 5], 1, 64, 16, 91)
    ws = T.workspace(T.tf_kvcache_workspace_bytes(c))
    before, data = book_of(c), c.data.clone()

    def refused(code=T.TF_E_INVALID_ARG):
        assert T.tf_workspace_status(ws) == code
        assert book_of(c) == before and torch.equal(c.data, data)

    for seqs, start in [([0, 0], [0, 1, 2]), ([3], [0, 1]), ([-1], [0, 1]), ([0], [2, 1]), ([0], [0, 9]), ([0], [-1, 2])]:
        slots, _ = T.tf_kvcache_extend(c, i32(seqs), i32(start), 4, ws=ws)
        assert (slots == -1).all()
        refused()
    T.tf_kvcache_extend(c, i32([1]), i32([0, 64]), 64, ws=ws)  # past max_pages
    refused()
    for parent in ([0, 1, 3], [0, -2, 2]):
        T.tf_kvcache_fork(c, i32(parent), ws=ws)
        refused()
    for seqs, start, keep, n in [([0], [0, 3], [0, 2, 1], [3]), ([0], [0, 3], [1, 1, 0], [2]), ([0], [0, 3], [0, 3, 0], [2]),
                                 ([0], [0, 3], [-1, 0, 0], [1]), ([0], [0, 3], [0, 1, 2], [4]), ([0], [0, 3], [0, 1, 2], [-1]),
                                 ([2], [0, 6], list(range(6)), [1]), ([4], [0, 3], [0, 1, 2], [1]), ([0], [0, 4], [0, 1, 2], [1])]:
        T.tf_kvcache_keep(c, i32(seqs), i32(start), i32(keep), i32(n), ws=ws)
        refused()
    T.tf_kvcache_keep(c, i32([0, 1, 0]), i32([0, 1, 2, 3]), i32([0, 0, 0]), i32([0, 0, 0]), ws=ws)
    refused()
    # a block on a page that another slot holds too
    T.tf_kvcache_fork(c, i32([0, 1, 1]), ws=ws)  # slot 2 shares slot 1's two full pages
    assert T.tf_workspace_status(ws) == T.TF_OK
    before, data = book_of(c), c.data.clone()
    T.tf_kvcache_keep(c, i32([2]), i32([0, 5]), i32([0, 1, 2, 3, 4]), i32([1]), ws=ws)
    refused()
    # one sequence refused, the other done
    T.tf_kvcache_keep(c, i32([2, 0]), i32([0, 5, 7]), i32([0] * 5 + [1, 0]), i32([1, 1]), ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG
    assert c.len.tolist() == [19, 33, 33]


def test_reset_empties_the_book(T):
    c = filled_cache(T, [20, 33, 5], 1, 64, 16, 92)
    T.tf_kvcache_reset(c)
    assert book_of(c) == R.Book(3, c.n_pages, c.max_pages, 16).flat()


# ---------------------------------------------------------------- log probabilities

def lp_close(got, ref, scale):
    """Sums in fp32: up to N / 2048 terms in a row in a thread's four partial sums, then a tree,
    and 2^-22 an exponential: 2^-16 of the whole is above that for N up to 200,000. Differences of
    logits are rounded to 2^-24 of their size."""
    got, ref = R.f64(got), np.asarray(ref)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
    np.testing.assert_array_equal(np.isneginf(got), np.isneginf(ref))
    ok = np.isfinite(ref)
    err = np.abs(got[ok] - ref[ok])
    assert (err <= 2.0 ** -16 * scale + 2.0 ** -22 * np.abs(ref[ok])).all(), float(err.max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,k,nt", [(1, 1, 1, 1), (1, 2, 2, 1), (3, 7, 7, 2), (1, 151936, 8, 1), (9, 151936, 32, 3),
                                      (40, 1000, 20, 1), (2, 33000, 0, 1), (200, 131, 5, 0), (2, 200001, 32, 33), (17, 9999, 1, 1)])
def test_logprobs(T, dtype, M, N, k, nt):
    g = torch.Generator(device="cuda").manual_seed(M * 7 + N)
    wide = (torch.randn((M, N + 5), generator=g, device="cuda") * 4).to(dtype)
    v = wide[:, 3:3 + N]  # rows that start anywhere
    targets = torch.randint(-1, N, (M, nt), generator=g, device="cuda").int() if nt else None
    ws = T.workspace(T.tf_logprobs_workspace_bytes(M, N, k))
    lp, ent, idx, tlp = T.tf_logprobs_rows(v, targets, k, ws=ws)
    ref = R.logprobs(R.f64(v), targets.cpu().numpy() if nt else np.zeros((M, 0), int), k)
    assert T.tf_workspace_status(ws) == T.TF_OK
    if nt:
        lp_close(lp, ref[0], 1.0)
    lp_close(ent, ref[1], 1.0)
    if k:
        np.testing.assert_array_equal(idx.cpu().numpy(), ref[2])
        lp_close(tlp, ref[3], 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [40, 5001, 70000])
def test_logprobs_masks_ties_and_what_is_not_a_number(T, dtype, N):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(dtype).min
    g = torch.Generator(device="cuda").manual_seed(N)
    v = (torch.randn((12, N), generator=g, device="cuda") * 3).to(dtype)
    v[0] = 1.5                      # every value the same
    v[1] = -inf                     # nothing left
    v[2, torch.arange(N, device="cuda") % 7 != 3] = -inf   # a grammar's mask
    v[3, torch.arange(N, device="cuda") % 5 != 1] = low    # the same with the type's lowest value
    v[4] = low
    v[5, N // 2] = nan
    v[6] = nan
    v[6, [3, 17]] = 2.0
    v[7, N - 1] = inf
    v[8] = v[8].round()             # many ties
    v[9] = -inf
    v[9, N - 2] = 3.0               # one certain token
    v[10, 5] = 0.0
    v[10, 6] = -0.0
    v[10] = v[10].clamp(max=0)
    v[11] = 0.0
    v[11, 11] = 60.0                # nearly certain: the entropy is all in the rest
    k = 21
    targets = torch.tensor([[0, N - 2, -1, N, -7]] * 12, dtype=torch.int32, device="cuda")
    ws = T.workspace(T.tf_logprobs_workspace_bytes(12, N, k))
    lp, ent, idx, tlp = T.tf_logprobs_rows(v, targets, k, ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG  # the targets N and -7
    ref = R.logprobs(R.f64(v), targets.cpu().numpy(), k)
    np.testing.assert_array_equal(idx.cpu().numpy(), ref[2])
    for a, b in ((lp, ref[0]), (ent, ref[1]), (tlp, ref[3])):
        lp_close(a, b, 1.0)
    # relative, where the value is small: the rest's own sum (2^-16), not the whole's
    for a, b in ((float(ent[11]), ref[1][11]), (float(tlp[11, 0]), ref[3][11, 0])):
        assert abs(a - b) <= 2.0 ** -15 * abs(b)


def test_logprobs_sorted_rows(T):
    """Rows in which one thread's share holds nearly all of the largest values."""
    v = torch.zeros((3, 60000), device="cuda")
    v[0] = torch.arange(60000, device="cuda") * 1e-3
    v[1] = -v[0]
    v[2, 512 * 4 * torch.arange(20, device="cuda")] = torch.arange(20, device="cuda") + 1.0
    v[2, 1 + 512 * 4 * torch.arange(20, device="cuda")] = torch.arange(20, device="cuda") + 1.5
    _, _, idx, _ = T.tf_logprobs_rows(v, None, 32)
    np.testing.assert_array_equal(idx.cpu().numpy(), R.logprobs(R.f64(v), np.zeros((3, 0), int), 32)[2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,k", [(700, 1, 1), (1300, 40, 32), (700, 5001, 7), (613, 33000, 20), (650, 70000, 0)])
def test_logprobs_of_many_rows(T, dtype, M, N, k):
    """More rows than the GPU holds blocks at once, of every kind among them."""
    inf, nan, low = float("inf"), float("nan"), torch.finfo(dtype).min
    g = torch.Generator(device="cuda").manual_seed(N + k)
    v = (torch.randn((M, N + 9), generator=g, device="cuda") * 3).to(dtype)[:, 5:5 + N]
    at = torch.arange(N, device="cuda")
    for i, rows in enumerate([v[j::50] for j in range(9)]):
        if i == 0:
            rows[:] = 1.5
        elif i == 1:
            rows[:] = -inf
        elif i in (2, 3):
            rows[:, at % 7 != 3] = -inf if i == 2 else low
        elif i == 4:
            rows[:, N // 2] = nan
        elif i == 5:
            rows[:, N - 1] = inf
        elif i == 6:
            rows[:] = rows.round()
        elif i == 7:
            rows[:] = (at * 1e-3).to(dtype)
        else:
            rows[:] = (at // 1024 % 2 * 5).to(dtype)  # many threads' largest in one batch, or none
    t = torch.randint(-1, N, (M, 2), generator=g, device="cuda").int()
    ws = T.workspace(T.tf_logprobs_workspace_bytes(M, N, k))
    lp, ent, idx, tlp = T.tf_logprobs_rows(v, t, k, ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_OK
    ref = R.logprobs(R.f64(v), t.cpu().numpy(), k)
    lp_close(lp, ref[0], 1.0)
    lp_close(ent, ref[1], 1.0)
    if k:
        np.testing.assert_array_equal(idx.cpu().numpy(), ref[2])
        lp_close(tlp, ref[3], 1.0)


def test_logprobs_agrees_with_argmax_and_repeats_in_a_graph(T):
    v = rand((8, 151936), 5, 3.0)
    t = i32(list(range(8)))
    want = T.tf_logprobs_rows(v, t, 4)
    assert torch.equal(want[2][:, 0], T.tf_argmax_rows(v))
    out = [torch.empty_like(x) for x in want]
    ws = T.workspace(T.tf_logprobs_workspace_bytes(8, 151936, 4))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        T.tf_logprobs_rows(v, t, 4, *out, ws=ws)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- refusals of the binding

def test_the_binding_refuses_tensors_that_do_not_fit(T):
    c = filled_cache(T, [20], 2, 128, 16, 93)
    q, s, st = rand((2, 512), 1), i32([0]), i32([0, 2])
    for bad in [dict(q=q.float()), dict(q=q.t()), dict(q=q[:, :200]), dict(seqs=s.long()), dict(q_start=i32([0])),
                dict(masks=mask_tensor([1])), dict(masks=i32([1, 1])), dict(out=torch.empty(2, 512, device="cuda")),
                dict(out=torch.empty(2, 256, dtype=torch.bfloat16, device="cuda")), dict(seqs=s.cpu())]:
        kw = dict(q=q, seqs=s, q_start=st, masks=None, out=None)
        kw.update(bad)
        with pytest.raises(ValueError):
            T.tf_tree_attn_run(kw["q"], c, 0, kw["seqs"], kw["q_start"], masks=kw["masks"], max_rows=2, out=kw["out"])
    with pytest.raises(T.TfqError):
        T.tf_tree_attn_run(q, c, 2, s, st, max_rows=2)
    with pytest.raises(T.TfqError):
        T.tf_tree_attn_run(q, c, 0, s, st, max_rows=2, out=q)
    with pytest.raises(ValueError):
        T.KVCache(c.data[:, :1], c.book, 1, 3)
    with pytest.raises(T.TfqError):
        T.KVCache(c.data, c.book[:4].clone(), 1, 3)
    with pytest.raises(ValueError):
        T.tf_logprobs_rows(rand((2, 8), 1), i32([1]), 1)
    with pytest.raises(ValueError):
        T.tf_kvcache_fork(c, i32([]))
