"""The cache of 8 bits against 64-bit references: norm, rotation and store as e4m3 codes, attention over them, and the page
operations that move them."""
import numpy as np
import pytest
import torch

import cache8_ref as Q
import cached_ref as R

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


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


def within(got, ref, tol):
    err = np.abs(got - ref)
    bad = ~((err <= tol) | (np.isnan(got) & np.isnan(ref)))
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside: worst {np.nanmax(err / tol)}, at {np.argwhere(bad)[:3].tolist()}"


def paged(T, lens, n_kv, hd, page, seed, layers=2, spare=3, dtype=E4M3, sizes=True):
    """A cache whose slots hold `lens` tokens on scattered pages, everything in it random."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    n_pages, max_pages = sum(need) + spare, max(need + [1]) + 2
    c = T.KVCache.create(layers, n_kv, hd, page, n_pages, len(lens), max_pages, dtype=dtype)
    if dtype == E4M3:
        Q.fill(c, seed, sizes)
    else:
        c.data.copy_(rand(c.data.shape, seed))
    order = rng.permutation(n_pages).tolist()
    table = np.full((len(lens), max_pages), -1, np.int32)
    for s, n in enumerate(need):
        table[s, :n] = [order.pop() for _ in range(n)]
    c.len.copy_(i32(lens))
    c.refs.copy_(torch.from_numpy(np.bincount(table[table >= 0], minlength=n_pages).astype(np.int32)))
    c.table.copy_(torch.from_numpy(table))
    return c


def slots_of(c, s, first, rows):
    at = torch.arange(first, first + rows, device="cuda")
    return (c.table[s].long()[at // c.page_size] * c.page_size + at % c.page_size).int()


def tokens(c, vals, layer, kv, s):
    r = np.arange(int(c.len[s]))
    return vals[layer, kv][c.table[s].cpu().numpy()[r // c.page_size], :, r % c.page_size]


# ---------------------------------------------------------------- norm, rotation and store

def check_store(c, before, after, e0, e1, codes0, codes1, layer, kv, slots, x, tol):
    """Values x [rows, heads, hd] at `slots`: scales by their definition, codes half a step from x, the block's other rows
    rounded to the new scale, everything else as it was."""
    blocks = {}
    for m, s in enumerate(slots):
        if s >= 0:
            blocks.setdefault((s // c.page_size, s % c.page_size // 16), []).append(m)
    same = np.ones(e0.shape[2:], bool)
    for (p, b), rows in blocks.items():
        same[p, :, b] = False
        offs = [slots[m] % 16 for m in rows]
        for h in range(c.n_kv):
            most = max((np.abs(x[m, h][np.isfinite(x[m, h])]).max(initial=0.0) for m in rows), default=0.0)
            # fp32 values may fall to either side of a power's border
            fine = {Q.least_exponent(most * (1 - 2.0 ** -18)), Q.least_exponent(most * (1 + 2.0 ** -18))}
            if 0 not in offs:
                fine = {max(e, int(np.clip(e0[layer, kv, p, h, b], Q.LEAST, Q.MOST))) for e in fine}
            e = int(e1[layer, kv, p, h, b])
            assert e in fine, (p, b, h, e, fine)
            got = after[layer, kv, p, h, b * 16:b * 16 + 16]
            for m, off in zip(rows, offs):
                ref = x[m, h]
                want = np.where(np.isnan(ref), np.nan, np.clip(ref, -448 * 2.0 ** e, 448 * 2.0 ** e))
                room = tol[m, h] + Q.E4M3_HALF * np.abs(want) + 2.0 ** (e - 10)
                within(got[off], want, np.where(np.isfinite(room), room, 0.0))
            if 0 not in offs:
                rest = [r for r in range(16) if r not in offs]
                d = int(np.clip(e0[layer, kv, p, h, b], Q.LEAST, Q.MOST)) - e
                old = codes0[layer, kv, p, h, b * 16:b * 16 + 16][rest]
                np.testing.assert_array_equal(codes1[layer, kv, p, h, b * 16:b * 16 + 16][rest], Q.e4m3(old * 2.0 ** d) if d else old)
    np.testing.assert_array_equal(e0[layer, kv][same], e1[layer, kv][same])
    keep = np.repeat(same, 16, -1)
    np.testing.assert_array_equal(codes0[layer, kv][keep], codes1[layer, kv][keep])


def snapshot(c):
    return Q.values(c), Q.exponents(c), R.f64(c.data.float())


@pytest.mark.parametrize("seqs,n_q,n_kv,hd,rot,pairs,norm,page", [
    ([(0, 1)], 16, 8, 128, 128, False, True, 16),                        # the first row of a sequence
    ([(15, 1)], 16, 8, 128, 128, False, True, 16),                       # the last of a block
    ([(16, 1), (17, 1), (31, 1), (5, 1)], 5, 1, 128, 64, False, True, 32),
    ([(13, 8), (0, 8), (30, 8), (64, 3)], 4, 2, 64, 64, True, True, 64),  # blocks of drafts over borders
    ([(7, 130)], 3, 3, 256, 256, False, True, 128),
    ([(0, 9)], 2, 1, 256, 16, True, False, 16),
    ([(3, 300), (0, 1), (250, 17), (9, 64), (16, 16)], 16, 8, 128, 0, False, True, 64),
    ([(5, 1500)], 4, 2, 128, 128, True, True, 16),
    ([(i % 40, 1) for i in range(300)], 2, 2, 64, 48, False, False, 16),  # a served batch
    ([(i % 23, 1 + i % 5) for i in range(90)], 8, 2, 128, 128, False, True, 32),
])
def test_norm_rope_into_8_bits(T, seqs, n_q, n_kv, hd, rot, pairs, norm, page):
    lens = [a + r for a, r in seqs]
    c = paged(T, lens, n_kv, hd, page, 5 + sum(lens), layers=2)
    rows = sum(r for _, r in seqs)
    M = rows + 2
    cols = (n_q + 2 * n_kv) * hd
    qkv = rand((M, cols + 24), 1, 2.0)[:, 8:8 + cols]
    qkv[: M // 2] *= 8  # some blocks' scales grow, some do not
    qg, kg = (rand((hd,), 2) + 1, rand((hd,), 3) + 1) if norm else (None, None)
    none = i32([-1])
    slots = torch.cat([none] + [slots_of(c, s, a, r) for s, (a, r) in enumerate(seqs)] + [none])
    pos = np.random.default_rng(rows).integers(-5, 200000, M).astype(np.int32)
    inv = 1e6 ** (-np.arange(0, rot, 2) / max(rot, 1))
    rope, ws = T.RopeTable(inv, pairs=pairs), T.workspace(256)
    kw = dict(q_gamma=qg, k_gamma=kg, eps=1e-5, n_q=n_q)
    v0, e0, c0 = snapshot(c)
    q = T.tf_qk_norm_rope_run(qkv, c, 1, torch.from_numpy(pos).cuda(), slots, rope, ws=ws, **kw)
    v1, e1, c1 = snapshot(c)
    assert T.tf_workspace_status(ws) == T.TF_OK
    x = R.f64(qkv).reshape(M, -1, hd)
    ref, size = R.norm_rope(x[:, :n_q], None if qg is None else R.f64(qg), 1e-5, pos, inv, pairs)
    within(R.f64(q).reshape(M, n_q, hd), ref, R.rope_tol(ref, size))
    ref, size = R.norm_rope(x[:, n_q:n_q + n_kv], None if kg is None else R.f64(kg), 1e-5, pos, inv, pairs)
    sl = slots.tolist()
    check_store(c, v0, v1, e0, e1, c0, c1, 1, 0, sl, ref, 2.0 ** -19 * size)
    check_store(c, v0, v1, e0, e1, c0, c1, 1, 1, sl, x[:, n_q + n_kv:], np.zeros_like(ref))
    np.testing.assert_array_equal(e0[0], e1[0])
    np.testing.assert_array_equal(c0[0], c1[0])
    # the same call again changes nothing
    T.tf_qk_norm_rope_run(qkv, c, 1, torch.from_numpy(pos).cuda(), slots, rope, ws=ws, **kw)
    v2, e2, c2 = snapshot(c)
    np.testing.assert_array_equal(c1, c2)
    np.testing.assert_array_equal(e1, e2)


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_store_of_what_is_not_ordinary(T, hd):
    """Infinities and NaN, zeros, values past the scales' bounds, bytes of earlier tenants."""
    c = paged(T, [16 * 12], 1, hd, 16, 3, layers=1)
    c.scales.view(torch.uint8).fill_(255)  # what memory may hold
    rows = []
    x = torch.zeros((12, hd), dtype=torch.bfloat16, device="cuda")
    x[1] = 1.0
    x[1, 3], x[1, 7] = float("inf"), float("-inf")
    x[2] = float("nan")
    x[3, 0] = float("nan")
    x[3, 1] = 3.0
    x[4] = 1e30
    x[5] = 1e-30
    x[6, 5] = 448.0
    x[7, 5] = 450.0   # bf16: 450, above 448
    x[8, 5] = -1.75 * 2 ** -5
    x[9] = float("inf")
    x[10] = torch.linspace(-1, 1, hd).bfloat16()
    x[11, 0], x[11, 1] = 448.0, 2.0 ** -6
    qkv = torch.cat([x, x, x], 1)
    slots = torch.cat([slots_of(c, 0, 16 * i, 1) for i in range(12)])
    T.tf_qk_norm_rope_run(qkv, c, 0, i32([0] * 12), slots, T.RopeTable([]), n_q=1)
    e, code = Q.exponents(c), R.f64(c.data.float())
    for i, s in enumerate(slots.tolist()):
        y = R.f64(x[i])
        most = np.abs(y[np.isfinite(y)]).max(initial=0.0)
        for kv in (0, 1):
            assert e[0, kv, s // 16, 0, 0] == Q.least_exponent(most), i
            np.testing.assert_array_equal(code[0, kv, s // 16, 0, 0], Q.e4m3(y * 2.0 ** -Q.least_exponent(most)))
    # a larger row joins: what is there is rounded to the new scale
    old = code.copy()
    again = torch.cat([x * 0 + 100.0] * 3, 1)
    again[9], again[2] = 1.0, 1.0
    T.tf_qk_norm_rope_run(again, c, 0, i32([0] * 12), slots + 1, T.RopeTable([]), n_q=1)
    e2, code2 = Q.exponents(c), R.f64(c.data.float())
    for i, s in enumerate(slots.tolist()):
        d = e[0, 0, s // 16, 0, 0] - e2[0, 0, s // 16, 0, 0]
        assert d <= 0
        np.testing.assert_array_equal(code2[0, 0, s // 16, 0, 0], Q.e4m3(old[0, 0, s // 16, 0, 0] * 2.0 ** d))


def test_store_in_steps_is_the_store_at_once_but_for_rounding(T):
    """Rows of one prompt appended in calls of any length: scales as at once, or larger where an early row fell later."""
    c1, c2 = (paged(T, [203], 2, 128, 32, 9, layers=1) for _ in range(2))
    qkv = rand((203, 6 * 128), 4) * torch.exp2(torch.arange(203, device="cuda") % 9).bfloat16()[:, None]
    pos, slots, rope = torch.arange(203, dtype=torch.int32, device="cuda"), slots_of(c1, 0, 0, 203), T.RopeTable(1e4 ** (-np.arange(64) / 64))
    T.tf_qk_norm_rope_run(qkv, c1, 0, pos, slots, rope, n_q=2)
    at = 0
    for n in [1, 1, 7, 30, 16, 1, 64, 3, 40, 40]:
        T.tf_qk_norm_rope_run(qkv[at:at + n], c2, 0, pos[at:at + n], slots[at:at + n], rope, n_q=2)
        at += n
    assert at == 203
    e1, e2 = Q.exponents(c1), Q.exponents(c2)
    used = np.zeros(e1.shape[2:], bool)
    for s in slots.tolist():
        used[s // 32, :, s % 32 // 16] = True
    np.testing.assert_array_equal(e1[0][:, used], e2[0][:, used])
    rows = np.repeat(used, 16, -1)
    for s in range(c1.n_pages):  # rows of the prompt alone
        for r in range(32):
            if s * 32 + r not in set(slots.tolist()):
                rows[s, :, r] = False
    a, b = Q.values(c1)[0][:, rows], Q.values(c2)[0][:, rows]
    step = 2.0 ** np.repeat(e1, 16, -1)[0][:, rows] * 2.0 ** -9  # of e4m3's subnormals, where a code may have been rounded twice
    within(b, a, step[..., None] * 1.0 + 0 * a)


def test_store_repeats_in_a_graph_on_another_stream_and_reports(T):
    c = paged(T, [100, 40], 2, 128, 16, 21)
    qkv, pos = rand((9, 8 * 128), 5), i32(list(range(9)))
    slots = torch.cat([slots_of(c, 0, 92, 8), slots_of(c, 1, 39, 1)])
    rope, ws = T.RopeTable(1e4 ** (-np.arange(64) / 64)), T.workspace(256)
    data0, scales0 = c.data.clone(), c.scales.clone()
    want_q = T.tf_qk_norm_rope_run(qkv, c, 1, pos, slots, rope, ws=ws)
    want, want_s = c.data.view(torch.uint8).clone(), c.scales.view(torch.uint8).clone()
    side = torch.cuda.Stream()
    for how in ("stream", "graph"):
        c.data.copy_(data0)
        c.scales.copy_(scales0)
        torch.cuda.synchronize()
        if how == "stream":
            q = T.tf_qk_norm_rope_run(qkv, c, 1, pos, slots, rope, ws=ws, stream=side, flags=T.TF_RUN_PDL)
        else:
            q, g = torch.empty_like(want_q), torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                T.tf_qk_norm_rope_run(qkv, c, 1, pos, slots, rope, ws=ws, out=q)
            c.data.copy_(data0)
            c.scales.copy_(scales0)
            g.replay()
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, want_q) and torch.equal(c.data.view(torch.uint8), want) and torch.equal(c.scales.view(torch.uint8), want_s)
    slots[3] = c.n_pages * 16 + 5
    T.tf_qk_norm_rope_run(qkv, c, 1, pos, slots, rope, ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG


def test_sums_of_squares_past_fp32_give_what_a_bf16_cache_gets(T):
    """Finite rows whose squares overflow: 0; with an infinity among them, NaN where it is and where it is turned to."""
    qkv = rand((6, 4 * 64), 40, 2.0)
    qkv[1] *= 2.0 ** 100
    qkv[2, 5] = 2.0 ** 90
    qkv[3, 64 + 7] = float("inf")
    qkv[4, 128 + 9] = float("inf")
    gamma = rand((64,), 41) * 2.0 ** 40
    rope = T.RopeTable(1e4 ** (-np.arange(32) / 32))
    got = []
    for dtype in (E4M3, torch.bfloat16):
        c = T.KVCache.create(1, 1, 64, 16, 1, 1, 1, dtype=dtype)
        q = T.tf_qk_norm_rope_run(qkv, c, 0, i32([0] * 6), i32(list(range(6))), rope, q_gamma=gamma, k_gamma=gamma)
        k = c.data[0, 0, 0, 0, :6].float()
        got.append((q.float().cpu(), k.cpu()))
    (q8, k8), (q16, k16) = got
    assert torch.equal(q8.isnan(), q16.isnan()) and torch.equal(k8.isnan(), k16.isnan())
    assert q8[3].isnan().any() and k8[4].isnan().any() and not q8[:3].isnan().any()
    for i in (1, 2):  # row 2's first head alone
        assert (q8[i, :64] == 0).all() and (q16[i, :64] == 0).all()
    assert (k8[1] == 0).all() and (k16[1] == 0).all()


# ---------------------------------------------------------------- attention

def chain(rows):
    return [(1 << (i + 1)) - 1 for i in range(rows)]


def tree(rows, rng):
    out = []
    for i in range(rows):
        out.append((1 << i) | (out[rng.integers(i)] if i else 0))
    return out


def run_attn(T, c, layer, seqs, rows, masks, n_q, seed, scale=None, lead=0, q=None):
    start = np.cumsum([lead] + rows)
    M = int(start[-1]) + 3
    q = rand((M, n_q * c.head_dim), seed, 2.0) if q is None else q
    out = torch.full((M, n_q * c.head_dim), 5.0, dtype=torch.bfloat16, device="cuda")
    m = None
    if masks is not None:
        m = mask_tensor([0] * lead + [b for x in masks for b in x] + [0] * 3)
    most = max(max(rows), 1)
    ws = T.workspace(T.tf_tree_attn_workspace_bytes(c, n_q, len(seqs), most))
    for _ in range(2):  # the second call finds the workspace as the first left it
        T.tf_tree_attn_run(q, c, layer, i32(seqs), i32(start.tolist()), masks=m, max_rows=most, scale=scale, out=out, ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_OK
    assert (out[:lead] == 5).all() and (out[int(start[-1]):] == 5).all()
    return q, out, start


def seen(n, rows, bits):
    see = np.ones((rows, n), bool)
    for i in range(rows):
        for j in range(rows):
            see[i, n - rows + j] = bits[i] >> j & 1
    return see


def check_attn(T, c, layer, seqs, rows, masks, n_q, seed, scale=None, lead=0, q=None, which=None):
    q, out, start = run_attn(T, c, layer, seqs, rows, masks, n_q, seed, scale, lead, q)
    hd, vals = c.head_dim, Q.values(c)
    for b in range(len(seqs)) if which is None else which:
        qq = R.f64(q[start[b]:start[b + 1]]).reshape(rows[b], n_q, hd)
        k, v = tokens(c, vals, layer, 0, seqs[b]), tokens(c, vals, layer, 1, seqs[b])
        bits = chain(rows[b]) if masks is None else masks[b]
        ref, spread, size = Q.attn(qq, k, v, seen(len(k), rows[b], bits), hd ** -0.5 if scale is None else scale, Q.scales_of(c, layer, seqs[b]))
        within(R.f64(out[start[b]:start[b + 1]]).reshape(rows[b], n_q, hd), ref, Q.attn_tol(ref, spread, size))


SHAPES = [
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
    ([1100, 70], [20, 9], 4, 1, 64, 64),             # 80 query rows
    ([900], [9], 8, 1, 128, 32),                     # 72
    ([5000], [40], 8, 2, 64, 16),                    # 160
]


@pytest.mark.parametrize("lens,rows,n_q,n_kv,hd,page", SHAPES)
def test_attention_over_8_bits(T, lens, rows, n_q, n_kv, hd, page):
    rng = np.random.default_rng(sum(lens))
    c = paged(T, lens, n_kv, hd, page, 11 + sum(lens))
    seqs = rng.permutation(len(lens)).tolist()
    rr = [rows[s] for s in seqs]
    check_attn(T, c, 1, seqs, rr, None, n_q, 21)
    check_attn(T, c, 0, seqs, rr, [tree(r, rng) for r in rr], n_q, 22, scale=0.05, lead=2)


@pytest.mark.parametrize("n,rows", [(40000, 1), (9001, 8), (5000, 40), (3000, 64)])
def test_attention_over_8_bits_long(T, n, rows):
    c = paged(T, [n, 3, 777], 2, 128, 16, n)
    check_attn(T, c, 1, [0, 1, 2], [rows, 1, min(rows, 700)], None, 4, 5)


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
@pytest.mark.parametrize("rows,n_q,hd", [(3, 4, 128), (40, 8, 64), (64, 16, 128)])
def test_scales_of_every_size_and_sign(T, rows, n_q, hd, scale):
    """Blocks whose scales lie 2^20 apart, and rows of q from 2^-40 to 2^2."""
    c = paged(T, [333], 2, hd, 16, 8)
    g = torch.Generator(device="cuda").manual_seed(1)
    v = c.scales.view(torch.uint8)
    v[:, 1] = torch.randint(127 - 25, 127 - 4, v[:, 1].shape, generator=g, device="cuda").to(torch.uint8)
    v[:, 0] = 127 - 7
    q = rand((rows + 3, n_q * hd), 3)
    for i, e in enumerate([0, -40, 2, -3]):
        q[i::4] *= 2.0 ** e
    check_attn(T, c, 0, [0], [rows], None, n_q, 3, scale=scale, q=q)


@pytest.mark.parametrize("rows,n_q", [(1, 4), (40, 4), (64, 16)])
def test_the_scales_bounds(T, rows, n_q):
    """A value of 2^-32's block beside one of 2^32's, and bytes out of bounds, which count as the bound."""
    c = paged(T, [200], 2, 128, 16, 8, sizes=False)
    v = c.scales.view(torch.uint8)
    v[0, 1] = 127 - 32
    v[0, 1, ::2] = 127 + 32
    v[1, 1] = 0
    v[1, 1, 1::3] = 255
    for layer in (0, 1):
        check_attn(T, c, layer, [0], [rows], None, n_q, 4)


@pytest.mark.parametrize("n_q,hd,rows", [(2, 128, 1), (4, 64, 7), (1, 256, 3), (40, 128, 3)])
def test_attention_over_8_bits_the_most_sequences(T, n_q, hd, rows):
    lens = [1 + 7 * i % 90 for i in range(40)]
    c = paged(T, lens, 1, hd, 16, 101)
    rng = np.random.default_rng(rows)
    seqs = rng.integers(0, 40, 1024).tolist()
    rr = [int(min(rng.integers(0, rows + 1), lens[s])) for s in seqs]
    check_attn(T, c, 1, seqs, rr, None, n_q, 6, which=rng.permutation(1024)[:60].tolist() + [0, 1023])


@pytest.mark.parametrize("hd,rows", [(128, 4), (64, 20), (256, 6), (128, 50)])
def test_rows_that_see_nothing_are_zero(T, hd, rows):
    c = paged(T, [rows, 100 + rows], 2, hd, 16, 31)
    masks = [[0 if i % 2 else chain(rows)[i] for i in range(rows)], [0] * rows]
    check_attn(T, c, 0, [0, 1], [rows, rows], masks, 4, 7)
    q, out, start = run_attn(T, c, 0, [0], [rows], [[0] * rows], 4, 8)
    assert int(torch.count_nonzero(out[:rows])) == 0


@pytest.mark.parametrize("hd,rows,n_q", [(128, 6, 4), (64, 40, 4), (256, 9, 2), (128, 30, 16), (128, 12, 4)])
def test_what_a_row_does_not_see_takes_no_part(T, hd, rows, n_q):
    n = 150 + rows
    c = paged(T, [n, 40], 2, hd, 16, 41)
    rng = np.random.default_rng(rows)
    bits = [b & ~8 if i != 3 else b for i, b in enumerate(tree(rows, rng))]  # row 3 is seen by itself alone
    clean = run_attn(T, c, 1, [0], [rows], [bits], n_q, 9)[1]
    codes = c.data.view(torch.uint8)
    page, off = int(c.table[0, (n - rows + 3) // 16]), (n - rows + 3) % 16
    codes[1, :, page, :, off] = 0x7F
    codes[1, 1, page, :, off, 5:] = 0x35  # some of its values alone are NaN
    last = int(c.table[0, (n - 1) // 16])
    if n % 16:
        codes[1, :, last, :, n % 16:] = 0xFF
    codes[1, :, c.refs == 0] = 0x7F
    c.scales.view(torch.uint8)[1, :, c.refs == 0] = 255
    dirty = run_attn(T, c, 1, [0], [rows], [bits], n_q, 9)[1]
    others = [i for i in range(rows) if i != 3]
    assert torch.equal(clean[others], dirty[others])
    assert not torch.isfinite(dirty[3]).any()  # its keys make its scores NaN


@pytest.mark.parametrize("hd,rows,n_q", [(128, 6, 4), (64, 40, 4), (256, 9, 2), (128, 30, 16), (128, 12, 4)])
def test_values_that_are_nan_reach_those_who_see_them_in_their_columns(T, hd, rows, n_q):
    n = 150 + rows
    c = paged(T, [n], 2, hd, 16, 43)
    codes = c.data.view(torch.uint8)
    t = n - rows + 2
    codes[0, 1, int(c.table[0, t // 16]), 1, t % 16, 7] = 0xFF
    q, out, start = run_attn(T, c, 0, [0], [rows], None, n_q, 9)
    nan = torch.isnan(out[:rows].view(rows, n_q, hd))
    want = torch.zeros_like(nan)
    want[2:, n_q // 2:, 7] = True
    assert torch.equal(nan, want)


def test_attention_over_8_bits_reports_what_does_not_hold(T):
    c = paged(T, [40, 5], 2, 128, 16, 51)
    q = rand((8, 512), 1)
    for seqs, start, rows, zero, same in [([2], [0, 3], 4, range(0, 3), range(3, 8)), ([1], [0, 6], 8, range(0, 6), range(6, 8)),
                                          ([0], [5, 3], 4, [], range(8)), ([0], [2, 9], 8, [], range(8))]:
        ws = T.workspace(T.tf_tree_attn_workspace_bytes(c, 4, 1, rows))
        out = torch.full((8, 512), 5.0, dtype=torch.bfloat16, device="cuda")
        T.tf_tree_attn_run(q, c, 0, i32(seqs), i32(start), max_rows=rows, out=out, ws=ws)
        assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG, (seqs, start)
        assert (out[list(zero)] == 0).all() and (out[list(same)] == 5).all(), (seqs, start)
    c.table[0, 1] = 99  # a page out of range counts as zeros
    vals = Q.values(c)
    k, v = np.zeros((40, 2, 128)), np.zeros((40, 2, 128))
    for r in [*range(16), *range(32, 40)]:
        p = int(c.table[0, r // 16])
        k[r], v[r] = vals[0, 0, p, :, r % 16], vals[0, 1, p, :, r % 16]
    for rows in (1, 30):
        ws = T.workspace(T.tf_tree_attn_workspace_bytes(c, 8, 1, rows))
        q = rand((rows, 1024), 2)
        out = T.tf_tree_attn_run(q, c, 0, i32([0]), i32([0, rows]), max_rows=rows, ws=ws)
        assert T.tf_workspace_status(ws) == T.TF_E_INVALID_ARG
        ref, spread, size = Q.attn(R.f64(q).reshape(rows, 8, 128), k, v, seen(40, rows, chain(rows)), 128 ** -0.5,
                                      np.full((40, 2), 2.0 ** Q.exponents(c)[0, 1].max()))
        within(R.f64(out).reshape(rows, 8, 128), ref, Q.attn_tol(ref, spread, size))


def test_attention_over_8_bits_same_bits_in_a_graph_and_on_streams(T):
    c = paged(T, [3000, 70, 901], 2, 128, 16, 71)
    for rows, n_q in ((8, 4), (14, 16)):
        q, seqs, start = rand((14, n_q * 128), 3, 2.0), i32([0, 1, 2] if rows == 8 else [0]), i32([0, 8, 9, 14] if rows == 8 else [0, 14])
        B = seqs.numel()
        want = T.tf_tree_attn_run(q, c, 1, seqs, start, max_rows=rows)
        need = T.tf_tree_attn_workspace_bytes(c, n_q, B, rows)
        streams, wss = [torch.cuda.Stream() for _ in range(2)], [T.workspace(need) for _ in range(2)]
        outs = [[torch.empty_like(q) for _ in range(8)] for _ in range(2)]
        torch.cuda.synchronize()
        for n in range(8):
            for i in (0, 1):
                T.tf_tree_attn_run(q, c, 1, seqs, start, max_rows=rows, out=outs[i][n], ws=wss[i], stream=streams[i])
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for x in outs for o in x)
        ws, out = wss[0], torch.empty_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            T.tf_tree_attn_run(q, c, 1, seqs, start, max_rows=rows, out=out, ws=ws)
        for _ in range(3):
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        old = int(c.len[0])
        c.len[0] = 100
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, T.tf_tree_attn_run(q, c, 1, seqs, start, max_rows=rows))
        c.len[0] = old


@pytest.mark.parametrize("rows,n_q", [(3, 16), (40, 32)])
def test_8_bits_past_32_bit_offsets(T, rows, n_q):
    """5.4 GB of codes: the last layer's values start beyond 2^32 bytes."""
    c = T.KVCache.create(2, 8, 128, 16, 82000, 1, 60, dtype=E4M3)
    n = 700
    c.refs[:81956] = 1
    slots = T.tf_kvcache_extend(c, i32([0]), i32([0, n]), n)[0]
    at = torch.arange(n, device="cuda")
    assert torch.equal(slots, (81956 * 16 + at).int())
    kv = rand((n, (1 + 16) * 128), 7)
    T.tf_qk_norm_rope_run(kv, c, 1, at.int(), slots, T.RopeTable([]), n_q=1)
    x = R.f64(kv).reshape(n, 17, 128)
    # the 44 pages alone as a cache of their own: the same codes, the same attention
    small = T.KVCache.create(1, 8, 128, 16, 44, 1, 60, dtype=E4M3)
    T.tf_kvcache_extend(small, i32([0]), i32([0, n]), n)
    T.tf_qk_norm_rope_run(kv, small, 0, at.int(), slots - 81956 * 16, T.RopeTable([]), n_q=1)
    assert torch.equal(small.data[0].view(torch.uint8), c.data[1, :, 81956:].view(torch.uint8))
    assert torch.equal(small.scales[0].view(torch.uint8), c.scales[1, :, 81956:].view(torch.uint8))
    vals = Q.values(small)
    e = np.repeat(Q.exponents(small), 16, -1)
    for kv_ in (0, 1):
        got = tokens(small, vals, 0, kv_, 0)
        scale = 2.0 ** tokens(small, e[..., None].astype(float), 0, kv_, 0)
        ref = x[:, 1 + 8 * kv_:9 + 8 * kv_]
        within(got, ref, Q.E4M3_HALF * np.abs(ref) + scale * 2.0 ** -10)
    check_attn(T, small, 0, [0], [rows], None, n_q, 8)
    q, out, _ = run_attn(T, small, 0, [0], [rows], None, n_q, 8)
    assert torch.equal(out, run_attn(T, c, 1, [0], [rows], None, n_q, 8)[1])


# ---------------------------------------------------------------- page operations

@pytest.mark.parametrize("page,hd,n_kv,layers,seed", [(16, 64, 3, 2, 1), (32, 128, 2, 1, 2), (64, 256, 1, 3, 3), (128, 64, 5, 1, 4)])
def test_keep_moves_codes_to_their_new_blocks_scales(T, page, hd, n_kv, layers, seed):
    rng = np.random.default_rng(seed)
    rows = [64, 1, 20, 33, 7, 0, 16, 50]
    lens = [r + int(rng.integers(0, 70)) for r in rows]
    lens[4] = 7  # nothing before the block
    c = paged(T, lens, n_kv, hd, page, seed, layers=layers)
    start = np.cumsum([2] + rows).tolist()
    keep, n_keep, kept = [0] * (start[-1] + 1), [], []
    for b, r in enumerate(rows):
        k = sorted(rng.permutation(r)[:rng.integers(0, r + 1)].tolist())
        if b in (0, 3):
            k = list(range(min(3, r))) + [i for i in k if i >= 3]  # some stay in their places
        if b == 7:
            k = list(range(20, 50))  # the first row of every block it reaches moves in
        kept.append(k)
        n_keep.append(len(k))
        keep[start[b]:start[b] + len(k)] = k
    v0, e0, c0 = snapshot(c)
    e0 = np.clip(e0, Q.LEAST, Q.MOST)
    table = c.table.cpu().numpy().copy()
    ws = T.workspace(T.tf_kvcache_workspace_bytes(c))
    T.tf_kvcache_keep(c, i32(list(range(len(rows)))), i32(start), i32(keep), i32(n_keep), ws=ws)
    assert T.tf_workspace_status(ws) == T.TF_OK
    v1, e1, c1 = snapshot(c)
    assert c.len.tolist() == [n - r + k for n, r, k in zip(lens, rows, n_keep)]
    for b, k in enumerate(kept):
        base = lens[b] - rows[b]
        place = lambda i: (table[b, i // page], i % page)  # noqa: E731
        e = {}  # the model: block -> exponents [layers, 2, heads]
        for j, i in enumerate(k):
            if i != j:
                (p, r), (ps, rs) = place(base + j), place(base + i)
                was = e.get((p, r // 16), e0[:, :, p, :, r // 16] if r % 16 else None)
                theirs = e0[:, :, ps, :, rs // 16]
                e[p, r // 16] = theirs if was is None else np.maximum(was, theirs)
        for (p, blk), want in e.items():
            np.testing.assert_array_equal(e1[:, :, p, :, blk], want)
        for t in range(base + len(k)):
            (p, r), (ps, rs) = place(t), place(base + k[t - base] if t >= base else t)
            now, then = e1[:, :, p, :, r // 16], e0[:, :, ps, :, rs // 16]
            d = (then - now)[..., None]
            np.testing.assert_array_equal(c1[:, :, p, :, r], Q.e4m3(c0[:, :, ps, :, rs] * 2.0 ** d))
            assert (d <= 0).all()


def test_fork_copies_codes_and_scales(T):
    c = paged(T, [70, 33, 64, 5], 3, 64, 32, 6, spare=6)
    vals = Q.values(c)
    before = [[tokens(c, vals, l, kv, s) for s in range(4)] for l in range(2) for kv in range(2)]
    parent = [1, 0, 0, 0]
    T.tf_kvcache_fork(c, i32(parent))
    vals = Q.values(c)
    assert c.len.tolist() == [33, 70, 70, 70]
    for i in range(4):
        for s, p in enumerate(parent):
            np.testing.assert_array_equal(tokens(c, vals, i // 2, i % 2, s), before[i][p])
    # a token appended to one of the takers changes nobody else's values
    slots, pos = T.tf_kvcache_extend(c, i32([2]), i32([0, 1]), 1)
    T.tf_qk_norm_rope_run(rand((1, 7 * 64), 1, 500.0), c, 0, pos, slots, T.RopeTable([]), n_q=1)
    vals = Q.values(c)
    for i in range(4):
        for s in (0, 1, 3):
            np.testing.assert_array_equal(tokens(c, vals, i // 2, i % 2, s), before[i][parent[s]])


def test_reset_and_the_binding(T):
    c = paged(T, [70, 33], 2, 64, 16, 6)
    T.tf_kvcache_reset(c)
    assert c.len.tolist() == [0, 0] and int(c.refs.sum()) == 0 and (c.table == -1).all()
    data, scales = c.data, c.scales
    for d, s in [(data, None), (data.float().bfloat16(), scales), (data, scales.view(torch.uint8)), (data, scales[:1]), (data[:, :, ::2], scales)]:
        with pytest.raises(ValueError):
            T.KVCache(d, c.book, 2, c.max_pages, scales=s)
    with pytest.raises(T.TfqError):  # an odd number of scales, and no room for the word's end
        T.KVCache(data[:1, :, :1, :1].contiguous(), c.book, 2, 1, scales=scales[:1, :, :1, :1].clone().contiguous())


def test_one_workspace_for_calls_of_all_shapes(T):
    """The largest of them, over both kinds of cache: each finds it as the others left it."""
    cs = [paged(T, [4000, 900], 2, 64, 16, 77, dtype=dtype) for dtype in (E4M3, torch.bfloat16)]
    calls = [(c, rows) for c in cs for rows in (1, 16, 64, 5, 2)]
    need = max(T.tf_tree_attn_workspace_bytes(c, 16, 2, rows) for c, rows in calls)
    prompt_need = max(T.tf_prompt_attn_workspace_bytes(c, 16, 2) for c in cs)
    ws, prompt_ws = T.workspace(need), T.workspace(prompt_need)
    q = rand((128, 16 * 64), 79)

    def run(c, rows, w):
        return T.tf_tree_attn_run(q[: 2 * rows], c, 0, i32([0, 1]), i32([0, rows, 2 * rows]), max_rows=rows, ws=w)

    def prompt(c, w):
        return T.tf_prompt_attn_run(q, c, 0, i32([0, 1]), i32([0, 90, 128]), ws=w)

    want = [run(c, rows, T.workspace(need)) for c, rows in calls]
    want_prompt = [prompt(c, T.workspace(prompt_need)) for c in cs]
    for _ in range(2):
        for (c, rows), w in zip(calls, want):
            assert torch.equal(run(c, rows, ws), w)
        for c, w in zip(cs, want_prompt):
            assert torch.equal(prompt(c, prompt_ws), w)
    assert T.tf_workspace_status(ws) == T.TF_OK and T.tf_workspace_status(prompt_ws) == T.TF_OK
