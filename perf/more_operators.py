"""Operators of serving from an 8-bit cache, in their plain form and as the library's calls.

Three operators: norms of queries and keys with the position rotation, whose keys and values are
appended to a paged cache of 8-bit codes; attention of drafted tokens over that cache; and causal
attention of whole prompts (or chunks of them) of different lengths over the cache, held in 8 bits
or in bf16.

The 8-bit cache is a pool of e4m3 codes [layers, 2 (K, V), pages, kv heads, page rows, head dim] and
of one power of two (e8m0) for each 16 rows of a page and head [layers, 2, pages, kv heads,
page rows / 16]; a value is code * scale. A block's scale is the least with which its largest
finite value is at most 448, kept within 2^-32 .. 2^32. Rows that join a block which holds others
raise its scale where they have to, and the others are rounded to the new one; a call that stores a
block's first row begins it anew.
"""
import math
import random
from types import SimpleNamespace

import numpy as np
import torch

own = False
DEV = "cuda"

THETA = 1e6
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token of the 28-layer decoder step's heads (16 query, 8 key/value, 128 wide): latency
        dict(name="append8_one_token", op="append8", B=1, T=1, L=4099, n_q=16, n_kv=8, hd=128, rot=128, pairs=False, norm=True, page=16),
        # a served batch, one token to each of 64 sequences of different lengths
        dict(name="append8_batch", op="append8", B=64, T=1, L=8003, n_q=16, n_kv=8, hd=128, rot=128, pairs=False, norm=True, page=64),
        # a long prompt's chunk behind a context, an odd number of rows, beginning inside a block
        dict(name="append8_prompt", op="append8", B=1, T=8191, L=1003, n_q=16, n_kv=8, hd=128, rot=128, pairs=False, norm=True, page=64),
        # one token of one sequence over a medium context: latency
        dict(name="attn8_one_token", op="attn8", B=1, T=1, L=4097, ragged=False, n_q=16, n_kv=8, hd=128, page=16, tree="chain"),
        # one sequence's verify block of 8 rows over a long context
        dict(name="attn8_verify_long", op="attn8", B=1, T=8, L=32771, ragged=False, n_q=16, n_kv=8, hd=128, page=64, tree="chain"),
        # a served batch: ragged contexts and blocks, drafts from several occurrences of the prompt
        dict(name="attn8_batch_ragged", op="attn8", B=64, T=8, L=8190, ragged=True, n_q=16, n_kv=8, hd=128, page=32, tree="lookup"),
        # wide trees of drafts and eight query heads to a key/value head: the arithmetic counts
        dict(name="attn8_wide_tree", op="attn8", B=8, T=64, L=16001, ragged=False, n_q=32, n_kv=4, hd=128, page=64, tree="wide"),
        # one short prompt, bf16 cache: latency
        dict(name="prompt_short", op="prompt", B=1, T=333, L=0, n_q=16, n_kv=8, hd=128, page=16, bits=16),
        # prompts of different lengths served together, bf16 cache
        dict(name="prompt_packed", op="prompt", B=24, T=2047, L=0, n_q=16, n_kv=8, hd=128, page=32, bits=16),
        # one long prompt, bf16 cache: the arithmetic
        dict(name="prompt_long", op="prompt", B=1, T=8191, L=0, n_q=16, n_kv=8, hd=128, page=64, bits=16),
        # the next chunk of a long document over an 8-bit cache, eight query heads to a key/value head
        dict(name="prompt_chunk8", op="prompt", B=1, T=1500, L=14001, n_q=32, n_kv=4, hd=128, page=64, bits=8),
        # chunks of several documents over an 8-bit cache, heads of 64
        dict(name="prompt_packed8", op="prompt", B=8, T=1001, L=3001, n_q=16, n_kv=4, hd=64, page=32, bits=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append8", "attn8", "prompt"])
    n_kv = rng.choice([1, 2, 4, 8])
    if op == "append8":
        hd = rng.choice([64, 128, 128, 256])
        n_q = n_kv * rng.choice([1, 2, 4, 5])
        B = _log_int(rng, 1, 64)
        T = _log_int(rng, 1, max(1, min(8191, 8191 * 4096 // (B * hd * (n_q + 2 * n_kv)))))
        return dict(op=op, B=B, T=T, L=_log_int(rng, 1, 20000), n_q=n_q, n_kv=n_kv, hd=hd, rot=rng.choice([hd, hd, hd // 2]),
                    pairs=rng.random() < 0.3, norm=rng.random() < 0.8, page=rng.choice([16, 32, 64, 128]))
    if op == "attn8":
        n_q = n_kv * rng.choice([1, 2, 4, 8])
        hd = rng.choice([64, 128, 128])
        B, T = _log_int(rng, 1, 64), rng.choice([1, 1, 2, 5, 8, 16, 33, 64])
        # at most the bytes of the served batch and the arithmetic of the wide trees
        most = min(64 * 4096 * 8 // (B * n_kv), 8 * 64 * 16001 * 32 // (B * T * n_q))
        L = _log_int(rng, 1, max(1, min(40000, most)))
        return dict(op=op, B=B, T=T, L=L, ragged=rng.random() < 0.6, n_q=n_q, n_kv=n_kv, hd=hd,
                    page=rng.choice([16, 32, 64]), tree=rng.choice(["chain", "lookup", "wide"]))
    n_q = n_kv * rng.choice([1, 2, 3, 4, 8])
    B, L = _log_int(rng, 1, 32), rng.choice([0, 0, _log_int(rng, 1, 16000)])
    # at most the scores of the long prompt
    scores = 8191 * 8191 * 16 // (B * n_q)
    T = _log_int(rng, 1, max(1, min(8191, int((math.sqrt(L * L + 4 * scores) - L) / 2))))
    return dict(op=op, B=B, T=T, L=L, n_q=n_q, n_kv=n_kv, hd=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64]),
                bits=rng.choice([8, 16]))


# ---------------------------------------------------------------- sizes that follow from a case

def _spread(b):
    """Places that fill (0, 1) evenly, 0.5 the first."""
    return (0.5 + b * 0.6180339887498949) % 1.0


def _sizes(c):
    """(context length, rows) of each sequence."""
    B, L, T = c["B"], c["L"], c["T"]
    if c["op"] == "attn8":
        if not c["ragged"]:
            return [L] * B, [T] * B
        return [1 + int((L - 1) * _spread(b)) for b in range(B)], [1 + (5 * b + T - 1) % T for b in range(B)]
    if B == 1:
        return [L], [T]
    return [int(L * _spread(b)) for b in range(B)], [1 + int((T - 1) * _spread(3 * b + 1)) for b in range(B)]


def _tree_masks(kind, rows, rng):
    """Each drafted row's visible drafted rows, as bits: its ancestors and itself."""
    masks = []
    for i in range(rows):
        if kind == "lookup":  # a root and chains of 3 behind it, as proposed from several places of a prompt
            parent = -1 if i == 0 else (0 if (i - 1) % 3 == 0 else i - 1)
        else:  # "wide": each row behind a random earlier one
            parent = -1 if i == 0 else rng.randrange(i)
        masks.append((1 << i) | (masks[parent] if parent >= 0 else 0))
    return masks


def work(case):
    c = case
    ctx, rows = _sizes(c)
    n, hd, n_q, n_kv = sum(rows), c["hd"], c["n_q"], c["n_kv"]
    if c["op"] == "append8":
        blocks = sum((x + t + 15) // 16 - x // 16 for x, t in zip(ctx, rows))
        return {"bytes": n * hd * (4 * n_q + 6 * n_kv) + blocks * 2 * n_kv + 8 * n, "flops": 6 * n * (n_q + n_kv) * hd}
    tokens = sum(x + t for x, t in zip(ctx, rows))
    row = hd * 2 if c["op"] == "prompt" and c["bits"] == 16 else hd + 1 / 16
    pairs = sum(t * (x + t) if c["op"] == "attn8" else t * x + t * (t + 1) // 2 for x, t in zip(ctx, rows))
    return {"bytes": tokens * 2 * n_kv * row + n * n_q * hd * 4, "flops": 4 * hd * n_q * pairs}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _randn(shape, g, scale=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, scale, generator=g)


def _least_exponent(most):
    """The least e with most <= 448 * 2^e, within -32 .. 32."""
    bits = most.float().view(torch.int32)
    return ((bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(-32, 32)


def _two_to(e):
    return ((e.int() + 127) << 23).view(torch.float32)


def _pool8(g, n_pages, n_kv, page, hd):
    """Codes and scale bytes of random values, one layer at a time; layer 1 is the one in use."""
    codes = torch.empty((2, 2, n_pages, n_kv, page, hd), dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty((2, 2, n_pages, n_kv, page // 16), dtype=torch.uint8, device=DEV)
    for at in ((0, 0), (0, 1), (1, 0), (1, 1)):
        x = _randn((n_pages, n_kv, page // 16, 16, hd), g)
        # heads of different size, as trained ones are
        x *= torch.exp2(torch.arange(n_kv, device=DEV) % 5 - 2)[None, :, None, None, None].bfloat16()
        e = _least_exponent(x.abs().amax((-1, -2)))
        codes[at] = (x.float() * _two_to(-e)[..., None, None]).to(torch.float8_e4m3fn).view(n_pages, n_kv, page, hd)
        scales[at] = (e + 127).to(torch.uint8)
    return codes, scales.view(torch.float8_e8m0fnu)


def _private_table(g, lens, page, max_pages, spare):
    """A table in which every sequence has pages of its own, scattered over the pool."""
    need = [-(-int(n) // page) for n in lens]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g, device=DEV).int()
    at = torch.arange(max_pages, device=DEV)[None, :]
    need_t = torch.tensor(need, device=DEV)[:, None]
    first = torch.cumsum(need_t, 0) - need_t
    table = torch.where(at < need_t, order[(first + at).clamp(max=n_pages - 1)], -1).int()
    return table, n_pages


def _book(lens, table, n_pages):
    return torch.cat([lens, torch.bincount(table[table >= 0].long(), minlength=n_pages).int(), table.reshape(-1)])


def prepare(case, seed):
    c, g, s = case, _gen(seed), SimpleNamespace()
    s.op, s.c = c["op"], c
    B, n_q, n_kv, hd, page = c["B"], c["n_q"], c["n_kv"], c["hd"], c["page"]
    ctx, rows = _sizes(c)
    M = sum(rows)
    if s.op == "append8":
        # the pages that the rows go to, the one with the context's end among them: what lies before is not touched
        held = [x % page for x in ctx]
        lens = [h + t for h, t in zip(held, rows)]
        table, n_pages = _private_table(g, lens, page, -(-max(lens) // page), 3)
        s.codes, s.scales = _pool8(g, n_pages, n_kv, page, hd)
        s.book = _book(_i32(lens), table, n_pages)
        at = torch.cat([torch.arange(h, n, device=DEV) for h, n in zip(held, lens)])
        b = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(rows, device=DEV))
        s.slots = (table[b, at // page] * page + at % page).int()
        s.positions = (at + _i32([x - h for x, h in zip(ctx, held)])[b]).int()
        s.qkv = _randn((M, (n_q + 2 * n_kv) * hd), g)
        s.q_gamma = (1 + _randn((hd,), g, 0.1, torch.float32)).bfloat16() if c["norm"] else None
        s.k_gamma = (1 + _randn((hd,), g, 0.1, torch.float32)).bfloat16() if c["norm"] else None
        s.inv_freq = THETA ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / c["rot"])
        s.out = torch.empty((M, n_q * hd), dtype=torch.bfloat16, device=DEV)
    else:
        lens = [x + t for x, t in zip(ctx, rows)]
        table, n_pages = _private_table(g, lens, page, -(-max(lens) // page) + 5, 7)
        if s.op == "prompt" and c["bits"] == 16:
            s.codes, s.scales = _randn((2, 2, n_pages, n_kv, page, hd), g), None
        else:
            s.codes, s.scales = _pool8(g, n_pages, n_kv, page, hd)
        s.book = _book(_i32(lens), table, n_pages)
        s.lens, s.table, s.most_rows, s.most_len = _i32(lens), table, max(rows), max(lens)
        s.seqs = torch.randperm(B, generator=g, device=DEV).int()
        rows = [rows[b] for b in s.seqs.tolist()]
        s.q_start = _i32([0] + np.cumsum(rows).tolist())
        s.masks = None
        if s.op == "attn8" and c["tree"] != "chain":
            rng = random.Random(seed)
            bits = [m for r in rows for m in _tree_masks(c["tree"], r, rng)]
            s.masks = torch.from_numpy(np.array(bits, dtype=np.uint64).view(np.int64)).to(DEV)
        # queries longer than the keys: a few places stand out, as trained heads have it
        s.q = _randn((M, n_q * hd), g, 2.0)
        s.out = torch.empty_like(s.q)
    if own:
        from skinny_gemm_bit_gb300 import tfq
        s.cache = tfq.KVCache(s.codes, s.book, n_seqs=B, max_pages=table.shape[1], scales=s.scales)
        if s.op == "append8":
            s.rope = tfq.RopeTable(s.inv_freq.cpu().numpy(), pairs=c["pairs"])
            s.ws = tfq.workspace(256)
        elif s.op == "attn8":
            s.ws = tfq.workspace(tfq.tf_tree_attn_workspace_bytes(s.cache, n_q, B, c["T"]))
        else:
            s.ws = tfq.workspace(tfq.tf_prompt_attn_workspace_bytes(s.cache, n_q, B))
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    if own:
        from skinny_gemm_bit_gb300 import tfq
        if s.op == "append8":
            tfq.tf_qk_norm_rope_run(s.qkv, s.cache, 1, s.positions, s.slots, s.rope, q_gamma=s.q_gamma,
                                    k_gamma=s.k_gamma, eps=EPS, out=s.out, ws=s.ws)
            return s.out, s.codes, s.scales
        if s.op == "attn8":
            return tfq.tf_tree_attn_run(s.q, s.cache, 1, s.seqs, s.q_start, masks=s.masks, max_rows=s.c["T"],
                                        out=s.out, ws=s.ws)
        return tfq.tf_prompt_attn_run(s.q, s.cache, 1, s.seqs, s.q_start, out=s.out, ws=s.ws)
    return _plain_append8(s) if s.op == "append8" else _plain_attn(s)


# ---------------------------------------------------------------- plain forms

def _plain_norm(x, gamma):
    return x if gamma is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.float()


def _plain_rotate(x, cos, sin, rot, pairs):
    """x [M, heads, hd]; cos, sin [M, 1, rot / 2]."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., : rot // 2], x[..., rot // 2 : rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1), x[..., rot:]], -1)


def _plain_store(codes, scales, x, block, row):
    """Rows x [M, heads, hd] to the rows `row` of the blocks `block` of codes [blocks, heads, 16, hd] and scales [blocks, heads]."""
    n, heads = scales.shape
    most = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    most = torch.zeros((n, heads), device=DEV).index_reduce_(0, block, most, "amax")
    e = _least_exponent(most)
    was = scales.int().sub(127).clamp(-32, 32)
    hit = torch.zeros(n, dtype=torch.bool, device=DEV).index_fill_(0, block, True)
    anew = torch.zeros(n, dtype=torch.bool, device=DEV).index_fill_(0, block[row == 0], True)
    e = torch.where(anew[:, None], e, torch.maximum(e, was))
    kept = (codes.float() * _two_to(was - e)[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    codes.copy_(torch.where((hit & ~anew)[:, None, None, None], kept.view(torch.uint8), codes.view(torch.uint8)).view(torch.float8_e4m3fn))
    scales.copy_(torch.where(hit[:, None], (e + 127).to(torch.uint8), scales))
    codes[block, :, row] = (x * _two_to(-e)[block][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes, scales


def _plain_append8(s):
    c = s.c
    n_q, n_kv, hd, page = c["n_q"], c["n_kv"], c["hd"], c["page"]
    M = s.qkv.shape[0]
    x = s.qkv.float().view(M, n_q + 2 * n_kv, hd)
    angle = s.positions.double()[:, None, None] * s.inv_freq
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _plain_rotate(_plain_norm(x[:, :n_q], s.q_gamma), cos, sin, c["rot"], c["pairs"])
    k = _plain_rotate(_plain_norm(x[:, n_q : n_q + n_kv], s.k_gamma), cos, sin, c["rot"], c["pairs"])
    block, row = (s.slots // 16).long(), (s.slots % 16).long()
    pages = s.codes.shape[2]
    codes, scales = s.codes[1].view(2, pages, n_kv, page // 16, 16, hd), s.scales[1].view(torch.uint8)
    # the pool by blocks: [2, pages * blocks of a page, heads, 16, hd]
    codes, scales = codes.transpose(2, 3).flatten(1, 2), scales.transpose(2, 3).flatten(1, 2)
    kc, ks = _plain_store(codes[0], scales[0], k, block, row)
    vc, vs = _plain_store(codes[1], scales[1], x[:, n_q + n_kv :], block, row)
    s.codes[1].copy_(torch.stack([kc, vc]).view(2, pages, page // 16, n_kv, 16, hd).transpose(2, 3).reshape(2, pages, n_kv, page, hd))
    s.scales[1].view(torch.uint8).copy_(torch.stack([ks, vs]).view(2, pages, page // 16, n_kv).transpose(2, 3))
    s.out.copy_(q.reshape(M, -1))
    return s.out, s.codes, s.scales


def _plain_rows(s, kv, at, off):
    """The keys or values at pages `at`, rows `off` of them, in fp32: [B, tokens, heads, hd]."""
    x = s.codes[1, kv][at, :, off].float()
    if s.scales is None:
        return x
    e = s.scales[1, kv].view(torch.uint8)[at, :, off // 16].int() - 127
    return x * _two_to(e)[..., None]


def _plain_attn(s):
    c = s.c
    n_q, n_kv, hd, page = c["n_q"], c["n_kv"], c["hd"], c["page"]
    M, G = s.q.shape[0], n_q // n_kv
    lens = s.lens[s.seqs.long()].long()
    rows = (s.q_start[1:] - s.q_start[:-1]).long()
    base = lens - rows
    # every sequence's keys and values, gathered to the longest one's length
    pos = torch.arange(s.most_len, device=DEV)
    at = s.table[s.seqs.long()][:, pos // page].long().clamp(min=0)
    off = (pos % page)[None, :].expand_as(at)
    k = _plain_rows(s, 0, at, off)
    v = torch.where((pos[None, :] < lens[:, None])[:, :, None, None], _plain_rows(s, 1, at, off), 0.0)
    # the queries, padded to the most rows of a sequence
    t = torch.arange(s.most_rows, device=DEV)
    row = (s.q_start[:-1, None] + t).clamp(max=M - 1).long()
    q = s.q.float().view(M, n_kv, G, hd)[row]
    mine = pos[None, :] - base[:, None]  # the sequence's own row at a place, if 0 <= mine < rows
    if s.masks is None:
        see = mine[:, None, :] <= t[None, :, None]
    else:
        see = ((s.masks[row][:, :, None] >> mine[:, None, :].clamp(0, 63)) & 1).bool()
    vis = (mine < 0)[:, None, :] | (see & (mine < rows[:, None])[:, None, :])
    p = torch.einsum("bthgd,blhd->bhtgl", q, k).mul_(hd ** -0.5)
    p = p.masked_fill_(~vis[:, None, :, None, :], -math.inf)
    m = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1)
    o = torch.einsum("bhtgl,blhd->bhtgd", p, v) / torch.where(total > 0, total, 1.0)[..., None]
    b = torch.searchsorted(s.q_start, torch.arange(M, device=DEV, dtype=torch.int32), right=True) - 1
    mt = torch.arange(M, device=DEV) - s.q_start[b]
    s.out.copy_(o[b, :, mt].reshape(M, n_q * hd))
    return s.out


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    n_q, n_kv, hd, page = c["n_q"], c["n_kv"], c["hd"], c["page"]
    G = n_q // n_kv
    scale_of = lambda byte: 2.0 ** (byte.double() - 127)  # noqa: E731
    if s.op != "append8":
        out = torch.empty(s.q.shape, dtype=torch.float64, device=DEV)
        starts, seqs, lens = s.q_start.tolist(), s.seqs.tolist(), s.lens.tolist()
        for b, seq in enumerate(seqs):
            lo, hi, n = starts[b], starts[b + 1], lens[seq]
            r = hi - lo
            pages = s.table[seq, : -(-n // page)].long()
            if s.masks is None:
                seen = torch.ones((r, r), dtype=torch.bool, device=DEV).tril()
            else:
                bits = s.masks[lo:hi].tolist()
                seen = torch.tensor([[v >> j & 1 for j in range(r)] for v in bits], dtype=torch.bool, device=DEV)
            seen = torch.cat([torch.ones((r, n - r), dtype=torch.bool, device=DEV), seen], 1)
            for h in range(n_kv):
                kv = []
                for i in range(2):
                    x = s.codes[1, i, pages, h].double()
                    if s.scales is not None:
                        x = x.view(len(pages), page // 16, 16, hd) * scale_of(s.scales[1, i, pages, h].view(torch.uint8))[..., None, None]
                    kv.append(x.reshape(-1, hd)[:n])
                for gr in range(G):  # a head at a time, for the memory's sake
                    at = slice((h * G + gr) * hd, (h * G + gr + 1) * hd)
                    w = (s.q[lo:hi, at].double() @ kv[0].T) / math.sqrt(hd)
                    w[~seen] = -math.inf
                    out[lo:hi, at] = torch.softmax(w, -1) @ kv[1]
        return out
    x = s.qkv.double().view(-1, n_q + 2 * n_kv, hd)
    q, k, v = x[:, :n_q], x[:, n_q : n_q + n_kv], x[:, n_q + n_kv :]
    turned = []
    for y, gamma in ((q, s.q_gamma), (k, s.k_gamma)):
        if gamma is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / hd + EPS).sqrt() * gamma.double()
        i = torch.arange(c["rot"] // 2, device=DEV)
        a, b = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + c["rot"] // 2)
        w = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s.positions.double()[:, None] * s.inv_freq)[:, None]
        z = torch.complex(y[..., a], y[..., b]) * w
        y = y.clone()
        y[..., a], y[..., b] = z.real, z.imag
        turned.append(y)
    codes, scales = s.codes.cpu().float().numpy().astype(np.float64), s.scales.view(torch.uint8).cpu().numpy().astype(np.int64) - 127
    slots = s.slots.cpu().numpy()
    for i, y in enumerate((turned[1], v)):
        y = y.cpu().numpy()
        m = 0
        while m < len(slots):  # the rows of one block
            p, r0 = slots[m] // page, slots[m] % page
            blk, end = r0 // 16, m + 1
            while end < len(slots) and slots[end] // 16 == slots[m] // 16:
                end += 1
            most = np.abs(y[m:end]).max((0, 2))
            e = np.clip(np.ceil(np.log2(np.maximum(most, 1e-300) / 448)), -32, 32).astype(np.int64)
            held = codes[1, i, p, :, blk * 16 : blk * 16 + 16]  # a view
            if r0 % 16:
                was = scales[1, i, p, :, blk]
                e = np.maximum(e, was)
                held[:] = _nearest_e4m3(held * 2.0 ** (was - e)[:, None, None])
            held[:, r0 % 16 : r0 % 16 + end - m] = _nearest_e4m3(y[m:end].transpose(1, 0, 2) * 2.0 ** -e[:, None, None])
            scales[1, i, p, :, blk] = e
            m = end
    return turned[0].reshape(len(slots), -1), torch.from_numpy(codes), torch.from_numpy(2.0 ** scales)


def _nearest_e4m3(x):
    """The nearest number with three bits behind the first and exponents -6 .. 8, ties to the even one."""
    step = 2.0 ** (np.clip(np.frexp(x)[1] - 1, -6, 8) - 3)
    return np.clip(np.rint(x / step) * step, -448, 448)
