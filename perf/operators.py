"""Operators of cached decoding, in their plain form and as the library's calls.

Four operators of the path around the packed projections: norms of queries and keys for each
head with the position rotation (keys and values go to the paged cache), attention of drafted
tokens over that cache, the cache's own page operations (fork with copying and freeing, and
compaction of the accepted drafts), and log probabilities of given tokens with entropy and
top alternatives.

The cache is one bf16 pool [layers, 2 (K, V), pages, kv heads, page rows, head dim] and one
int32 book: the lengths [seqs], the pages' reference counts [pages] and the page table
[seqs, max pages] (-1: none), in that order.
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
        dict(name="rope_one_token", op="rope", rows=1, n_q=16, n_kv=8, hd=128, rot=128, pairs=False, norm=True, page=16),
        # sixteen sequences' verify blocks of 8 rows
        dict(name="rope_blocks", op="rope", rows=128, n_q=16, n_kv=8, hd=128, rot=128, pairs=False, norm=True, page=32),
        # a long prompt's chunk, an odd number of rows
        dict(name="rope_prompt", op="rope", rows=8191, n_q=16, n_kv=8, hd=128, rot=128, pairs=False, norm=True, page=64),
        # one token of one sequence over a medium context: latency
        dict(name="attn_one_token", op="attn", B=1, T=1, L=4097, ragged=False, n_q=16, n_kv=8, hd=128, page=16, tree="chain"),
        # one sequence's verify block of 8 rows over a long context
        dict(name="attn_verify_long", op="attn", B=1, T=8, L=32771, ragged=False, n_q=16, n_kv=8, hd=128, page=64, tree="chain"),
        # a served batch: ragged contexts and blocks, drafts from several occurrences of the prompt
        dict(name="attn_batch_ragged", op="attn", B=64, T=8, L=8190, ragged=True, n_q=16, n_kv=8, hd=128, page=32, tree="lookup"),
        # wide trees of drafts and eight query heads to a key/value head: the arithmetic counts
        dict(name="attn_wide_tree", op="attn", B=8, T=64, L=16001, ragged=False, n_q=32, n_kv=4, hd=128, page=64, tree="wide"),
        # the accepted chains of 64 sequences' drafts moved up, in all 28 layers
        dict(name="keep_accepted", op="keep", B=64, chains=4, depth=7, L=100, layers=28, n_kv=8, hd=128, page=16),
        # a beam step: every slot takes its parent's pages, the unfilled ones copied, some slots end
        dict(name="fork_beams", op="fork", groups=4, width=8, L=500, layers=28, n_kv=8, hd=128, page=64),
        # one row of the readout's logits
        dict(name="logp_one_row", op="logp", rows=1, vocab=151936, f32=False, top=8, targets=1),
        # a verify block's logits in fp32, each row scored for several tokens
        dict(name="logp_block_f32", op="logp", rows=8, vocab=151936, f32=True, top=5, targets=4),
        # scoring a prompt: a thousand rows
        dict(name="logp_prompt", op="logp", rows=1000, vocab=151936, f32=False, top=20, targets=1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "keep", "fork", "logp"])
    if op == "rope":
        hd = rng.choice([64, 128, 128, 256])
        n_kv = rng.choice([1, 2, 4, 8])
        n_q = n_kv * rng.choice([1, 2, 4, 5])
        rows = _log_int(rng, 1, max(1, min(8191, 8191 * 4096 // (hd * (n_q + 2 * n_kv)))))
        return dict(op=op, rows=rows, n_q=n_q, n_kv=n_kv, hd=hd, rot=rng.choice([hd, hd, hd // 2]),
                    pairs=rng.random() < 0.3, norm=rng.random() < 0.8, page=rng.choice([16, 32, 64]))
    if op == "attn":
        n_kv = rng.choice([1, 2, 4, 8])
        n_q = n_kv * rng.choice([1, 2, 4, 8])
        hd = rng.choice([64, 128, 128])
        B, T = _log_int(rng, 1, 64), rng.choice([1, 1, 2, 5, 8, 16, 33, 64])
        # at most the bytes of the served batch and the arithmetic of the wide trees
        most = min(64 * 4096 * 8 // (B * n_kv), 8 * 64 * 16001 * 32 // (B * T * n_q))
        L = _log_int(rng, 1, max(1, min(40000, most)))
        return dict(op=op, B=B, T=T, L=L, ragged=rng.random() < 0.6, n_q=n_q, n_kv=n_kv, hd=hd,
                    page=rng.choice([16, 32, 64]), tree=rng.choice(["chain", "lookup", "wide"]))
    if op == "keep":
        return dict(op=op, B=_log_int(rng, 1, 64), chains=rng.choice([2, 3, 4, 8]), depth=rng.choice([1, 3, 7]),
                    L=_log_int(rng, 1, 100), layers=rng.choice([1, 7, 28]), n_kv=rng.choice([1, 4, 8]),
                    hd=rng.choice([64, 128]), page=rng.choice([16, 32]))
    if op == "fork":
        return dict(op=op, groups=rng.choice([1, 2, 4]), width=rng.choice([2, 3, 5, 8]), L=_log_int(rng, 1, 500),
                    layers=rng.choice([1, 7, 28]), n_kv=rng.choice([1, 4, 8]), hd=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64]))
    vocab = _log_int(rng, 100, 200000)
    f32 = rng.random() < 0.4
    rows = _log_int(rng, 1, max(1, min(4000, 1000 * 151936 // (vocab * (2 if f32 else 1)))))
    return dict(op=op, rows=rows, vocab=vocab, f32=f32, top=rng.choice([1, 4, 10, 20, 32]), targets=rng.choice([1, 1, 3]))


# ---------------------------------------------------------------- sizes that follow from a case

def _attn_sizes(c):
    """(context length, drafted rows) of each sequence."""
    B, L, T = c["B"], c["L"], c["T"]
    if not c["ragged"]:
        return [L] * B, [T] * B
    ctx = [1 + int((L - 1) * ((0.5 + b * 0.6180339887498949) % 1.0)) for b in range(B)]
    return ctx, [1 + (5 * b + T - 1) % T for b in range(B)]


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


def _keep_sizes(c):
    """(base length, kept rows, the chain that was accepted) of each sequence."""
    B = c["B"]
    base = [1 + int((c["L"] - 1) * ((0.5 + b * 0.6180339887498949) % 1.0)) for b in range(B)]
    return base, [1 + (3 * b + 2) % (c["depth"] + 1) for b in range(B)], [1 + b % (c["chains"] - 1) for b in range(B)]


def _fork_sizes(c):
    """(length, parent) of each slot: beams of a group take a beam of the group; every eleventh slot ends."""
    S = c["groups"] * c["width"]
    rng = random.Random(S * 1000 + c["L"])
    lens = [max(1, c["L"] - 7 * (s // c["width"])) for s in range(S)]
    parent = [s // c["width"] * c["width"] + rng.randrange(c["width"]) for s in range(S)]
    return lens, [-1 if s % 11 == 10 else p for s, p in enumerate(parent)]


def _fork_copies(c):
    """(slot, rows) of each copied page: the keeper of a parent's unfilled page is the parent where it keeps
    itself, else the lowest slot that takes it; the other takers get a copy."""
    lens, parent = _fork_sizes(c)
    seen, out = set(p for s, p in enumerate(parent) if p == s), []
    for s, p in enumerate(parent):
        if p < 0 or p == s or lens[p] % c["page"] == 0:
            continue
        if p in seen:
            out.append((s, lens[p] % c["page"]))
        seen.add(p)
    return out


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["rows"] * (c["n_q"] + 2 * c["n_kv"]) * c["hd"]
        return {"bytes": 4 * n, "flops": 6 * c["rows"] * (c["n_q"] + c["n_kv"]) * c["hd"]}
    if c["op"] == "attn":
        ctx, rows = _attn_sizes(c)
        kv = sum(x + t for x, t in zip(ctx, rows)) * c["n_kv"] * c["hd"] * 4
        return {"bytes": kv + sum(rows) * c["n_q"] * c["hd"] * 4,
                "flops": 4 * c["hd"] * c["n_q"] * sum(t * (x + t) for x, t in zip(ctx, rows))}
    if c["op"] == "keep":
        _, kept, _ = _keep_sizes(c)
        return {"bytes": 4 * sum(k - 1 for k in kept) * c["layers"] * 2 * c["n_kv"] * c["hd"] + 8 * c["B"], "flops": 0}
    if c["op"] == "fork":
        rows = sum(r for _, r in _fork_copies(c))
        lens, _ = _fork_sizes(c)
        table = sum(-(-n // c["page"]) for n in lens)
        return {"bytes": 4 * rows * c["layers"] * 2 * c["n_kv"] * c["hd"] + 8 * table, "flops": 0}
    n = c["rows"] * c["vocab"]
    return {"bytes": n * (4 if c["f32"] else 2) + c["rows"] * (8 + 8 * c["top"] + 8 * c["targets"]), "flops": 5 * n}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _randn(shape, g, scale=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, scale, generator=g)


def _cache(g, layers, n_pages, n_kv, page, hd, lens, table):
    """The pool, the book, and with `own` the library's handle over them."""
    pool = _randn((layers, 2, n_pages, n_kv, page, hd), g)
    refs = torch.bincount(table[table >= 0].long(), minlength=n_pages).int()
    book = torch.cat([lens, refs, table.reshape(-1)])
    handle = None
    if own:
        from skinny_gemm_bit_gb300 import tfq
        handle = tfq.KVCache(pool, book, n_seqs=lens.numel(), max_pages=table.shape[1])
    return pool, book, handle


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


def prepare(case, seed):
    c, g, s = case, _gen(seed), SimpleNamespace()
    s.op, s.c = c["op"], c
    if own:
        from skinny_gemm_bit_gb300 import tfq
    if s.op == "rope":
        M, n_q, n_kv, hd, page = c["rows"], c["n_q"], c["n_kv"], c["hd"], c["page"]
        s.qkv = _randn((M, (n_q + 2 * n_kv) * hd), g)
        s.q_gamma = (1 + _randn((hd,), g, 0.1, torch.float32)).bfloat16() if c["norm"] else None
        s.k_gamma = (1 + _randn((hd,), g, 0.1, torch.float32)).bfloat16() if c["norm"] else None
        # one stretch of a sequence: positions behind a context, rows scattered over the pool's pages
        ctx = 1 + (seed * 7919) % 20000
        s.positions = _i32([ctx]) + torch.arange(M, dtype=torch.int32, device=DEV)
        lens = _i32([M])
        table, n_pages = _private_table(g, [M], page, -(-M // page), 3)
        s.pool, _, s.cache = _cache(g, 2, n_pages, n_kv, page, hd, lens, table)
        row = torch.arange(M, device=DEV)
        s.slots = (table[0, row // page] * page + row % page).int()
        s.inv_freq = THETA ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / c["rot"])
        s.out = torch.empty((M, n_q * hd), dtype=torch.bfloat16, device=DEV)
        s.rope = tfq.RopeTable(s.inv_freq.cpu().numpy(), pairs=c["pairs"]) if own else None
        s.ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    elif s.op == "attn":
        ctx, rows = _attn_sizes(c)
        lens = [x + t for x, t in zip(ctx, rows)]
        max_pages = -(-(c["L"] + c["T"]) // c["page"]) + 5
        table, n_pages = _private_table(g, lens, c["page"], max_pages, 7)
        s.pool, s.book, s.cache = _cache(g, 2, n_pages, c["n_kv"], c["page"], c["hd"], _i32(lens), table)
        s.lens, s.table = _i32(lens), table
        s.seqs = torch.randperm(c["B"], generator=g, device=DEV).int()
        rows = [rows[b] for b in s.seqs.tolist()]
        s.q_start = _i32([0] + np.cumsum(rows).tolist())
        M = sum(rows)
        rng = random.Random(seed)
        s.masks = None
        if c["tree"] != "chain":
            bits = [m for r in rows for m in _tree_masks(c["tree"], r, rng)]
            s.masks = torch.from_numpy(np.array(bits, dtype=np.uint64).view(np.int64)).to(DEV)
        # queries twice as long as the keys: a few places stand out, as trained heads have it
        s.q = _randn((M, c["n_q"] * c["hd"]), g, 2.0)
        s.out = torch.empty_like(s.q)
        if own:
            s.ws = tfq.workspace(tfq.tf_tree_attn_workspace_bytes(s.cache, c["n_q"], c["B"], c["T"]))
    elif s.op == "keep":
        base, kept, chain = _keep_sizes(c)
        T = 1 + c["chains"] * c["depth"]
        lens = [b + T for b in base]
        table, n_pages = _private_table(g, lens, c["page"], -(-max(lens) // c["page"]) + 2, 16)
        s.pool, s.book, s.cache = _cache(g, c["layers"], n_pages, c["n_kv"], c["page"], c["hd"], _i32(lens), table)
        s.book0 = s.book.clone()
        s.n_seqs, s.max_pages = c["B"], table.shape[1]
        s.seqs = torch.arange(c["B"], dtype=torch.int32, device=DEV)
        s.q_start = torch.arange(c["B"] + 1, dtype=torch.int32, device=DEV) * T
        # the root and the first rows of one of the later chains: no row that moves is another's place
        keep = [[0] + [1 + ch * c["depth"] + j for j in range(c["depth"])] + [0] * (T - 1 - c["depth"]) for ch in chain]
        s.keep, s.n_keep = _i32(keep).reshape(-1), _i32(kept)
        s.T = T
        if own:
            s.ws = tfq.workspace(tfq.tf_kvcache_workspace_bytes(s.cache))
    elif s.op == "fork":
        lens, parent = _fork_sizes(c)
        S, page = len(lens), c["page"]
        pages = [-(-n // page) for n in lens]
        tail = [min(2, n) for n in pages]  # a group's beams share all pages but their last two
        max_pages = max(pages) + 3
        firsts = sum(pages[gr * c["width"]] - tail[gr * c["width"]] for gr in range(c["groups"]))
        n_pages = firsts + sum(tail) + S + 5
        order = torch.randperm(n_pages, generator=g, device=DEV).tolist()
        rows, shared = [], []
        for i in range(S):
            if i % c["width"] == 0:
                shared = [order.pop() for _ in range(pages[i] - tail[i])]
            mine = shared + [order.pop() for _ in range(tail[i])]
            rows.append(mine + [-1] * (max_pages - len(mine)))
        table = _i32(rows)
        s.pool, s.book, s.cache = _cache(g, c["layers"], n_pages, c["n_kv"], page, c["hd"], _i32(lens), table)
        s.book0 = s.book.clone()
        s.n_seqs, s.max_pages = S, max_pages
        s.parent = _i32(parent)
        if own:
            s.ws = tfq.workspace(tfq.tf_kvcache_workspace_bytes(s.cache))
    else:
        M, N = c["rows"], c["vocab"]
        # logits of spread 3 with a few tokens well above the rest, rounded as the readout stores them
        x = _randn((M, N), g, 3.0, torch.float32)
        hot = torch.randint(0, N, (M, 6), generator=g, device=DEV)
        x.scatter_add_(1, hot, _randn((M, 6), g, 4.0, torch.float32).abs() + 6.0)
        s.logits = x if c["f32"] else x.bfloat16()
        s.targets = torch.randint(0, N, (M, c["targets"]), generator=g, device=DEV).int()
        s.targets[:, 0] = hot[:, 0].int()
        s.logp = torch.empty((M, c["targets"]), dtype=torch.float32, device=DEV)
        s.entropy = torch.empty((M,), dtype=torch.float32, device=DEV)
        s.top_idx = torch.empty((M, c["top"]), dtype=torch.int32, device=DEV)
        s.top_logp = torch.empty((M, c["top"]), dtype=torch.float32, device=DEV)
        if own:
            s.ws = tfq.workspace(tfq.tf_logprobs_workspace_bytes(M, N, c["top"]))
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    if own:
        from skinny_gemm_bit_gb300 import tfq
        if s.op == "rope":
            tfq.tf_qk_norm_rope_run(s.qkv, s.cache, 1, s.positions, s.slots, s.rope, q_gamma=s.q_gamma,
                                    k_gamma=s.k_gamma, eps=EPS, out=s.out, ws=s.ws)
            return s.out, s.pool
        if s.op == "attn":
            return tfq.tf_tree_attn_run(s.q, s.cache, 1, s.seqs, s.q_start, masks=s.masks, max_rows=s.c["T"],
                                        out=s.out, ws=s.ws)
        if s.op == "keep":
            s.book.copy_(s.book0)  # the lengths and pages as they were when the drafts were made
            tfq.tf_kvcache_keep(s.cache, s.seqs, s.q_start, s.keep, s.n_keep, ws=s.ws)
            return s.book, s.pool
        if s.op == "fork":
            s.book.copy_(s.book0)
            tfq.tf_kvcache_fork(s.cache, s.parent, ws=s.ws)
            return s.book, s.pool
        return tfq.tf_logprobs_rows(s.logits, s.targets, s.c["top"], logp=s.logp, entropy=s.entropy,
                                    top_idx=s.top_idx, top_logp=s.top_logp, ws=s.ws)
    return {"rope": _plain_rope, "attn": _plain_attn, "keep": _plain_keep, "fork": _plain_fork, "logp": _plain_logp}[s.op](s)


# ---------------------------------------------------------------- plain forms

def _plain_norm(x, gamma):
    return x if gamma is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.float()


def _plain_rotate(x, cos, sin, rot, pairs):
    """x [M, heads, hd]; cos, sin [M, 1, rot / 2]."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., : rot // 2], x[..., rot // 2 : rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1), x[..., rot:]], -1)


def _plain_rope(s):
    c = s.c
    M, n_q, n_kv, hd, page = c["rows"], c["n_q"], c["n_kv"], c["hd"], c["page"]
    x = s.qkv.float().view(M, n_q + 2 * n_kv, hd)
    angle = s.positions.double()[:, None, None] * s.inv_freq
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _plain_rotate(_plain_norm(x[:, :n_q], s.q_gamma), cos, sin, c["rot"], c["pairs"])
    k = _plain_rotate(_plain_norm(x[:, n_q : n_q + n_kv], s.k_gamma), cos, sin, c["rot"], c["pairs"])
    at, off = (s.slots // page).long(), (s.slots % page).long()
    s.pool[1, 0, at, :, off] = k.bfloat16()
    s.pool[1, 1, at, :, off] = x[:, n_q + n_kv :].bfloat16()
    s.out.copy_(q.reshape(M, -1))
    return s.out, s.pool


def _plain_attn(s):
    c = s.c
    n_q, n_kv, hd, page, T, B = c["n_q"], c["n_kv"], c["hd"], c["page"], c["T"], c["B"]
    M, G = s.q.shape[0], n_q // n_kv
    lens = s.lens[s.seqs.long()].long()
    rows = (s.q_start[1:] - s.q_start[:-1]).long()
    base = lens - rows
    # every sequence's keys and values, gathered to the longest one's length
    pos = torch.arange(c["L"] + T, device=DEV)
    at = s.table[s.seqs.long()][:, pos // page].long().clamp(min=0)
    off = (pos % page)[None, :].expand_as(at)
    k = s.pool[1, 0][at, :, off].float()
    v = torch.where((pos[None, :] < lens[:, None])[:, :, None, None], s.pool[1, 1][at, :, off].float(), 0.0)
    # the queries, padded to T rows for each sequence
    t = torch.arange(T, device=DEV)
    row = (s.q_start[:-1, None] + t).clamp(max=M - 1).long()
    q = s.q.float().view(M, n_kv, G, hd)[row]
    mine = pos[None, :] - base[:, None]  # the drafted row at a place, if 0 <= mine < rows
    if s.masks is None:
        see = mine[:, None, :] <= t[None, :, None]
    else:
        see = ((s.masks[row][:, :, None] >> mine[:, None, :].clamp(0, 63)) & 1).bool()
    vis = (mine < 0)[:, None, :] | (see & (mine < rows[:, None])[:, None, :])
    p = torch.einsum("bthgd,blhd->bhtgl", q, k) * hd ** -0.5
    p = p.masked_fill_(~vis[:, None, :, None, :], -math.inf)
    m = p.amax(-1, keepdim=True)
    p = (p - torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1)
    o = torch.einsum("bhtgl,blhd->bhtgd", p, v) / torch.where(total > 0, total, 1.0)[..., None]
    b = torch.searchsorted(s.q_start, torch.arange(M, device=DEV, dtype=torch.int32), right=True) - 1
    mt = torch.arange(M, device=DEV) - s.q_start[b]
    s.out.copy_(o[b, :, mt].reshape(M, n_q * hd))
    return s.out


def _book(s):
    S, P = s.n_seqs, s.pool.shape[2]
    return s.book[:S], s.book[S : S + P], s.book[S + P :].view(S, s.max_pages)


def _plain_keep(s):
    page, B, T = s.c["page"], s.c["B"], s.T
    s.book.copy_(s.book0)
    lens, refs, table = _book(s)
    seqs = s.seqs.long()
    base = lens[seqs].long() - T
    j = torch.arange(T, device=DEV)
    kept = j[None, :] < s.n_keep[:, None]
    src = base[:, None] + torch.where(kept, s.keep.view(B, T).long(), j)
    dst = base[:, None] + j
    rows = s.pool[:, :, table[seqs[:, None], src // page].long(), :, src % page]
    s.pool[:, :, table[seqs[:, None], dst // page].long(), :, dst % page] = rows
    new = base + s.n_keep
    col = torch.arange(s.max_pages, device=DEV)[None, :]
    gone = (table[seqs] >= 0) & (col >= ((new + page - 1) // page)[:, None])
    refs.scatter_add_(0, table[seqs].clamp(min=0).long().reshape(-1), -gone.int().reshape(-1))
    table[seqs] = torch.where(gone, -1, table[seqs])
    lens[seqs] = new.int()
    return s.book, s.pool


def _plain_fork(s):
    page, S = s.c["page"], s.n_seqs
    s.book.copy_(s.book0)
    lens, refs, table = _book(s)
    me = torch.arange(S, device=DEV)
    parent, p = s.parent.long(), s.parent.long().clamp(min=0)
    changed, old = parent != me, table.clone()
    fill = lens[p] % page
    # who keeps a parent's unfilled page: the parent itself, else the lowest taker
    rank = torch.where(parent == me, -1, me)
    first = torch.full((S,), S, device=DEV).scatter_reduce_(0, p, torch.where(parent >= 0, rank, S), "amin")
    copy = changed & (parent >= 0) & (fill > 0) & (first[p] != me)
    free = torch.argsort((refs != 0).int(), stable=True)
    fresh = free[torch.cumsum(copy, 0) - 1].int()
    col = torch.arange(s.max_pages, device=DEV)[None, :]
    last = (lens[p] // page).long()[:, None]  # the column of an unfilled page
    new = torch.where((parent >= 0)[:, None], old[p], -1)
    new = torch.where(copy[:, None] & (col == last), fresh[:, None], new)
    for t, sign in ((old, -1), (new, 1)):
        live = changed[:, None] & (t >= 0)
        refs.scatter_add_(0, t.clamp(min=0).long().reshape(-1), sign * live.int().reshape(-1))
    # the copies; a slot without one writes a page that is in use onto itself
    idle = old[p, last[:, 0].clamp(max=s.max_pages - 1)]
    idle = torch.where(idle >= 0, idle, old.max()).long()
    src, dst = idle, torch.where(copy, fresh.long(), idle)
    mine = copy[:, None] & (torch.arange(page, device=DEV)[None, :] < fill[:, None])
    s.pool[:, :, dst] = torch.where(mine[:, None, :, None], s.pool[:, :, src], s.pool[:, :, dst])
    lens.copy_(torch.where(changed, torch.where(parent >= 0, lens[p], 0), lens))
    table.copy_(torch.where(changed[:, None], new, old))
    return s.book, s.pool


def _plain_logp(s):
    x = s.logits.float()
    val, idx = torch.sort(x, dim=-1, descending=True, stable=True)
    m = val[:, :1]
    z = x - m
    # the largest value's own 1 stays out of the sum: a sure row's entropy is all in the rest
    e = z.exp().scatter_(1, idx[:, :1], 0.0)
    rest = e.sum(-1, keepdim=True)
    log_total = torch.log1p(rest)
    s.entropy.copy_((log_total - (e * z).sum(-1, keepdim=True) / (1.0 + rest))[:, 0])
    s.logp.copy_(x.gather(1, s.targets.long()) - m - log_total)
    k = s.c["top"]
    s.top_idx.copy_(idx[:, :k])
    s.top_logp.copy_(val[:, :k] - m - log_total)
    return s.logp, s.entropy, s.top_idx, s.top_logp


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c, dev = case, DEV
    if s.op == "rope":
        hd, n_q, n_kv, rot, page = c["hd"], c["n_q"], c["n_kv"], c["rot"], c["page"]
        heads = s.qkv.double().view(c["rows"], -1, hd)
        pool = s.pool.double()
        phase = torch.outer(s.positions.double(), s.inv_freq)
        turn = torch.complex(phase.cos(), phase.sin())

        def head(x, gamma):
            if gamma is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / hd + EPS) * gamma.double()
            y = x.clone()
            one, two = (slice(0, rot, 2), slice(1, rot, 2)) if c["pairs"] else (slice(0, rot // 2), slice(rot // 2, rot))
            z = torch.complex(x[:, one].contiguous(), x[:, two].contiguous()) * turn
            y[:, one], y[:, two] = z.real, z.imag
            return y

        q = torch.cat([head(heads[:, h], s.q_gamma) for h in range(n_q)], 1)
        pages, offs = torch.div(s.slots, page, rounding_mode="floor").long(), torch.remainder(s.slots, page).long()
        for h in range(n_kv):
            pool[1, 0, pages, h, offs] = head(heads[:, n_q + h], s.k_gamma)
            pool[1, 1, pages, h, offs] = heads[:, n_q + n_kv + h]
        return q, pool
    if s.op == "attn":
        n_kv, hd, page = c["n_kv"], c["hd"], c["page"]
        G = c["n_q"] // n_kv
        out = torch.empty(s.q.shape, dtype=torch.float64, device=dev)
        starts, seqs, lens = s.q_start.tolist(), s.seqs.tolist(), s.lens.tolist()
        for b, seq in enumerate(seqs):
            lo, hi, n = starts[b], starts[b + 1], lens[seq]
            r = hi - lo
            pages = s.table[seq, : -(-n // page)].long()
            bits = [(1 << (i + 1)) - 1 for i in range(r)] if s.masks is None else [int(v) for v in s.masks[lo:hi].tolist()]
            seen = torch.tensor([[v >> j & 1 for j in range(r)] for v in bits], dtype=torch.bool, device=dev)
            seen = torch.cat([torch.ones((r, n - r), dtype=torch.bool, device=dev), seen], 1)
            for h in range(n_kv):
                kk = s.pool[1, 0, pages, h].reshape(-1, hd)[:n].double()
                vv = s.pool[1, 1, pages, h].reshape(-1, hd)[:n].double()
                qq = s.q[lo:hi, h * G * hd : (h + 1) * G * hd].double().reshape(r * G, hd)
                w = (qq @ kk.T) / math.sqrt(hd)
                w[~seen.repeat_interleave(G, 0)] = -math.inf
                out[lo:hi, h * G * hd : (h + 1) * G * hd] = (torch.softmax(w, -1) @ vv).reshape(r, G * hd)
        return out
    if s.op == "keep":
        page, T = c["page"], s.T
        lens, refs, table = (t.clone() for t in _book(s))
        lens, refs, table = lens.tolist(), refs.tolist(), table.tolist()
        pool = s.pool.clone()
        keep, n_keep = s.keep.view(-1, T).tolist(), s.n_keep.tolist()
        for b in range(c["B"]):
            base = lens[b] - T
            for j in range(n_keep[b]):
                a, z = base + keep[b][j], base + j
                pool[:, :, table[b][z // page], :, z % page] = s.pool[:, :, table[b][a // page], :, a % page]
            for i in range(-(-(base + n_keep[b]) // page), -(-lens[b] // page)):
                refs[table[b][i]] -= 1
                table[b][i] = -1
            lens[b] = base + n_keep[b]
        return torch.tensor(lens + refs + [p for r in table for p in r], dtype=torch.int32, device=dev), pool.float()
    if s.op == "fork":
        page = c["page"]
        lens, refs, table = (t.tolist() for t in _book(s))
        parent = s.parent.tolist()
        pool = s.pool.clone()
        free = iter([i for i, r in enumerate(refs) if r == 0])
        new_lens, new_table, left = list(lens), [list(r) for r in table], list(refs)
        copies = dict(_fork_copies(c))
        for i, p in enumerate(parent):
            if p == i:
                continue
            for a in table[i]:
                if a >= 0:
                    left[a] -= 1
            new_lens[i], new_table[i] = (0, [-1] * s.max_pages) if p < 0 else (lens[p], list(table[p]))
            if i in copies:
                k, to = lens[p] // page, next(free)
                pool[:, :, to, :, : copies[i]] = s.pool[:, :, table[p][k], :, : copies[i]]
                new_table[i][k] = to
            for a in new_table[i]:
                if a >= 0:
                    left[a] += 1
        return torch.tensor(new_lens + left + [p for r in new_table for p in r], dtype=torch.int32, device=dev), pool.float()
    x = s.logits.double()
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[:, None])
    ent = -(p * (x - lse[:, None])).sum(-1)  # 2^-53 of a logit: far inside a sure row's entropy
    logp = x.gather(1, s.targets.long()) - lse[:, None]
    # one whole number for each value that orders by value, then by the lower place
    i = s.logits.float().view(torch.int32).long()
    order = torch.where(i < 0, -(i & 0x7FFFFFFF), i) * (1 << 20) + ((1 << 20) - 1 - torch.arange(c["vocab"], device=dev))
    best = torch.topk(order, c["top"], dim=-1).indices
    return logp, ent, best.int(), x.gather(1, best) - lse[:, None]
