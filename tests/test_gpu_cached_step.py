"""The decoder step over a paged cache, and the cached-decoding operators in a run as they are used:
room is made, a step runs, tokens are scored, the accepted drafts are kept."""
import numpy as np
import pytest
import torch

from parity import dev_bf16, pack
from skinny_gemm_bit_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    from skinny_gemm_bit_gb300 import build
    build.build()
    from skinny_gemm_bit_gb300 import tfq
    return tfq


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def mask_tensor(bits):
    return torch.from_numpy(np.array(bits, dtype=np.uint64).view(np.int64)).cuda()


class Model:
    def __init__(self, T, seed, n_layers, d_model, d_ff, n_q, n_kv, hd, vocab, bits=4, code="mlx", norms=True, pairs=False):
        cfg = synth.decoder(seed=seed, n_layers=n_layers, d_model=d_model, d_ff=d_ff, n_q_heads=n_q, n_kv_heads=n_kv,
                            head_dim=hd, vocab=vocab, M=8, bits=bits, code=code)
        pk = (lambda w: T.tf_qlinear_pack_nvfp4(w["codes"], w["scales"], float(w["gscale"]))) if code == "nvfp4" else \
            (lambda w: pack(T, w))
        layers = [{k: (dev_bf16(v) if k.endswith("norm") else pk(v)) for k, v in L.items()} for L in cfg["layers"]]
        self.dec = T.Decoder(layers, dev_bf16(cfg["final_norm"]), pk(cfg["readout"]), d_model, d_ff, n_q * hd, n_kv * hd,
                             cfg["eps"])
        g = torch.Generator(device="cuda").manual_seed(seed)
        gam = lambda: (1 + 0.1 * torch.randn(hd, generator=g, device="cuda")).bfloat16()  # noqa: E731
        self.rope = T.RopeTable(1e4 ** (-np.arange(0, hd, 2) / hd), pairs=pairs)
        self.attn = T.Attention([(gam(), gam()) if norms else (None, None) for _ in range(n_layers)], n_q, hd, self.rope)
        self.dims = (n_layers, n_kv, hd)
        self.x = dev_bf16(cfg["x"])
        self.vocab = vocab

    def cache(self, T, page, n_pages, n_seqs, max_pages):
        return T.KVCache.create(*self.dims, page, n_pages, n_seqs, max_pages)

    def embed(self, T, tokens):
        return T.tf_embed_rows(self.dec.readout, tokens)

    def separately(self, T, c, x, seqs, q_start, slots, positions, masks):
        """The step as the separate calls a user would make."""
        h, a = x, self.attn
        for l, L in enumerate(self.dec.layers):
            qkv = T.tf_qlinear_run(L["qkv"], h, gamma=L["attn_norm"], eps=self.dec.desc.eps)
            q = T.tf_qk_norm_rope_run(qkv, c, l, positions, slots, self.rope, q_gamma=a.norms[l][0], k_gamma=a.norms[l][1],
                                      eps=a.desc.eps)
            o = T.tf_tree_attn_run(q, c, l, seqs, q_start, masks=masks, max_rows=x.shape[0])
            h1 = T.tf_qlinear_run(L["o"], o, residual=h)
            h = T.tf_qlinear_run(L["down"], T.tf_qmlp_gateup_run(L["gate"], L["up"], h1, gamma=L["mlp_norm"], eps=self.dec.desc.eps),
                                 residual=h1)
        return T.tf_qlinear_run(self.dec.readout, h, gamma=self.dec.final_norm, eps=self.dec.desc.eps)


@pytest.mark.parametrize("kw,page", [
    (dict(seed=1, n_layers=3, d_model=256, d_ff=384, n_q=4, n_kv=2, hd=64, vocab=1000), 16),
    (dict(seed=2, n_layers=2, d_model=512, d_ff=640, n_q=8, n_kv=1, hd=128, vocab=777, bits=8, pairs=True), 32),
    (dict(seed=3, n_layers=2, d_model=256, d_ff=256, n_q=2, n_kv=1, hd=256, vocab=500, norms=False), 16),
    (dict(seed=4, n_layers=2, d_model=256, d_ff=384, n_q=4, n_kv=4, hd=64, vocab=1000, code="nvfp4"), 64),
])
def test_the_step_is_the_separate_calls_bit_for_bit(T, kw, page):
    m = Model(T, **kw)
    c, c2 = m.cache(T, page, 40, 4, 10), m.cache(T, page, 40, 4, 10)
    ws = T.workspace(T.tf_decode_step_attn_workspace_bytes(m.dec, c, m.attn))
    for seqs, rows, masks in [([2], [1], None), ([0, 2], [5, 3], None), ([1, 0, 2], [2, 4, 2], [1, 3, 1, 3, 5, 11, 1, 2]),
                              ([2], [8], [1, 3, 5, 9, 19, 35, 69, 137])]:
        start, M = np.cumsum([0] + rows).tolist(), sum(rows)
        mt = None if masks is None else mask_tensor(masks)
        x = m.x[:M].contiguous()
        got = []
        for cc in (c, c2):
            slots, pos = T.tf_kvcache_extend(cc, i32(seqs), i32(start), M, masks=mt)
            args = (i32(seqs), i32(start), slots, pos)
            got.append(T.tf_decode_step_attn_run(m.dec, cc, m.attn, x, *args, masks=mt, ws=ws) if cc is c else
                       m.separately(T, cc, x, *args, mt))
        assert T.tf_workspace_status(ws) == T.TF_OK
        assert torch.equal(got[0], got[1])
        assert torch.equal(c.data, c2.data) and torch.equal(c.book, c2.book)
        assert bool(torch.isfinite(got[0]).all())


def test_a_verified_tree_leaves_the_cache_of_plain_decoding(T):
    """The accepted path of a tree of drafts, kept, holds in the first layer (whose keys and values
    depend on a token and its position alone) exactly what token-by-token decoding stored."""
    m = Model(T, seed=5, n_layers=2, d_model=256, d_ff=384, n_q=4, n_kv=2, hd=64, vocab=1000)
    tokens = [11, 500, 7, 999, 42, 3, 250, 8, 77, 600, 5]
    plain = m.cache(T, 16, 6, 1, 4)
    for t in tokens:
        slots, pos = T.tf_kvcache_extend(plain, i32([0]), i32([0, 1]), 1)
        T.tf_decode_step_attn_run(m.dec, plain, m.attn, m.embed(T, i32([t])), i32([0]), i32([0, 1]), slots, pos)
    c = m.cache(T, 16, 6, 2, 4)
    at = 0
    for block, masks, path in [
            ([11, 500, 33, 7, 999, 1], [1, 3, 5, 11, 27, 37], [0, 1, 3, 4]),     # 11 -> 500 -> 7 -> 999, others beside
            ([42, 9, 3, 4, 250, 2, 8, 1], [1, 3, 5, 9, 21, 37, 85, 133], [0, 2, 4, 6]),
            ([77, 600, 5], [1, 3, 7], [0, 1, 2])]:
        M = len(block)
        mt = mask_tensor(masks)
        slots, pos = T.tf_kvcache_extend(c, i32([1]), i32([0, M]), M, masks=mt)
        T.tf_decode_step_attn_run(m.dec, c, m.attn, m.embed(T, i32(block)), i32([1]), i32([0, M]), slots, pos, masks=mt)
        T.tf_kvcache_keep(c, i32([1]), i32([0, M]), i32(path + [0] * (M - len(path))), i32([len(path)]))
        assert [block[i] for i in path] == tokens[at:at + len(path)]
        at += len(path)
    assert c.len.tolist() == [0, len(tokens)] and plain.len.tolist() == [len(tokens)]
    r = torch.arange(len(tokens), device="cuda")
    for kv in range(2):
        a = plain.data[0, kv, plain.table[0].long()[r // 16], :, r % 16]
        b = c.data[0, kv, c.table[1].long()[r // 16], :, r % 16]
        assert torch.equal(a, b)


def test_a_captured_step_decodes_on_over_page_ends(T):
    """Extend, step, log probabilities and the next token's embedding in one graph, replayed: the
    sequence grows by a token each time, over page ends, as in separate calls."""
    m = Model(T, seed=6, n_layers=2, d_model=256, d_ff=384, n_q=4, n_kv=2, hd=64, vocab=1000)
    runs = []
    for captured in (False, True):
        c = m.cache(T, 16, 8, 2, 6)
        seqs, start = i32([1]), i32([0, 1])
        slots, pos, token = i32([0]), i32([0]), i32([17])
        kws = T.workspace(T.tf_kvcache_workspace_bytes(c))
        sws = T.workspace(T.tf_decode_step_attn_workspace_bytes(m.dec, c, m.attn))
        ews, lws = T.workspace(256), T.workspace(256)
        logits = torch.empty((1, m.vocab), dtype=torch.bfloat16, device="cuda")
        lp, ent = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        top, tlp = torch.empty((1, 3), dtype=torch.int32, device="cuda"), torch.empty((1, 3), device="cuda")
        seen = torch.zeros(64, dtype=torch.int32, device="cuda")
        n = torch.zeros(1, dtype=torch.long, device="cuda")

        def step():
            T.tf_kvcache_extend(c, seqs, start, 1, slots=slots, positions=pos, ws=kws)
            x = T.tf_embed_rows(m.dec.readout, token, ws=ews)
            T.tf_decode_step_attn_run(m.dec, c, m.attn, x, seqs, start, slots, pos, out=logits, ws=sws)
            T.tf_logprobs_rows(logits, token, 3, lp, ent, top, tlp, ws=lws)
            token.copy_(top[:, 0])
            seen[n] = token
            n.add_(1)

        if captured:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            g = torch.cuda.CUDAGraph()
            with torch.cuda.stream(s):
                with torch.cuda.graph(g, stream=s):
                    step()
            torch.cuda.current_stream().wait_stream(s)
            for _ in range(40):
                g.replay()
        else:
            for _ in range(40):
                step()
        torch.cuda.synchronize()
        for w in (kws, sws, ews, lws):
            assert T.tf_workspace_status(w) == T.TF_OK
        assert c.len.tolist() == [0, 40]
        runs.append((seen.tolist(), logits.clone(), c.data.clone(), c.book.clone(), lp.clone(), ent.clone(), tlp.clone()))
    assert runs[0][0] == runs[1][0]
    for a, b in zip(runs[0][1:], runs[1][1:]):
        assert torch.equal(a, b)


def test_the_step_refuses_what_does_not_fit(T):
    m = Model(T, seed=7, n_layers=2, d_model=256, d_ff=256, n_q=4, n_kv=2, hd=64, vocab=500)
    c = m.cache(T, 16, 4, 2, 2)
    x, s, st = m.x[:2].contiguous(), i32([0]), i32([0, 2])
    slots, pos = T.tf_kvcache_extend(c, s, st, 2)
    with pytest.raises(T.TfqError):  # a cache of other heads
        T.tf_decode_step_attn_run(m.dec, T.KVCache.create(2, 1, 64, 16, 4, 2, 2), m.attn, x, s, st, slots, pos)
    with pytest.raises(T.TfqError):  # too few layers
        T.tf_decode_step_attn_run(m.dec, T.KVCache.create(1, 2, 64, 16, 4, 2, 2), m.attn, x, s, st, slots, pos)
    with pytest.raises(T.TfqError):  # more sequences than rows
        T.tf_decode_step_attn_run(m.dec, c, m.attn, x[:1], i32([0, 1]), i32([0, 1, 1]), slots, pos)
    with pytest.raises(T.TfqError):
        T.tf_decode_step_attn_run(m.dec, c, m.attn, x, s, st, slots, pos, ws=T.workspace(256))
    with pytest.raises(ValueError):
        T.tf_decode_step_attn_run(m.dec, c, T.Attention([(None, None)], 4, 64, m.rope), x, s, st, slots, pos)
    with pytest.raises(ValueError):  # described for other heads, or elsewhere
        T.tf_decode_step_attn_run(m.dec, c, T.Attention([(None, None)] * 2, 4, 128, m.rope), x, s, st, slots, pos)
    with pytest.raises(ValueError):
        T.tf_decode_step_attn_run(m.dec, c, T.Attention([(None, None)] * 2, 4, 64, T.RopeTable([1.0], device="cpu")), x, s, st, slots,
                                  pos)
    with pytest.raises(ValueError):
        T.tf_decode_step_attn_run(m.dec, c, m.attn, x, s, st, slots[:1], pos)
