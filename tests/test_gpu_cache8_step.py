"""The decoder step over a cache of 8 bits: the separate calls' results, and a run of steps with drafts."""
import numpy as np
import pytest
import torch

from test_gpu_cache8 import E4M3, i32, mask_tensor
from test_gpu_cached_step import Model

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    from skinny_gemm_bit_gb300 import build
    build.build()
    from skinny_gemm_bit_gb300 import tfq
    return tfq


def cache8(T, m, page, n_pages, n_seqs, max_pages):
    return T.KVCache.create(*m.dims, page, n_pages, n_seqs, max_pages, dtype=E4M3)


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("kw,page", [
    (dict(seed=1, n_layers=3, d_model=256, d_ff=384, n_q=4, n_kv=2, hd=64, vocab=1000), 16),
    (dict(seed=2, n_layers=2, d_model=512, d_ff=640, n_q=8, n_kv=1, hd=128, vocab=777, bits=8, pairs=True), 32),
    (dict(seed=3, n_layers=2, d_model=256, d_ff=256, n_q=2, n_kv=1, hd=256, vocab=500, norms=False), 16),
    (dict(seed=4, n_layers=2, d_model=256, d_ff=384, n_q=4, n_kv=4, hd=64, vocab=1000, code="nvfp4"), 64),
])
def test_the_step_over_8_bits_is_the_separate_calls_bit_for_bit(T, kw, page):
    m = Model(T, **kw)
    c, c2 = cache8(T, m, page, 40, 4, 10), cache8(T, m, page, 40, 4, 10)
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
        assert torch.equal(got[0], got[1]) and bool(torch.isfinite(got[0]).all())
        assert same(c.data, c2.data) and same(c.scales, c2.scales) and torch.equal(c.book, c2.book)


def test_a_captured_step_over_8_bits_decodes_on(T):
    """A graph of extend and step, replayed over page and block ends, gives what the calls give."""
    m = Model(T, seed=6, n_layers=2, d_model=256, d_ff=384, n_q=4, n_kv=2, hd=64, vocab=1000)
    c, c2 = cache8(T, m, 16, 10, 2, 6), cache8(T, m, 16, 10, 2, 6)
    seqs, start, x = i32([1, 0]), i32([0, 2, 3]), m.x[:3].contiguous()
    slots, pos = i32([0] * 3), i32([0] * 3)
    ws, wsc = T.workspace(T.tf_decode_step_attn_workspace_bytes(m.dec, c, m.attn)), T.workspace(T.tf_kvcache_workspace_bytes(c))
    out = torch.empty((3, 1000), dtype=torch.bfloat16, device="cuda")

    def step():
        T.tf_kvcache_extend(c, seqs, start, 3, slots=slots, positions=pos, ws=wsc)
        T.tf_decode_step_attn_run(m.dec, c, m.attn, x, seqs, start, slots, pos, out=out, ws=ws)

    step()
    T.tf_kvcache_reset(c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in range(20):
        x.copy_(torch.roll(m.x[:3], n, 1))
        g.replay()
        sl, ps = T.tf_kvcache_extend(c2, seqs, start, 3)
        want = T.tf_decode_step_attn_run(m.dec, c2, m.attn, x, seqs, start, sl, ps)
        torch.cuda.synchronize()
        assert torch.equal(out, want), n
    used = c.refs > 0
    assert torch.equal(c.book, c2.book) and same(c.data[:, :, used], c2.data[:, :, used]) and same(c.scales[:, :, used], c2.scales[:, :, used])
    assert T.tf_workspace_status(ws) == T.TF_OK and T.tf_workspace_status(wsc) == T.TF_OK


def test_8_bits_stay_near_bf16(T):
    """The same tokens through both caches: logits within what e4m3's half step of 2^-4 of keys and values makes of them."""
    m = Model(T, seed=7, n_layers=2, d_model=256, d_ff=384, n_q=4, n_kv=2, hd=64, vocab=1000)
    a, b = m.cache(T, 16, 10, 1, 6), cache8(T, m, 16, 10, 1, 6)
    for n in range(30):
        x = m.embed(T, i32([37 * n % 1000]))
        got = []
        for c in (a, b):
            slots, pos = T.tf_kvcache_extend(c, i32([0]), i32([0, 1]), 1)
            got.append(T.tf_decode_step_attn_run(m.dec, c, m.attn, x, i32([0]), i32([0, 1]), slots, pos).double())
        assert float((got[0] - got[1]).norm() / got[0].norm()) < 2.0 ** -3
