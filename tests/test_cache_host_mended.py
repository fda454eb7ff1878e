"""What the cached-decoding entry points once let through on the host."""
import ctypes

import pytest

from skinny_gemm_bit_gb300 import build as tfq_build

FAKE = 0x10000  # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def T():
    tfq_build.build()
    from skinny_gemm_bit_gb300 import tfq
    return tfq


class Step:
    """A decoder step over a cache on made-up addresses."""
    D, F, n_q, n_kv, hd, V, page, n_pages, n_seqs, max_pages = 256, 256, 4, 2, 64, 500, 16, 10, 4, 8

    def __init__(self, T, data=0x100000000, book=0x200000000):
        self.T, self.L = T, T.lib()
        D, F, n_q, n_kv, hd, V = self.D, self.F, self.n_q, self.n_kv, self.hd, self.V
        self.layers = (T.tf_decoder_layer * 2)()
        for l in self.layers:
            l.qkv, l.o, l.gate = self.weight((n_q + 2 * n_kv) * hd, D), self.weight(D, n_q * hd), self.weight(F, D)
            l.up, l.down = self.weight(F, D), self.weight(D, F)
            l.attn_norm = l.mlp_norm = FAKE
        self.dec = T.tf_decoder_desc()
        d = self.dec
        d.n_layers, d.d_model, d.d_ff, d.q_dim, d.kv_dim, d.vocab = 2, D, F, n_q * hd, n_kv * hd, V
        d.layers, d.final_norm, d.readout = ctypes.cast(self.layers, ctypes.POINTER(T.tf_decoder_layer)), FAKE, self.weight(V, D)
        self.cache = T.tf_kvcache()
        assert self.L.tf_kvcache_init(2, n_kv, hd, self.page, self.n_pages, self.n_seqs, self.max_pages, data, 1 << 40, book,
                                      1 << 30, ctypes.byref(self.cache)) == T.TF_OK
        self.norms = (T.tf_attn_layer * 2)()
        self.attn = T.tf_attn_desc()
        a = self.attn
        a.n_q, a.eps, a.scale, a.rot_dim, a.turns = n_q, 1e-6, 0.1, 64, FAKE
        a.layers = ctypes.cast(self.norms, ctypes.POINTER(T.tf_attn_layer))

    def weight(self, N, K):
        d = self.T.tf_qweight()
        d.magic, d.version, d.bits, d.group, d.batch, d.N, d.K = 0x31515446, self.T.TF_PACK_VERSION, 4, 64, 1, N, K
        d.code, d.global_scale, d.n_pad, d.tile_bytes, d.data = self.T.TF_CODE_AFFINE, 1.0, (N + 15) // 16 * 16, 576, 0x20000
        d.matrix_bytes = d.n_pad // 16 * (K // 64) * d.tile_bytes
        return d

    def need(self):
        return self.L.tf_decode_step_attn_workspace_bytes(ctypes.byref(self.dec), ctypes.byref(self.cache), ctypes.byref(self.attn))

    def run(self, M=2, B=1, logits=0x300000000, ws=FAKE, wsb=1 << 40):
        return self.L.tf_decode_step_attn_run(ctypes.byref(self.dec), ctypes.byref(self.cache), ctypes.byref(self.attn), FAKE, M,
                                              FAKE, FAKE, B, None, FAKE, FAKE, logits, ws, wsb, 0, None)


def test_the_step_refuses_a_max_rows_out_of_range(T):
    s = Step(T)
    want = s.need()
    for rows in (0, 1, 3, 8):
        s.attn.max_rows = rows
        assert s.need() == want > 0  # one workspace for them all
        assert s.run(wsb=want - 1) == T.TF_E_WORKSPACE_TOO_SMALL
    for rows in (-1, 9, 64):
        s.attn.max_rows = rows
        assert s.need() == 0
        assert s.run() == T.TF_E_UNSUPPORTED_SHAPE


def test_outputs_over_the_cache_or_the_inputs_are_refused(T):
    data, book, x, y, ints = 0x100000000, 0x200000000, 0x300000000, 0x400000000, 0x500000000
    s = Step(T, data, book)
    L, c = s.L, ctypes.byref(s.cache)
    data_end = data + L.tf_kvcache_data_bytes(2, s.n_kv, s.hd, s.page, s.n_pages)
    book_end = book + 4 * L.tf_kvcache_book_elems(s.n_pages, s.n_seqs, s.max_pages)

    def extend(slots, positions):
        return L.tf_kvcache_extend(c, ints, ints + 4096, 2, 5, None, slots, positions, FAKE, 1 << 20, None)

    for at in (book - 16, book, book_end - 4, data - 16, data_end - 4):
        assert extend(at, None) == extend(at, x) == extend(x, at) == T.TF_E_INVALID_ARG

    for at in (data - 4 * s.V + 4, data, data_end - 2, book, book_end - 2, book - 4 * s.V + 2):
        assert s.run(logits=at) == T.TF_E_INVALID_ARG

    def rope(q, pos=ints, slots=ints + 64, turns=ints + 128, qg=ints + 512, kg=ints + 1024):  # 3 rows of 2 heads of 64
        return L.tf_qk_norm_rope_run(x, 384, 3, 2, qg, kg, 0.0, pos, turns, 64, 0, q, c, 0, slots, FAKE, 256, 0, None)

    for kw in (dict(pos=y + 764), dict(slots=y - 8), dict(turns=y - 248), dict(turns=y + 760), dict(qg=y + 752), dict(kg=y - 112)):
        assert rope(y, **kw) == T.TF_E_INVALID_ARG, kw

    def attn(o, seqs=ints, start=ints + 64, masks=None):  # 3 rows of 2 heads of 64, 2 sequences
        ws = L.tf_tree_attn_workspace_bytes(c, 2, 2, 3)
        return L.tf_tree_attn_run(x, 128, 3, 2, c, 0, seqs, start, 2, 3, masks, 0.1, o, FAKE, ws, 0, None)

    for kw in (dict(seqs=y - 4), dict(seqs=y + 764), dict(start=y - 8), dict(masks=y - 16), dict(masks=y + 760)):
        assert attn(y, **kw) == T.TF_E_INVALID_ARG, kw
