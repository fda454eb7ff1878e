"""The 8-bit cache's and the prompt attention's entry points refuse bad arguments on the host, before anything reaches the GPU."""
import ctypes
import math

import pytest

from skinny_gemm_bit_gb300 import build as tfq_build

FAKE, DATA, SCALES, BOOK, OUT = 0x10000, 0x100000000, 0x180000000, 0x200000000, 0x300000000  # never dereferenced


@pytest.fixture(scope="module")
def T():
    tfq_build.build()
    from skinny_gemm_bit_gb300 import tfq
    return tfq


def cache(T, **kw):
    a = dict(layers=2, n_kv=2, hd=128, page=32, n_pages=10, n_seqs=4, max_pages=8, data=DATA, db=1 << 40, scales=SCALES, sb=1 << 30, book=BOOK,
             be=1 << 30)
    a.update(kw)
    d = T.tf_kvcache()
    rc = T.lib().tf_kvcache_init_e4m3(a["layers"], a["n_kv"], a["hd"], a["page"], a["n_pages"], a["n_seqs"], a["max_pages"], a["data"], a["db"],
                                      a["scales"], a["sb"], a["book"], a["be"], ctypes.byref(d))
    return rc, d


def test_sizes(T):
    L = T.lib()
    assert L.tf_kvcache_e4m3_bytes(28, 8, 128, 16, 100) == 28 * 2 * 100 * 8 * 16 * 128
    assert L.tf_kvcache_scale_bytes(28, 8, 64, 100) == 28 * 2 * 100 * 8 * 4
    assert L.tf_kvcache_scale_bytes(1, 1, 16, 3) == 8  # 6, its end rounded up
    assert L.tf_kvcache_e4m3_bytes(1, 8, 96, 16, 1) == 0 and L.tf_kvcache_scale_bytes(1, 8, 24, 1) == 0


def test_init_refuses(T):
    rc, d = cache(T)
    assert rc == T.TF_OK and d.code == T.TF_KV_E4M3 and d.scales == SCALES
    need = T.lib().tf_kvcache_e4m3_bytes(2, 2, 128, 32, 10)
    assert cache(T, db=need)[0] == T.TF_OK and cache(T, sb=2 * 2 * 10 * 2 * 2)[0] == T.TF_OK
    for kw, want in [(dict(hd=80), T.TF_E_UNSUPPORTED_SHAPE), (dict(page=20), T.TF_E_UNSUPPORTED_SHAPE), (dict(n_seqs=2000), T.TF_E_UNSUPPORTED_SHAPE),
                     (dict(data=None), T.TF_E_INVALID_ARG), (dict(data=DATA + 8), T.TF_E_INVALID_ARG), (dict(scales=None), T.TF_E_INVALID_ARG),
                     (dict(scales=SCALES + 2), T.TF_E_INVALID_ARG), (dict(book=BOOK + 2), T.TF_E_INVALID_ARG),
                     (dict(db=need - 1), T.TF_E_WORKSPACE_TOO_SMALL), (dict(sb=2 * 2 * 10 * 2 * 2 - 1), T.TF_E_WORKSPACE_TOO_SMALL)]:
        rc, d = cache(T, **kw)
        assert rc == want and d.magic == 0, kw
    assert T.lib().tf_kvcache_init_e4m3(2, 2, 128, 32, 10, 4, 8, DATA, 1 << 40, SCALES, 1 << 30, BOOK, 1 << 30, None) == T.TF_E_INVALID_ARG


def test_a_descriptor_that_does_not_hold_is_refused(T):
    L, big = T.lib(), 1 << 30
    for change in (dict(code=2), dict(code=-1), dict(code=T.TF_KV_BF16), dict(scales=None), dict(scales=SCALES + 1)):
        _, d = cache(T)
        for k, v in change.items():
            setattr(d, k, v)
        c = ctypes.byref(d)
        assert L.tf_kvcache_workspace_bytes(c) == 0 and L.tf_kvcache_reset(c, None) == T.TF_E_INVALID_ARG, change
        assert L.tf_kvcache_extend(c, FAKE, FAKE, 1, 1, None, OUT, None, FAKE, big, None) == T.TF_E_INVALID_ARG
        assert L.tf_kvcache_fork(c, FAKE, FAKE, big, None) == T.TF_E_INVALID_ARG
        assert L.tf_kvcache_keep(c, FAKE, FAKE, FAKE, FAKE, 1, 1, FAKE, big, None) == T.TF_E_INVALID_ARG
        assert L.tf_prompt_attn_run(FAKE, 512, 1, 4, c, 0, FAKE, FAKE, 1, 0.1, OUT, FAKE, big, 0, None) == T.TF_E_INVALID_ARG


def test_outputs_over_the_codes_or_the_scales_are_refused(T):
    L = T.lib()
    _, d = cache(T)
    c, big = ctypes.byref(d), 1 << 30
    data_end, scale_end = DATA + L.tf_kvcache_e4m3_bytes(2, 2, 128, 32, 10), SCALES + 2 * 2 * 10 * 2 * 2
    row = 4 * 128 * 2

    def attn(o, prompt):
        return L.tf_prompt_attn_run(FAKE, 512, 1, 4, c, 0, FAKE + 4096, FAKE + 8192, 1, 0.1, o, FAKE, 0, 0, None) if prompt else \
            L.tf_tree_attn_run(FAKE, 512, 1, 4, c, 0, FAKE + 4096, FAKE + 8192, 1, 1, None, 0.1, o, FAKE, 0, 0, None)

    def rope(q):
        return L.tf_qk_norm_rope_run(FAKE << 8, 1024, 1, 4, None, None, 0.0, FAKE, None, 0, 0, q, c, 0, FAKE, FAKE, 256, 0, None)

    for prompt in (False, True):
        for o in (DATA, data_end - 16, DATA - row + 16, SCALES, (scale_end - 1) // 16 * 16, SCALES - row + 16, BOOK, FAKE):
            assert attn(o, prompt) == T.TF_E_INVALID_ARG, (hex(o), prompt)
        for o in (data_end, DATA - row, (scale_end + 15) // 16 * 16, SCALES - row):  # beside them: only the workspace is missing
            assert attn(o, prompt) == T.TF_E_WORKSPACE_TOO_SMALL, (hex(o), prompt)
    for q in (DATA, data_end - 16, SCALES, BOOK):
        assert rope(q) == T.TF_E_INVALID_ARG
    assert L.tf_kvcache_extend(c, FAKE, FAKE, 1, 1, None, SCALES, None, FAKE, big, None) == T.TF_E_INVALID_ARG


def test_prompt_attention_refuses(T):
    L = T.lib()
    bf = T.tf_kvcache()
    assert L.tf_kvcache_init(2, 2, 128, 32, 10, 4, 8, DATA, 1 << 40, BOOK, 1 << 30, ctypes.byref(bf)) == T.TF_OK and bf.code == T.TF_KV_BF16
    _, wide = cache(T, hd=256)
    for d in (bf, cache(T)[1]):
        def run(c=d, q=FAKE, ldq=512, M=3, n_q=4, layer=1, seqs=FAKE + 8192, qs=FAKE + 12288, B=2, scale=0.1, o=OUT, ws=FAKE, wsb=1 << 40):
            return L.tf_prompt_attn_run(q, ldq, M, n_q, ctypes.byref(c), layer, seqs, qs, B, scale, o, ws, wsb, 0, None)

        arg, shape = T.TF_E_INVALID_ARG, T.TF_E_UNSUPPORTED_SHAPE
        for kw, rc in [(dict(q=None), arg), (dict(o=None), arg), (dict(seqs=None), arg), (dict(qs=None), arg), (dict(q=FAKE + 8), arg),
                       (dict(o=OUT + 8), arg), (dict(ldq=516), arg), (dict(ldq=504), arg), (dict(layer=2), arg), (dict(layer=-1), arg),
                       (dict(scale=math.nan), arg), (dict(scale=math.inf), arg), (dict(o=FAKE), arg), (dict(o=FAKE + 512 * 2 * 2), arg),
                       (dict(o=FAKE + 8192), arg), (dict(ws=None), arg), (dict(ws=FAKE + 16), arg), (dict(c=T.tf_kvcache()), arg),
                       (dict(n_q=3), shape), (dict(n_q=0), shape), (dict(n_q=130, ldq=130 * 128), shape), (dict(B=0), shape),
                       (dict(B=1025), shape), (dict(M=0), shape), (dict(M=1 << 21, ldq=512), shape),
                       (dict(M=1 << 20, n_q=64, ldq=64 * 128, o=OUT << 8), shape), (dict(c=wide, n_q=4, ldq=1024), shape),
                       (dict(wsb=100), T.TF_E_WORKSPACE_TOO_SMALL)]:
            assert run(**kw) == rc, kw
        assert L.tf_prompt_attn_workspace_bytes(ctypes.byref(d), 4, 3) > 256
        for bad in ((3, 1), (0, 1), (4, 0), (4, 1025), (130, 1)):
            assert L.tf_prompt_attn_workspace_bytes(ctypes.byref(d), *bad) == 0, bad
    assert L.tf_prompt_attn_workspace_bytes(ctypes.byref(wide), 2, 1) == 0
