"""The cached-decoding entry points refuse bad arguments on the host, before anything reaches
the GPU, and the host-only calls give what they say."""
import ctypes
import math

import numpy as np
import pytest

from skinny_gemm_bit_gb300 import build as tfq_build

FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10002)
OUT = ctypes.c_void_p(0x40000000)


@pytest.fixture(scope="module")
def T():
    tfq_build.build()
    from skinny_gemm_bit_gb300 import tfq
    return tfq


def _cache(T, **kw):
    a = dict(layers=2, n_kv=2, hd=128, page=16, n_pages=10, n_seqs=4, max_pages=8, data=FAKE, book=FAKE, db=1 << 40, be=1 << 30)
    a.update(kw)
    d = T.tf_kvcache()
    rc = T.lib().tf_kvcache_init(a["layers"], a["n_kv"], a["hd"], a["page"], a["n_pages"], a["n_seqs"], a["max_pages"],
                                 a["data"], a["db"], a["book"], a["be"], ctypes.byref(d))
    return rc, d


def test_cache_sizes(T):
    L = T.lib()
    assert L.tf_kvcache_data_bytes(28, 8, 128, 16, 100) == 28 * 2 * 100 * 8 * 16 * 128 * 2
    assert L.tf_kvcache_book_elems(100, 4, 9) == 4 + 100 + 36
    for bad in [(0, 8, 128, 16, 1), (1, 0, 128, 16, 1), (1, 257, 128, 16, 1), (1, 8, 96, 16, 1), (1, 8, 128, 24, 1),
                (1, 8, 128, 8, 1), (1, 8, 128, 16, 0), (1, 1, 128, 16, 1 << 27), (64, 64, 128, 16, 1 << 15)]:
        assert L.tf_kvcache_data_bytes(*bad) == 0, bad
    for bad in [(0, 4, 9), (10, 0, 9), (10, 1025, 9), (10, 4, 0), (10, 4, 1 << 27)]:
        assert L.tf_kvcache_book_elems(*bad) == 0, bad


def test_cache_init_refuses(T):
    assert _cache(T)[0] == T.TF_OK
    for kw, want in [(dict(hd=80), T.TF_E_UNSUPPORTED_SHAPE), (dict(page=20), T.TF_E_UNSUPPORTED_SHAPE),
                     (dict(n_seqs=2000), T.TF_E_UNSUPPORTED_SHAPE), (dict(max_pages=1 << 28), T.TF_E_UNSUPPORTED_SHAPE),
                     (dict(data=None), T.TF_E_INVALID_ARG), (dict(data=ctypes.c_void_p(0x10008)), T.TF_E_INVALID_ARG),
                     (dict(book=ODD), T.TF_E_INVALID_ARG), (dict(db=100), T.TF_E_WORKSPACE_TOO_SMALL),
                     (dict(be=10), T.TF_E_WORKSPACE_TOO_SMALL)]:
        rc, d = _cache(T, **kw)
        assert rc == want and d.magic == 0, kw


def test_page_operations_refuse(T):
    L = T.lib()
    _, d = _cache(T)
    c, big = ctypes.byref(d), 1 << 20
    blank = ctypes.byref(T.tf_kvcache())
    assert L.tf_kvcache_workspace_bytes(c) > 256
    assert L.tf_kvcache_workspace_bytes(blank) == 0
    assert L.tf_kvcache_reset(blank, None) == T.TF_E_INVALID_ARG

    def extend(cc=c, seqs=FAKE, qs=FAKE, B=1, M=1, slots=FAKE, ws=FAKE, wsb=big):
        return L.tf_kvcache_extend(cc, seqs, qs, B, M, None, slots, None, ws, wsb, None)

    def keep(cc=c, seqs=FAKE, qs=FAKE, k=FAKE, n=FAKE, B=1, M=1, ws=FAKE, wsb=big):
        return L.tf_kvcache_keep(cc, seqs, qs, k, n, B, M, ws, wsb, None)

    for f in (extend, keep):
        assert f(cc=blank) == T.TF_E_INVALID_ARG
        assert f(seqs=None) == T.TF_E_INVALID_ARG
        assert f(qs=None) == T.TF_E_INVALID_ARG
        assert f(B=0) == f(B=5) == f(M=0) == f(M=1 << 31) == T.TF_E_UNSUPPORTED_SHAPE
        assert f(ws=None) == f(ws=ctypes.c_void_p(0x10010)) == T.TF_E_INVALID_ARG
        assert f(wsb=256) == T.TF_E_WORKSPACE_TOO_SMALL
    assert extend(slots=None) == T.TF_E_INVALID_ARG
    assert keep(k=None) == keep(n=None) == T.TF_E_INVALID_ARG
    assert L.tf_kvcache_fork(c, None, FAKE, big, None) == T.TF_E_INVALID_ARG
    assert L.tf_kvcache_fork(c, FAKE, FAKE, 100, None) == T.TF_E_WORKSPACE_TOO_SMALL


def test_norm_rope_refuses(T):
    L = T.lib()
    _, d = _cache(T)

    def run(qkv=FAKE, ld=1024, M=1, n_q=4, qg=None, kg=None, eps=1e-6, pos=FAKE, turns=FAKE, rot=128, q=OUT, layer=0,
            slots=FAKE, ws=FAKE, wsb=256, c=d):
        return L.tf_qk_norm_rope_run(qkv, ld, M, n_q, qg, kg, eps, pos, turns, rot, 0, q, ctypes.byref(c), layer, slots, ws,
                                     wsb, 0, None)

    for kw in [dict(qkv=None), dict(qkv=ODD), dict(ld=1023), dict(ld=1020), dict(qg=ODD), dict(kg=ODD), dict(eps=-1.0),
               dict(eps=math.nan), dict(pos=None), dict(turns=None), dict(q=None), dict(q=ODD), dict(q=ctypes.c_void_p(0x10000 + 1008)), dict(layer=2), dict(layer=-1),
               dict(slots=None), dict(ws=None), dict(c=T.tf_kvcache())]:
        assert run(**kw) == T.TF_E_INVALID_ARG, kw
    for kw in [dict(M=0), dict(M=1 << 25), dict(n_q=0), dict(n_q=1025), dict(rot=24), dict(rot=144), dict(rot=-16)]:
        assert run(**kw) == T.TF_E_UNSUPPORTED_SHAPE, kw
    assert run(wsb=100) == T.TF_E_WORKSPACE_TOO_SMALL


def test_tree_attn_refuses(T):
    L = T.lib()
    _, d = _cache(T)

    def run(q=FAKE, ldq=512, M=1, n_q=4, layer=0, seqs=FAKE, qs=FAKE, B=1, rows=1, scale=0.1, o=OUT, ws=FAKE, wsb=1 << 30,
            c=d):
        return L.tf_tree_attn_run(q, ldq, M, n_q, ctypes.byref(c), layer, seqs, qs, B, rows, None, scale, o, ws, wsb, 0, None)

    for kw in [dict(q=None), dict(q=ODD), dict(ldq=511), dict(ldq=500), dict(layer=2), dict(seqs=None), dict(qs=None),
               dict(scale=math.inf), dict(scale=math.nan), dict(o=None), dict(o=ODD), dict(o=FAKE), dict(o=ctypes.c_void_p(0x10000 - 1008)), dict(ws=None), dict(c=T.tf_kvcache())]:
        assert run(**kw) == T.TF_E_INVALID_ARG, kw
    for kw in [dict(M=0), dict(M=1 << 21), dict(n_q=3), dict(n_q=0), dict(n_q=130), dict(B=0), dict(B=1025), dict(rows=0),
               dict(rows=65)]:
        assert run(**kw) == T.TF_E_UNSUPPORTED_SHAPE, kw
    assert run(wsb=16) == T.TF_E_WORKSPACE_TOO_SMALL
    assert L.tf_tree_attn_workspace_bytes(ctypes.byref(d), 4, 1, 8) >= 256
    assert L.tf_tree_attn_workspace_bytes(ctypes.byref(d), 5, 1, 8) == 0


def test_logprobs_refuses(T):
    L = T.lib()

    def run(v=FAKE, dt=0, ld=100, M=1, N=100, t=FAKE, nt=1, k=4, lp=FAKE, ti=FAKE, tl=FAKE, ws=FAKE, wsb=1 << 20):
        return L.tf_logprobs_rows(v, dt, ld, M, N, t, nt, k, lp, None, ti, tl, ws, wsb, None)

    for kw in [dict(v=None), dict(v=ctypes.c_void_p(0x10001)), dict(dt=1, v=ODD), dict(dt=2), dict(t=None), dict(lp=None),
               dict(ti=None), dict(tl=None), dict(ws=None)]:
        assert run(**kw) == T.TF_E_INVALID_ARG, kw
    for kw in [dict(ld=99), dict(M=0), dict(M=1 << 25), dict(N=0), dict(k=33), dict(k=-1), dict(N=3), dict(nt=-1), dict(nt=1025)]:
        assert run(**kw) == T.TF_E_UNSUPPORTED_SHAPE, kw
    assert run(wsb=0) == T.TF_E_WORKSPACE_TOO_SMALL
    assert L.tf_logprobs_workspace_bytes(1, 100, 4) >= 256
    assert L.tf_logprobs_workspace_bytes(1, 3, 4) == 0


def test_rope_turns(T):
    f = np.array([1.0, 0.5, 1e-6, -0.25, 0.0, 6.28, 2.0 ** -40])
    turns = np.zeros(f.size, np.uint64)
    assert T.lib().tf_rope_turns(f.ctypes.data, f.size, turns.ctypes.data) == T.TF_OK
    for x, t in zip(f, turns):
        t = int(t)
        t = t - (1 << 64) if x < 0 else t
        # inv_freq / 2 pi in fp64 (two roundings) and the cut to 2^-64
        assert abs(t / 2.0 ** 64 - x / (2 * math.pi)) <= 2.0 ** -52 * abs(x) + 2.0 ** -64, x
    for bad in (math.inf, math.nan, 6.3, -7.0):
        assert T.lib().tf_rope_turns(np.array([bad]).ctypes.data, 1, turns.ctypes.data) == T.TF_E_INVALID_ARG
    assert T.lib().tf_rope_turns(None, 1, turns.ctypes.data) == T.TF_E_INVALID_ARG
    assert T.lib().tf_rope_turns(None, 0, None) == T.TF_OK


def test_cache_full_has_a_name(T):
    assert T.status_str(T.TF_E_CACHE_FULL) == "TF_E_CACHE_FULL" == T.status_str(8)


def _at(a):
    return ctypes.c_void_p(a)


def test_outputs_over_the_cache_or_over_one_another_are_refused(T):
    L = T.lib()
    d0, b0, x0, y0 = 0x100000000, 0x200000000, 0x300000000, 0x400000000
    _, d = _cache(T, data=_at(d0), book=_at(b0))
    c = ctypes.byref(d)
    data_end, book_end = d0 + L.tf_kvcache_data_bytes(2, 2, 128, 16, 10), b0 + 4 * L.tf_kvcache_book_elems(10, 4, 8)

    def rope(qkv, q):  # 3 rows of 4 + 2 * 2 heads, 2048 bytes each; q 1024 bytes a row
        return L.tf_qk_norm_rope_run(_at(qkv), 1024, 3, 4, None, None, 0.0, FAKE, None, 0, 0, _at(q), c, 0, FAKE, FAKE, 256, 0, None)

    def attn(o):
        ws = L.tf_tree_attn_workspace_bytes(c, 4, 1, 3)
        return L.tf_tree_attn_run(_at(x0), 512, 3, 4, c, 0, FAKE, FAKE, 1, 3, None, 0.1, _at(o), FAKE, ws, 0, None)

    def extend(slots, pos, seqs=FAKE, qs=FAKE, masks=None):
        return L.tf_kvcache_extend(c, seqs, qs, 2, 5, masks, slots, pos, FAKE, 1 << 20, None)

    for a in (d0 - 3 * 2048 + 16, d0, data_end - 16, b0 - 3 * 2048 + 16, book_end // 16 * 16 - 16):
        assert rope(a, y0) == T.TF_E_INVALID_ARG
    for a in (d0 - 3 * 1024 + 16, d0, data_end - 16, b0 - 3 * 1024 + 16, book_end // 16 * 16 - 16):
        assert rope(x0, a) == T.TF_E_INVALID_ARG
        assert attn(a) == T.TF_E_INVALID_ARG
    assert extend(_at(x0), _at(x0 + 16)) == T.TF_E_INVALID_ARG
    for out in ((_at(x0), None), (_at(y0), _at(x0))):
        assert extend(*out, seqs=_at(x0 + 16)) == T.TF_E_INVALID_ARG
        assert extend(*out, qs=_at(x0 - 8)) == T.TF_E_INVALID_ARG
        assert extend(*out, masks=_at(x0 - 32)) == T.TF_E_INVALID_ARG

    def logp(v=x0, t=0x500000000, lp=0x600000000, en=0x700000000, ti=0x800000000, tl=0x900000000):
        return L.tf_logprobs_rows(_at(v), 0, 100, 3, 90, _at(t), 2, 4, _at(lp), _at(en), _at(ti), _at(tl), FAKE, 1 << 20, None)

    last = (2 * 100 + 90) * 2
    for kw in (dict(lp=x0), dict(en=x0 + last - 4), dict(ti=x0 - 44), dict(tl=x0 + 100), dict(lp=0x500000000),
               dict(en=0x500000000 + 20), dict(tl=0x800000000 + 44), dict(en=0x600000000 + 20), dict(ti=0x700000000)):
        assert logp(**kw) == T.TF_E_INVALID_ARG, kw


def test_decoder_step_over_a_cache_refuses(T):
    L = T.lib()

    def qw(N, K):
        d = T.tf_qweight()
        d.magic, d.version, d.bits, d.group, d.batch, d.N, d.K = 0x31515446, T.TF_PACK_VERSION, 4, 64, 1, N, K
        d.code, d.global_scale, d.n_pad, d.tile_bytes, d.data = T.TF_CODE_AFFINE, 1.0, (N + 15) // 16 * 16, 576, 0x20000
        d.matrix_bytes = d.n_pad // 16 * (K // 64) * d.tile_bytes
        return d

    D, F, n_q, n_kv, hd, V = 256, 256, 4, 2, 64, 500
    layers = (T.tf_decoder_layer * 2)()
    for l in layers:
        l.qkv, l.o, l.gate, l.up, l.down = qw((n_q + 2 * n_kv) * hd, D), qw(D, n_q * hd), qw(F, D), qw(F, D), qw(D, F)
        l.attn_norm = l.mlp_norm = FAKE.value
    dec = T.tf_decoder_desc()
    dec.n_layers, dec.d_model, dec.d_ff, dec.q_dim, dec.kv_dim, dec.vocab = 2, D, F, n_q * hd, n_kv * hd, V
    dec.layers, dec.final_norm, dec.readout = ctypes.cast(layers, ctypes.POINTER(T.tf_decoder_layer)), FAKE.value, qw(V, D)

    def attn(**kw):
        a = dict(n_q=n_q, eps=1e-6, scale=0.1, rot_dim=64, turns=FAKE.value, layers=None, norms=(None, None))
        a.update(kw)
        arr = (T.tf_attn_layer * 2)()
        arr[1].q_norm, arr[1].k_norm = a["norms"]
        d = T.tf_attn_desc()
        d.n_q, d.eps, d.scale, d.rot_dim, d.turns = a["n_q"], a["eps"], a["scale"], a["rot_dim"], a["turns"]
        d.layers = ctypes.cast(arr, ctypes.POINTER(T.tf_attn_layer)) if a["layers"] is None else a["layers"]
        return d

    def cache(**kw):
        return _cache(T, hd=hd, **kw)[1]

    def need(a, c=None):
        return L.tf_decode_step_attn_workspace_bytes(ctypes.byref(dec), ctypes.byref(cache() if c is None else c), ctypes.byref(a))

    good = need(attn())
    assert good > 0

    def run(a=None, c=None, x=FAKE, M=2, seqs=FAKE, qs=FAKE, B=1, slots=FAKE, pos=FAKE, out=OUT, ws=FAKE, wsb=good):
        return L.tf_decode_step_attn_run(ctypes.byref(dec), ctypes.byref(cache() if c is None else c),
                                         ctypes.byref(attn() if a is None else a), x, M, seqs, qs, B, None, slots, pos, out, ws,
                                         wsb, 0, None)

    shape, arg = T.TF_E_UNSUPPORTED_SHAPE, T.TF_E_INVALID_ARG
    nowhere = ctypes.POINTER(T.tf_attn_layer)()
    for kw, rc in [(dict(n_q=2), shape), (dict(n_q=0), shape), (dict(rot_dim=24), shape), (dict(rot_dim=80), shape),
                   (dict(rot_dim=-16), shape), (dict(turns=None), arg), (dict(turns=0x10004), arg), (dict(eps=-1.0), arg),
                   (dict(eps=math.nan), arg), (dict(scale=math.inf), arg), (dict(norms=(0x10008, None)), arg),
                   (dict(norms=(None, 0x10002)), arg), (dict(layers=nowhere), arg)]:
        assert need(attn(**kw)) == 0, kw
        assert run(attn(**kw)) == rc, kw
    for kw, rc in [(dict(c=cache(n_kv=1)), shape), (dict(c=cache(layers=1)), shape), (dict(c=T.tf_kvcache()), arg), (dict(M=0), shape),
                   (dict(M=9), shape), (dict(B=0), shape), (dict(B=3), shape), (dict(x=None), arg), (dict(x=ODD), arg),
                   (dict(seqs=None), arg), (dict(qs=None), arg), (dict(slots=None), arg), (dict(pos=None), arg),
                   (dict(out=None), arg), (dict(ws=None), arg), (dict(wsb=good - 1), T.TF_E_WORKSPACE_TOO_SMALL)]:
        assert run(**kw) == rc, kw


def test_the_attention_description_refuses_norms_that_do_not_fit(T):
    import torch
    rope = T.RopeTable([1.0, 0.5] * 16, device="cpu")
    good = torch.ones(64, dtype=torch.bfloat16)
    T.Attention([(good, None), (None, good)], 2, 64, rope)
    for bad in (good.float(), good[:32], torch.ones(128, dtype=torch.bfloat16)[::2]):
        with pytest.raises(ValueError):
            T.Attention([(good, good), (None, bad)], 2, 64, rope)
