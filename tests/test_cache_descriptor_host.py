"""The descriptor of a bf16 cache is what it was before caches of 8 bits: 48 bytes, behind which no call looks or writes."""
import ctypes

import pytest

from skinny_gemm_bit_gb300 import build as tfq_build

FAKE, DATA, SCALES, BOOK, OUT = 0x10000, 0x100000000, 0x180000000, 0x200000000, 0x300000000  # never dereferenced
BIG, BF16_BYTES = 1 << 40, 48


@pytest.fixture(scope="module")
def T():
    tfq_build.build()
    from skinny_gemm_bit_gb300 import tfq
    return tfq


def init(T, junk):
    """A bf16 descriptor whose memory held `junk` before."""
    buf = (ctypes.c_uint8 * ctypes.sizeof(T.tf_kvcache))(*[junk] * ctypes.sizeof(T.tf_kvcache))
    d = T.tf_kvcache.from_buffer(buf)
    assert T.lib().tf_kvcache_init(2, 2, 128, 32, 10, 4, 8, DATA, BIG, BOOK, 1 << 30, ctypes.byref(d)) == T.TF_OK
    return buf, d


@pytest.mark.parametrize("junk", [0x00, 0x01, 0xA5, 0xFF])
def test_a_bf16_descriptor_ends_behind_the_book(T, junk):
    L = T.lib()
    assert T.tf_kvcache.code.offset == BF16_BYTES
    buf, d = init(T, junk)
    assert d.magic == T.TF_KVCACHE_MAGIC and list(buf[BF16_BYTES:]) == [junk] * (len(buf) - BF16_BYTES)
    c, clean = ctypes.byref(d), ctypes.byref(init(T, 0)[1])
    assert L.tf_kvcache_workspace_bytes(c) == L.tf_kvcache_workspace_bytes(clean) > 256
    assert L.tf_tree_attn_workspace_bytes(c, 4, 3, 8) == L.tf_tree_attn_workspace_bytes(clean, 4, 3, 8) > 256
    assert L.tf_prompt_attn_workspace_bytes(c, 4, 3) == L.tf_prompt_attn_workspace_bytes(clean, 4, 3) > 256
    # past the descriptor's checks: what is missing is the workspace
    assert L.tf_kvcache_extend(c, FAKE, FAKE, 1, 1, None, OUT, None, FAKE, 0, None) == T.TF_E_WORKSPACE_TOO_SMALL
    assert L.tf_tree_attn_run(FAKE, 512, 1, 4, c, 0, FAKE + 4096, FAKE + 8192, 1, 1, None, 0.1, OUT, FAKE, 0, 0, None) == T.TF_E_WORKSPACE_TOO_SMALL
    # the data is bf16's, twice the bytes of codes: an output in its second half lies in the cache
    half = DATA + L.tf_kvcache_e4m3_bytes(2, 2, 128, 32, 10)
    assert L.tf_tree_attn_run(FAKE, 512, 1, 4, c, 0, FAKE + 4096, FAKE + 8192, 1, 1, None, 0.1, half, FAKE, 0, 0, None) == T.TF_E_INVALID_ARG


def test_a_cache_of_8_bits_is_named_by_its_magic(T):
    L, d = T.lib(), T.tf_kvcache()
    assert L.tf_kvcache_init_e4m3(2, 2, 128, 32, 10, 4, 8, DATA, BIG, SCALES, BIG, BOOK, 1 << 30, ctypes.byref(d)) == T.TF_OK
    assert d.magic == T.TF_KVCACHE_MAGIC_E4M3 != T.TF_KVCACHE_MAGIC and d.code == T.TF_KV_E4M3 and d.scales == SCALES
    # the scales are known to be the cache's
    assert L.tf_tree_attn_run(FAKE, 512, 1, 4, ctypes.byref(d), 0, FAKE + 4096, FAKE + 8192, 1, 1, None, 0.1, SCALES, FAKE, 0, 0, None) == T.TF_E_INVALID_ARG
    d.magic = 0x334B5654
    assert L.tf_kvcache_workspace_bytes(ctypes.byref(d)) == 0
