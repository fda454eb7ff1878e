"""Plain 64-bit forms of the operators over a cache of 8 bits and of prompt attention, for the GPU parity tests."""
import numpy as np
import torch

import cached_ref as R

F16_HALF, E4M3_HALF = 2.0 ** -11, 2.0 ** -4  # roundings, relative to the value
LEAST, MOST = -32, 32                        # exponents of a block's scale


def e4m3(x):
    """Nearest e4m3 number, ties to the even one, +-448 where larger; NaN stays."""
    with np.errstate(invalid="ignore"):
        e = np.clip(np.frexp(np.where(np.isfinite(x), x, 1.0))[1] - 1, -6, 8)
        step = 2.0 ** (e - 3)
        return np.where(np.isnan(x), np.nan, np.clip(np.where(np.isinf(x), np.sign(x) * 448, np.rint(x / step) * step), -448, 448))


def least_exponent(most):
    return int(np.clip(np.ceil(np.log2(most / 448)), LEAST, MOST)) if most > 0 else LEAST


def exponents(c):
    """[layers, 2, pages, heads, blocks] of a cache."""
    return c.scales.view(torch.uint8).int().cpu().numpy() - 127


def values(c):
    """[layers, 2, pages, heads, rows, hd] fp64: codes times scales, which count as within their bounds."""
    e = np.clip(exponents(c), LEAST, MOST)
    return R.f64(c.data.float()) * 2.0 ** np.repeat(e, 16, -1)[..., None]


def fill(c, seed, sizes=True):
    """Random codes and scales in all of a cache; heads and blocks of different size."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = c.scales.shape
    x = torch.randn((*shape, 16, c.head_dim), generator=g, device="cuda")
    e = torch.randint(-6, 7, shape, generator=g, device="cuda") if sizes else torch.zeros(shape, dtype=torch.int64, device="cuda")
    c.data.copy_((x * 100).clamp(-448, 448).view(c.data.shape).to(torch.float8_e4m3fn))
    c.scales.view(torch.uint8).copy_((127 - 7 + e).to(torch.uint8))


def scales_of(c, layer, s):
    """[len, n_kv]: the scale of each value of a slot; None for a bf16 cache."""
    if c.scales is None:
        return None
    r, page = np.arange(int(c.len[s])), c.page_size
    e = np.clip(exponents(c)[layer, 1], LEAST, MOST)
    return 2.0 ** e[c.table[s].cpu().numpy()[r // page], :, r % page // 16]


def attn(q, k, v, see, scale, vs=None):
    """q [T, n_q, hd], k, v [n, n_kv, hd], see [T, n] bool, vs [n, n_kv] the values' scales (None: bf16): (o, spread = sum p |v|,
    (the largest sum of a seen score's |terms|, what weights too small for fp16 may be worth)), zeros for rows that see nothing."""
    T, n_q, hd = q.shape
    G = n_q // k.shape[1]
    o, spread, size, lost = np.zeros_like(q), np.zeros_like(q), np.zeros((T, n_q, 1)), np.zeros((T, n_q, 1))
    vis = see[:, None, :]
    for h in range(k.shape[1]):
        at = slice(h * G, (h + 1) * G)
        s = np.where(vis, np.einsum("tgd,nd->tgn", q[:, at], k[:, h]) * scale, -np.inf)
        m = s.max(-1, keepdims=True)
        p = np.exp(s - np.where(np.isinf(m), 0, m))
        t = p.sum(-1, keepdims=True)
        p = p / np.where(t > 0, t, 1)
        o[:, at] = np.einsum("tgn,nd->tgd", p, v[:, h])
        spread[:, at] = np.einsum("tgn,nd->tgd", p, np.abs(v[:, h]))
        size[:, at, 0] = np.where(vis, np.einsum("tgd,nd->tgn", np.abs(q[:, at]), np.abs(k[:, h])) * abs(scale), 0).max(-1)
        if vs is not None:
            lost[:, at, 0] = len(k) * 2.0 ** -32 * 448 * (p * vs[:, h]).max(-1)
    return o, spread, (size, lost)


def attn_tol(ref, spread, more, e8=True):
    """The weights' rounding to fp16 (bf16 over a bf16 cache), half a step of each, and the output's to bf16. Scores: head_dim
    exact products added in fp32, 16 at a time, so up to 17 roundings of 2^-23 of the terms' size, and three more for the
    factor, the reference and 2^x: 2^-18 of the size is above them; a weight is off by as much, and again through the sum.
    fp16 weights w = p vs end at 2^-24, so they are off by 2^-25 beside the half step: the reference's is 2^7, the largest
    at least that, so by 2^-32 of the largest w, times a code of 448 at most, each of the n tokens."""
    size, lost = more
    return ((F16_HALF if e8 else R.BF16_HALF) + 2.0 ** -17 * size + 2.0 ** -19) * spread + R.BF16_HALF * np.abs(ref) + lost + 1e-30
