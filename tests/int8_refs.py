"""Plain references of serving from an INT8 cache (numpy, no library code).

append_f32 follows the documented order of fp32 operations and is compared bit
for bit; the attentions are the definitions in 64 bits, with the elementwise
error bounds that the kernels' roundings allow.
"""
from __future__ import annotations

import numpy as np

from tests import refs, verify_refs as V

SCALE_MIN, SCALE_MAX = np.float32(2.0 ** -60), np.float32(2.0 ** 60)


# ---- pages --------------------------------------------------------------------
def page_bytes(bs, hkv, d):
    return (bs * hkv * d + 4 * hkv + 127) // 128 * 128


def codes(cache: np.ndarray, bs, hkv, d):
    """int8 view [page, head, row, dim] of a flat uint8 cache."""
    n = hkv * bs * d
    return cache.view(np.int8).reshape(-1, page_bytes(bs, hkv, d))[:, :n].reshape(-1, hkv, bs, d)


def codes_view(cache: np.ndarray, bs, hkv, d):
    """The same as a view that can be written."""
    pages = cache.view(np.int8).reshape(-1, page_bytes(bs, hkv, d))
    return np.lib.stride_tricks.as_strided(
        pages, (pages.shape[0], hkv, bs, d), (pages.strides[0], bs * d, d, 1))


def scales(cache: np.ndarray, bs, hkv, d):
    """float32 view [page, head] of a flat uint8 cache."""
    n = hkv * bs * d
    return cache.reshape(-1, page_bytes(bs, hkv, d))[:, n:n + 4 * hkv].view(np.float32)


def random_cache(rng, nb, bs, hkv, d, spread=3.0):
    """nb pages of random codes, their scales spread over 2^(+-spread)."""
    cache = rng.integers(0, 256, nb * page_bytes(bs, hkv, d), dtype=np.uint8)
    c = codes_view(cache, bs, hkv, d)
    c[:] = rng.integers(-127, 128, c.shape, dtype=np.int8)
    scales(cache, bs, hkv, d)[:] = 2.0 ** rng.uniform(-spread, spread, (nb, hkv)) / 64
    return cache


def values(cache, table_row, length, bs, hkv, d):
    """One sequence's rows [length, head, dim] in 64 bits."""
    at = table_row[:(length + bs - 1) // bs]
    x = codes(cache, bs, hkv, d)[at].astype(np.float64) * \
        scales(cache, bs, hkv, d)[at].astype(np.float64)[..., None, None]
    return x.transpose(0, 2, 1, 3).reshape(-1, hkv, d)[:length]


def paging(lens, bs, rng, spare=2):
    """(tables int32 [B, MBS] with -1 behind a sequence's pages, pages of the pool)."""
    pages = [(int(n) + bs - 1) // bs for n in lens]
    total = sum(pages) + spare
    perm = rng.permutation(total)
    table = np.full((len(lens), max(1, max(pages, default=1))), -1, np.int32)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = perm[at:at + p]
        at += p
    return table, total


# ---- append -------------------------------------------------------------------
def rotate_f32(x, cos_sin, positions, interleaved):
    """fp32 [T, H, D], every operation rounded once."""
    rot = cos_sin.shape[1]
    cs = cos_sin[positions][:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    a, b = V._pairs(x, rot, interleaved)
    y = V._unpair(a * c - b * s, b * c + a * s, x[..., rot:], interleaved)
    assert y.dtype == np.float32
    return y


def quantise(x, factor):
    """fp32 -> int8: rint(x * factor) clamped to +-127, NaN to 0."""
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.rint(np.asarray(x, np.float32) * np.float32(factor))
    return np.where(np.isnan(y), 0, np.clip(y, -127, 127)).astype(np.int8)


def append_f32(qkv_bits, cu_q, seq_lens, cos_sin, k_cache, v_cache, tables, hq, hkv, d, bs, *,
               positions=None, interleaved=False):
    """Appends to the caches in place; returns (q bits, k bits) [T, H, D]."""
    T = qkv_bits.shape[0]
    x = V.f32(qkv_bits)[:, :(hq + 2 * hkv) * d].reshape(T, hq + 2 * hkv, d)
    pos = np.zeros(T, np.int64)
    for b in range(len(seq_lens)):
        n = cu_q[b + 1] - cu_q[b]
        pos[cu_q[b]:cu_q[b + 1]] = np.arange(seq_lens[b] - n, seq_lens[b])
    turned = rotate_f32(x[:, :hq + hkv], cos_sin, pos if positions is None else positions,
                        interleaved)
    for cache, rows in ((k_cache, turned[:, hq:]), (v_cache, x[:, hq + hkv:])):
        cc, ss = codes_view(cache, bs, hkv, d), scales(cache, bs, hkv, d)
        for b in range(len(seq_lens)):
            n = cu_q[b + 1] - cu_q[b]
            if n == 0:
                continue
            first = seq_lens[b] - n
            for p in range(first // bs, (seq_lens[b] + bs - 1) // bs):
                lo, hi = max(first, p * bs), min(seq_lens[b], (p + 1) * bs)
                page = tables[b][p]
                for g in range(hkv):
                    new = rows[cu_q[b] + lo - first:cu_q[b] + hi - first, g]
                    fin = np.abs(np.where(np.isfinite(new), new, np.float32(0)))
                    want = min(max(np.float32(fin.max()) / np.float32(127), SCALE_MIN), SCALE_MAX)
                    have, r0 = ss[page, g], lo - p * bs
                    scale = want if r0 == 0 or want > have else have
                    if r0 and want > have:
                        cc[page, g, :r0] = quantise(cc[page, g, :r0], have / scale)
                    cc[page, g, r0:hi - p * bs] = quantise(new, np.float32(1) / scale)
                    ss[page, g] = scale
    return V.bf16_bits(turned[:, :hq]), V.bf16_bits(turned[:, hq:])


# ---- attention ----------------------------------------------------------------
def decode_f64(q_bits, k_cache, v_cache, tables, seq_lens, hkv, bs, scale, *, window=0,
               lost=-25):
    """(out, bound) [B, Hq, D]. The bound: weights times value scales rounded to
    f16, small ones off by up to 2^lost of the largest; scores with D fp32
    additions, each off by at most a full fp32 step of the terms' magnitude, four
    roundings of the score and its factors, log2 of a value scale off by 2^-22 of
    itself, the exponential within 2^-20, one rounding of the output."""
    B, hq, d = q_bits.shape
    G = hq // hkv
    q = refs.bf16_to_f64(q_bits)
    out, bound = np.zeros((B, hq, d)), np.zeros((B, hq, d))
    for b in range(B):
        L = int(seq_lens[b])
        if L == 0:
            continue
        lo = max(0, L - window) if window else 0
        K = values(k_cache, tables[b], L, bs, hkv, d)[lo:]
        W = values(v_cache, tables[b], L, bs, hkv, d)[lo:]
        vs = scales(v_cache, bs, hkv, d).astype(np.float64)[tables[b][np.arange(lo, L) // bs]]
        for h in range(hq):
            g = h // G
            k, v, sv = K[:, g], W[:, g], vs[:, g]
            s = k @ q[b, h] * scale
            p = np.exp(s - s.max())
            l = p.sum()
            o = p @ v / l
            terms = (np.abs(k) @ np.abs(q[b, h])).max() * abs(scale)
            dt = 2 * d * V.HALF_F32 * terms + 4 * V.HALF_F32 * np.abs(s).max() * 1.5 + \
                np.abs(np.log2(sv)).max() * 2.0 ** -22 + \
                V.HALF_F32 * np.abs(s * 1.4427 + np.log2(sv)).max()
            small = 2.0 ** lost * (p * sv).max() * (np.abs(v) / sv[:, None]).sum(0) / l
            out[b, h] = o
            bound[b, h] = (V.HALF_F16 + 2 * dt + 2.0 ** -20) * (p @ np.abs(v) / l) + small + \
                V.HALF_BF16 * np.abs(o)
    return out, bound * 1.01 + 1e-30


def packed_f64(q_bits, k_bits, v_bits, cu_q, scale, *, causal=True, window=0):
    """(out, bound) [T, Hq, D] of prompts over their own rows; the bound as
    verify_refs.tree_f64's with bf16 weights."""
    T, hq, d = q_bits.shape
    hkv = k_bits.shape[1]
    q, k, v = (refs.bf16_to_f64(x) for x in (q_bits, k_bits, v_bits))
    out, bound = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    for b in range(len(cu_q) - 1):
        r0, r1 = int(cu_q[b]), int(cu_q[b + 1])
        n = r1 - r0
        if n == 0:
            continue
        i = np.arange(n)[:, None] if causal else np.full((n, 1), n - 1)
        j = np.arange(n)
        see = j <= i
        if window:
            see &= i - j < window
        for h in range(hq):
            kk, vv, qq = k[r0:r1, h * hkv // hq], v[r0:r1, h * hkv // hq], q[r0:r1, h]
            s = np.where(see, qq @ kk.T * scale, -np.inf)
            p = np.exp(s - s.max(-1, keepdims=True))
            w = p / p.sum(-1, keepdims=True)
            o = w @ vv
            terms = np.where(see, np.abs(qq) @ np.abs(kk).T, 0.0).max(-1, keepdims=True)
            ds = 2 * d * V.HALF_F32 * terms * abs(scale)
            out[r0:r1, h] = o
            bound[r0:r1, h] = (V.HALF_BF16 + 2 * ds + 2.0 ** -20) * (w @ np.abs(vv)) + \
                V.HALF_BF16 * np.abs(o)
    return out, bound * 1.01 + 1e-30
