"""Plain references of the draft-and-verify operators (numpy, no library code).

norm_rope_f32 follows the documented order of fp32 operations and is compared
bit for bit; norm_rope_f64 and tree_f64 are the definitions in 64 bits, with
the elementwise error bounds that the kernels' roundings allow.
"""
from __future__ import annotations

import numpy as np

from tests import refs

HALF_BF16 = 2.0 ** -8    # half a step of bf16, relative to the value
HALF_F16 = 2.0 ** -11
HALF_F32 = 2.0 ** -24


# ---- norm + rotation --------------------------------------------------------
def rope_table_f64(max_position, rot_dim, base=10000.0):
    i = np.arange(rot_dim // 2)
    ang = np.arange(max_position)[:, None] * base ** (-2.0 * i / rot_dim)
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1)


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """float32 -> bf16 bit patterns, nearest even (finite inputs)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def f32(bits):
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32)


def _pairs(x, rot, interleaved):
    half = rot // 2
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :half], x[..., half:rot])


def _unpair(a, b, rest, interleaved):
    if interleaved:
        turned = np.stack([a, b], -1).reshape(*a.shape[:-1], -1)
    else:
        turned = np.concatenate([a, b], -1)
    return np.concatenate([turned, rest], -1)


def norm_rope_f32(x_bits, weight_bits, cos_sin, positions, *, eps, offset, interleaved):
    """bf16 bits [T, H, D] -> bf16 bits, every fp32 operation rounded once."""
    x = f32(x_bits)
    d = x.shape[-1]
    if weight_bits is not None:
        s = x * x
        while s.shape[-1] > 1:
            s = s[..., 0::2] + s[..., 1::2]
        inv = np.float32(1) / np.sqrt(s * np.float32(1.0 / d) + np.float32(eps))
        x = (x * inv) * (f32(weight_bits) + np.float32(offset))
    rot = cos_sin.shape[1]
    cs = cos_sin[positions][:, None]
    c, sn = cs[..., :rot // 2], cs[..., rot // 2:]
    a, b = _pairs(x, rot, interleaved)
    y = _unpair(a * c - b * sn, b * c + a * sn, x[..., rot:], interleaved)
    assert y.dtype == np.float32
    return bf16_bits(y)


def norm_rope_f64(x_bits, weight_bits, positions, rot, *, eps, offset, interleaved, base=10000.0):
    """The definition in 64 bits, and how far a bf16 result may be from it: half
    a bf16 step, and the fp32 steps before it: 9 levels of the sum and eps at
    half weight (a square root), then root, reciprocal, two products and an add
    of the norm, the table's own rounding, product and sum: 13 half steps of
    |a cos| + |b sin|."""
    x = f32(x_bits).astype(np.float64)
    if weight_bits is not None:
        ms = (x * x).mean(-1, keepdims=True)
        x = x / np.sqrt(ms + eps) * (f32(weight_bits).astype(np.float64) + offset)
    ang = positions[:, None] * base ** (-2.0 * np.arange(rot // 2) / rot)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = _pairs(x, rot, interleaved)
    y = _unpair(a * c - b * s, b * c + a * s, x[..., rot:], interleaved)
    mag = _unpair(np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s),
                  np.abs(x[..., rot:]), interleaved)
    return y, HALF_BF16 * np.abs(y) + 13 * HALF_F32 * mag


# ---- draft trees --------------------------------------------------------------
def random_tree(rng, n):
    """Masks (python ints) of a random tree of n nodes, and its parents."""
    masks, parents = [], []
    for i in range(n):
        p = -1 if i == 0 else (i - 1 if rng.random() < 0.5 else int(rng.integers(0, i)))
        parents.append(p)
        masks.append((masks[p] if p >= 0 else 0) | (1 << i))
    return masks, parents


def chain(n):
    return [(2 << i) - 1 for i in range(n)]


def masks_to_i64(masks):
    return np.array(masks, dtype=np.uint64).view(np.int64) if len(masks) else np.zeros(0, np.int64)


def visible(masks, prefix, window=0, sinks=0):
    """bool [n, prefix + n]: what each node of one sequence sees."""
    n = len(masks)
    masks = [m & ((1 << n) - 1) for m in masks]
    depth = [max(bin(m).count("1") - 1, 0) for m in masks]
    see = np.zeros((n, prefix + n), bool)
    pos = np.concatenate([np.arange(prefix), prefix + np.array(depth, dtype=np.int64)])
    for i in range(n):
        tree = np.array([True] * prefix + [bool((masks[i] >> j) & 1) for j in range(n)])
        near = (window == 0) | (prefix + depth[i] - pos < window) | (pos < sinks)
        see[i] = tree & near
    return see


def tree_f64(q_bits, cu_q, masks, kpages, vpages, block_tables, seq_lens, scale, *, window=0,
             sinks=0, kv_dtype=0):
    """(out, bound) float64 [total_q, Hq, D]; masks: python ints, all nodes in
    order. The bound: P rounded to bf16 (f16 for the widened forms, whose small
    P also lose up to 2^-25 of the row's largest), scores with D fp32 additions,
    each off by at most a full fp32 step of the terms' magnitude, the
    exponential within 2^-20, one rounding of the output."""
    T, Hq, D = q_bits.shape
    hkv = kpages.shape[2]
    g = Hq // hkv
    q = refs.bf16_to_f64(q_bits)
    out, bound = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for b in range(len(seq_lens)):
        r0, r1, L = int(cu_q[b]), int(cu_q[b + 1]), int(seq_lens[b])
        if r1 == r0:
            continue
        see = visible(masks[r0:r1], L - (r1 - r0), window, sinks)
        K = refs.gather_sequence(kpages, block_tables[b], L)
        V = refs.gather_sequence(vpages, block_tables[b], L)
        for h in range(Hq):
            k, v = K[:, h // g], V[:, h // g]
            k = np.where(see.any(0)[:, None], k, 0.0)
            v = np.where(see.any(0)[:, None], v, 0.0)
            s = np.where(see, q[r0:r1, h] @ k.T * scale, -np.inf)
            top = s.max(-1, keepdims=True)
            p = np.where(see, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
            l = p.sum(-1, keepdims=True)
            w = p / np.where(l > 0, l, 1.0)
            o = w @ v
            out[r0:r1, h] = o
            mag = w @ np.abs(v)
            terms = np.where(see, np.abs(q[r0:r1, h]) @ np.abs(k).T, 0.0).max(-1, keepdims=True)
            ds = 2 * D * HALF_F32 * terms * abs(scale)
            half_p = HALF_BF16 if kv_dtype == 0 else HALF_F16
            small = 0.0 if kv_dtype == 0 else 2.0 ** -25 * (see @ np.abs(v)) / np.where(l > 0, l, 1.0)
            bound[r0:r1, h] = (half_p + 2 * ds + 2.0 ** -20) * mag + small + HALF_BF16 * np.abs(o)
    return out, bound * 1.01 + 1e-30  # second-order terms
