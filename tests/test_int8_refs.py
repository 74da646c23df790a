"""The INT8 references against simpler statements of what they compute."""
import numpy as np
import pytest

from tests import int8_refs as R, verify_refs as V


def _bits(rng, shape, std=1.0):
    return V.bf16_bits((rng.standard_normal(shape) * std).astype(np.float32))


@pytest.mark.parametrize("steps", [[37], [1] * 37, [5, 1, 11, 20]])
def test_append_error_within_half_steps(steps):
    """A value is off by half its page's scale, and half of each scale the page
    grew to after it went in."""
    rng = np.random.default_rng(len(steps))
    hq, hkv, d, bs = 2, 2, 32, 16
    n = sum(steps)
    cos_sin = V.rope_table_f64(64, 16).astype(np.float32)
    tables, nb = R.paging([n], bs, rng)
    k = np.zeros(nb * R.page_bytes(bs, hkv, d), np.uint8)
    v = np.zeros_like(k)
    qkv = _bits(rng, (n, (hq + 2 * hkv) * d))
    off = np.zeros((n, hkv))           # what each row may be off by (v)
    at = 0
    for m in steps:
        before = R.scales(v, bs, hkv, d).copy()
        R.append_f32(qkv[at:at + m], [0, m], [at + m], cos_sin, k, v, tables, hq, hkv, d, bs)
        after = R.scales(v, bs, hkv, d)
        for i in range(at + m):
            page = tables[0][i // bs]
            if i >= at or (after[page] > before[page]).any():
                grew = (i >= at) | (after[page] > before[page])
                off[i] += np.where(grew, after[page] / 2, 0)
        at += m
    want = V.f32(qkv).reshape(n, -1, d)[:, hq + hkv:].astype(np.float64)
    got = R.values(v, tables[0], n, bs, hkv, d)
    # the product with the reciprocal: 127 codes, three roundings
    assert (np.abs(got - want) <= (off * (1 + 127 * 4 * 2.0 ** -23))[..., None]).all()
    assert np.abs(R.codes(v, bs, hkv, d)[tables[0][0]]).max() == 127


def test_special_values():
    x = np.array([np.nan, np.inf, -np.inf, 0.0, 1e30, -0.4, 0.5, 1.5, 2.5], np.float32)
    assert R.quantise(x, 1.0).tolist() == [0, 127, -127, 0, 127, 0, 0, 2, 2]


def test_decode_single_key():
    rng = np.random.default_rng(0)
    tables, nb = R.paging([1], 16, rng)
    k, v = (R.random_cache(rng, nb, 16, 1, 64) for _ in range(2))
    out, bound = R.decode_f64(_bits(rng, (1, 2, 64)), k, v, tables, [1], 1, 16, 0.1)
    assert np.allclose(out[0, 0], R.values(v, tables[0], 1, 16, 1, 64)[0, 0], rtol=1e-14)
    assert (bound < 0.01 * np.abs(out).max() + 1e-30).all()


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3), (False, 3)])
def test_packed_against_softmax(causal, window):
    rng = np.random.default_rng(1)
    q, k, v = _bits(rng, (9, 2, 16)), _bits(rng, (9, 1, 16)), _bits(rng, (9, 1, 16))
    out, _ = R.packed_f64(q, k, v, [0, 4, 4, 9], 0.25, causal=causal, window=window)
    for r0, r1 in ((0, 4), (4, 9)):
        for t in range(r0, r1):
            last = t if causal else r1 - 1
            keys = range(max(r0, last - window + 1) if window else r0, last + 1)
            e = np.array([np.exp(0.25 * float(V.f32(q[t, 1]).astype(float) @ V.f32(k[j, 0])))
                          for j in keys])
            want = (e[:, None] * np.array([V.f32(v[j, 0]) for j in keys])).sum(0) / e.sum()
            assert np.allclose(out[t, 1], want, rtol=1e-9, atol=1e-12)
