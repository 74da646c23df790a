"""INT8 pages whose value scales lie far apart, where the page of the large scale
holds zeros: what is left there is the small scales' part, and it has to be right.

Weights times value scales are rounded to f16. Half a step of its smallest numbers is
2^-25; the kernels put the largest weight at 2^15 (decode, chunks at head_dim 256 and on
the cross-check: off by up to 2^-40 of the largest) or between 2^7 and 2^15 (chunks at
head_dim 64 and 128: 2^-32). All other roundings are relative: int8_refs.decode_f64."""
import numpy as np
import pytest
import torch

from tests import int8_refs as R, verify_refs as V
from tests.test_gpu_int8_decode import SMS, Case, _cuda, chunk  # noqa: F401

pytestmark = pytest.mark.gpu


def small_beside_large(d, octaves, hq=8, hkv=2):
    """Value scales 2^-octaves of one page's, whose codes are zero in half of head_dim."""
    c = Case([250, 90], hq, hkv, d, 16, seed=d + octaves, spread=0.5, q_std=0.5)
    cv, sv = R.codes_view(c.v, 16, hkv, d), R.scales(c.v, 16, hkv, d)
    sv[:] *= np.float32(2.0 ** -octaves)
    for b, at in ((0, 7), (1, 0)):
        page = c.tables[b][at]
        cv[page, :, :, d // 2:] = 0
        sv[page] *= np.float32(2.0 ** octaves)
    return c


def check(c, got, qb, tables, lens, lost):
    want, bound = R.decode_f64(qb, c.k, c.v, tables, lens, c.hkv, c.bs, c.scale, lost=lost)
    err = np.abs(got - want)
    assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(err > bound)[:3])
    # the bound says something of the small values: not met by leaving them out
    half = slice(c.d // 2, None)
    assert (bound[..., half] < 0.5 * np.abs(want[..., half]).mean()).all()


@pytest.mark.parametrize("octaves", [12, 20, 27])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_decode(d, octaves):
    c = small_beside_large(d, octaves)
    for got in (c.split(1), c.split(3), c.balanced(SMS), c.balanced(3)):
        check(c, V.f32(got), c.q, c.tables, c.lens, -40)


def test_decode_of_wide_groups():
    for d in (64, 256):
        c = small_beside_large(d, 20, hq=16, hkv=1)
        check(c, V.f32(c.split(2)), c.q, c.tables, c.lens, -40)


@pytest.mark.parametrize("octaves", [12, 20, 22])
@pytest.mark.parametrize("d,crosscheck", [(64, False), (128, False), (256, False), (128, True)])
def test_chunks(d, crosscheck, octaves):
    c = small_beside_large(d, octaves)
    q_lens = [40, 3]
    qb, cu, got = chunk(c, q_lens, crosscheck=crosscheck)
    for b, n in enumerate(q_lens):
        for i in range(0, n, 3):
            at = cu[b] + i
            check(c, got[at][None], qb[at][None], c.tables[b][None],
                  [int(c.lens[b]) - n + i + 1], -40 if d == 256 or crosscheck else -32)
