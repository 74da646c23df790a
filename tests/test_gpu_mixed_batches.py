"""One long prompt among thousands of short ones, for the kernels that find their work
on the device (pd_prefill_packed, pd_prefill over INT8 pages): every row against the
cross-check kernel, and the call takes about what its parts take. The search for work
goes level by level of the longest prompt; were each level to pass over all sequences,
the mixed batch would take thirteen times its parts and more."""
import numpy as np
import pytest
import torch

from tests import gpu_util as U
from tests.test_gpu_int8_decode import Case as Int8Case
from tests.test_gpu_prefill_packed import Case as PackedCase, _cuda  # noqa: F401

pytestmark = pytest.mark.gpu


def least_us(call, n=7):
    for _ in range(2):
        call()
    best = float("inf")
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


def packed(lens, hq, hkv, d, window=0, crosscheck=False):
    c = PackedCase(lens, hq, hkv, d, seed=len(lens))
    q, k, v = c.views(U.bf16_dev(c.rows))
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    cu = U.to_dev(c.cu)

    def call():
        U.pd().pd_prefill_packed(q, k, v, cu, out, max_q_len=max(c.lens), scale=c.scale,
                                 sliding_window=window, crosscheck=crosscheck)
        return out
    return call


def chunks(lens, hq, hkv, d, window=0, crosscheck=False, bs=32):
    """Every row of a sequence in one chunk."""
    c = Int8Case(lens, hq, hkv, d, bs, seed=len(lens))
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    q = torch.randn(int(cu[-1]), hq, d, generator=torch.Generator("cuda").manual_seed(len(lens)),
                    device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 7.0)
    dev = [U.to_dev(x) for x in (cu, c.k, c.v, c.tables, c.lens)]

    def call():
        U.pd().pd_prefill(q, *dev, out, max_q_len=int(max(lens)), sliding_window=window,
                          crosscheck=crosscheck, **c.args())
        return out
    return call


@pytest.mark.parametrize("make", [packed, chunks])
@pytest.mark.parametrize("place", [0, 1777, 4000])
def test_one_long_prompt_among_many(make, place):
    """8192 tokens (128 levels of 64) and 4000 prompts of one (126 warps of sequences)."""
    short = [1] * 4000
    mixed = short[:place] + [8192] + short[place:]
    shape = (4, 1, 64, 64)
    parts = least_us(make([8192], *shape)) + least_us(make(short, *shape))
    whole = least_us(make(mixed, *shape))
    assert whole < 4 * parts, (whole, parts)


LENS = {
    "one long": lambda r: np.r_[np.ones(255, int), 2048, np.ones(40, int)],
    "long ones apart": lambda r: np.where(np.arange(1100) % 300 == 7, 700, r.integers(0, 3, 1100)),
    "runs of several warps": lambda r: np.where(np.arange(2500) % 997 == 500,
                                                r.integers(300, 900, 2500), r.integers(0, 4, 2500)),
    "every length": lambda r: r.permutation(300),
    "long last, none between": lambda r: np.r_[np.zeros(1500, int), 400, np.zeros(99, int), 33],
}


@pytest.mark.parametrize("make,hq,hkv,d", [(packed, 16, 1, 64), (packed, 8, 4, 128),
                                           (packed, 4, 2, 256), (chunks, 16, 1, 64),
                                           (chunks, 8, 4, 128)])
@pytest.mark.parametrize("lens", LENS)
def test_every_row_is_some_item_s(lens, make, hq, hkv, d):
    lens = LENS[lens](np.random.default_rng(5))
    got = make(lens, hq, hkv, d)().float()
    want = make(lens, hq, hkv, d, crosscheck=True)().float()
    assert not (got == 7.0).all(-1).any()
    # both within their roundings of the definition: a few bf16 steps of V's size
    assert (got - want).abs().max() < 4 * 2.0 ** -8 * want.abs().max()
