"""pd_prefill_packed (and its CUDA-core cross-check) on the GPU against the
64-bit definition, every element, within the bound that its roundings allow."""
import numpy as np
import pytest
import torch

from tests import gpu_util as U, int8_refs as R, verify_refs as V

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_split_gb300 import binding
    binding.pd_device_status(reset=True)
    yield
    assert binding.pd_device_status(reset=True) == 0


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Case:
    def __init__(self, lens, hq, hkv, d, *, seed=0, std=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.lens = [int(n) for n in lens]
        self.cu = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32)
        T = int(self.cu[-1])
        self.hq, self.hkv, self.d = hq, hkv, d
        self.rows = V.bf16_bits((rng.standard_normal((T, (hq + 2 * hkv) * d)) *
                                 std).astype(np.float32))
        x = self.rows.reshape(T, hq + 2 * hkv, d)
        self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        self.scale = 1.0 / np.sqrt(d)

    def views(self, rows):
        x = rows.view(rows.shape[0], self.hq + 2 * self.hkv, self.d)
        return x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]

    def run(self, causal=True, window=0, packed=False, crosscheck=False, most=None, out=None, **kw):
        q, k, v = self.views(U.bf16_dev(self.rows))
        if packed:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        if out is None:
            out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        U.pd().pd_prefill_packed(q, k, v, U.to_dev(self.cu), out,
                                 max_q_len=max(self.lens) if most is None else most,
                                 scale=self.scale, causal=causal, sliding_window=window,
                                 crosscheck=crosscheck, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, causal=True, window=0):
        want, bound = R.packed_f64(self.q, self.k, self.v, self.cu, self.scale, causal=causal,
                                   window=window)
        err = np.abs(V.f32(bits(out)) - want)
        bad = ~(err <= bound)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], float((err / bound).max()))


SHAPES = [  # lens, hq, hkv, d
    ([1], 4, 2, 64),
    ([1, 2, 0, 3, 130, 64], 4, 2, 64),
    ([17, 200, 129], 32, 8, 128),
    ([128, 127, 256, 1], 8, 8, 128),
    ([300, 33], 12, 4, 64),
    ([257, 0, 90], 16, 1, 128),
    ([257, 90], 9, 3, 128),
    ([140, 65], 8, 4, 256),
    ([200, 31], 16, 1, 256),
    ([600], 5, 1, 64),
]


@pytest.mark.parametrize("crosscheck", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,hq,hkv,d", SHAPES)
def test_against_definition(lens, hq, hkv, d, causal, crosscheck):
    c = Case(lens, hq, hkv, d, seed=len(lens) + d)
    for window in (0, 1, 50, 130):
        c.check(c.run(causal, window, crosscheck=crosscheck), causal, window)


def test_packed_and_strided_rows_agree():
    c = Case([130, 257, 5], 8, 2, 128, seed=3)
    a = c.run()
    assert torch.equal(a, c.run(packed=True))
    T = a.shape[0]
    wide = torch.full((T, 8 * 128 + 40), 3.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :1024].unflatten(1, (8, 128))
    c.run(out=out)
    assert torch.equal(a, out.contiguous()) and (wide[:, 1024:] == 3.0).all()


def test_max_q_len_past_the_longest():
    c = Case([130, 20], 8, 2, 64, seed=4)
    assert torch.equal(c.run(), c.run(most=100000))


@pytest.mark.parametrize("std", [1e-15, 30.0])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_far_scores(std, d):
    """Scores near zero, and scores where one key takes the whole weight."""
    c = Case([150, 300], 4, 2, d, seed=5, std=std)
    c.check(c.run())


@pytest.mark.parametrize("scale", [0.0, -0.09, 1.5])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_any_scale(scale, d):
    c = Case([150, 300], 4, 2, d, seed=5)
    c.scale = scale
    c.check(c.run())
    c.check(c.run(window=40), window=40)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rising_scores(d):
    """Each key's score passes the one before: the reference moves in every tile."""
    c = Case([700], 2, 1, d, seed=6)
    x = c.rows.reshape(700, 4, d)
    x[:, :3] = 0
    x[:, :2, 0] = V.bf16_bits(np.full((700, 2), 8.0, np.float32))
    x[:, 2, 0] = V.bf16_bits(np.linspace(0.0, 300.0, 700).astype(np.float32))
    c.check(c.run())
    x[:, 2, 0] = x[::-1, 2, 0].copy()                     # and the other way round
    c.check(c.run())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_other_sequences_do_not_leak(d):
    """NaN and infinities in the rows before, after and between."""
    c = Case([70, 200, 3, 90], 4, 2, d, seed=7)
    a = c.run()
    c.rows[:c.cu[1]] = 0x7FC0
    c.rows[c.cu[2]:c.cu[3]] = 0x7F80
    g = c.run()
    for b in (1, 3):
        assert torch.equal(a[c.cu[b]:c.cu[b + 1]], g[c.cu[b]:c.cu[b + 1]])


def test_bad_counts():
    B = U.pd()
    c = Case([40, 130, 20], 4, 2, 64, seed=8)
    good = c.run()
    out = c.run(most=100)
    assert B.pd_device_status(reset=True) == 2
    assert torch.equal(out[:40], good[:40]) and torch.equal(out[170:], good[170:])
    assert (out[40:170] == 7.0).all()
    c.cu = np.array([0, 40, 170, 191], np.int32)           # a row past the last
    out = c.run()
    assert B.pd_device_status(reset=True) == 2
    assert torch.equal(out[:170], good[:170]) and (out[170:] == 7.0).all()
    c.cu = np.array([0, 40, 30, 190], np.int32)            # a negative count
    c.lens = [40, 0, 160]
    out = c.run(most=200)
    assert B.pd_device_status(reset=True) == 2


def test_rows_of_no_sequence_stay():
    c = Case([40, 60], 4, 2, 64, seed=9)
    c.cu = np.array([8, 40, 90], np.int32)
    out = c.run()
    assert (out[:8] == 7.0).all() and (out[90:] == 7.0).all()
    want, bound = R.packed_f64(c.q, c.k, c.v, c.cu, c.scale)
    err = np.abs(V.f32(bits(out)) - want)[8:90]
    assert (err <= bound[8:90]).all()


def test_many_sequences():
    rng = np.random.default_rng(10)
    c = Case(rng.integers(0, 30, 700), 4, 2, 64, seed=10)
    c.check(c.run())


def test_graph_follows_lengths():
    c = Case([130, 257, 13], 8, 2, 128, seed=11)
    q, k, v = c.views(U.bf16_dev(c.rows))
    cu = U.to_dev(c.cu)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")

    def call():
        U.pd().pd_prefill_packed(q, k, v, cu, out, max_q_len=400, scale=c.scale)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([400, 0, 0], [0, 1, 399], [130, 257, 13]):
        c.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        cu.copy_(U.to_dev(c.cu))
        g.replay()
        torch.cuda.synchronize()
        c.check(out)


def test_long_prompt_against_crosscheck():
    c = Case([3333, 1500], 8, 2, 128, seed=12)
    a, b = c.run().float(), c.run(crosscheck=True).float()
    # two roundings of the output and the rounded weights: a few bf16 steps of V's size
    assert (a - b).abs().max() < 4 * 2.0 ** -8 * b.abs().max()


@pytest.mark.parametrize("hq,hkv,d", [(16, 1, 64), (8, 8, 128), (12, 2, 256)])
@pytest.mark.parametrize("count,longest", [(1, 2500), (31, 500), (32, 700), (33, 700), (64, 300),
                                           (65, 300), (200, 90)])
def test_every_item_is_found(count, longest, hq, hkv, d):
    """Many levels, lengths that repeat, sequences of none, more than a warp of them:
    each row of each sequence is some CTA's, and no other row is touched."""
    rng = np.random.default_rng(count)
    lens = rng.integers(0, longest, count)
    lens[rng.integers(0, count)] = longest
    lens[::5] = lens[0]
    c = Case(np.concatenate([lens, [9]]), hq, hkv, d, seed=count)
    c.cu = c.cu[:-1]
    a, b = c.run().float(), c.run(crosscheck=True).float()
    assert (a[-9:] == 7.0).all() and (b[-9:] == 7.0).all()
    assert (a - b).abs().max() < 4 * 2.0 ** -8 * b.abs().max()
