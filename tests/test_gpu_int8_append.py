"""pd_rope_append_int8 on the GPU against the documented order of operations,
bit for bit: q and k rows, codes, scales, and every byte that stays."""
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


class Batch:
    """Sequences with `old` cached rows each and `new` tokens to append."""

    def __init__(self, old, new, hq, hkv, d, bs, *, rot=None, inter=False, seed=0, far=2048, pad=0,
                 std=1.0, spread=3.0):
        self.hq, self.hkv, self.d, self.bs, self.inter = hq, hkv, d, bs, inter
        rng = self.rng = np.random.default_rng(seed)
        self.new = list(new)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.lens = (np.array(old) + np.array(new)).astype(np.int32)
        self.tables, self.nb = R.paging(self.lens, bs, rng)
        T = int(self.cu[-1])
        self.qkv = V.bf16_bits((rng.standard_normal((T, (hq + 2 * hkv) * d + pad)) *
                                std).astype(np.float32))
        self.k = R.random_cache(rng, self.nb, bs, hkv, d, spread)
        self.v = R.random_cache(rng, self.nb, bs, hkv, d, spread)
        B = U.pd()
        self.cos_dev = torch.empty(far, rot or d, device="cuda")
        B.pd_rope_table(self.cos_dev)
        self.cos = self.cos_dev.cpu().numpy()

    def geom(self):
        return dict(num_kv_heads=self.hkv, block_size=self.bs, num_blocks=self.nb)

    def dev(self):
        return (U.bf16_dev(self.qkv), U.to_dev(self.k), U.to_dev(self.v), U.to_dev(self.tables),
                U.to_dev(self.lens), U.to_dev(self.cu))

    def run(self, positions=None, keep_k=True, most=None, **kw):
        B = U.pd()
        qkv, k, v, tables, lens, cu = self.dev()
        T = qkv.shape[0]
        q = torch.full((T, self.hq, self.d), 7.0, dtype=torch.bfloat16, device="cuda")
        ko = torch.full((T, self.hkv, self.d), 7.0, dtype=torch.bfloat16,
                        device="cuda") if keep_k else None
        B.pd_rope_append_int8(qkv, q, k, v, tables, lens, cu, self.cos_dev,
                              max_q_len=max(self.new) if most is None else most, k_out=ko,
                              positions=None if positions is None else U.to_dev(positions),
                              interleaved=self.inter, **self.geom(), **kw)
        torch.cuda.synchronize()
        return q, ko, k, v

    def want(self, positions=None):
        k, v = self.k.copy(), self.v.copy()
        q, ko = R.append_f32(self.qkv, self.cu, self.lens, self.cos, k, v, self.tables, self.hq,
                             self.hkv, self.d, self.bs, positions=positions, interleaved=self.inter)
        return q, ko, k, v

    def check(self, got, want):
        for name, g, w in zip(("q", "k rows"), got[:2], want[:2]):
            if g is not None:
                assert np.array_equal(bits(g), w), name
        for name, g, w in zip(("k cache", "v cache"), got[2:], want[2:]):
            g = g.cpu().numpy()
            assert np.array_equal(R.scales(g, self.bs, self.hkv, self.d),
                                  R.scales(w, self.bs, self.hkv, self.d)), name
            assert np.array_equal(g, w), (name, int((g != w).sum()))


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


SHAPES = [  # hq, hkv, d, bs, rot, interleaved
    (4, 2, 64, 16, 64, False), (4, 2, 64, 32, 32, True), (32, 8, 128, 16, 128, False),
    (64, 8, 128, 32, 128, True), (6, 1, 128, 16, 48, False), (3, 3, 128, 32, 16, True),
    (8, 4, 256, 16, 256, False), (8, 4, 256, 32, 128, True), (16, 2, 512, 16, 512, False),
    (16, 2, 512, 32, 64, False), (5, 5, 64, 16, 48, False), (2, 1, 512, 32, 512, True),
]


@pytest.mark.parametrize("hq,hkv,d,bs,rot,inter", SHAPES)
@pytest.mark.parametrize("old,new", [
    ([0], [1]),
    ([5, 0, 15, 16, 31, 32, 100], [1] * 7),             # a decode step
    ([5, 7, 33], [1, 0, 1]),                            # with an idle sequence
    ([0, 3, 15, 9, 16], [7, 2, 1, 0, 40]),              # short chunks
    ([0, 11], [97, 64]),                                # prompts
])
def test_bits(old, new, hq, hkv, d, bs, rot, inter):
    b = Batch(old, new, hq, hkv, d, bs, rot=rot, inter=inter, seed=len(old) * 31 + d + bs)
    b.check(b.run(), b.want())


@pytest.mark.parametrize("old,new", [([5, 15, 30], [1, 1, 1]), ([5, 15, 30], [4, 18, 3])])
@pytest.mark.parametrize("std", [1e-30, 1e-3, 1.0, 1e4, 1e30])
def test_scales_grow_and_stay(old, new, std):
    """Pages whose scale stays, grows a little, grows so far that old codes vanish,
    and values past both ends of the scale's range."""
    b = Batch(old, new, 4, 2, 128, 16, std=std, seed=3, spread=12.0)
    b.check(b.run(keep_k=False), b.want())


@pytest.mark.parametrize("new", [[1, 1], [20, 5]])
def test_special_values(new):
    b = Batch([3, 14], new, 4, 2, 64, 16, seed=4)
    flat = b.qkv.reshape(-1)
    at = b.rng.permutation(flat.size)[:flat.size // 20]
    flat[at] = b.rng.choice(np.array([0x7F80, 0xFF80, 0x7FC0, 0x0001, 0x8000, 0x7F7F],
                                     np.uint16), at.size)
    q, _, k, v = b.run()
    with np.errstate(all="ignore"):
        wq, _, wk, wv = b.want()
    # rotated NaNs have no one bit pattern; the caches have to agree
    b.check((None, None, k, v), (None, None, wk, wv))
    got, nan = V.f32(bits(q)), np.isnan(V.f32(wq))
    assert np.array_equal(np.isnan(got), nan)
    assert np.array_equal(got[~nan], V.f32(wq)[~nan])


def test_zero_rows():
    b = Batch([0, 4], [3, 1], 4, 2, 64, 16, seed=5)
    b.qkv[:] = 0
    got = b.run()
    b.check(got, b.want())
    s = R.scales(got[3].cpu().numpy(), 16, 2, 64)
    assert (s[b.tables[0][0]] == 2.0 ** -60).all()


@pytest.mark.parametrize("new", [[1, 1, 1], [9, 30, 2]])
def test_given_positions_and_longer_rows(new):
    b = Batch([7, 0, 40], new, 8, 2, 128, 16, seed=6, pad=24)
    pos = b.rng.integers(0, 2048, int(b.cu[-1])).astype(np.int32)
    b.check(b.run(positions=pos), b.want(positions=pos))


@pytest.mark.parametrize("new", [[1, 1, 1], [9, 30, 2]])
def test_in_place(new):
    b = Batch([7, 0, 40], new, 8, 2, 128, 16, seed=7, pad=8)
    B = U.pd()
    qkv, k, v, tables, lens, cu = b.dev()
    B.pd_rope_append_int8_(qkv, k, v, tables, lens, cu, b.cos_dev, max_q_len=max(new),
                           num_q_heads=8, head_dim=128, **b.geom())
    wq, wk, wkc, wvc = b.want()
    T = len(wq)
    rows = bits(qkv)
    assert np.array_equal(rows[:, :8 * 128].reshape(T, 8, 128), wq)
    assert np.array_equal(rows[:, 8 * 128:10 * 128].reshape(T, 2, 128), wk)
    assert np.array_equal(rows[:, 10 * 128:], b.qkv[:, 10 * 128:])
    b.check((None, None, k, v), (None, None, wkc, wvc))


def test_outputs_in_wider_rows_and_other_stream():
    b = Batch([7, 0, 40], [9, 30, 2], 8, 2, 128, 16, seed=8)
    B = U.pd()
    qkv, k, v, tables, lens, cu = b.dev()
    T = qkv.shape[0]
    buf = torch.full((T, 8 * 128 + 2 * 128 + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    q_out = buf[:, :1024].unflatten(1, (8, 128))
    k_out = buf[:, 1024:1280].unflatten(1, (2, 128))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    B.pd_rope_append_int8(qkv, q_out, k, v, tables, lens, cu, b.cos_dev, max_q_len=30, k_out=k_out,
                          stream=st, **b.geom())
    st.synchronize()
    b.check((q_out.contiguous(), k_out.contiguous(), k, v), b.want())
    assert (buf[:, 1280:] == 3.0).all()


def test_token_by_token_in_a_graph():
    """A captured step follows the lengths and tables on the device."""
    b = Batch([13, 0, 31], [1, 1, 1], 4, 2, 64, 16, seed=9)
    B = U.pd()
    tables = np.full((3, 4), -1, np.int32)
    tables[:, :] = b.rng.permutation(12).reshape(3, 4)
    nb = 12
    rng = b.rng
    k = R.random_cache(rng, nb, 16, 2, 64)
    v = R.random_cache(rng, nb, 16, 2, 64)
    kd, vd, td, ld = U.to_dev(k), U.to_dev(v), U.to_dev(tables), U.to_dev(b.lens)
    qkv = U.bf16_dev(b.qkv)
    q = torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    cu = U.to_dev(b.cu)

    def step():
        B.pd_rope_append_int8(qkv, q, kd, vd, td, ld, cu, b.cos_dev, max_q_len=1, num_kv_heads=2,
                              block_size=16, num_blocks=nb)
        ld.add_(1)
    step()
    wk, wv = k.copy(), v.copy()
    lens = b.lens.copy()
    R.append_f32(b.qkv, b.cu, lens, b.cos, wk, wv, tables, 4, 2, 64, 16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(20):
        rows = V.bf16_bits(rng.standard_normal(b.qkv.shape).astype(np.float32))
        qkv.copy_(U.bf16_dev(rows))
        g.replay()
        lens = lens + 1
        R.append_f32(rows, b.cu, lens, b.cos, wk, wv, tables, 4, 2, 64, 16)
    torch.cuda.synchronize()
    assert np.array_equal(kd.cpu().numpy(), wk) and np.array_equal(vd.cpu().numpy(), wv)


@pytest.mark.parametrize("most", [1, 8])
def test_bad_counts_pages_and_positions(most):
    """A sequence that does not fit is skipped, a page outside the pool keeps its
    rows out of the cache, a position past the table is clamped; all are flagged."""
    B = U.pd()
    one = most == 1
    new = [1, 1, 1, 1] if one else [3, 5, 2, 8]
    b = Batch([4, 20, 3, 16], new, 4, 2, 64, 16, seed=10)
    kinds = {"counts": 2, "page": 1, "position": 64}
    for kind, flag in kinds.items():
        lens, tables, cu, positions = b.lens.copy(), b.tables.copy(), b.cu, None
        if kind == "counts":
            lens[1] = tables.shape[1] * 16 + 1
        elif kind == "page":
            tables[1, lens[1] - 1 >> 4] = b.nb
        else:
            positions = np.arange(b.cu[-1]).astype(np.int32)
            positions[b.cu[1]] = 2048
        qkv, k, v, _, _, _ = b.dev()
        q = torch.full((int(b.cu[-1]), 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        B.pd_rope_append_int8(qkv, q, k, v, U.to_dev(tables), U.to_dev(lens), U.to_dev(cu),
                              b.cos_dev, max_q_len=most,
                              positions=None if positions is None else U.to_dev(positions),
                              **b.geom())
        assert B.pd_device_status(reset=True) == flag, kind
        if positions is not None:
            positions[b.cu[1]] = 2047
        wq, _, wk, wv = b.want(positions=positions)
        rows = slice(int(b.cu[1]), int(b.cu[2]))
        if kind == "counts":
            wq[rows] = V.bf16_bits(np.full((1,), 7.0, np.float32))[0]
        assert np.array_equal(bits(q), wq), kind
        for got, want, before in ((k, wk, b.k), (v, wv, b.v)):
            if kind != "position":  # sequence 1's pages are as they were
                at = [p for p in b.tables[1] if p >= 0]
                if kind == "page":
                    at = [b.tables[1][(b.lens[1] - 1) // 16]]
                pb = R.page_bytes(16, 2, 64)
                for p in at:
                    want[p * pb:(p + 1) * pb] = before[p * pb:(p + 1) * pb]
            assert np.array_equal(got.cpu().numpy(), want), kind


def test_counts_past_max_q_len():
    B = U.pd()
    b = Batch([4, 20], [3, 9], 4, 2, 64, 16, seed=11)
    q, _, k, v = b.run(most=8)
    assert B.pd_device_status(reset=True) == 2
    assert (q[3:] == 7.0).all()
    pb = R.page_bytes(16, 2, 64)
    for p in b.tables[1]:
        if p >= 0:
            assert np.array_equal(k.cpu().numpy()[p * pb:(p + 1) * pb], b.k[p * pb:(p + 1) * pb])
