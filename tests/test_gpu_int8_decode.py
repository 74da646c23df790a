"""Decode attention over INT8 pages on the GPU against the 64-bit definition,
every element, within the bound that its roundings allow: both schedules and the
CUDA-core kernel."""
import numpy as np
import pytest
import torch

from tests import gpu_util as U, int8_refs as R, verify_refs as V

pytestmark = pytest.mark.gpu
SMS = 152


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_split_gb300 import binding
    binding.pd_device_status(reset=True)
    yield
    assert binding.pd_device_status(reset=True) == 0


class Case:
    def __init__(self, lens, hq, hkv, d, bs, *, seed=0, spread=3.0, q_std=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.lens = np.array(lens, np.int32)
        self.hq, self.hkv, self.d, self.bs = hq, hkv, d, bs
        self.tables, self.nb = R.paging(self.lens, bs, rng)
        self.q = V.bf16_bits((rng.standard_normal((len(lens), hq, d)) * q_std).astype(np.float32))
        self.k = R.random_cache(rng, self.nb, bs, hkv, d, 0.5)
        self.v = R.random_cache(rng, self.nb, bs, hkv, d, spread)
        # scores of a few units: codes are about 73 in size
        R.scales(self.k, bs, hkv, d)[:] *= np.float32(64 / 73 / np.sqrt(1.0))
        self.scale = 1.0 / np.sqrt(d)

    def args(self):
        return dict(num_kv_heads=self.hkv, block_size=self.bs, num_blocks=self.nb,
                    scale=self.scale, kv_dtype="int8")

    def split(self, num_splits, window=0, crosscheck=False, **kw):
        B = U.pd()
        q = U.bf16_dev(self.q)
        out = torch.full_like(q, 7.0)
        B.pd_decode(q, U.to_dev(self.k), U.to_dev(self.v), U.to_dev(self.tables),
                    U.to_dev(self.lens), out, num_splits=num_splits, sliding_window=window,
                    crosscheck=crosscheck, **self.args(), **kw)
        torch.cuda.synchronize()
        return bits(out)

    def plan(self, sms, window=0):
        return U.pd().pd_balanced_plan(
            self.lens, num_q_heads=self.hq, num_kv_heads=self.hkv, head_dim=self.d,
            block_size=self.bs, max_blocks_per_seq=self.tables.shape[1], sliding_window=window,
            kv_dtype="int8", num_sms=sms)

    def balanced(self, sms, window=0, plan=None):
        B = U.pd()
        plan = self.plan(sms, window) if plan is None else plan
        q = U.bf16_dev(self.q)
        out = torch.full_like(q, 7.0)
        B.pd_decode_balanced(q, U.to_dev(self.k), U.to_dev(self.v), U.to_dev(self.tables),
                             plan.to("cuda"), plan, out, sliding_window=window, **self.args())
        torch.cuda.synchronize()
        return bits(out)

    def check(self, got, window=0):
        want, bound = R.decode_f64(self.q, self.k, self.v, self.tables, self.lens, self.hkv,
                                   self.bs, self.scale, window=window)
        err = np.abs(V.f32(got) - want)
        bad = ~(err <= bound)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], float((err / bound).max()))


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


SHAPES = [  # lens, hq, hkv, d, bs, window
    ([1], 4, 2, 64, 16, 0),
    ([40, 17, 0, 1, 300], 4, 2, 64, 16, 0),
    ([40, 17, 64, 65, 300], 6, 1, 64, 32, 0),
    ([700, 1, 16, 1000, 0, 63], 32, 8, 128, 16, 0),
    ([700, 1, 32, 1000, 31, 95], 64, 8, 128, 32, 0),
    ([130, 513], 16, 1, 128, 16, 0),                    # groups of 16: two column tiles
    ([130, 513, 0], 12, 1, 64, 32, 0),
    ([200, 77], 5, 5, 128, 16, 0),                      # one q head a kv head
    ([700, 20, 260], 8, 4, 256, 16, 100),
    ([700, 20, 260], 32, 2, 256, 32, 0),
    ([300, 41], 16, 2, 512, 16, 0),
    ([300, 41], 16, 1, 512, 32, 77),
    ([700, 20, 260], 32, 8, 128, 16, 100),
    ([700, 20, 260], 4, 2, 64, 32, 1),
]


@pytest.mark.parametrize("lens,hq,hkv,d,bs,window", SHAPES)
def test_against_definition(lens, hq, hkv, d, bs, window):
    c = Case(lens, hq, hkv, d, bs, seed=len(lens) + d)
    for s in (1, 3, 0):
        c.check(c.split(s, window), window)
    c.check(c.split(2, window, crosscheck=True), window)
    for sms in (1, 3, SMS):
        c.check(c.balanced(sms, window), window)


def test_long_context():
    c = Case([9000, 2500], 8, 2, 128, 16, seed=5)
    c.check(c.split(0))
    c.check(c.balanced(SMS))


def test_many_short_sequences():
    rng = np.random.default_rng(6)
    c = Case(rng.integers(0, 40, 500), 4, 2, 64, 16, seed=6)
    c.check(c.split(0))
    c.check(c.balanced(SMS))


@pytest.mark.parametrize("spread", [0.0, 30.0])
@pytest.mark.parametrize("d", [128, 256])
def test_value_scales_far_apart(spread, d):
    """Pages whose value scales differ by 2^60, zero pages at the smallest scale, and
    heads where the keys that matter lie in a zero page."""
    c = Case([500, 80], 8, 2, d, 16, seed=7, spread=spread)
    cv, sv = R.codes_view(c.v, 16, 2, d), R.scales(c.v, 16, 2, d)
    sk = R.scales(c.k, 16, 2, d)
    first = c.tables[0][0]
    cv[first] = 0
    sv[first] = 2.0 ** -60
    sk[first] *= 20
    c.check(c.split(3))
    c.check(c.balanced(3))


@pytest.mark.parametrize("q_std", [1e-20, 1e4])
def test_far_queries(q_std):
    """Tiny scores (the mean of V) and scores that one key takes."""
    c = Case([300, 20], 8, 2, 128, 16, seed=8, q_std=q_std)
    c.check(c.split(2))


def test_rows_that_no_one_sees_may_hold_anything():
    """Bytes behind a sequence's last row, and all of pages outside its window."""
    c = Case([37, 300], 8, 2, 128, 16, seed=9)
    window = 50
    a = c.split(3, window)
    pb = R.page_bytes(16, 2, 128)
    for cache in (c.k, c.v):
        cc = R.codes_view(cache, 16, 2, 128)
        cc[c.tables[0][2], :, 37 - 32:] = -128
        for p in range(0, (300 - window) // 16):
            at = c.tables[1][p]
            cache[at * pb:(at + 1) * pb] = 0xFF          # NaN scales
    assert np.array_equal(a, c.split(3, window))


def test_schedules_and_halves_agree():
    c = Case([700, 33, 260], 32, 8, 128, 16, seed=10)
    B = U.pd()
    q, k, v = U.bf16_dev(c.q), U.to_dev(c.k), U.to_dev(c.v)
    tables, lens = U.to_dev(c.tables), U.to_dev(c.lens)
    ws = torch.empty(B.pd_decode_workspace_bytes(3, 32, 128, 4), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    B.pd_decode_partial(q, k, v, tables, lens, ws, num_splits=4, **c.args())
    B.pd_decode_combine(ws, lens, out, block_size=16, max_blocks_per_seq=tables.shape[1],
                        num_splits=4)
    c.check(bits(out))
    # strided rows, bit for bit
    rows = torch.zeros(3, 32 * 128 + 64, dtype=torch.bfloat16, device="cuda")
    rows[:, :4096] = q.view(3, -1)
    orows = torch.full_like(rows, 5.0)
    B.pd_decode_strided(rows, k, v, tables, lens, orows, num_q_heads=32, head_dim=128, num_splits=4,
                        **c.args())
    assert np.array_equal(bits(orows[:, :4096].contiguous()).reshape(3, 32, 128), c.split(4))
    assert (orows[:, 4096:] == 5.0).all()
    plan = c.plan(3)
    orows.fill_(5.0)
    B.pd_decode_balanced_strided(rows, k, v, tables, plan.to("cuda"), plan, orows, num_q_heads=32,
                                 head_dim=128, **c.args())
    assert np.array_equal(bits(orows[:, :4096].contiguous()).reshape(3, 32, 128), c.balanced(3))


def test_e4m3_output():
    c = Case([300, 20], 8, 2, 128, 16, seed=11)
    B = U.pd()
    out = torch.empty(2, 8, 128, dtype=torch.uint8, device="cuda")
    B.pd_decode_e4m3_out(U.bf16_dev(c.q), U.to_dev(c.k), U.to_dev(c.v), U.to_dev(c.tables),
                         U.to_dev(c.lens), out, out_scale=0.25, num_splits=2, **c.args())
    want, bound = R.decode_f64(c.q, c.k, c.v, c.tables, c.lens, 2, 16, c.scale)
    got = out.view(torch.float8_e4m3fn).double().cpu().numpy() * 0.25
    half = np.maximum(np.abs(want) * 2.0 ** -4, 0.25 * 2.0 ** -10)
    assert (np.abs(got - want) <= half * 1.07 + bound).all()


def test_bad_pages_and_lengths():
    c = Case([100, 50], 4, 2, 64, 16, seed=12)
    B = U.pd()
    keep = c.tables.copy()
    c.tables[0][2] = c.nb
    got = c.split(2)
    assert B.pd_device_status(reset=True) == 1
    # the page's keys drop out: the other keys alone
    order = [0, 1, 3, 4, 5, 6]
    short = Case([84, 50], 4, 2, 64, 16, seed=12)
    short.k, short.v, short.q = c.k, c.v, c.q
    short.tables = keep.copy()
    short.tables[0][:6] = keep[0][order]
    short.lens = np.array([84, 50], np.int32)
    short.nb = c.nb
    short.check(got)
    c.tables = keep
    c.lens = np.array([100, keep.shape[1] * 16 + 5], np.int32)
    c.tables[1] = np.where(c.tables[1] < 0, 0, c.tables[1])
    c.split(2)
    assert B.pd_device_status(reset=True) == 2


PREFILL = [  # lens, q lens, hq, hkv, d, bs, window
    ([40, 17, 300, 5], [3, 17, 65, 0], 4, 2, 64, 16, 0),
    ([130, 700, 64], [30, 100, 1], 32, 8, 128, 16, 0),
    ([130, 700, 64], [30, 100, 64], 12, 1, 128, 32, 60),
    ([200, 333], [77, 40], 8, 4, 256, 16, 0),
    ([200, 333], [20, 333], 16, 2, 64, 32, 100),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,q_lens,hq,hkv,d,bs,window", PREFILL)
def test_chunks_of_prompts(lens, q_lens, hq, hkv, d, bs, window, causal):
    """pd_prefill over the cache: each query row is decode over the keys it sees."""
    c = Case(lens, hq, hkv, d, bs, seed=21)
    T = sum(q_lens)
    qb = V.bf16_bits(c.rng.standard_normal((T, hq, d)).astype(np.float32))
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = U.bf16_dev(qb)
    out = torch.full_like(q, 7.0)
    U.pd().pd_prefill(q, U.to_dev(cu), U.to_dev(c.k), U.to_dev(c.v), U.to_dev(c.tables),
                      U.to_dev(c.lens), out, max_q_len=max(q_lens), causal=causal,
                      sliding_window=window, **c.args())
    torch.cuda.synchronize()
    got = V.f32(bits(out))
    for b, n in enumerate(q_lens):
        for i in range(0, n, 7):
            pos = lens[b] - n + i if causal else lens[b] - 1
            want, bound = R.decode_f64(qb[cu[b] + i][None], c.k, c.v, c.tables[b][None], [pos + 1],
                                       hkv, bs, c.scale, window=window)
            err = np.abs(got[cu[b] + i] - want[0])
            assert (err <= bound[0]).all(), (b, i, float((err / bound[0]).max()))


def test_graph_follows_lengths():
    c = Case([300, 500], 8, 2, 128, 16, seed=13)
    B = U.pd()
    q, k, v = U.bf16_dev(c.q), U.to_dev(c.k), U.to_dev(c.v)
    tables, lens = U.to_dev(c.tables), U.to_dev(c.lens)
    ws = torch.empty(B.pd_decode_workspace_bytes(2, 8, 128, 5), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def step():
        B.pd_decode(q, k, v, tables, lens, out, num_splits=5, workspace=ws, **c.args())
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in ([300, 500], [1, 499], [0, 17], [299, 64]):
        c.lens = np.array(n, np.int32)
        lens.copy_(U.to_dev(c.lens))
        g.replay()
        torch.cuda.synchronize()
        c.check(bits(out))


def test_waits_that_run_out():
    """Consumer waits made to give up: the call returns, says so, and the next one
    is right."""
    B = U.pd()
    for d in (128, 256):
        c = Case([900, 300], 8, 2, d, 16, seed=14)
        try:
            B.pd_test_set_consumer_wait_ns(0)
            c.split(3)
            c.balanced(3)
        finally:
            B.pd_test_set_consumer_wait_ns(0xFFFFFFFF)
        assert B.pd_device_status(reset=True) == 8
        c.check(c.split(3))
        c.check(c.balanced(3))


def test_other_calls_refuse_the_form():
    B = U.pd()
    c = Case([20], 4, 2, 64, 16, seed=15)
    q, k, v = U.bf16_dev(c.q), U.to_dev(c.k), U.to_dev(c.v)
    tables, lens = U.to_dev(c.tables), U.to_dev(c.lens)
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    geom = dict(num_kv_heads=2, block_size=16, num_blocks=c.nb, kv_dtype="int8")
    calls = [
        lambda: B.pd_reshape_and_cache(q[:, :2].contiguous(), q[:, :2].contiguous(), k, v, lens,
                                       num_blocks=c.nb, block_size=16, kv_dtype="int8"),
        lambda: B.pd_decode_tree(q, cu, k, v, tables, lens, torch.empty_like(q), max_q_len=1,
                                 scale=1.0, workspace=torch.empty(1 << 20, dtype=torch.uint8,
                                                                  device="cuda"), **geom),
        lambda: B.pd_compact_tree(k, v, tables, lens, cu, cu[None, :1].contiguous(), lens,
                                  torch.empty_like(lens), num_kv_heads=2, head_dim=64, block_size=16,
                                  num_blocks=c.nb, kv_dtype="int8"),
    ]
    for call in calls:
        with pytest.raises(B.PdError) as e:
            call()
        assert e.value.status == 2


@pytest.mark.parametrize("d", [64, 128, 256])
def test_chunk_ends_inside_a_stage(d):
    """The places of a stage that no page is copied to hold what was there before,
    here NaN from another kernel's rows: no part of the result."""
    B = U.pd()
    foul = torch.full((4096, 16, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.pd_prefill_packed(foul, foul[:, :8], foul[:, :8], U.to_dev(np.array([0, 4096], np.int32)),
                        torch.empty_like(foul), max_q_len=4096, scale=1.0)
    lens = [5 + 16 * (i % 7) for i in range(64)]
    c = Case(lens, 16, 8, d, 16, seed=22)
    qb = V.bf16_bits(c.rng.standard_normal((len(lens), 16, d)).astype(np.float32))
    cu = np.arange(len(lens) + 1, dtype=np.int32)
    q = U.bf16_dev(qb)
    out = torch.full_like(q, 7.0)
    U.pd().pd_prefill(q, U.to_dev(cu), U.to_dev(c.k), U.to_dev(c.v), U.to_dev(c.tables),
                      U.to_dev(c.lens), out, max_q_len=1, **c.args())
    torch.cuda.synchronize()
    want, bound = R.decode_f64(qb, c.k, c.v, c.tables, lens, 8, 16, c.scale)
    assert (np.abs(V.f32(bits(out)) - want) <= bound).all()


def test_the_call_s_scales_are_not_read():
    """k_scale and v_scale are FP8's."""
    c = Case([300, 41], 8, 2, 128, 16, seed=23)
    B = U.pd()
    for kw in (dict(), dict(crosscheck=True)):
        assert np.array_equal(c.split(2, **kw), c.split(2, k_scale=3.0, v_scale=0.0, **kw))
    q, k, v = U.bf16_dev(c.q), U.to_dev(c.k), U.to_dev(c.v)
    cu = U.to_dev(np.arange(3, dtype=np.int32))
    outs = []
    for ks, vs in ((1.0, 1.0), (3.0, 0.0)):
        out = torch.empty_like(q)
        B.pd_prefill(q, cu, k, v, U.to_dev(c.tables), U.to_dev(c.lens), out, max_q_len=1,
                     k_scale=ks, v_scale=vs, **c.args())
        outs.append(out)
    assert torch.equal(*outs)


def chunk(c, q_lens, out=7.0, flags=0, scale=None, seed=0, most=None, **kw):
    """pd_prefill of the case's newest q_lens tokens: (q bits, first rows, outputs)."""
    B = U.pd()
    rng = np.random.default_rng(seed)
    qb = V.bf16_bits(rng.standard_normal((sum(q_lens) + 3, c.hq, c.d)).astype(np.float32))
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = U.bf16_dev(qb)
    out = torch.full_like(q, 7.0)
    args = c.args()
    args["scale"] = c.scale if scale is None else scale
    B.pd_prefill(q, U.to_dev(cu), U.to_dev(c.k), U.to_dev(c.v), U.to_dev(c.tables),
                 U.to_dev(c.lens), out, max_q_len=max(q_lens) if most is None else most, **args, **kw)
    torch.cuda.synchronize()
    assert B.pd_device_status(reset=True) == flags
    return qb, cu, V.f32(bits(out))


@pytest.mark.parametrize("hq,hkv,d,bs", [(16, 2, 128, 16), (4, 4, 64, 32), (16, 1, 64, 16)])
@pytest.mark.parametrize("count", [31, 33, 70])
def test_chunks_of_many_prompts(count, hq, hkv, d, bs):
    rng = np.random.default_rng(count)
    q_lens = rng.integers(0, 90, count)
    q_lens[::4] = q_lens[0]
    lens = q_lens + rng.integers(0, 300, count)
    c = Case(lens, hq, hkv, d, bs, seed=count)
    qb, cu, got = chunk(c, q_lens.tolist(), most=130)
    assert (got[cu[-1]:] == 7.0).all()       # rows of no sequence
    assert not (got[:cu[-1]] == 7.0).all(axis=(1, 2)).any()
    for b in range(count):
        for i in {0, int(q_lens[b]) // 2, int(q_lens[b]) - 1}:
            if 0 <= i < q_lens[b]:
                want, bound = R.decode_f64(qb[cu[b] + i][None], c.k, c.v, c.tables[b][None],
                                           [lens[b] - q_lens[b] + i + 1], hkv, bs, c.scale)
                assert (np.abs(got[cu[b] + i] - want[0]) <= bound[0]).all(), (b, i)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_chunks_at_any_scale(scale, d):
    c = Case([300, 41], 8, 2, d, 16, seed=31)
    q_lens = [100, 41]
    qb, cu, got = chunk(c, q_lens, scale=scale)
    for b in range(2):
        for i in range(0, q_lens[b], 9):
            want, bound = R.decode_f64(qb[cu[b] + i][None], c.k, c.v, c.tables[b][None],
                                       [int(c.lens[b]) - q_lens[b] + i + 1], 2, 16, scale)
            assert (np.abs(got[cu[b] + i] - want[0]) <= bound[0]).all(), (b, i)


@pytest.mark.parametrize("d", [64, 128])
def test_chunks_with_bad_pages_and_counts(d):
    """A page outside the pool: its keys are left out, as if the sequence had not had
    them. Counts that do not fit: nothing is written, the others are right."""
    c = Case([160, 90, 50], 4, 2, d, 16, seed=32)
    keep = c.tables.copy()
    c.tables[0][2] = c.nb + 7
    c.tables[0][9] = -1                     # the last page: a row's own keys
    qb, cu, got = chunk(c, [20, 30, 50], flags=1)
    order = [0, 1, 3, 4, 5, 6, 7, 8]
    few = keep.copy()
    few[0][:8] = keep[0][order]
    for b, n in ((0, 20), (1, 30), (2, 50)):
        for i in range(0, n, 3):
            pos = int(c.lens[b]) - n + i
            keys = min(pos, 143) + 1 - 16 if b == 0 else pos + 1
            want, bound = R.decode_f64(qb[cu[b] + i][None], c.k, c.v, few[b][None], [keys], 2, 16,
                                       c.scale)
            assert (np.abs(got[cu[b] + i] - want[0]) <= bound[0]).all(), (b, i)
    c.tables = keep
    lens = c.lens.copy()
    for bad, q_lens, most in (([160, 20, 50], [20, 30, 50], None),          # fewer keys than rows
                              ([160, keep.shape[1] * 16 + 1, 50], [20, 30, 50], None),
                              ([160, 90, 50], [20, 30, 25], 25)):           # more than max_q_len
        c.lens = np.array(bad, np.int32)
        qb, cu, got = chunk(c, q_lens, flags=2, most=most)
        assert (got[cu[1]:cu[2]] == 7.0).all()
        for b in (0, 2):
            want, bound = R.decode_f64(qb[cu[b]][None], c.k, c.v, keep[b][None],
                                       [int(lens[b]) - q_lens[b] + 1], 2, 16, c.scale)
            assert (np.abs(got[cu[b]] - want[0]) <= bound[0]).all()


def test_chunk_graph_follows_lengths():
    c = Case([300, 500, 64], 8, 2, 128, 16, seed=33)
    B = U.pd()
    T = 200
    qb = V.bf16_bits(c.rng.standard_normal((T, 8, 128)).astype(np.float32))
    q, k, v = U.bf16_dev(qb), U.to_dev(c.k), U.to_dev(c.v)
    tables, lens = U.to_dev(c.tables), U.to_dev(c.lens)
    cu = U.to_dev(np.array([0, 60, 136, 200], np.int32))
    out = torch.empty_like(q)

    def call():
        B.pd_prefill(q, cu, k, v, tables, lens, out, max_q_len=200, **c.args())
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for ls, qs in (([300, 500, 64], [60, 76, 64]), ([5, 320, 0], [0, 200, 0]),
                   ([290, 77, 1], [199, 0, 1])):
        lens.copy_(U.to_dev(np.array(ls, np.int32)))
        cq = np.concatenate([[0], np.cumsum(qs)]).astype(np.int32)
        cu.copy_(U.to_dev(cq))
        g.replay()
        torch.cuda.synchronize()
        got = V.f32(bits(out))
        for b in range(3):
            for i in range(0, qs[b], 11):
                want, bound = R.decode_f64(qb[cq[b] + i][None], c.k, c.v, c.tables[b][None],
                                           [ls[b] - qs[b] + i + 1], 2, 16, c.scale)
                assert (np.abs(got[cq[b] + i] - want[0]) <= bound[0]).all(), (b, i)


@pytest.mark.parametrize("hq,hkv,d,bs,window", [(8, 2, 128, 16, 0), (12, 1, 64, 32, 50)])
def test_chunks_on_the_crosscheck(hq, hkv, d, bs, window):
    c = Case([200, 77], hq, hkv, d, bs, seed=41)
    qb, cu, got = chunk(c, [90, 77], crosscheck=True, sliding_window=window)
    for b, n in ((0, 90), (1, 77)):
        for i in range(0, n, 7):
            want, bound = R.decode_f64(qb[cu[b] + i][None], c.k, c.v, c.tables[b][None],
                                       [int(c.lens[b]) - n + i + 1], hkv, bs, c.scale, window=window)
            assert (np.abs(got[cu[b] + i] - want[0]) <= bound[0]).all(), (b, i)
