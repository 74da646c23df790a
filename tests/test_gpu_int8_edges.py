"""What calls that are flagged leave of the other sequences, and the edges of batches:
rows of no sequence, the most sequences, the same call twice."""
import numpy as np
import pytest
import torch

from tests import gpu_util as U, int8_refs as R, verify_refs as V
from tests.test_gpu_int8_append import Batch, bits as append_bits
from tests.test_gpu_int8_decode import SMS, Case, _cuda, chunk  # noqa: F401
from tests.test_gpu_mixed_batches import packed
from tests.test_gpu_prefill_packed import Case as PackedCase, bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
def test_packed_negative_count(d):
    """The sequence before and the one behind are right, but for the rows that both
    have."""
    c = PackedCase([40, 0, 160], 4, 2, d, seed=8)
    c.rows = c.rows[:190]
    x = c.rows.reshape(190, 8, d)
    c.q, c.k, c.v = x[:, :4], x[:, 4:6], x[:, 6:]
    c.cu = np.array([0, 40, 30, 190], np.int32)
    for crosscheck in (False, True):
        got = V.f32(bits(c.run(most=200, crosscheck=crosscheck)))
        assert U.pd().pd_device_status(reset=True) == 2
        for cu, rows in (([0, 40], slice(0, 30)), ([30, 190], slice(40, 190))):
            want, bound = R.packed_f64(c.q, c.k, c.v, cu, c.scale)
            assert (np.abs(got - want) <= bound)[rows].all()


@pytest.mark.parametrize("d,bs", [(64, 16), (128, 32), (256, 16), (512, 16)])
def test_decode_length_past_the_table(d, bs):
    """Clamped to the block table's rows; the others are as they were. Negative: none."""
    B = U.pd()
    c = Case([100, 50, 70], 4, 2, d, bs, seed=12)
    cap = c.tables.shape[1] * bs
    c.tables[1] = np.where(c.tables[1] < 0, c.tables[0][0], c.tables[1])
    c.lens[1] = cap + 5
    c.lens[2] = -3
    for kw in (dict(), dict(crosscheck=True)):
        got = c.split(2, **kw)
        assert B.pd_device_status(reset=True) == 2
        want, bound = R.decode_f64(c.q, c.k, c.v, c.tables, [100, cap, 0], 2, bs, c.scale)
        assert (np.abs(V.f32(got) - want) <= bound).all()
        assert (V.f32(got)[2] == 0).all()


@pytest.mark.parametrize("new", [[1, 0, 1], [5, 0, 20]])
def test_append_rows_of_no_sequence(new):
    """Rows before the first sequence and behind the last: neither read into a cache nor
    written."""
    b = Batch([7, 3, 40], new, 4, 2, 64, 16, seed=7)
    B = U.pd()
    wq, wk, wkc, wvc = b.want()
    qkv, k, v, tables, lens, _ = b.dev()
    T = len(wq)
    wide = torch.full((T + 9, qkv.shape[1]), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[4:4 + T] = qkv
    q = torch.full((T + 9, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((T + 9, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    B.pd_rope_append_int8(wide, q, k, v, tables, lens, U.to_dev((b.cu + 4).astype(np.int32)),
                          b.cos_dev, max_q_len=max(new), k_out=ko, **b.geom())
    torch.cuda.synchronize()
    for t in (q, ko):
        assert (t[:4] == 7.0).all() and (t[4 + T:] == 7.0).all()
    b.check((q[4:4 + T].contiguous(), ko[4:4 + T].contiguous(), k, v), (wq, wk, wkc, wvc))


def test_most_sequences():
    """65535 of one or two tokens, one longer; one more is refused."""
    lens = np.random.default_rng(1).integers(1, 3, 65535)
    lens[40000] = 300
    got, want = (packed(lens, 2, 1, 64, crosscheck=x)().float() for x in (False, True))
    assert not (got == 7.0).all(-1).any()
    assert (got - want).abs().max() < 4 * 2.0 ** -8 * want.abs().max()
    with pytest.raises(U.pd().PdError) as e:
        packed(np.ones(65536, int), 2, 1, 64)()
    assert e.value.status == 1


@pytest.mark.parametrize("d", [64, 128, 256])
def test_the_same_call_twice_gives_the_same_bits(d):
    c = Case([700, 33, 260], 8, 2, d, 16, seed=10)
    for f in (lambda: c.split(3), lambda: c.balanced(SMS), lambda: chunk(c, [90, 33, 1])[2]):
        first = f()
        for _ in range(5):
            assert np.array_equal(first, f())
    p = PackedCase([700, 33, 260], 8, 2, d, seed=10)
    first = p.run()
    for _ in range(5):
        assert torch.equal(first, p.run())


@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_decode_on_another_stream(d):
    """The call follows its stream argument, its workspace too."""
    B = U.pd()
    c = Case([300, 41], 8, 2, d, 16, seed=3)
    want = c.split(3)
    st = torch.cuda.Stream()
    q, out = U.bf16_dev(c.q), torch.full((2, 8, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v, tables, lens = (U.to_dev(x) for x in (c.k, c.v, c.tables, c.lens))
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        B.pd_decode(q, k, v, tables, lens, out, num_splits=3, **c.args())
    B.pd_decode(q, k, v, tables, lens, torch.empty_like(out), num_splits=3, stream=st, **c.args())
    st.synchronize()
    assert np.array_equal(append_bits(out), want)


@pytest.mark.parametrize("lens,hq,hkv,d", [([300, 1, 77, 130], 8, 2, 128), ([257, 90], 9, 3, 128),
                                           ([5, 600, 64], 4, 4, 64), ([200, 31], 16, 1, 256)])
def test_packed_in_place(lens, hq, hkv, d):
    """The q heads of fused rows replaced by the outputs; k and v heads stay."""
    c = PackedCase(lens, hq, hkv, d, seed=9)
    want = c.run()
    for crosscheck in (False, True):
        alone = c.run(crosscheck=crosscheck)
        rows = U.bf16_dev(c.rows)
        before = rows.clone()
        q, k, v = c.views(rows)
        U.pd().pd_prefill_packed(q, k, v, U.to_dev(c.cu), q, max_q_len=max(lens), scale=c.scale,
                                 crosscheck=crosscheck)
        torch.cuda.synchronize()
        assert torch.equal(q, alone)
        assert torch.equal(rows[:, hq * d:], before[:, hq * d:])
    assert torch.equal(want, c.run())
