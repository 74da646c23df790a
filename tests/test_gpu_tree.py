"""pd_decode_tree on the GPU (and its CUDA-core cross-check) against the 64-bit
definition, every element, within the bound that its roundings allow."""
import numpy as np
import pytest
import torch

from paged_kv_split_gb300 import inputs
from tests import gpu_util as U, refs, verify_refs as V

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_split_gb300 import binding
    binding.pd_device_status(reset=True)
    yield
    assert binding.pd_device_status(reset=True) == 0


def build(lens, nodes, hq, hkv, d, bs, kv_dtype, seed, kind="tree", extra_blocks=0):
    """(case, masks, caches on the device, their dequantised pages, scales)."""
    case = inputs.make_prefill_case("t", lens, nodes, hq, hkv, d, bs, seed=seed,
                                    extra_blocks=extra_blocks)
    rng = np.random.default_rng(seed)
    masks = []
    for n in nodes:
        m = V.chain(n) if kind == "chain" else V.random_tree(rng, n)[0]
        if kind == "padded" and n > 1:
            m[-1] = 0                       # a padding node: sees the prefix only
            m[0] |= 1 << 63 if n < 64 else 0  # a bit past the tree
        masks += m
    ks, vs = (0.011, 0.012) if kv_dtype == 1 else (1.0, 1.0)
    kc, vc = U.gpu_write_cache(case, kv_dtype, ks, vs)
    pages = [refs.dequant_pages(c.cpu().numpy(), kv_dtype, case.num_blocks, bs, hkv, d, s)
             for c, s in ((kc, ks), (vc, vs))]
    return case, masks, (kc, vc), pages, (ks, vs)


def call(case, masks, caches, scales, kv_dtype, window=0, sinks=0, crosscheck=False, out=None,
         most=None, **kw):
    B = U.pd()
    q = U.bf16_dev(case.q)
    out = torch.full_like(q, 7.0) if out is None else out
    B.pd_decode_tree(q, U.to_dev(case.extra["cu_q"]), *caches, U.to_dev(case.block_tables),
                     U.to_dev(case.seq_lens), out,
                     tree_mask=None if masks is None else U.to_dev(V.masks_to_i64(masks)),
                     max_q_len=int(max(case.extra["q_lens"], default=0)) if most is None else most,
                     num_kv_heads=case.num_kv_heads,
                     block_size=case.block_size, num_blocks=case.num_blocks, scale=case.scale,
                     sliding_window=window, num_sinks=sinks, kv_dtype=kv_dtype, k_scale=scales[0],
                     v_scale=scales[1], crosscheck=crosscheck, **kw)
    torch.cuda.synchronize()
    return out.view(torch.int16).cpu().numpy().view(np.uint16)


def check(case, masks, pages, got, kv_dtype, window=0, sinks=0):
    want, bound = V.tree_f64(case.q, case.extra["cu_q"], masks, *pages, case.block_tables,
                             case.seq_lens, case.scale, window=window, sinks=sinks,
                             kv_dtype=kv_dtype)
    err = np.abs(V.f32(got) - want)
    assert np.all(np.isfinite(V.f32(got)))
    bad = err > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], float((err / bound).max()))


SHAPES = [
    # lens, nodes, hq, hkv, d, bs, window, sinks, kind
    ([1], [1], 4, 2, 64, 16, 0, 0, "tree"),
    ([40, 17, 1, 300], [3, 1, 1, 9], 4, 2, 64, 16, 0, 0, "tree"),
    ([130, 700, 64, 65], [16, 5, 16, 1], 32, 8, 128, 16, 0, 0, "tree"),
    ([513, 20, 0, 90], [33, 20, 0, 0], 12, 4, 64, 32, 0, 0, "padded"),
    ([2000, 64], [64, 64], 16, 4, 128, 32, 0, 0, "tree"),
    ([900, 333], [64, 50], 64, 8, 128, 16, 0, 0, "padded"),
    ([1500], [64], 16, 1, 128, 16, 0, 0, "tree"),
    ([777, 100], [7, 2], 5, 5, 128, 16, 0, 0, "tree"),
    ([257, 400], [24, 11], 8, 4, 256, 16, 0, 0, "tree"),
    ([257, 40], [9, 40], 16, 2, 512, 16, 0, 0, "tree"),
    ([130, 700, 64, 65], [16, 5, 16, 1], 32, 8, 128, 16, 100, 4, "tree"),
    ([2500, 1000, 90], [1, 1, 1], 32, 8, 128, 16, 512, 4, "chain"),
    ([600, 350], [12, 30], 4, 2, 64, 16, 5, 3, "tree"),
    ([600, 350, 70], [40, 30, 20], 4, 2, 64, 32, 1, 0, "tree"),
    ([600, 350, 70], [40, 30, 20], 8, 1, 128, 32, 64, 70, "padded"),
    ([3000], [24], 8, 4, 256, 16, 700, 16, "tree"),
    ([300], [24], 2, 2, 256, 32, 33, 200, "tree"),
    ([500, 80], [3, 70 - 10], 16, 2, 512, 32, 90, 2, "tree"),
    ([5, 3, 64], [5, 3, 64], 32, 8, 128, 16, 0, 0, "tree"),
    ([5, 3, 64], [5, 3, 64], 6, 3, 64, 16, 3, 1, "padded"),
    (list(range(1, 150, 5)), [min(n, 1 + n % 7) for n in range(1, 150, 5)], 8, 2, 128, 16, 0, 0,
     "tree"),
    ([70, 333, 0, 33], [20, 64, 0, 33], 5, 5, 512, 16, 0, 0, "padded"),
    ([901], [31], 12, 4, 512, 32, 200, 35, "tree"),
    ([700, 41, 0, 3], [4, 2, 0, 3], 8, 4, 256, 16, 0, 0, "padded"),
    ([1200, 95], [1, 1], 16, 2, 256, 32, 300, 4, "chain"),
]


@pytest.mark.parametrize("kv_dtype", [0, 1, 2])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_against_the_definition(i, kv_dtype):
    lens, nodes, hq, hkv, d, bs, window, sinks, kind = SHAPES[i]
    case, masks, caches, pages, scales = build(lens, nodes, hq, hkv, d, bs, kv_dtype, 300 + i, kind)
    for cross in (True, False):
        got = call(case, masks, caches, scales, kv_dtype, window, sinks, cross)
        check(case, masks, pages, got, kv_dtype, window, sinks)
    if kind == "chain":  # no mask: a chain
        again = call(case, None, caches, scales, kv_dtype, window, sinks)
        assert np.array_equal(again, got)


def test_a_node_that_sees_nothing_is_zero():
    case, _, caches, _, scales = build([4, 70], [4, 3], 8, 2, 128, 16, 0, 1)
    got = call(case, [0, 2, 0, 15, 1, 3, 7], caches, scales, 0)
    assert not got[0].any() and not got[2].any() and got[1].any() and got[3].any()


@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 8), (64, 4, 2), (256, 8, 4), (512, 4, 2),
                                      (512, 8, 2)])
@pytest.mark.parametrize("kv_dtype", [0, 1])
def test_what_no_node_sees_may_be_nan(kv_dtype, d, hq, hkv):
    """Rows past the length, before every window, and padding nodes' own rows
    hold NaN codes; the output is the one without them."""
    bs = 16
    case, masks, caches, pages, scales = build([210, 19], [6, 5], hq, hkv, d, bs, kv_dtype, 77)
    masks[4] = masks[4] & ~(1 << 5)
    masks = [m & ~(1 << 2) if i < 6 else m for i, m in enumerate(masks)]  # node 2 of sequence 0
    got = call(case, masks, caches, scales, kv_dtype, window=60, sinks=3)
    row_bytes = caches[0].numel() // (case.num_blocks * bs)
    seen = [V.visible(masks[:6], 204, 60, 3).any(0), V.visible(masks[6:], 14, 60, 3).any(0)]
    for b in range(2):
        n_pages = (int(case.seq_lens[b]) + bs - 1) // bs
        for r in range(n_pages * bs):
            if r >= case.seq_lens[b] or not seen[b][r]:
                at = int(case.block_tables[b, r // bs]) * bs + r % bs
                for c in caches:
                    c.view(-1, row_bytes)[at] = 0x7F if kv_dtype == 1 else 0xFF
    assert np.array_equal(call(case, masks, caches, scales, kv_dtype, window=60, sinks=3), got)


@pytest.mark.parametrize("cross", [True, False])
def test_bad_lengths_and_pages_are_flagged(cross):
    B = U.pd()
    case, masks, caches, pages, scales = build([50, 40, 60], [4, 4, 4], 8, 2, 128, 16, 0, 5,
                                               extra_blocks=2)
    good = call(case, masks, caches, scales, 0, crosscheck=cross)
    case.seq_lens = case.seq_lens.copy()
    case.seq_lens[1] = 3                       # fewer rows than nodes
    got = call(case, masks, caches, scales, 0, crosscheck=cross)
    assert B.pd_device_status(reset=True) == 2
    assert np.array_equal(got[:4], good[:4]) and np.array_equal(got[8:], good[8:])
    assert (V.f32(got[4:8]) == 7).all()        # not written
    case.seq_lens[1] = 40
    got = call(case, masks, caches, scales, 0, crosscheck=cross, most=3)
    assert B.pd_device_status(reset=True) == 2
    assert (V.f32(got) == 7).all()
    bt = case.block_tables
    case.block_tables = bt.copy()
    case.block_tables[0, 1] = case.num_blocks + 5
    case.block_tables[2, 0] = -3
    got = call(case, masks, caches, scales, 0, crosscheck=cross)
    assert B.pd_device_status(reset=True) == 1
    assert np.array_equal(got[4:8], good[4:8])
    # the rows of a bad page drop out of the softmax
    for b, page in ((0, 1), (2, 0)):
        keep = [r for r in range(int(case.seq_lens[b])) if r // 16 != page]
        q = refs.bf16_to_f64(case.q)[4 * b:4 * b + 4]
        K = refs.gather_sequence(pages[0], bt[b], int(case.seq_lens[b]))[keep]
        Vv = refs.gather_sequence(pages[1], bt[b], int(case.seq_lens[b]))[keep]
        see = V.visible(masks[4 * b:4 * b + 4], int(case.seq_lens[b]) - 4)[:, keep]
        for h in range(8):
            s = np.where(see, q[:, h] @ K[:, h // 4].T * case.scale, -np.inf)
            p = np.exp(s - s.max(-1, keepdims=True))
            want = p / p.sum(-1, keepdims=True) @ Vv[:, h // 4]
            U.assert_close(got[4 * b:4 * b + 4, h], V.bf16_bits(want.astype(np.float32)))


@pytest.mark.parametrize("kv_dtype", [0, 1, 2])
def test_strided_rows_and_other_streams(kv_dtype):
    B = U.pd()
    hq, hkv, d = 32, 8, 128
    case, masks, caches, _, scales = build([300, 41], [7, 12], hq, hkv, d, 16, kv_dtype, 8)
    want = call(case, masks, caches, scales, kv_dtype)
    T = case.q.shape[0]
    rows = torch.full((T, (hq + 2 * hkv) * d), float("nan"), dtype=torch.bfloat16, device="cuda")
    rows[:, :hq * d] = U.bf16_dev(case.q).view(T, -1)
    out = torch.full((T, hq * d + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    args = [U.to_dev(case.extra["cu_q"]), *caches, U.to_dev(case.block_tables),
            U.to_dev(case.seq_lens)]
    mask = U.to_dev(V.masks_to_i64(masks))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        B.pd_decode_tree_strided(rows, *args, out, tree_mask=mask, num_q_heads=hq, head_dim=d,
                                 max_q_len=12, num_kv_heads=hkv, block_size=16,
                                 num_blocks=case.num_blocks, scale=case.scale, kv_dtype=kv_dtype,
                                 k_scale=scales[0], v_scale=scales[1])
    st.synchronize()
    got = out[:, :hq * d].contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    assert np.array_equal(got.reshape(want.shape), want)
    assert (out[:, hq * d:] == 3).all()


def test_permuted_pages_and_repeats_give_the_same_bits():
    B = U.pd()
    case, masks, caches, _, scales = build([3000, 1200, 40], [16, 9, 1], 32, 8, 128, 16, 0, 9)
    want = call(case, masks, caches, scales, 0)
    assert np.array_equal(call(case, masks, caches, scales, 0), want)
    perm = np.random.default_rng(1).permutation(case.num_blocks)
    inv = U.to_dev(np.argsort(perm))
    moved = [c.view(case.num_blocks, -1)[inv].contiguous().view(-1) for c in caches]
    case.block_tables = np.where(case.block_tables >= 0, perm[case.block_tables], -1).astype(np.int32)
    assert np.array_equal(call(case, masks, moved, scales, 0), want)
    assert B.pd_device_status() == 0


@pytest.mark.parametrize("kv_dtype", [0, 2])
@pytest.mark.parametrize("d,scale", [(128, -0.7), (128, 0.0), (64, 3.0), (256, -0.5), (512, 2.0)])
def test_any_scale(d, scale, kv_dtype):
    """A negative scale, none, and one that makes the softmax nearly one-hot."""
    case, masks, caches, pages, scales = build([700, 130], [6, 9], 8, 2, d, 16, kv_dtype, 12)

    class Scaled:
        def __getattr__(self, name):
            return scale if name == "scale" else getattr(case, name)

    s = Scaled()
    check(s, masks, pages, call(s, masks, caches, scales, kv_dtype), kv_dtype)


LONG = [
    # lens, nodes, hq, hkv, d, bs, window, sinks: tens of tiles a CTA, many times round its buffers
    ([9000] * 24, [3] * 24, 8, 8, 64, 16, 0, 0),
    ([12000] * 16, [1] * 16, 16, 8, 128, 16, 0, 0),
    ([12000] * 16, [5] * 16, 16, 8, 128, 32, 9000, 4),
    ([20000, 16000], [64, 40], 32, 8, 128, 16, 0, 0),
    ([9000] * 16, [5] * 16, 16, 8, 256, 16, 0, 0),
    ([6000] * 8, [9] * 8, 16, 2, 512, 16, 0, 0),
    ([9000, 4000], [40, 64], 8, 4, 512, 32, 3000, 20),
    ([9000] * 4, [2] * 4, 16, 2, 512, 16, 0, 0),
    ([9000] * 6, [4] * 6, 8, 4, 256, 16, 0, 0),
]


@pytest.mark.parametrize("kv_dtype", [0, 1, 2])
@pytest.mark.parametrize("i", range(len(LONG)))
def test_long_sequences(i, kv_dtype):
    """Against the CUDA-core kernel, itself compared with the definition above.
    Both are within the definition's bound: P to 16 bits and the output to bf16
    are 2^-8 of values that average |v| <= 1 in the mean square, halved by the
    averaging over thousands of keys; outputs here are below 2^-3."""
    B = U.pd()
    lens, nodes, hq, hkv, d, bs, window, sinks = LONG[i]
    g = torch.Generator(device="cuda").manual_seed(i)
    rng = np.random.default_rng(i)
    pages = [(n + bs - 1) // bs for n in lens]
    nb = sum(pages)
    perm = rng.permutation(nb).astype(np.int32)
    bt = np.full((len(lens), max(pages)), -1, np.int32)
    at = 0
    for b, p in enumerate(pages):
        bt[b, :p] = perm[at:at + p]
        at += p
    caches = [B.empty_cache(kv_dtype, nb, bs, hkv, d) for _ in range(2)]
    slots = torch.arange(nb * bs, dtype=torch.int32, device="cuda")
    kv = [torch.randn(nb * bs, hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2)]
    B.pd_reshape_and_cache(*kv, *caches, slots, num_blocks=nb, block_size=bs, kv_dtype=kv_dtype,
                           k_scale=0.0125, v_scale=0.0125)
    T = sum(nodes)
    masks = [m for n in nodes for m in V.random_tree(rng, n)[0]]
    q = torch.randn(T, hq, d, generator=g, device="cuda").bfloat16()
    outs = []
    for cross in (False, True):
        out = torch.empty_like(q)
        B.pd_decode_tree(q, U.to_dev(np.cumsum([0] + nodes).astype(np.int32)), *caches, U.to_dev(bt),
                         U.to_dev(np.array(lens, np.int32)), out,
                         tree_mask=U.to_dev(V.masks_to_i64(masks)), max_q_len=max(nodes),
                         num_kv_heads=hkv, block_size=bs, num_blocks=nb, scale=d ** -0.5,
                         sliding_window=window, num_sinks=sinks, kv_dtype=kv_dtype, k_scale=0.0125,
                         v_scale=0.0125, crosscheck=cross)
        outs.append(out.float())
    assert B.pd_device_status() == 0
    got, want = outs
    assert float((got - want).abs().max()) <= 2 * 2.0 ** -8 * 2.0 ** -2
    assert float(want.abs().max()) > 2.0 ** -6


def test_many_sequences():
    """More sequences than a CTA has threads, most of them idle or tiny."""
    rng = np.random.default_rng(4)
    nodes = rng.integers(0, 4, 700)
    lens = np.where(nodes > 0, nodes + rng.integers(0, 90, 700), rng.integers(0, 2, 700) * 33)
    case, masks, caches, pages, scales = build(lens, nodes, 4, 2, 64, 16, 0, 10)
    check(case, masks, pages, call(case, masks, caches, scales, 0), 0)


def test_refusals():
    B = U.pd()
    case, masks, caches, _, scales = build([30], [4], 8, 2, 128, 16, 0, 11)
    with pytest.raises(B.PdError):
        call(case, masks, caches, scales, 0, most=65)
    with pytest.raises(ValueError):
        call(case, masks[:3], caches, scales, 0)
    with pytest.raises(B.PdError):
        call(case, masks, caches, scales, 0,
             workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert B.pd_device_status() == 0
