"""pd_qk_norm_rope_cache and pd_rope_table on the GPU: bit for bit against the
documented order of fp32 operations (q rows, and cache bytes through the
oracle's cache write), and within the derived bound of the 64-bit definition."""
import numpy as np
import pytest
import torch

from paged_kv_split_gb300 import inputs
from tests import gpu_util as U, verify_refs as V

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_split_gb300 import binding
    binding.pd_device_status(reset=True)
    yield
    assert binding.pd_device_status(reset=True) == 0


def _table(n, rot, base=10000.0):
    return U.pd().pd_rope_table(torch.empty(n, rot, device="cuda"), base)


@pytest.mark.parametrize("n,rot,base", [(1, 16, 1e4), (5000, 128, 1e4), (131072, 64, 5e5),
                                        (700, 48, 1e4), (33, 512, 1e6)])
def test_table(n, rot, base):
    got = _table(n, rot, base).cpu().numpy()
    want = V.rope_table_f64(n, rot, base)
    # half an fp32 step, and the two 64-bit angles' difference: some 2^-52 steps of the angle
    bound = V.HALF_F32 * np.abs(want) + 8 * 2.0 ** -52 * n
    assert np.all(np.abs(got - want) <= bound)


def _inputs(seed, T, hq, hkv, d, nb, bs, far, extra=0, pad=True):
    rng = np.random.default_rng(seed)
    qkv = inputs.normal_bf16(seed, (T, (hq + 2 * hkv) * d + extra))
    slots = rng.permutation(nb * bs)[:T].astype(np.int32)
    if pad and T > 2:
        slots[rng.integers(0, T)] = -1
    pos = rng.integers(0, far, T).astype(np.int32)
    w = [V.bf16_bits(rng.standard_normal(d).astype(np.float32) * 0.3 + 1) for _ in range(2)]
    return qkv, slots, pos, w


CASES = [
    # T, hq, hkv, d, bs, rot, interleaved, norm, offset
    (1, 4, 2, 64, 16, 64, False, True, 0.0),
    (37, 32, 8, 128, 16, 128, False, True, 0.0),
    (37, 32, 8, 128, 32, 128, True, True, 1.0),
    (19, 5, 5, 128, 16, 48, False, True, 0.0),
    (19, 6, 1, 64, 32, 16, True, False, 0.0),
    (23, 8, 4, 256, 16, 256, False, True, 1.0),
    (23, 8, 4, 256, 16, 96, True, True, 0.0),
    (11, 16, 2, 512, 16, 512, False, True, 0.0),
    (11, 16, 2, 512, 32, 272, False, True, 0.0),
    (11, 3, 1, 512, 16, 496, True, False, 0.0),
    (700, 3, 1, 64, 16, 64, False, True, 0.0),
    (9, 1, 7, 64, 16, 32, False, False, 0.0),
]


@pytest.mark.parametrize("kv_dtype", [0, 1, 2])
@pytest.mark.parametrize("T,hq,hkv,d,bs,rot,inter,norm,offset", CASES)
def test_bits_and_bound(orc, kv_dtype, T, hq, hkv, d, bs, rot, inter, norm, offset):
    B = U.pd()
    nb, far = T // bs + 3, 4000
    qkv, slots, pos, (qw, kw) = _inputs(100 + T + d, T, hq, hkv, d, nb, bs, far)
    table = _table(far, rot)
    kc = torch.full((B.pd_cache_bytes(kv_dtype, nb, bs, hkv, d),), U.SENTINEL, dtype=torch.uint8,
                    device="cuda")
    vc = kc.clone()
    q_out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    ks, vs = 0.013, 0.021
    kw_args = dict(q_weight=U.bf16_dev(qw), k_weight=U.bf16_dev(kw)) if norm else {}
    args = dict(num_kv_heads=hkv, block_size=bs, num_blocks=nb, eps=1e-5, weight_offset=offset,
                interleaved=inter, kv_dtype=kv_dtype, k_scale=ks, v_scale=vs, **kw_args)
    B.pd_qk_norm_rope_cache(U.bf16_dev(qkv), q_out, kc, vc, U.to_dev(pos), U.to_dev(slots), table,
                            **args)
    # in place, rows with a tail that stays
    wide = np.concatenate([qkv, np.full((T, 24), 0x1234, np.uint16)], 1)
    rows = U.bf16_dev(wide)
    kc2, vc2 = torch.full_like(kc, U.SENTINEL), torch.full_like(vc, U.SENTINEL)
    B.pd_qk_norm_rope_cache_(rows, kc2, vc2, U.to_dev(pos), U.to_dev(slots), table,
                             num_q_heads=hq, head_dim=d, **args)
    torch.cuda.synchronize()
    x = qkv.reshape(T, hq + 2 * hkv, d)
    kwr = dict(eps=1e-5, offset=offset, interleaved=inter)
    cs = table.cpu().numpy()
    q_want = V.norm_rope_f32(x[:, :hq], qw if norm else None, cs, pos, **kwr)
    k_want = V.norm_rope_f32(x[:, hq:hq + hkv], kw if norm else None, cs, pos, **kwr)
    got = q_out.view(torch.int16).cpu().numpy().view(np.uint16)
    assert np.array_equal(got, q_want)
    okc = np.full(kc.numel(), U.SENTINEL, np.uint8)
    ovc = okc.copy()
    orc.reshape_and_cache(np.ascontiguousarray(k_want), np.ascontiguousarray(x[:, hq + hkv:]), okc,
                          ovc, slots, hkv, d, bs, nb, kv_dtype, ks, vs)
    assert np.array_equal(kc.cpu().numpy(), okc)
    assert np.array_equal(vc.cpu().numpy(), ovc)
    f, bound = V.norm_rope_f64(x[:, :hq], qw if norm else None, pos, rot, **kwr)
    assert np.all(np.abs(V.f32(got) - f) <= bound)
    r = rows.view(torch.int16).cpu().numpy().view(np.uint16)
    assert np.array_equal(r[:, :hq * d], q_want.reshape(T, -1))
    assert np.array_equal(r[:, hq * d:], wide[:, hq * d:])
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


@pytest.mark.parametrize("kv_dtype", [0, 1, 2])
@pytest.mark.parametrize("scale", [1.0, 1.7, 3.14159 / 448, 2.0 ** -20, 1e6])
def test_every_bf16_pattern_as_v(orc, kv_dtype, scale):
    """All 65536 patterns (NaN payloads, infinities, subnormals) through the V
    write, bit for bit as the oracle's cache write."""
    if kv_dtype != 1 and scale != 1.0:
        pytest.skip("the scale is FP8's")
    B = U.pd()
    d, bs, T = 128, 16, 512
    v = np.arange(65536, dtype=np.uint32).astype(np.uint16).reshape(T, 1, d)
    x = np.zeros((T, 3, d), np.uint16)
    x[:, 2:] = v
    nb = T // bs
    slots = np.arange(T, dtype=np.int32)
    kc = B.empty_cache(kv_dtype, nb, bs, 1, d).zero_()
    vc = kc.clone()
    out = torch.empty(T, 1, d, dtype=torch.bfloat16, device="cuda")
    B.pd_qk_norm_rope_cache(U.bf16_dev(x.reshape(T, -1)), out, kc, vc, U.to_dev(slots * 0),
                            U.to_dev(slots), _table(1, d), num_kv_heads=1, block_size=bs,
                            num_blocks=nb, kv_dtype=kv_dtype, k_scale=scale, v_scale=scale)
    okc, ovc = (np.zeros(kc.numel(), np.uint8) for _ in range(2))
    orc.reshape_and_cache(np.zeros_like(v), v, okc, ovc, slots, 1, d, bs, nb, kv_dtype, scale, scale)
    assert np.array_equal(vc.cpu().numpy(), ovc)


def test_zero_rows_infinities_and_nan():
    """A zero head stays zero, a NaN element spoils its own head alone."""
    B = U.pd()
    T, hq, hkv, d, bs = 3, 2, 1, 128, 16
    x = np.zeros((T, 4, d), np.uint16)
    x[1] = V.bf16_bits(np.ones((4, d), np.float32))
    x[1, 0, 5] = 0x7FC0
    x[2] = V.bf16_bits(np.full((4, d), 2.0 ** 70, np.float32))  # x^2 overflows: the head becomes 0
    one = U.bf16_dev(V.bf16_bits(np.ones(d, np.float32)))
    kc = B.empty_cache(0, 1, bs, hkv, d).zero_()
    vc = kc.clone()
    out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    B.pd_qk_norm_rope_cache(U.bf16_dev(x.reshape(T, -1)), out, kc, vc,
                            torch.zeros(T, dtype=torch.int32, device="cuda"),
                            torch.arange(T, dtype=torch.int32, device="cuda"), _table(4, d),
                            num_kv_heads=hkv, block_size=bs, num_blocks=1, q_weight=one,
                            k_weight=one)
    o = out.float().cpu()
    assert torch.all(o[0] == 0) and torch.all(o[2] == 0)
    assert torch.isnan(o[1, 0]).all() and torch.allclose(o[1, 1], torch.ones(d), atol=1e-2)
    k = kc.view(torch.bfloat16).view(bs, d).float().cpu()
    assert torch.all(k[0] == 0) and torch.allclose(k[1], torch.ones(d), atol=1e-2)


def test_bad_positions_and_slots_are_flagged():
    B = U.pd()
    T, hq, hkv, d, bs, nb = 4, 2, 1, 64, 16, 2
    qkv, _, _, _ = _inputs(9, T, hq, hkv, d, nb, bs, 8)
    table = _table(8, d)
    pos = np.array([3, -5, 100, 7], np.int32)
    slots = np.array([0, 1, 2, nb * bs], np.int32)
    kc = torch.full((B.pd_cache_bytes(0, nb, bs, hkv, d),), U.SENTINEL, dtype=torch.uint8,
                    device="cuda")
    vc = kc.clone()
    out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    B.pd_qk_norm_rope_cache(U.bf16_dev(qkv), out, kc, vc, U.to_dev(pos), U.to_dev(slots), table,
                            num_kv_heads=hkv, block_size=bs, num_blocks=nb)
    assert B.pd_device_status(reset=True) == 64 | 4
    want = V.norm_rope_f32(qkv.reshape(T, 4, d)[:, :hq], None, table.cpu().numpy(),
                           np.clip(pos, 0, 7), eps=0, offset=0, interleaved=False)
    assert np.array_equal(out.view(torch.int16).cpu().numpy().view(np.uint16), want)
    assert (kc.view(nb * bs, -1)[3:] == U.SENTINEL).all()


def test_no_tokens_and_refusals():
    B = U.pd()
    d, bs, nb = 64, 16, 1
    kc = B.empty_cache(0, nb, bs, 1, d)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    table = _table(8, d)
    out = torch.empty(0, 2, d, dtype=torch.bfloat16, device="cuda")
    qkv = torch.empty(0, 4 * d, dtype=torch.bfloat16, device="cuda")
    args = dict(num_kv_heads=1, block_size=bs, num_blocks=nb)
    B.pd_qk_norm_rope_cache(qkv, out, kc, kc, e, e, table, **args)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        B.pd_qk_norm_rope_cache(qkv, out, kc, kc, e, e, table, q_weight=w, **args)
    with pytest.raises(ValueError):
        B.pd_qk_norm_rope_cache(qkv[:, :3 * d], out, kc, kc, e, e, table, **args)
    with pytest.raises(ValueError):
        B.pd_qk_norm_rope_cache(qkv, out, kc, kc, e.long(), e, table, **args)
    with pytest.raises(B.PdError):
        B.pd_qk_norm_rope_cache(qkv, out, kc, kc, e, e, _table(8, 80), **args)
