"""The INT8 cache and packed prompts past 2^31 elements and 2^32 bytes: pages at
the end of a large pool, rows that lie far apart. The same rows near by give the
same bits."""
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


@pytest.mark.parametrize("d,bs,hkv", [(64, 32, 8), (128, 16, 8), (256, 16, 4)])
def test_pages_at_the_end_of_a_large_pool(d, bs, hkv):
    B = U.pd()
    hq, lens, new = 16, [300, 77, 131], [70, 1, 131]
    rng = np.random.default_rng(d)
    tables, nb = R.paging(lens, bs, rng)
    page = B.pd_cache_bytes(B.PD_KV_INT8, 1, bs, hkv, d)
    far = (5 << 30) // page           # the first page behind 5 GiB
    cos = torch.empty(512, d, device="cuda")
    B.pd_rope_table(cos)
    qkv = U.bf16_dev(V.bf16_bits(rng.standard_normal((sum(new), (hq + 2 * hkv) * d)).astype(np.float32)))
    cu = U.to_dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    steps = U.to_dev(np.arange(len(lens) + 1, dtype=np.int32))
    dlens = U.to_dev(np.array(lens, np.int32))
    more = U.to_dev(np.array(lens, np.int32) - 1)
    start = [U.to_dev(R.random_cache(rng, nb, bs, hkv, d)) for _ in range(2)]
    plan = B.pd_balanced_plan(np.array(lens, np.int32), num_q_heads=hq, num_kv_heads=hkv,
                              head_dim=d, block_size=bs, max_blocks_per_seq=tables.shape[1],
                              kv_dtype="int8", num_sms=152)
    results = []
    for shift in (0, far):
        caches = [torch.empty((nb + shift) * page, dtype=torch.uint8, device="cuda")
                  for _ in range(2)]
        for c, s in zip(caches, start):
            c[shift * page:] = s
        bt = U.to_dev((tables + shift).astype(np.int32))
        geom = dict(num_kv_heads=hkv, block_size=bs, num_blocks=nb + shift)
        q = torch.empty(sum(new), hq, d, dtype=torch.bfloat16, device="cuda")
        B.pd_rope_append_int8(qkv, q, *caches, bt, dlens, cu, cos, max_q_len=max(new), **geom)
        rows = torch.zeros_like(q)
        B.pd_prefill(q, cu, *caches, bt, dlens, rows, max_q_len=max(new), scale=d ** -0.5,
                     kv_dtype="int8", **geom)
        one = q[:len(lens)].contiguous()
        B.pd_rope_append_int8(qkv[:len(lens)], one, *caches, bt, more, steps, cos, max_q_len=1, **geom)
        out = [torch.empty_like(one) for _ in range(3)]
        args = dict(scale=d ** -0.5, kv_dtype="int8", **geom)
        B.pd_decode(one, *caches, bt, more, out[0], num_splits=2, **args)
        B.pd_decode_balanced(one, *caches, bt, plan.to("cuda"), plan, out[1], **args)
        B.pd_decode(one, *caches, bt, more, out[2], num_splits=2, crosscheck=True, **args)
        torch.cuda.synchronize()
        results.append([q, rows, one, *out, *(c[shift * page:].clone() for c in caches)])
        del caches
    for i, (near, off) in enumerate(zip(*results)):
        assert torch.equal(near.view(torch.uint8), off.view(torch.uint8)), i


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_far_apart(d):
    B = U.pd()
    hq, hkv, wide, T = 8, 4, 65536, 40000   # 2.6e9 elements
    buf = torch.empty(T, wide, dtype=torch.bfloat16, device="cuda")
    n = (hq + 2 * hkv) * d
    gen = torch.Generator(device="cuda").manual_seed(d)
    buf[:, :n] = torch.randn(T, n, device="cuda", generator=gen)
    near = buf[:, :n].contiguous()
    cu = U.to_dev(np.array([0, 5, 5, 39000, 39700], np.int32))

    def parts(rows):
        return (rows[:, :hq * d].unflatten(1, (hq, d)),
                rows[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                rows[:, (hq + hkv) * d:n].unflatten(1, (hkv, d)))
    out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    far_out = buf[:, n:n + hq * d].unflatten(1, (hq, d))
    far_out.fill_(7.0)
    kw = dict(max_q_len=38995, scale=d ** -0.5, sliding_window=300)
    B.pd_prefill_packed(*parts(near), cu, out, **kw)
    B.pd_prefill_packed(*parts(buf), cu, far_out, **kw)
    torch.cuda.synchronize()
    assert torch.equal(out, far_out)
    assert (out[39700:] == 7.0).all() and not (out[:39700] == 7.0).all(dim=(1, 2)).any()

    # the same rows into a cache
    bs, lens = 16, [5, 0, 38995, 700]
    tables, nb = R.paging(lens, bs, np.random.default_rng(0))
    page = B.pd_cache_bytes(B.PD_KV_INT8, 1, bs, hkv, d)
    cos = torch.empty(40000, d, device="cuda")
    B.pd_rope_table(cos)
    got = []
    for rows in (near, buf):
        k, v = (torch.zeros(nb * page, dtype=torch.uint8, device="cuda") for _ in range(2))
        q = out if rows is near else far_out
        B.pd_rope_append_int8(rows, q, k, v, U.to_dev(tables), U.to_dev(np.array(lens, np.int32)),
                              cu, cos, max_q_len=38995, num_kv_heads=hkv, block_size=bs,
                              num_blocks=nb)
        torch.cuda.synchronize()
        got.append((k, v, q))
    for a, b in zip(*got):
        assert torch.equal(a, b)
