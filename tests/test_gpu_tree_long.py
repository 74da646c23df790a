"""Tree attention over long caches, tens of tiles a CTA, against the definition in
64 bits within the bound of its roundings: whole sequences of a batch, every
element, so that a few keys lost or counted twice in a ring turned many times show."""
import numpy as np
import pytest
import torch

from tests import gpu_util as U, refs, verify_refs as V
from tests.test_gpu_tree import LONG

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_split_gb300 import binding
    binding.pd_device_status(reset=True)
    yield
    assert binding.pd_device_status(reset=True) == 0


@pytest.mark.parametrize("kv_dtype", [0, 1, 2])
@pytest.mark.parametrize("i", range(len(LONG)))
def test_against_the_definition(i, kv_dtype):
    B = U.pd()
    lens, nodes, hq, hkv, d, bs, window, sinks = LONG[i]
    g = torch.Generator(device="cuda").manual_seed(100 + i)
    rng = np.random.default_rng(100 + i)
    pages = [(n + bs - 1) // bs for n in lens]
    nb = sum(pages)
    perm = rng.permutation(nb).astype(np.int32)
    first = np.concatenate([[0], np.cumsum(pages)])
    bt = np.full((len(lens), max(pages)), -1, np.int32)
    for b, p in enumerate(pages):
        bt[b, :p] = perm[first[b]:first[b] + p]
    scale = 0.0125
    caches = [B.empty_cache(kv_dtype, nb, bs, hkv, d) for _ in range(2)]
    kv = [torch.randn(nb * bs, hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2)]
    B.pd_reshape_and_cache(*kv, *caches, torch.arange(nb * bs, dtype=torch.int32, device="cuda"),
                           num_blocks=nb, block_size=bs, kv_dtype=kv_dtype, k_scale=scale,
                           v_scale=scale)
    del kv
    cu = np.cumsum([0] + nodes).astype(np.int32)
    masks = [m for n in nodes for m in V.random_tree(rng, n)[0]]
    # scores of some spread, so that single keys count
    q = (torch.randn(int(cu[-1]), hq, d, generator=g, device="cuda") * 2).bfloat16()
    out = B.pd_decode_tree(q, U.to_dev(cu), *caches, U.to_dev(bt), U.to_dev(np.array(lens, np.int32)),
                           torch.empty_like(q), tree_mask=U.to_dev(V.masks_to_i64(masks)),
                           max_q_len=max(nodes), num_kv_heads=hkv, block_size=bs, num_blocks=nb,
                           scale=d ** -0.5, sliding_window=window, num_sinks=sinks,
                           kv_dtype=kv_dtype, k_scale=scale, v_scale=scale)
    bits = [x.view(torch.int16).cpu().numpy().view(np.uint16) for x in (q, out)]
    for b in sorted({0, len(lens) // 2, len(lens) - 1}):
        own = U.to_dev(bt[b, :pages[b]].astype(np.int64))
        kp, vp = (refs.dequant_pages(c.view(nb, -1)[own].contiguous().view(-1).cpu().numpy(), kv_dtype,
                                     pages[b], bs, hkv, d, scale if kv_dtype == 1 else 1.0)
                  for c in caches)
        rows = slice(cu[b], cu[b + 1])
        want, bound = V.tree_f64(bits[0][rows], [0, nodes[b]], masks[rows], kp, vp,
                                 np.arange(pages[b], dtype=np.int32)[None], [lens[b]], d ** -0.5,
                                 window=window, sinks=sinks, kv_dtype=kv_dtype)
        err = np.abs(V.f32(bits[1][rows]) - want)
        assert (err <= bound).all(), (b, int((err > bound).sum()), float((err / bound).max()))
