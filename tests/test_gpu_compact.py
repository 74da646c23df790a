"""pd_compact_tree on the GPU, byte for byte against a row-by-row move."""
import numpy as np
import pytest
import torch

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


def _rows(form, page_bytes, hkv, d, bs):
    """Byte indices [bs, row bytes] of a page's rows."""
    if form < 2:
        return np.arange(page_bytes).reshape(bs, -1)
    data = (np.arange(hkv)[:, None, None] * bs + np.arange(bs)[:, None]) * (d // 2) + np.arange(d // 2)
    sc = (bs * hkv * d // 2 + (np.arange(hkv)[:, None, None] * bs + np.arange(bs)[:, None]) *
          (d // 16) + np.arange(d // 16))
    return np.concatenate([data, sc], 2).transpose(1, 0, 2).reshape(bs, -1)


def _batch(seed, B, bs, most):
    rng = np.random.default_rng(seed)
    nodes = rng.integers(0, most + 1, B)
    lens = nodes + rng.integers(0, 3 * bs, B)
    pages = (lens + bs - 1) // bs
    nb = int(pages.sum()) + 2
    perm = rng.permutation(nb)
    bt = np.full((B, max(1, int(pages.max()))), -1, np.int32)
    at = 0
    for b in range(B):
        bt[b, :pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
    acc = np.full((B, most), -7, np.int32)  # entries past the path are not read
    num = np.zeros(B, np.int32)
    for b in range(B):
        k = int(rng.integers(0, nodes[b] + 1))
        path = np.sort(rng.permutation(nodes[b])[:k])
        acc[b, :k], num[b] = path, k
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    return lens.astype(np.int32), nodes, bt, nb, acc, num, cu


def _want(caches, form, bs, hkv, d, pb, bt, lens, nodes, acc, num):
    out = caches.copy()
    rows = _rows(form, pb, hkv, d, bs)
    for b in range(len(lens)):
        p = lens[b] - nodes[b]
        for i in range(num[b]):
            s, t = p + acc[b, i], p + i
            out[:, bt[b, t // bs] * pb + rows[t % bs]] = caches[:, bt[b, s // bs] * pb + rows[s % bs]]
    return out


@pytest.mark.parametrize("form", [0, 1, 2])
@pytest.mark.parametrize("B,layers,hkv,d,bs,most,pad", [
    (1, 1, 2, 64, 16, 5, 0), (7, 3, 8, 128, 16, 17, 64), (5, 2, 4, 256, 32, 64, 0),
    (3, 4, 2, 512, 16, 40, 16), (33, 1, 1, 64, 32, 64, 0)])
def test_moves(form, B, layers, hkv, d, bs, most, pad):
    P = U.pd()
    lens, nodes, bt, nb, acc, num, cu = _batch(B * 10 + d, B, bs, most)
    pb = P.pd_page_bytes(form, bs, hkv, d)
    rng = np.random.default_rng(1)
    kc, vc = (rng.integers(0, 256, (layers, nb * pb + pad), dtype=np.uint8) for _ in range(2))
    k, v = U.to_dev(kc), U.to_dev(vc)
    new = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    P.pd_compact_tree(k, v, U.to_dev(bt), U.to_dev(lens), U.to_dev(cu), U.to_dev(acc),
                      U.to_dev(num), new, num_kv_heads=hkv, head_dim=d, block_size=bs,
                      num_blocks=nb, kv_dtype=form)
    want = [_want(x, form, bs, hkv, d, pb, bt, lens, nodes, acc, num) for x in (kc, vc)]
    assert np.array_equal(k.cpu().numpy(), want[0])
    assert np.array_equal(v.cpu().numpy(), want[1])
    assert np.array_equal(new.cpu().numpy(), lens - nodes + num)


def test_bad_paths_move_nothing():
    P = U.pd()
    hkv, d, bs, nb = 2, 64, 16, 8
    pb = P.pd_page_bytes(0, bs, hkv, d)
    rng = np.random.default_rng(2)
    kc = rng.integers(0, 256, nb * pb, dtype=np.uint8)
    bt = np.arange(8, dtype=np.int32).reshape(8, 1)
    lens = np.full(8, 12, np.int32)
    lens[6], lens[7] = 99, 12            # beyond the table; fine
    cu = (np.arange(9) * 6).astype(np.int32)
    acc = np.array([[0, 2, 1], [0, 0, 3], [0, 6, 0], [-1, 2, 3], [0, 1, 2], [0, 2, 5], [0, 2, 5],
                    [1, 3, 5]], np.int32)
    num = np.array([3, 3, 2, 2, 4, -1, 3, 3], np.int32)
    k, v = U.to_dev(kc), U.to_dev(kc)
    new = torch.full((8,), -1, dtype=torch.int32, device="cuda")
    P.pd_compact_tree(k, v, U.to_dev(bt), U.to_dev(lens), U.to_dev(cu), U.to_dev(acc),
                      U.to_dev(num), new, num_kv_heads=hkv, head_dim=d, block_size=bs,
                      num_blocks=nb)
    assert P.pd_device_status(reset=True) == 128 | 2
    assert new.cpu().tolist() == [6] * 6 + [16, 9]
    want = kc.copy()
    rows = _rows(0, pb, hkv, d, bs)
    for i, a in enumerate([1, 3, 5]):
        want[7 * pb + rows[6 + i]] = kc[7 * pb + rows[6 + a]]
    assert np.array_equal(k.cpu().numpy(), want) and np.array_equal(v.cpu().numpy(), want)


def test_pages_outside_the_pool_are_skipped():
    P = U.pd()
    hkv, d, bs, nb = 1, 64, 16, 4
    pb = P.pd_page_bytes(1, bs, hkv, d)
    kc = np.arange(nb * pb, dtype=np.int64).astype(np.uint8)
    bt = np.array([[0, 9]], np.int32)
    k, v = U.to_dev(kc), U.to_dev(kc)
    new = torch.empty(1, dtype=torch.int32, device="cuda")
    P.pd_compact_tree(k, v, U.to_dev(bt), U.to_dev(np.array([20], np.int32)),
                      U.to_dev(np.array([0, 8], np.int32)),
                      U.to_dev(np.array([[1, 3, 7]], np.int32)),
                      U.to_dev(np.array([3], np.int32)), new, num_kv_heads=hkv, head_dim=d,
                      block_size=bs, num_blocks=nb, kv_dtype=1)
    assert P.pd_device_status(reset=True) == 1
    want = kc.copy()
    rows = _rows(1, pb, hkv, d, bs)
    for i, a in enumerate([1, 3]):  # the third comes from the bad page
        want[rows[12 + i]] = kc[rows[12 + a]]
    assert np.array_equal(k.cpu().numpy(), want)
    assert new.cpu().tolist() == [15]


def test_refusals():
    P = U.pd()
    kc = torch.zeros(2, 1024, dtype=torch.uint8, device="cuda")
    i1 = torch.zeros(1, dtype=torch.int32, device="cuda")
    i2 = torch.zeros(2, dtype=torch.int32, device="cuda")
    t = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    geom = dict(num_kv_heads=1, head_dim=64, block_size=16, num_blocks=1)
    with pytest.raises(P.PdError):  # a layer's cache is 2048 bytes
        P.pd_compact_tree(kc, kc.clone(), t, i1, i2, t, i1, i1.clone(), **geom)
    with pytest.raises(ValueError):
        P.pd_compact_tree(kc, kc[:1], t, i1, i2, t, i1, i1.clone(), **geom)
    with pytest.raises(ValueError):
        P.pd_compact_tree(kc, kc.clone(), t, i1, i1, t, i1, i1.clone(), **geom)
    big = torch.zeros(2, 2048, dtype=torch.uint8, device="cuda")
    with pytest.raises(P.PdError):  # lengths are read by every layer while one writes them
        P.pd_compact_tree(big, big.clone(), t, i1, i2, t, i1, i1, **geom)
