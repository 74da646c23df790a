"""Tree attention's bounded waits, made to run out on purpose: with a limit of 0
the wait for a piece's first copies is a single probe, so a kernel gives up at the
first piece whose keys (or q rows) have not landed. The call ends, reports PD_DEV_TIMEOUT and leaves the
device usable; the next ordinary call gives the bits of the one before. A call
that reports nothing has found everything landed (some forms are slower than their
copies) and gives the same bits too. Nothing here faults the GPU or waits
without a limit."""
import time

import numpy as np
import pytest
import torch

from tests import gpu_util as U, verify_refs as V

pytestmark = pytest.mark.gpu

PD_DEV_TIMEOUT = 8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_split_gb300 import binding
    binding.pd_device_status(reset=True)
    yield
    binding.pd_test_set_consumer_wait_ns(0xFFFFFFFF)


# seqs, length, nodes, hq, hkv, d, bs
SPLIT = [(8, 6000, 2, 8, 4, 256, 16), (8, 6000, 1, 16, 2, 256, 32), (8, 5000, 1, 16, 2, 512, 16),
         (6, 5000, 7, 8, 2, 512, 32)]

# the tcgen05 kernel: few and many rows, both ways its groups share them, long rings
UMMA = [(24, 4000, 3, 8, 8, 64, 16), (16, 6000, 4, 32, 8, 128, 16), (2, 16000, 40, 32, 8, 128, 32),
        (8, 6000, 24, 8, 4, 256, 16), (4, 5000, 16, 16, 2, 512, 16)]


def run_out(seqs, length, nodes, hq, hkv, d, bs, kv_dtype):
    B = U.pd()
    g = torch.Generator(device="cuda").manual_seed(d)
    rng = np.random.default_rng(d)
    pages = (length + bs - 1) // bs
    nb = seqs * pages
    bt = rng.permutation(nb).astype(np.int32).reshape(seqs, pages)
    caches = [B.empty_cache(kv_dtype, nb, bs, hkv, d) for _ in range(2)]
    kv = [torch.randn(nb * bs, hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2)]
    B.pd_reshape_and_cache(*kv, *caches, torch.arange(nb * bs, dtype=torch.int32, device="cuda"),
                           num_blocks=nb, block_size=bs, kv_dtype=kv_dtype, k_scale=0.0125,
                           v_scale=0.0125)
    masks = [m for _ in range(seqs) for m in V.random_tree(rng, nodes)[0]]
    q = torch.randn(seqs * nodes, hq, d, generator=g, device="cuda").bfloat16()
    args = (U.to_dev(np.arange(0, (seqs + 1) * nodes, nodes).astype(np.int32)), *caches,
            U.to_dev(bt), U.to_dev(np.full(seqs, length, np.int32)))
    kw = dict(tree_mask=U.to_dev(V.masks_to_i64(masks)), max_q_len=nodes, num_kv_heads=hkv,
              block_size=bs, num_blocks=nb, scale=d ** -0.5, kv_dtype=kv_dtype, k_scale=0.0125,
              v_scale=0.0125)
    want = B.pd_decode_tree(q, *args, torch.empty_like(q), **kw)
    assert B.pd_device_status(reset=True) == 0
    prev = B.pd_test_set_consumer_wait_ns(0)
    try:
        seen = 0
        for _ in range(8):
            start = time.monotonic()
            out = B.pd_decode_tree(q, *args, torch.full_like(q, float("nan")), **kw)
            flags = B.pd_device_status(reset=True)
            # (whatever a CTA still waits for at its end comes; a wait alone would take 2 s)
            assert time.monotonic() - start < 1
            assert flags in (0, PD_DEV_TIMEOUT)
            assert flags or torch.equal(out, want)
            seen |= flags
        # BF16 keys of these widths come no faster than they are used: some have not landed
        assert seen or kv_dtype > 0 or d not in (128, 256)
    finally:
        B.pd_test_set_consumer_wait_ns(0xFFFFFFFF)
    assert prev == 2_000_000_000
    for _ in range(2):
        assert torch.equal(B.pd_decode_tree(q, *args, torch.empty_like(q), **kw), want)
    assert B.pd_device_status(reset=True) == 0


@pytest.mark.parametrize("kv_dtype", [0, 1, 2])
@pytest.mark.parametrize("i", range(len(SPLIT)))
def test_waits_run_out_and_the_device_recovers(i, kv_dtype):
    run_out(*SPLIT[i], kv_dtype)


@pytest.mark.parametrize("kv_dtype", [0, 1, 2])
@pytest.mark.parametrize("i", range(len(UMMA)))
def test_on_tcgen05(i, kv_dtype):
    run_out(*UMMA[i], kv_dtype)
