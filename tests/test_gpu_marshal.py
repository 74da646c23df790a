"""The draft-and-verify calls with CUDA tensors that they refuse: an ordinary
error each time, whichever side of the binding finds it."""
import pytest
import torch

from tests import gpu_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def i32(*shape):
    return z(*shape, dtype=torch.int32)


GEOM = dict(num_kv_heads=2, block_size=16, num_blocks=4)
ROWS = dict(num_q_heads=4, head_dim=64)


def strided(q, out, **kw):
    args = dict(max_q_len=2, scale=1.0, workspace=z(1 << 22, dtype=torch.uint8), **GEOM)
    args.update({**ROWS, **kw})
    return U.pd().pd_decode_tree_strided(q, i32(2), z(1 << 14), z(1 << 14), i32(1, 4), i32(1), out,
                                         **args)


def test_rows_of_the_wrong_rank():
    for q in (z(), z(256), z(2, 4, 64)):
        with pytest.raises(ValueError, match="q_rows"):
            strided(q, q)
    with pytest.raises(ValueError, match="out_rows"):
        strided(z(2, 256), z())


@pytest.mark.parametrize("kw", [dict(head_dim=0), dict(head_dim=0, num_q_heads=99),
                                dict(head_dim=None, num_q_heads=None)])
def test_packed_tensors_are_not_rows(kw):
    """3-D tensors belong to pd_decode_tree, whatever head_dim says."""
    q = z(2, 4, 64)
    with pytest.raises(ValueError, match="q_rows"):
        strided(q, q, **kw)


def test_tensors_without_an_address():
    """Inside vmap a tensor has no address to give."""
    with pytest.raises((ValueError, RuntimeError)):
        torch.vmap(lambda q: strided(q, z(2, 256)))(z(3, 2, 256))
    with pytest.raises((ValueError, RuntimeError)):
        torch.vmap(lambda k: U.pd().pd_compact_tree(
            k, z(1 << 14), i32(1, 4), i32(1), i32(2), i32(1, 2), i32(1), i32(1), head_dim=64,
            **GEOM))(z(3, 1 << 14))
    assert U.pd().pd_device_status() == 0
