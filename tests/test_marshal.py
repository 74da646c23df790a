"""The native marshalling of the draft-and-verify calls: it declines, without a
call, whatever it does not take as it is (the Python binding then says why)."""
import pytest
import torch

from paged_kv_split_gb300 import binding as B

M = B._marshal
X = torch.zeros(4, 4)
COUNTS = {"norm_rope": 21, "decode_tree": 22, "compact_tree": 14}


@pytest.mark.parametrize("name,count", sorted(COUNTS.items()))
def test_declines(name, count):
    f = getattr(M, name)
    assert f() is None
    assert f(*[X] * (count - 1)) is None
    assert f(*[X] * count) is None                     # not on a GPU
    assert f(*[None] * count) is None
    assert f(*["text"] * count) is None
    assert f(*[1 << 80] * count) is None
    assert f(*[X] * (count // 2), *[object()] * (count - count // 2)) is None


def test_the_binding_names_what_was_declined():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.pd_decode_tree(q, X, X, X, X, X, q, max_q_len=2, num_kv_heads=2, block_size=16,
                         num_blocks=1, scale=1.0)
    with pytest.raises(ValueError, match="qkv must be"):
        B.pd_qk_norm_rope_cache(q, q, X, X, X, X, X, num_kv_heads=2, block_size=16, num_blocks=1)
    with pytest.raises(ValueError, match="cu_q|CUDA|match"):
        B.pd_compact_tree(X, X, X, X, X, X, X, X, num_kv_heads=2, head_dim=64, block_size=16,
                          num_blocks=1)
