"""The plain references of the draft-and-verify operators, pinned by other
routes: a single node is windowed decode, a chain is causal prefill, a tree's
node is a chain over its own path; the rotation keeps norms and turns by angle
differences."""
import numpy as np
import pytest

from paged_kv_split_gb300 import inputs
from tests import refs, verify_refs as V


def _case(q_lens, lens, seed=5):
    case = inputs.make_prefill_case("vr", lens, q_lens, 4, 2, 64, 16, seed=seed)
    kp = refs.bf16_to_f64(case.key)
    vp = refs.bf16_to_f64(case.value)
    pages = [np.zeros((case.num_blocks, 16, 2, 64)) for _ in range(2)]
    for p, x in zip(pages, (kp, vp)):
        p.reshape(-1, 2, 64)[case.slot_mapping] = x
    return case, pages


@pytest.mark.parametrize("window", [0, 7, 100])
def test_one_node_is_decode(window):
    case, (kp, vp) = _case([1, 1, 1], [1, 40, 130])
    out, _ = V.tree_f64(case.q, case.extra["cu_q"], [1, 1, 1], kp, vp, case.block_tables,
                        case.seq_lens, case.scale, window=window)
    want = refs.sdpa_f64(case.q, kp, vp, case.block_tables, case.seq_lens, case.scale, window)
    assert np.abs(out - want).max() < 1e-12


@pytest.mark.parametrize("window", [0, 9])
def test_a_chain_is_causal_prefill(window):
    n = [5, 17, 1]
    case, (kp, vp) = _case(n, [5, 60, 33])
    masks = [m for k in n for m in V.chain(k)]
    out, _ = V.tree_f64(case.q, case.extra["cu_q"], masks, kp, vp, case.block_tables,
                        case.seq_lens, case.scale, window=window)
    want = refs.prefill_f64(case.q, case.extra["cu_q"], kp, vp, case.block_tables, case.seq_lens,
                            case.scale, True, window)
    assert np.abs(out - want).max() < 1e-12


def test_a_node_sees_its_path_only():
    rng = np.random.default_rng(3)
    masks, parents = V.random_tree(rng, 12)
    see = V.visible(masks, 20, window=6, sinks=2)
    for i in range(12):
        path, j = [], i
        while j >= 0:
            path.append(j)
            j = parents[j]
        path = path[::-1]
        line = list(range(20)) + [20 + j for j in path]  # row at each position of the path
        want = np.zeros(32, bool)
        for pos, row in enumerate(line):
            if len(line) - 1 - pos < 6 or pos < 2:
                want[row] = True
        assert np.array_equal(see[i], want)


def test_empty_and_padding_nodes():
    see = V.visible([1, 0, 5], 4, window=0)
    assert see[1].tolist() == [True] * 4 + [False] * 3
    assert not V.visible([0], 0).any()
    assert V.visible([1 << 40 | 1], 0).tolist() == [[True]]  # bits past the tree are ignored


def test_rotation_turns_by_position_differences():
    rng = np.random.default_rng(4)
    x = V.bf16_bits(rng.standard_normal((1, 2, 64)).astype(np.float32))
    for inter in (False, True):
        def at(p):
            return V.norm_rope_f64(x, None, np.array([p]), 64, eps=0, offset=0, interleaved=inter)[0]
        for p, q in ((0, 5), (1000, 1005)):
            d = (at(p)[0, 0] * at(q)[0, 1]).sum()
            assert abs(d - (at(0)[0, 0] * at(5)[0, 1]).sum()) < 1e-9
        assert np.allclose(at(0), V.f32(x))


@pytest.mark.parametrize("inter", [False, True])
def test_f32_order_is_within_the_bound(inter):
    rng = np.random.default_rng(5)
    x = V.bf16_bits(rng.standard_normal((9, 3, 128)).astype(np.float32) * 3)
    w = V.bf16_bits(rng.standard_normal(128).astype(np.float32))
    pos = rng.integers(0, 3000, 9)
    table = V.rope_table_f64(3000, 96).astype(np.float32)
    got = V.f32(V.norm_rope_f32(x, w, table, pos, eps=1e-5, offset=1.0, interleaved=inter))
    want, bound = V.norm_rope_f64(x, w, pos, 96, eps=1e-5, offset=1.0, interleaved=inter)
    assert np.all(np.abs(got - want) <= bound)
