"""The draft-and-verify step as a program runs it (examples/draft_and_verify.py):
captured once, replayed while the lengths change on the device, and compared
with decoding the same tokens one at a time through pd_decode."""
import importlib.util
import os

import pytest
import torch

from tests import gpu_util as U

pytestmark = pytest.mark.gpu

# Both paths compute the same scores with differently rounded intermediates.
# Relative to a vector, rounding all its values to bf16 is an error of at most
# 2^-8 and, spread over values, of 2^-8 / sqrt(3); a layer has four (qkv, P,
# attention, its projection), the head one. A score is a dot of the unit-size
# hidden vector with a head column of norm 1: an error of sqrt(9) 2^-8 / sqrt(3)
# = 0.007 in the mean square, and 8 times that over all the scores compared,
# twice since both paths round. Where the cache is quantised, a difference of
# 2^-9 before it becomes a whole step (2^-3 of an FP8 value, 2^-1 of an NVFP4
# one) in that share of the values: sqrt(2^-9 2^-3) = 2^-6 and 2^-5 in the mean
# square, for K and V of two layers: 0.032 and 0.063 in place of 0.007.
TOLERANCE = {"bf16": 16 * 0.007, "fp8_e4m3": 16 * 0.032, "nvfp4": 16 * 0.063}
STEPS = 12


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "draft_and_verify.py")
    spec = importlib.util.spec_from_file_location("draft_and_verify", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def one_at_a_time(ex, model, tables, prompts, streams):
    """Scores before each token of streams [B][k], feeding them token by token:
    the prompts by pd_prefill, the rest by pd_decode."""
    B = U.pd()
    run = ex.DraftAndVerify(model, prompts, tables)
    got = [[run.scores[b]] for b in range(len(prompts))]
    lens = run.lens.clone()
    longest = max(len(s) for s in streams)
    for i in range(longest):
        live = torch.tensor([i < len(s) for s in streams], device=tables.device)
        tok = torch.tensor([s[i] if i < len(s) else 0 for s in streams], device=tables.device)
        seq = torch.arange(len(streams), device=tables.device)
        slots = torch.where(live, ex.slots_of(tables, lens.long(), seq, model.block_size), -1).int()
        positions = lens.clone()
        lens = lens + live.int()

        def attend(layer, rows, out):
            B.pd_decode_strided(rows, model.k[layer], model.v[layer], tables, lens, out,
                                num_q_heads=model.hq, head_dim=model.d, scale=model.d ** -0.5,
                                k_scale=model.kv_scale, v_scale=model.kv_scale, **model.shape())

        scores = model.forward(tok, positions, slots, attend)
        for b in range(len(streams)):
            if i < len(streams[b]):
                got[b].append(scores[b])
    return got, lens


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "nvfp4"])
@pytest.mark.parametrize("block_size", [16, 32])
def test_drafted_decoding_is_one_at_a_time_decoding(example, kv, block_size):
    ex, B = example, U.pd()
    B.pd_device_status(reset=True)
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, ex.Model.vocab, (n,), generator=g) for n in (1, 37, 64, 190)]
    tables = ex.block_tables(len(prompts), 20)
    model = ex.Model(tables.numel(), block_size, ex.KV[kv])
    run = ex.DraftAndVerify(model, prompts, tables)
    first = run.scores.clone()
    graph = run.capture()
    streams = [[] for _ in prompts]
    scores = [[first[b]] for b in range(len(prompts))]
    for _ in range(STEPS):
        graph.replay()
        torch.cuda.synchronize()
        for b, k in enumerate(run.num_emitted.tolist()):
            streams[b] += run.emitted[b, :k].tolist()
            scores[b] += list(run.scores[b, :k].clone())
    assert B.pd_device_status(reset=True) == 0
    assert [len(p) + len(s) for p, s in zip(prompts, streams)] == run.lens.tolist()
    taken = sum(len(s) for s in streams) / STEPS / len(streams)
    assert taken > 1.2                                    # drafts are accepted, and
    assert taken < run.depth + 1                          # not all of them
    fresh = ex.Model(tables.numel(), block_size, ex.KV[kv])
    want, lens = one_at_a_time(ex, fresh, tables, prompts, streams)
    assert torch.equal(lens, run.lens)
    for b, s in enumerate(streams):
        for i, (x, y) in enumerate(zip(scores[b], want[b])):
            assert float((x - y).abs().max()) <= TOLERANCE[kv], (b, i)
            if i < len(s):                                # the token taken is the greedy one
                assert float(y.max() - y[s[i]]) <= 2 * TOLERANCE[kv], (b, i)


def test_replays_are_repeatable(example):
    """The captured step and the eager one, from the same state: the same bits."""
    ex = example
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, ex.Model.vocab, (n,), generator=g) for n in (12, 90)]
    tables = ex.block_tables(2, 16)
    runs = []
    for captured in (False, True):
        model = ex.Model(tables.numel())
        run = ex.DraftAndVerify(model, prompts, tables)
        step = run.capture().replay if captured else run.step
        out = []
        for _ in range(5):
            step()
            out += [x.clone() for x in (run.emitted, run.num_emitted, run.lens, run.tokens)]
        runs.append(out)
    assert all(torch.equal(x, y) for x, y in zip(*runs))
