"""examples/draft_and_verify.py on the host: what does not fit its tables is
refused before anything reaches the device."""
import importlib.util
import os
import types

import pytest
import torch


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "draft_and_verify.py")
    spec = importlib.util.spec_from_file_location("draft_and_verify", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


MODEL = types.SimpleNamespace(block_size=16, max_position=4096, vocab=512)


def tokens(*lens):
    return [torch.zeros(n, dtype=torch.int64) for n in lens]


@pytest.mark.parametrize("prompts,pages,kw", [
    (tokens(65, 3), 4, {}),                                   # past the block table
    (tokens(1064), 64, dict(max_position=1000)),              # past the rotation table
    (tokens(8, 0), 4, {}),
    (tokens(8), 4, {}),                                       # fewer prompts than sequences
    ([torch.tensor([1, 512]), torch.tensor([3])], 4, {}),
    ([torch.tensor([1, -1]), torch.tensor([3])], 4, {}),
])
def test_prompts_that_do_not_fit(ex, prompts, pages, kw):
    model = types.SimpleNamespace(**{**vars(MODEL), **kw})
    rows = 1 if len(prompts) == 1 and kw else 2
    with pytest.raises(ValueError):
        ex.DraftAndVerify(model, prompts, torch.zeros(rows, pages, dtype=torch.int32))


@pytest.mark.parametrize("depth", [1, 4, 31])
def test_steps_that_fit_use_no_more_rows(ex, depth):
    """Against a walk in which every step accepts all it can."""
    for rows in range(1, 400, 7):
        for longest in (1, 20, 97):
            lens, steps = longest, 0
            while lens + 1 + 2 * depth <= rows:
                lens, steps = lens + depth + 1, steps + 1
            assert ex.steps_that_fit(longest, rows, depth) == steps
            if steps:
                assert ex.rows_needed(longest, steps, depth) <= rows
            assert ex.rows_needed(longest, steps + 1, depth) > rows


def test_steps_are_counted(ex, monkeypatch):
    """A step, captured or not, beyond the room is refused on the host."""
    monkeypatch.setattr(ex.DraftAndVerify, "_prompts", lambda self, prompts: None)
    run = ex.DraftAndVerify(MODEL, tokens(40, 3), torch.zeros(2, 4, dtype=torch.int32))
    taken = []
    monkeypatch.setattr(ex.DraftAndVerify, "_step", lambda self: taken.append(1))
    captured = ex.Captured(run, types.SimpleNamespace(replay=lambda: taken.append(2)))
    assert run.steps_left == 4                                # 40 + 3 * 5 + 9 rows of 64
    for step in (run.step, captured.replay, run.step, captured.replay):
        step()
    for step in (run.step, captured.replay, run.capture):
        with pytest.raises(ValueError):
            step()
    assert taken == [1, 2, 1, 2]


@pytest.mark.parametrize("steps,seqs", [(32, 8), (500, 8), (32, 150), (1, 1)])
def test_main_sizes_its_tables(ex, steps, seqs):
    lens = [20 + 7 * b for b in range(seqs)]
    pages, positions = ex.sizes(lens, steps, 4)
    assert ex.steps_that_fit(max(lens), min(pages * 16, positions), 4) >= steps


@pytest.mark.parametrize("argv", [["--steps", "0"], ["--seqs", "0"], ["--steps", "-3"],
                                  ["--steps", "100000000", "--seqs", "100"]])
def test_main_refuses(ex, argv, monkeypatch):
    monkeypatch.setattr(ex, "block_tables", lambda *a: pytest.fail("reached the device"))
    with pytest.raises(SystemExit):
        ex.main(argv)
