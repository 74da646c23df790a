"""The library without its native marshalling: not built, not buildable, or
built for another Python or torch."""
import os
import subprocess
import sys

import pytest

from paged_kv_split_gb300 import build

PKG = build.PKG

CALLS = """
import warnings
import torch
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    from paged_kv_split_gb300 import binding as B
assert B.__file__.startswith({root!r}), B.__file__
assert B._marshal is None and any("not used" in str(w.message) for w in said)
assert B.pd_fp8_scale(448.0) == 1.0 and B.pd_page_bytes("bf16", 16, 2, 64) == 4096
q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
X = torch.zeros(4, 4)
for f in (lambda: B.pd_decode_tree(q, X, X, X, X, X, q, max_q_len=2, num_kv_heads=2, block_size=16,
                                   num_blocks=1, scale=1.0),
          lambda: B.pd_qk_norm_rope_cache(q, q, X, X, X, X, X, num_kv_heads=2, block_size=16,
                                          num_blocks=1),
          lambda: B.pd_compact_tree(X, X, X, X, X, X, X, X, num_kv_heads=2, head_dim=64,
                                    block_size=16, num_blocks=1)):
    try:
        f()
    except ValueError:
        continue
    raise AssertionError("taken")
"""


@pytest.fixture
def copy(tmp_path):
    """The built package, by links, in a folder of its own."""
    build.build()
    (tmp_path / "paged_kv_split_gb300" / "_build").mkdir(parents=True)
    for sub, names in (("", [n for n in os.listdir(PKG) if n.endswith((".py", ".so"))]),
                       ("_build", ["marshal.abi"])):
        for name in names:
            os.symlink(os.path.join(PKG, sub, name), tmp_path / "paged_kv_split_gb300" / sub / name)
    return tmp_path


def run(copy, code):
    r = subprocess.run([sys.executable, "-c", code], cwd=copy, text=True, stdout=subprocess.PIPE,
                       stderr=subprocess.STDOUT, env={**os.environ, "PYTHONPATH": str(copy)})
    assert r.returncode == 0, r.stdout[-3000:]


def test_used_when_it_fits(copy):
    run(copy, "from paged_kv_split_gb300 import binding as B; assert B._marshal is not None")


@pytest.mark.parametrize("gone", ["_marshal.so", "_build/marshal.abi"])
def test_not_built(copy, gone):
    os.remove(copy / "paged_kv_split_gb300" / gone)
    run(copy, CALLS.format(root=str(copy)))


@pytest.mark.parametrize("other", ["cpython-39-sparc torch 2.11.0", ""])
def test_built_for_another_python_or_torch(copy, other):
    mark = copy / "paged_kv_split_gb300" / "_build" / "marshal.abi"
    os.remove(mark)
    mark.write_text(other)
    run(copy, CALLS.format(root=str(copy)))
    code = ("from paged_kv_split_gb300 import build as b; "
            "assert not b.is_stale() and b.marshal_is_stale()")
    run(copy, code)


def test_what_cannot_be_built_is_a_warning(tmp_path, monkeypatch):
    """libpd.so does not depend on the headers of torch and Python."""
    build.build()
    for name in ("MARSHAL", "MARSHAL_ABI"):
        monkeypatch.setattr(build, name, str(tmp_path / name))
    src = tmp_path / "broken.cpp"
    src.write_text("#error no headers\n")
    monkeypatch.setattr(build, "MARSHAL_SRC", str(src))
    with pytest.warns(UserWarning, match="was not built"):
        assert build.build() == build.LIB
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    with pytest.warns(UserWarning, match="was not built"):
        assert build.build() == build.LIB
    assert sorted(os.listdir(tmp_path)) == ["broken.cpp"]


def test_the_mark_names_python_and_torch():
    import torch
    assert build.marshal_abi().endswith(f"torch {torch.__version__}")
    assert "cpython-" in build.marshal_abi()
