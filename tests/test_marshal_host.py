"""The native marshalling on tensors it looks into: built here for CPU tensors,
the library's calls replaced by stubs that return a number. Whatever it does not
take, it declines; nothing that a tensor throws ends the process."""
import os
import subprocess
import sys

import pytest

from paged_kv_split_gb300 import build

STUBS = """
#define PD_MARSHAL_DEVICE at::kCPU
#include "%s"
#define STUB(name, code, ...) extern "C" int name(__VA_ARGS__) { return code; }
STUB(pd_qk_norm_rope_cache, 41, const void*, int64_t, const void*, const void*, float, float,
     const float*, int32_t, int32_t, int32_t, const int32_t*, const int32_t*, void*, int64_t, void*,
     void*, int32_t, int32_t, int32_t, int32_t, int32_t, int64_t, int32_t, float, float, void*)
STUB(pd_decode_tree, 42, const void*, int64_t, const int32_t*, const uint64_t*, const void*,
     const void*, const int32_t*, const int32_t*, void*, int64_t, int32_t, int32_t, int32_t, int32_t,
     int32_t, int32_t, int32_t, int32_t, int64_t, float, int32_t, int32_t, int32_t, float, float,
     void*, size_t, void*)
STUB(pd_compact_tree, 43, void*, void*, int64_t, int32_t, const int32_t*, const int32_t*,
     const int32_t*, const int32_t*, const int32_t*, int32_t, int32_t*, int32_t, int32_t, int32_t,
     int32_t, int32_t, int64_t, int32_t, void*)
"""

# one good call of each function; CASES change arguments by their place
SETUP = """
import sys
import torch
sys.path.insert(0, sys.argv[1])
import _marshal as M
bf, i32 = torch.bfloat16, torch.int32
z = torch.zeros
GOOD = {
    "norm_rope": [z(2, 512, dtype=bf), z(2, 4, 64, dtype=bf), 0, 0, z(64), z(64), z(2, dtype=i32),
                  z(2, dtype=i32), z(8, 64), 2, 16, 4, z(64, dtype=bf), z(64, dtype=bf), 1e-6, 0.0,
                  False, 0, 1.0, 1.0, 0],
    "decode_tree": [z(2, 4, 64, dtype=bf), z(2, 4, 64, dtype=bf), None, None, z(3, dtype=i32),
                    z(2, dtype=torch.int64), z(64), z(64), z(2, 4, dtype=i32), z(2, dtype=i32), 2, 2,
                    16, 4, 1.0, 0, 0, 0, 1.0, 1.0, z(64), 0],
    "compact_tree": [z(2, 64), z(2, 64), z(2, 4, dtype=i32), z(2, dtype=i32), z(3, dtype=i32),
                     z(2, 3, dtype=i32), z(2, dtype=i32), z(2, dtype=i32), 2, 64, 16, 4, 0, 0],
}
def call(name, **at):
    a = list(GOOD[name])
    for k, v in at.items():
        a[int(k[1:])] = v
    return getattr(M, name)(*a)
assert call("norm_rope") == 41 and call("decode_tree") == 42 and call("compact_tree") == 43
rows = z(2, 256, dtype=bf)
GOOD["decode_tree_rows"] = [rows, rows, 4, 64] + GOOD["decode_tree"][4:]
"""

CASES = {
    "rows": """
assert call("decode_tree_rows") == 42
assert call("norm_rope", _1=None, _2=4, _3=64) == 41
# neither form of the attention takes the other's tensors
q = GOOD["decode_tree"][0]
for hq, d in ((4, 64), (0, 0), (9999, 0), (None, None)):
    assert call("decode_tree_rows", _0=q, _1=q, _2=hq, _3=d) is None
    assert call("decode_tree", _0=rows, _1=rows, _2=hq, _3=d) is None
assert call("decode_tree_rows", _2=5) is None
assert call("decode_tree_rows", _2=-4, _3=-64) is None
assert call("decode_tree", _2=4, _3=64) is None""",
    "0-dim": """
for name, args in GOOD.items():
    for i, x in enumerate(args):
        if isinstance(x, torch.Tensor):
            r = call(name, **{f"_{i}": z((), dtype=x.dtype)})
            # caches and workspaces are taken in any shape
            assert r is None or x.dtype == torch.float32, (name, i, r)
s = z((), dtype=bf)
assert call("decode_tree", _0=s, _1=s) is None
assert call("decode_tree_rows", _0=s, _1=s) is None
assert call("decode_tree_rows", _1=s) is None""",
    "1-dim": """
s = z(256, dtype=bf)
assert call("decode_tree", _0=s, _1=s) is None
assert call("decode_tree_rows", _0=s, _1=s) is None""",
    "vmap": """
got = []
for name, args in GOOD.items():
    for i, x in enumerate(args):
        if isinstance(x, torch.Tensor):
            def f(y, name=name, i=i):
                got.append((name, i, call(name, **{f"_{i}": y})))
                return y
            torch.vmap(f)(torch.stack([x, x]))
assert len(got) == 35 and all(r is None for _, _, r in got), got""",
    "sparse": """
assert call("decode_tree", _0=GOOD["decode_tree"][0].to_sparse()) is None
assert call("compact_tree", _0=z(2, 64).to_sparse(), _1=z(2, 64).to_sparse()) is None""",
}


@pytest.fixture(scope="module")
def module_dir(tmp_path_factory):
    d = tmp_path_factory.mktemp("marshal")
    src = d / "host.cpp"
    src.write_text(STUBS % build.MARSHAL_SRC)
    subprocess.run(["g++", *build.marshal_cflags(), "-O0", "-shared", str(src), "-o",
                    str(d / "_marshal.so"), *build.marshal_ldflags()], check=True)
    return str(d)


@pytest.mark.parametrize("name", sorted(CASES))
def test_declines(module_dir, name):
    r = subprocess.run([sys.executable, "-c", SETUP + CASES[name], module_dir],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True,
                       cwd=os.path.dirname(module_dir))
    assert r.returncode == 0, r.stdout[-3000:]
