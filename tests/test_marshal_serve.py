"""The native marshalling of the serving calls: on tensors that it looks into
(built here for CPU tensors, the library's calls replaced by stubs that check what
they are given), and what it declines, without a call, for the binding to refuse."""
import os
import subprocess
import sys

import pytest
import torch

from paged_kv_split_gb300 import binding as B, build

COUNTS = {"rope_append": 18, "prefill_packed": 10, "decode": 17, "decode_balanced": 19}
X = torch.zeros(4, 4)

STUBS = """
#define PD_MARSHAL_DEVICE at::kCPU
#include "%s"
extern "C" {
size_t pd_decode_workspace_bytes(int32_t B, int32_t hq, int32_t d, int32_t s) {
  return B == 2 && hq == 4 && d == 64 ? 256 : 0;
}
int pd_choose_num_splits(int32_t B, int32_t hkv, int32_t mbs, int32_t bs, int32_t w, int32_t d,
                         int32_t f, int) {
  return B == 2 && hkv == 2 && mbs == 4 && bs == 16 && w == 7 && d == 64 ? (f == 3 ? 1 : -2) : -1;
}
size_t pd_cache_bytes(int32_t f, int64_t n, int32_t bs, int32_t h, int32_t d) {
  return f == 3 ? n * bs * h * d : 0;
}
int pd_rope_append_int8(const void* qkv, int64_t, const int32_t*, const int32_t*, const int32_t*,
                        const float*, int32_t, int32_t, int32_t, void* q, int64_t qs, void* k,
                        int64_t ks, void*, void*, const int32_t*, int32_t, int32_t, int32_t, int32_t,
                        int32_t, int32_t, int32_t, int32_t, int64_t, void*) {
  if (q == qkv) return (char*)k - (char*)q == 4 * 64 * 2 && qs == 512 && ks == 512 ? 51 : -1;
  return 100 + (int)qs + (int)ks;
}
int pd_prefill_packed(const void*, int64_t qs, const void*, int64_t ks, const void*, int64_t vs,
                      const int32_t*, void*, int64_t os, int32_t B, int32_t T, int32_t mq,
                      int32_t hq, int32_t hkv, int32_t d, float, int32_t, int32_t, void*) {
  return B == 2 && T == 3 && mq == 2 && hq == 4 && hkv == 2 && d == 64 ? (int)(qs + ks + vs + os) : -1;
}
int pd_decode(const void*, const void*, const void*, const int32_t*, const int32_t*, void*,
              int32_t B, int32_t hq, int32_t hkv, int32_t d, int32_t bs, int32_t mbs, int64_t nb,
              float, int32_t s, int32_t w, int32_t f, float, float, void*, size_t n, void*) {
  return B == 2 && hq == 4 && hkv == 2 && d == 64 && bs == 16 && mbs == 4 && nb == 4 && s == 1 &&
         w == 7 && f == 3 && n == 256 ? 53 : -1;
}
int pd_decode_balanced(const void*, const void*, const void*, const int32_t*, const void*,
                       size_t plan, void*, int32_t B, int32_t hq, int32_t hkv, int32_t d, int32_t bs,
                       int32_t mbs, int64_t nb, float, int32_t w, int32_t f, float, float, int32_t c,
                       int32_t p, void*, size_t n, void*) {
  return plan == 32 && B == 2 && hq == 4 && hkv == 2 && d == 64 && bs == 16 && mbs == 4 &&
         nb == 4 && w == 7 && f == 3 && c == 5 && p == 6 && n == 256 ? 54 : -1;
}
}
"""

SETUP = """
import sys
import torch
sys.path.insert(0, sys.argv[1])
import _marshal_serve as M
bf, i32 = torch.bfloat16, torch.int32
z = torch.zeros
cache = z(4 * 16 * 2 * 64, dtype=torch.uint8)
ws = z(256, dtype=torch.uint8)
q = z(2, 4, 64, dtype=bf)
fused = z(3, 8 * 64, dtype=bf)
part = fused.view(3, 8, 64)
GOOD = {
    "rope_append": [z(2, 512, dtype=bf), q, 0, 0, cache, cache, z(2, 4, dtype=i32),
                    z(2, dtype=i32), z(3, dtype=i32), z(8, 64), 1, 2, 16, 4, None, None, False, 0],
    "prefill_packed": [part[:, :4], part[:, 4:6], part[:, 6:], z(3, dtype=i32),
                       z(3, 4, 64, dtype=bf), 2, 1.0, True, 0, 0],
    "decode": [q, cache, cache, z(2, 4, dtype=i32), z(2, dtype=i32), z(2, 4, 64, dtype=bf), 2, 16,
               4, 1.0, 1, 7, 3, 1.0, 1.0, ws, 0],
    "decode_balanced": [q, cache, cache, z(2, 4, dtype=i32), z(8, dtype=i32),
                        z(2, 4, 64, dtype=bf), 2, 16, 4, 1.0, 7, 3, 1.0, 1.0, 5, 6, ws, 0, 0],
}
def call(name, **at):
    a = list(GOOD[name])
    for k, v in at.items():
        a[int(k[1:])] = v
    return getattr(M, name)(*a)
"""

CASES = {
    "taken": """
assert call("decode") == 53 and call("decode_balanced") == 54
assert call("decode", _15=None) == 53 and call("decode", _10=0, _15=None) == 53
assert call("decode", _10=0, _12=9, _15=None) is None       # no split count for the form
assert call("decode_balanced", _16=None, _17=256) == 54
assert call("prefill_packed") == 3 * 512 + 256
assert call("rope_append") == 100 + 256
assert call("rope_append", _1=None, _2=4, _3=64) == 51
wide = z(2, 1024, dtype=bf)
assert call("rope_append", _1=wide[:, :256].unflatten(1, (4, 64)),
            _15=wide[:, 256:384].unflatten(1, (2, 64))) == 100 + 2048
assert call("rope_append", _14=z(2, dtype=i32)) == 356""",
    "shapes": """
assert call("rope_append", _1=z(3, 4, 64, dtype=bf)) is None
assert call("rope_append", _15=z(2, 3, 64, dtype=bf)) is None
assert call("rope_append", _4=cache[1:]) is None            # too short
assert call("rope_append", _14=z(3, dtype=i32)) is None
assert call("rope_append", _0=z(2, 504, dtype=bf)) is None
assert call("rope_append", _1=None, _2=-4, _3=-64) is None
assert call("rope_append", _1=z(2, 64, 4, dtype=bf).transpose(1, 2)) is None
assert call("prefill_packed", _1=part[:, 4:7]) is None
assert call("prefill_packed", _3=z(0, dtype=i32)) is None
assert call("prefill_packed", _4=z(4, 4, 64, dtype=bf)) is None
assert call("prefill_packed", _0=part[:, ::2]) is None
assert call("prefill_packed", _0=part[:1, :4].expand(3, 4, 64)) is None
assert call("prefill_packed", _4=z(3, 4, 64)) is None
assert call("decode", _5=z(2, 4, 32, dtype=bf)) is None
assert call("decode", _3=z(3, 4, dtype=i32)) is None
assert call("decode", _4=z(3, dtype=i32)) is None
assert call("decode", _10=1 << 40) is None
assert call("decode_balanced", _4=z(8)) is None
assert call("decode_balanced", _16=None, _17=-1) is None""",
    "0-dim": """
for name, args in GOOD.items():
    for i, x in enumerate(args):
        if isinstance(x, torch.Tensor) and x.dtype != torch.uint8 and i != 4:
            assert call(name, **{f"_{i}": z((), dtype=x.dtype)}) is None, (name, i)""",
    "vmap": """
got = []
for name, args in GOOD.items():
    for i, x in enumerate(args):
        if isinstance(x, torch.Tensor):
            def f(y, name=name, i=i):
                got.append((name, i, call(name, **{f"_{i}": y})))
                return y
            torch.vmap(f)(torch.stack([x, x]))
assert len(got) == 27 and all(r is None for _, _, r in got), got""",
    "sparse": """
assert call("decode", _0=q.to_sparse()) is None
assert call("prefill_packed", _0=z(3, 4, 64, dtype=bf).to_sparse()) is None""",
}


@pytest.fixture(scope="module")
def module_dir(tmp_path_factory):
    d = tmp_path_factory.mktemp("marshal_serve")
    src = d / "host.cpp"
    src.write_text(STUBS % build.SERVE_SRC)
    subprocess.run(["g++", *build.marshal_cflags(), "-O0", "-shared", str(src), "-o",
                    str(d / "_marshal_serve.so"), *build.marshal_ldflags()], check=True)
    return str(d)


@pytest.mark.parametrize("name", sorted(CASES))
def test_host(module_dir, name):
    r = subprocess.run([sys.executable, "-c", SETUP + CASES[name], module_dir],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True,
                       cwd=os.path.dirname(module_dir))
    assert r.returncode == 0, r.stdout[-3000:]


@pytest.mark.parametrize("name,count", sorted(COUNTS.items()))
def test_declines(name, count):
    f = getattr(B._serve, name)
    assert f() is None
    assert f(*[X] * (count - 1)) is None
    assert f(*[X] * count) is None                     # not on a GPU
    assert f(*[None] * count) is None
    assert f(*["text"] * count) is None
    assert f(*[1 << 80] * count) is None


def test_the_binding_names_what_was_declined():
    bf = torch.bfloat16
    q, i = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(2, dtype=torch.int32)
    geom = dict(num_kv_heads=2, block_size=16, num_blocks=1)
    with pytest.raises(ValueError, match="qkv"):
        B.pd_rope_append_int8(q, q, X, X, X, i, i, X, max_q_len=1, **geom)
    with pytest.raises(ValueError, match="CUDA"):
        B.pd_rope_append_int8(torch.zeros(2, 512, dtype=bf), q, X, X, X, i, i, X, max_q_len=1, **geom)
    with pytest.raises(ValueError, match="CUDA|qkv"):
        B.pd_rope_append_int8_(torch.zeros(2, 512, dtype=bf), X, X, X, i, i, X, max_q_len=1,
                               num_q_heads=4, head_dim=64, **geom)
    with pytest.raises(ValueError, match="CUDA"):
        B.pd_prefill_packed(q, q, q, i, q, max_q_len=1, scale=1.0)
    with pytest.raises(ValueError, match="total_q"):
        B.pd_prefill_packed(q, q, q[:1], i, q, max_q_len=1, scale=1.0)


def test_without_the_module(monkeypatch):
    monkeypatch.setattr(build, "SERVE_ABI", "/nonexistent")
    assert not build.serve_fits() and build.serve_is_stale()
    with pytest.warns(UserWarning, match="not used"):
        assert B._load_marshal("_marshal_serve", build.SERVE, build.serve_fits) is None


def test_tensors_of_another_device(monkeypatch):
    class T:
        is_cuda, device = True, torch.device("cuda", 1)

        def get_device(self):
            return 1

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
        B.pd_prefill_packed(T(), T(), T(), T(), T(), max_q_len=1, scale=1.0)
    with pytest.raises(ValueError, match="current device"):
        B.pd_rope_append_int8(T(), T(), T(), T(), T(), T(), T(), T(), max_q_len=1, num_kv_heads=1,
                              block_size=16, num_blocks=1)
