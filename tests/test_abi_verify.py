"""Refusals and sizes of the draft-and-verify entry points, on the host: every
call fails a check or has nothing to do, so the placeholder pointers are never
touched (a valid call would launch on them)."""
import ctypes

import pytest

P, i32, i64, f32, f64 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                         ctypes.c_double)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from paged_kv_split_gb300 import build
    return ctypes.CDLL(build.build())


def _entry(lib, name, spec, kw):
    f = getattr(lib, name)
    f.argtypes = [t for _, t, _ in spec]
    f.restype = ctypes.c_int
    args = {k: v for k, _, v in spec}
    assert set(kw) <= set(args)
    args.update(kw)
    return f(*args.values())


TABLE = [("cs", P, 0x1000), ("n", i32, 64), ("rot", i32, 128), ("base", f64, 1e4), ("st", P, None)]


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), 0), (dict(n=-1), 1), (dict(rot=8), 2), (dict(rot=24), 2), (dict(rot=528), 2),
    (dict(base=1.0), 1), (dict(base=NAN), 1), (dict(base=INF), 1), (dict(cs=0), 1),
    (dict(cs=0x1004), 1),
])
def test_rope_table(lib, kw, code):
    assert _entry(lib, "pd_rope_table", TABLE, kw) == code


ROPE = [("qkv", P, 0x1000), ("qs", i64, 0), ("qw", P, 0x2000), ("kw", P, 0x3000),
        ("eps", f32, 1e-6), ("off", f32, 0.0), ("cs", P, 0x4000), ("maxp", i32, 512),
        ("rot", i32, 128), ("inter", i32, 0), ("pos", P, 0x5000), ("slots", P, 0x6000),
        ("qo", P, 0x7000), ("qos", i64, 0), ("kc", P, 0x8000), ("vc", P, 0x9000), ("T", i32, 4),
        ("Hq", i32, 8), ("Hkv", i32, 2), ("D", i32, 128), ("bs", i32, 16), ("nb", i64, 8),
        ("dt", i32, 0), ("ks", f32, 1.0), ("vs", f32, 1.0), ("st", P, None)]


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), 0), (dict(T=0, qkv=0, kc=0), 0), (dict(T=-1), 1), (dict(Hq=0), 1),
    (dict(Hkv=-2), 1), (dict(D=96), 2), (dict(bs=8), 2), (dict(dt=3), 2), (dict(rot=0), 2),
    (dict(rot=24), 2), (dict(rot=144), 2), (dict(nb=0), 1), (dict(nb=1 << 28), 1),
    (dict(maxp=0), 1), (dict(qw=0), 1), (dict(kw=0), 1), (dict(qw=0x2002), 1), (dict(eps=0.0), 1),
    (dict(eps=NAN), 1), (dict(off=INF), 1), (dict(dt=1, ks=0.0), 1), (dict(dt=1, vs=NAN), 1),
    (dict(qs=1528), 1), (dict(qs=1540), 1), (dict(qos=1016), 1), (dict(qos=1028), 1),
    (dict(qkv=0x1008), 1), (dict(qkv=0), 1), (dict(cs=0), 1), (dict(pos=0), 1),
    (dict(slots=0x6004), 1), (dict(qo=0), 1), (dict(kc=0x8001), 1), (dict(vc=0), 1),
    (dict(T=0, qw=0, kw=0, eps=0.0), 0),  # no norm: eps is not read
])
def test_norm_rope(lib, kw, code):
    assert _entry(lib, "pd_qk_norm_rope_cache", ROPE, kw) == code


TREE = [("q", P, 0x1000), ("qs", i64, 0), ("cu", P, 0x2000), ("mask", P, 0x3000), ("kc", P, 0x4000),
        ("vc", P, 0x5000), ("bt", P, 0x6000), ("sl", P, 0x7000), ("o", P, 0x8000), ("os", i64, 0),
        ("B", i32, 2), ("T", i32, 6), ("mq", i32, 4), ("Hq", i32, 8), ("Hkv", i32, 2),
        ("D", i32, 128), ("bs", i32, 16), ("mbs", i32, 8), ("nb", i64, 32), ("sc", f32, 0.088),
        ("W", i32, 0), ("sinks", i32, 0), ("dt", i32, 0), ("ks", f32, 1.0), ("vs", f32, 1.0),
        ("ws", P, 0x9000), ("wsb", ctypes.c_size_t, 1 << 28), ("st", P, None)]


@pytest.mark.parametrize("name", ["pd_decode_tree", "pd_decode_tree_crosscheck"])
@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 0), (dict(T=0), 0), (dict(mq=0), 0), (dict(T=0, q=0, ws=0), 0), (dict(B=-1), 1),
    (dict(B=70000), 1), (dict(T=-1), 1), (dict(mq=-1), 1), (dict(mq=65), 2), (dict(Hq=6, Hkv=4), 1),
    (dict(Hq=34, Hkv=2), 2), (dict(D=96), 2), (dict(bs=8), 2), (dict(dt=7), 2), (dict(mbs=0), 1),
    (dict(nb=0), 1), (dict(W=-1), 1), (dict(sinks=-1), 1), (dict(sc=INF), 1), (dict(sc=NAN), 1),
    (dict(dt=1, ks=-1.0), 1), (dict(dt=1, vs=INF), 1), (dict(qs=1016), 1), (dict(os=1028), 1),
    (dict(q=0), 1), (dict(q=0x1008), 1), (dict(cu=0), 1), (dict(mask=0x3004), 1), (dict(kc=0), 1),
    (dict(vc=0x5001), 1), (dict(bt=0), 1), (dict(sl=0), 1), (dict(o=0), 1), (dict(ws=0), 1),
])
def test_tree(lib, name, kw, code):
    assert _entry(lib, name, TREE, kw) == code


def test_tree_workspace_bytes(lib):
    f = lib.pd_decode_tree_workspace_bytes
    f.argtypes, f.restype = [i32] * 6, ctypes.c_size_t
    assert f(16, 32, 8, 128, 0, 152) > 0
    for d in (64, 128, 256, 512):
        for dt in (0, 1, 2):
            for n in (0, 1, 64):
                assert f(n, 32, 8, d, dt, 152) > 0
    for bad in ((65, 32, 8, 128, 0, 152), (-1, 32, 8, 128, 0, 152), (4, 30, 8, 128, 0, 152),
                (4, 34, 2, 128, 0, 152), (4, 32, 8, 96, 0, 152), (4, 32, 8, 128, 3, 152),
                (4, 32, 8, 128, 0, 0), (4, 32, 0, 128, 0, 152)):
        assert f(*bad) == 0


COMPACT = [("kc", P, 0x1000), ("vc", P, 0x2000), ("lb", i64, 0), ("layers", i32, 2),
           ("bt", P, 0x3000), ("sl", P, 0x4000), ("cu", P, 0x5000), ("acc", P, 0x6000),
           ("na", P, 0x7000), ("ma", i32, 8), ("new", P, 0x8000), ("B", i32, 2), ("Hkv", i32, 2),
           ("D", i32, 64), ("bs", i32, 16), ("mbs", i32, 4), ("nb", i64, 8), ("dt", i32, 0),
           ("st", P, None)]


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 0), (dict(layers=0), 0), (dict(B=-1), 1), (dict(B=70000), 1), (dict(layers=-1), 1),
    (dict(Hkv=0), 1), (dict(D=80), 2), (dict(bs=64), 2), (dict(dt=9), 2), (dict(ma=65), 2),
    (dict(ma=-1), 1), (dict(mbs=0), 1), (dict(nb=0), 1), (dict(nb=1 << 28), 1),
    (dict(mbs=1 << 27), 1),
    (dict(lb=8 * 16 * 2 * 64 * 2 - 16), 1), (dict(lb=8 * 16 * 2 * 64 * 2 + 8), 1),
    (dict(kc=0), 1), (dict(vc=0x2008), 1), (dict(bt=0), 1), (dict(sl=0), 1), (dict(cu=0), 1),
    (dict(acc=0), 1), (dict(na=0), 1), (dict(new=0), 1), (dict(new=0x4000), 1),
])
def test_compact(lib, kw, code):
    assert _entry(lib, "pd_compact_tree", COMPACT, kw) == code
