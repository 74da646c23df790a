"""Refusals and sizes of the INT8 serving calls, on the host: every call fails a
check or has nothing to do, so the placeholder pointers are never touched."""
import ctypes

import pytest

from tests.test_abi_verify import INF, NAN, P, _entry, f32, i32, i64
from tests.test_abi_verify import lib  # noqa: F401

APPEND = [("qkv", P, 0x1000), ("qs", i64, 0), ("cu", P, 0x2000), ("sl", P, 0x3000),
          ("pos", P, 0x4000), ("cs", P, 0x5000), ("maxp", i32, 512), ("rot", i32, 128),
          ("inter", i32, 0), ("qo", P, 0x6000), ("qos", i64, 0), ("ko", P, 0x7000), ("kos", i64, 0),
          ("kc", P, 0x8000), ("vc", P, 0x9000), ("bt", P, 0xa000), ("B", i32, 2), ("T", i32, 4),
          ("mq", i32, 2), ("Hq", i32, 8), ("Hkv", i32, 2), ("D", i32, 128), ("bs", i32, 16),
          ("mbs", i32, 4), ("nb", i64, 8), ("st", P, None)]


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 0), (dict(T=0), 0), (dict(mq=0), 0), (dict(T=0, qkv=0, kc=0), 0), (dict(B=-1), 1),
    (dict(B=70000), 1), (dict(T=-1), 1), (dict(mq=-1), 1), (dict(Hq=0), 1), (dict(Hkv=-2), 1),
    (dict(Hq=40000), 2), (dict(Hkv=4096), 2), (dict(D=96), 2), (dict(bs=8), 2), (dict(rot=0), 2),
    (dict(rot=24), 2), (dict(rot=144), 2), (dict(nb=0), 1), (dict(nb=1 << 28), 1),
    (dict(mbs=0), 1), (dict(mbs=1 << 27), 1), (dict(maxp=0), 1), (dict(qs=1528), 1),
    (dict(qs=1540), 1), (dict(qos=1016), 1), (dict(qos=1028), 1), (dict(kos=248), 1),
    (dict(kos=260), 1), (dict(qkv=0x1008), 1), (dict(qkv=0), 1), (dict(cu=0), 1), (dict(sl=0), 1),
    (dict(pos=0x4004), 1), (dict(cs=0), 1), (dict(qo=0), 1), (dict(ko=0x7002), 1), (dict(kc=0), 1),
    (dict(vc=0x9008), 1), (dict(bt=0), 1),
])
def test_append(lib, kw, code):  # noqa: F811
    assert _entry(lib, "pd_rope_append_int8", APPEND, kw) == code


PACKED = [("q", P, 0x1000), ("qs", i64, 0), ("k", P, 0x2000), ("ks", i64, 0), ("v", P, 0x3000),
          ("vs", i64, 0), ("cu", P, 0x4000), ("o", P, 0x5000), ("os", i64, 0), ("B", i32, 2),
          ("T", i32, 4), ("mq", i32, 2), ("Hq", i32, 8), ("Hkv", i32, 2), ("D", i32, 128),
          ("sc", f32, 0.088), ("causal", i32, 1), ("W", i32, 0), ("st", P, None)]


@pytest.mark.parametrize("name", ["pd_prefill_packed", "pd_prefill_packed_crosscheck"])
@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 0), (dict(T=0), 0), (dict(mq=0), 0), (dict(T=0, q=0), 0), (dict(B=-1), 1),
    (dict(B=70000), 1), (dict(T=-1), 1), (dict(mq=-1), 1), (dict(Hq=6, Hkv=4), 1),
    (dict(Hkv=0), 1), (dict(Hq=34), 2), (dict(D=96), 2), (dict(D=512), 2), (dict(W=-1), 1),
    (dict(sc=INF), 1), (dict(sc=NAN), 1), (dict(qs=1016), 1), (dict(qs=1028), 1),
    (dict(ks=248), 1), (dict(vs=260), 1), (dict(os=1028), 1), (dict(q=0), 1), (dict(k=0x2008), 1),
    (dict(v=0), 1), (dict(cu=0), 1), (dict(o=0x5002), 1), (dict(Hq=8192, Hkv=8192), 2),
])
def test_packed(lib, name, kw, code):  # noqa: F811
    assert _entry(lib, name, PACKED, kw) == code


def test_cache_bytes(lib):  # noqa: F811
    f = lib.pd_cache_bytes
    f.argtypes, f.restype = [i32, i64, i32, i32, i32], ctypes.c_size_t
    for bs, h, d in ((16, 1, 64), (16, 8, 128), (32, 2, 512), (32, 33, 64)):
        page = (bs * h * d + 4 * h + 127) // 128 * 128
        assert f(3, 37, bs, h, d) == 37 * page
    assert f(4, 1, 16, 1, 64) == 0


def test_plans_take_the_form(lib):  # noqa: F811
    from paged_kv_split_gb300 import binding as B
    kw = dict(num_q_heads=32, num_kv_heads=8, block_size=16, max_blocks_per_seq=256, head_dim=128,
              sliding_window=0, kv_dtype="int8", num_sms=152)
    plan = B.pd_balanced_plan([4096, 17, 0], **kw)
    assert plan.num_ctas > 0 and plan.num_pieces >= plan.num_ctas
    assert B.pd_prefer_balanced([4096, 17, 900], **kw) in (True, False)
    assert B.pd_plan_num_splits_for_lengths([4096] * 4, **kw) >= 1
