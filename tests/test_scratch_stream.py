"""The workspace a call allocates belongs to the stream the call runs on: what
takes the memory next is then ordered behind the call's kernels. On the host,
with stand-ins for the library, its tensors and torch's current stream; on the
GPU, with the next allocations of the current stream written while the call
still waits."""
import contextlib
import types

import numpy as np
import pytest
import torch

from paged_kv_split_gb300 import binding as B

DEV = torch.device("cuda", 0)


class Side:
    """A stream that is not torch's current one."""
    cuda_stream = 0x5150


class Current:
    cuda_stream = 0x1000


class T:
    """A CUDA tensor's shape."""
    is_cuda, device = True, DEV

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype = torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return 4

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x100


@pytest.fixture
def made(monkeypatch):
    """Handles of the streams that were current when memory was allocated."""
    stack, handles = [Current()], []

    @contextlib.contextmanager
    def on(stream):
        stack.append(stream)
        yield
        stack.pop()

    def empty(n, dtype=None, device=None):
        handles.append(stack[-1].cuda_stream)
        return T(n, dtype=dtype)

    def call(*args):
        return 0

    call.__name__ = "pd_decode_tree"

    class Lib:
        def __getattr__(self, name):
            return (lambda *a: 4096) if name.endswith("_bytes") else call

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stack[-1])
    monkeypatch.setattr(torch.cuda, "default_stream",
                        lambda device=None: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda handle, device=None: types.SimpleNamespace(cuda_stream=handle))
    monkeypatch.setattr(B, "_raw_stream", None)
    monkeypatch.setattr(B, "_lib", Lib())
    monkeypatch.setattr(B, "_tree_workspace", lambda *a: 4096)
    monkeypatch.setattr(B, "_num_sms", lambda device: 152)
    monkeypatch.setattr(B, "_marshal", types.SimpleNamespace(decode_tree=lambda *a: 0,
                                                               decode_tree_rows=lambda *a: 0))
    for name in ("_dev", "_ptr", "_cache_ptr"):
        monkeypatch.setattr(B, name, lambda *a: 0x100)
    return handles


X = T(4, 4)
PLAN = types.SimpleNamespace(workspace_bytes=64, num_ctas=1, num_pieces=1)
GEOM = dict(num_kv_heads=2, block_size=16, num_blocks=4, scale=1.0)
ROWS = dict(num_q_heads=4, head_dim=64)
CALLS = {
    "pd_decode": lambda s: B.pd_decode(T(4, 4, 64), X, X, X, T(4), T(4, 4, 64), num_splits=2,
                                       stream=s, **GEOM),
    "pd_decode_e4m3_out": lambda s: B.pd_decode_e4m3_out(T(4, 4, 64), X, X, X, T(4), T(4, 4, 64),
                                                         out_scale=1.0, num_splits=2, stream=s,
                                                         **GEOM),
    "pd_decode_strided": lambda s: B.pd_decode_strided(T(4, 256), X, X, X, T(4), T(4, 256),
                                                       num_splits=2, stream=s, **ROWS, **GEOM),
    "pd_decode_balanced": lambda s: B.pd_decode_balanced(T(4, 4, 64), X, X, X, X, PLAN,
                                                         T(4, 4, 64), stream=s, **GEOM),
    "pd_decode_balanced_strided": lambda s: B.pd_decode_balanced_strided(
        T(4, 256), X, X, X, X, PLAN, T(4, 256), stream=s, **ROWS, **GEOM),
    "pd_decode_tree": lambda s: B.pd_decode_tree(T(4, 4, 64), T(5), X, X, X, T(4), T(4, 4, 64),
                                                 max_q_len=1, stream=s, **GEOM),
    "pd_decode_tree, cross-check": lambda s: B.pd_decode_tree(
        T(4, 4, 64), T(5), X, X, X, T(4), T(4, 4, 64), max_q_len=1, stream=s, crosscheck=True,
        **GEOM),
    "pd_decode_tree_strided": lambda s: B.pd_decode_tree_strided(
        T(4, 256), T(5), X, X, X, T(4), T(4, 256), max_q_len=1, stream=s, **ROWS, **GEOM),
}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("stream,handle", [(Side(), 0x5150), (0x5150, 0x5150), (0, 0),
                                           (None, 0x1000), (Current(), 0x1000)])
def test_allocated_on_the_calls_stream(made, name, stream, handle):
    CALLS[name](stream)
    assert made == [handle]


@pytest.mark.parametrize("stream,handle", [(Side(), 0x5150), (0x5150, 0x5150), (0, 0),
                                           (None, 0x1000)])
def test_calibration_runs_on_one_stream(made, monkeypatch, stream, handle):
    """The zeroed maxima, the kernels and the copy back are in one stream's order."""
    seen = []
    real = torch.zeros

    def here():
        seen.append(torch.cuda.current_stream().cuda_stream)

    class Scales:
        def cpu(self):
            here()
            return real(2)

    def zeros(n, dtype=None, device=None):
        here()
        return real(n, dtype=dtype)

    monkeypatch.setattr(torch, "zeros", zeros)
    monkeypatch.setattr(torch, "empty_like", lambda t: Scales())
    monkeypatch.setattr(B, "pd_absmax_bf16", lambda x, m, s=None: seen.append(B._stream(s)))
    monkeypatch.setattr(B, "pd_fp8_scales_from_absmax", lambda a, x, s=None: seen.append(B._stream(s)))
    B.fp8_calibrate(T(8), T(8), stream)
    assert seen == [handle] * 5


@pytest.mark.gpu
@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("d", [128, 512])
def test_the_next_allocation_does_not_meet_the_call(d, as_handle):
    """The call waits behind a sleep on a side stream; blocks of its workspace's
    size are filled on the current stream meanwhile."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hq, hkv, bs, L, n = 8, 2, 16, 3000, 4
    g = torch.Generator(device="cuda").manual_seed(d)
    nb = (L + bs - 1) // bs
    caches = [torch.randn(nb * bs * hkv * d, generator=g, device="cuda").bfloat16().view(torch.uint8)
              for _ in range(2)]
    q = torch.randn(n, hq, d, generator=g, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (torch.tensor([0, n], **i32), *caches, torch.arange(nb, **i32)[None].contiguous(),
            torch.tensor([L], **i32))
    geom = dict(max_q_len=n, num_kv_heads=hkv, block_size=bs, num_blocks=nb, scale=d ** -0.5)
    want = B.pd_decode_tree(q, *args, torch.empty_like(q), **geom)
    out = torch.empty_like(q)
    size = B.pd_decode_tree_workspace_bytes(n, hq, hkv, d, 0, B._num_sms(0))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    B.pd_decode_tree(q, *args, out, stream=side.cuda_stream if as_handle else side, **geom)
    blocks = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    side.synchronize()
    assert torch.equal(out, want)
    assert all(bool((b == 0xFF).all()) for b in blocks)
    assert B.pd_device_status() == 0
