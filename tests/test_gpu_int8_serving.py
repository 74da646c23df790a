"""Serving from an INT8 cache, the calls as they are used together: prompts appended
and attended over their own rows, a later chunk of one over the cache, then steps of
one token each from one captured graph, whose lengths live on the device. Every
output against the 64-bit definitions over the rows and cache bytes of the numpy
reference, which the caches equal bit for bit all along."""
import numpy as np
import pytest
import torch

from tests import gpu_util as U, int8_refs as R, verify_refs as V

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS = 8, 2, 64, 16
ROW = (HQ + 2 * HKV) * D


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_split_gb300 import binding
    binding.pd_device_status(reset=True)
    yield
    assert binding.pd_device_status(reset=True) == 0


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def within(got, want, bound):
    err = np.abs(V.f32(got) - want)
    assert (err <= bound).all(), float((err / bound).max())


class Server:
    def __init__(self, prompts, most, seed):
        self.rng = np.random.default_rng(seed)
        self.lens = np.zeros(len(prompts), np.int32)
        self.tables, self.nb = R.paging([most] * len(prompts), BS, self.rng)
        self.k = R.random_cache(self.rng, self.nb, BS, HKV, D)   # what was there before
        self.v = R.random_cache(self.rng, self.nb, BS, HKV, D)
        self.kd, self.vd, self.td = U.to_dev(self.k), U.to_dev(self.v), U.to_dev(self.tables)
        self.cos_dev = torch.empty(most, D, device="cuda")
        U.pd().pd_rope_table(self.cos_dev)
        self.cos = self.cos_dev.cpu().numpy()
        self.geom = dict(num_kv_heads=HKV, block_size=BS, num_blocks=self.nb)
        self.scale = D ** -0.5

    def rows(self, T):
        return V.bf16_bits(self.rng.standard_normal((T, ROW)).astype(np.float32))

    def append_ref(self, rows, cu):
        self.lens = self.lens + np.diff(cu).astype(np.int32)
        return R.append_f32(rows, cu, self.lens, self.cos, self.k, self.v, self.tables, HQ, HKV, D,
                            BS)

    def same_caches(self):
        assert np.array_equal(self.kd.cpu().numpy(), self.k)
        assert np.array_equal(self.vd.cpu().numpy(), self.v)

    def append(self, qkv, lens, cu, most):
        U.pd().pd_rope_append_int8_(qkv, self.kd, self.vd, self.td, lens, cu, self.cos_dev,
                                    max_q_len=most, num_q_heads=HQ, head_dim=D, **self.geom)


def test_prompts_chunk_and_steps():
    B = U.pd()
    new = [37, 130, 1, 64]
    s = Server(new, 300, 1)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    rows = s.rows(int(cu[-1]))
    q, k = s.append_ref(rows, cu)
    qkv, lens, cu_d = U.bf16_dev(rows), U.to_dev(s.lens), U.to_dev(cu)
    # the prompts, their attention over their own rotated rows
    s.append(qkv, lens, cu_d, max(new))
    x = qkv.view(-1, HQ + 2 * HKV, D)
    out = torch.empty(len(rows), HQ, D, dtype=torch.bfloat16, device="cuda")
    B.pd_prefill_packed(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], cu_d, out, max_q_len=max(new),
                        scale=s.scale)
    s.same_caches()
    v = rows.reshape(-1, HQ + 2 * HKV, D)[:, HQ + HKV:]
    within(bits(out), *R.packed_f64(q, k, v, cu, s.scale))

    # a second chunk of two of them, over the cache
    new2 = [0, 50, 0, 21]
    cu2 = np.concatenate([[0], np.cumsum(new2)]).astype(np.int32)
    rows2 = s.rows(int(cu2[-1]))
    q2, _ = s.append_ref(rows2, cu2)
    qkv2, lens, cu2_d = U.bf16_dev(rows2), U.to_dev(s.lens), U.to_dev(cu2)
    s.append(qkv2, lens, cu2_d, max(new2))
    out2 = torch.empty(len(rows2), ROW, dtype=torch.bfloat16, device="cuda")
    B.pd_prefill_strided(qkv2, cu2_d, s.kd, s.vd, s.td, lens, out2, num_q_heads=HQ, head_dim=D,
                         max_q_len=max(new2), scale=s.scale, kv_dtype="int8", **s.geom)
    s.same_caches()
    got = bits(out2[:, :HQ * D]).reshape(-1, HQ, D)
    for b, n in enumerate(new2):
        for i in range(n):
            within(got[cu2[b] + i][None],
                   *R.decode_f64(q2[cu2[b] + i][None], s.k, s.v, s.tables[b][None],
                                 [s.lens[b] - n + i + 1], HKV, BS, s.scale))

    # steps of one token, one graph: append and decode, the lengths counted up in it
    n = len(new)
    cu1 = np.arange(n + 1, dtype=np.int32)
    qkv1 = torch.empty(n, ROW, dtype=torch.bfloat16, device="cuda")
    out1 = torch.empty(n, ROW, dtype=torch.bfloat16, device="cuda")
    cu1_d = U.to_dev(cu1)
    ws = torch.empty(B.pd_decode_workspace_bytes(n, HQ, D, 3), dtype=torch.uint8, device="cuda")

    def step():
        lens.add_(1)
        s.append(qkv1, lens, cu1_d, 1)
        B.pd_decode_strided(qkv1, s.kd, s.vd, s.td, lens, out1, num_q_heads=HQ, head_dim=D,
                            num_splits=3, scale=s.scale, kv_dtype="int8", workspace=ws, **s.geom)

    graph = torch.cuda.CUDAGraph()
    for i in range(40):
        rows1 = s.rows(n)
        qkv1.copy_(U.bf16_dev(rows1))
        if i == 0:
            step()
        else:
            if i == 1:
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        q1, _ = s.append_ref(rows1, cu1)
        assert np.array_equal(bits(qkv1[:, :HQ * D]).reshape(n, HQ, D), q1)
        within(bits(out1[:, :HQ * D]).reshape(n, HQ, D),
               *R.decode_f64(q1, s.k, s.v, s.tables, s.lens, HKV, BS, s.scale))
    s.same_caches()
    assert lens.tolist() == s.lens.tolist()


def test_two_streams_at_once():
    """Calls of two streams side by side give what each gives alone."""
    B = U.pd()
    sets = []
    for seed, new in ((2, [300, 64]), (3, [64, 290, 5])):
        s = Server(new, 320, seed)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        rows = s.rows(int(cu[-1]))
        sets.append((s, rows, cu, max(new)))

    def go(s, rows, cu, most, stream):
        with torch.cuda.stream(stream):
            qkv, cu_d = U.bf16_dev(rows), U.to_dev(cu)
            lens = U.to_dev(np.diff(cu).astype(np.int32))
            outs = []
            for _ in range(10):
                x = qkv.clone()
                s.append(x, lens, cu_d, most)
                h = x.view(-1, HQ + 2 * HKV, D)
                out = torch.empty(len(rows), HQ, D, dtype=torch.bfloat16, device="cuda")
                B.pd_prefill_packed(h[:, :HQ], h[:, HQ:HQ + HKV], h[:, HQ + HKV:], cu_d, out,
                                    max_q_len=most, scale=s.scale)
                last = x[(cu_d[1:] - 1).long(), :HQ * D].view(-1, HQ, D).contiguous()
                dec = torch.empty_like(last)
                B.pd_decode(last, s.kd, s.vd, s.td, lens, dec, num_splits=2, scale=s.scale,
                            kv_dtype="int8", **s.geom)
                outs += [out, dec]
        return outs

    alone = []
    for args in sets:
        alone.append(go(*args, torch.cuda.current_stream()))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    both = [go(*args, st) for args, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
