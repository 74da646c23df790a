"""Workloads of the draft-and-verify step of decoding over a paged KV cache.

Three operators, each in its plain form (elementary torch operations) and as
the library's call:

* rope:    per-head RMS norm of q and k, position rotation and the cache
           write, from fused QKV rows (``pd_qk_norm_rope_cache``);
* tree:    attention of drafted token trees (a single token and a chain are
           trees too) over the cache, with a sliding window and first tokens
           that stay visible (``pd_decode_tree``);
* compact: moving the K/V rows of the accepted nodes to consecutive positions
           in the caches of all layers (``pd_compact_tree``).

Cache layouts (include/pd.h): BF16 and FP8 pages are [block][head][dim]; an
NVFP4 page holds [head][block][dim / 2] packed E2M1 codes, then
[head][block][dim / 16] E4M3 scales, its stride rounded up to 128 bytes.
"""
import math

import numpy as np
import torch

own = False

BF16, FP8, NVFP4 = "bf16", "fp8", "nvfp4"
DEV = "cuda"
NEG = float("-inf")


# ---------------------------------------------------------------------------
# the cases
def _rope(**kw):
    c = dict(op="rope", tokens=8, hq=32, hkv=8, d=128, bs=16, form=BF16, rot=128,
             interleaved=False, norm=True, offset=0.0, far=32768, shape=1)
    c.update(kw)
    return c


def _tree(**kw):
    c = dict(op="tree", seqs=1, lo=1024, hi=4096, nodes_lo=1, nodes=16, hq=32, hkv=8, d=128,
             bs=16, window=0, sinks=0, form=BF16, holes=False, lengths="uniform", shape=1)
    c.update(kw)
    return c


def _compact(**kw):
    c = dict(op="compact", seqs=32, lo=17, hi=128, nodes=16, layers=4, hkv=8, d=128, bs=16,
             form=BF16, shape=1)
    c.update(kw)
    return c


def listed():
    return [
        # one new token for each of 8 sequences: the launch itself counts
        _rope(name="rope_step_b8", tokens=8, shape=11),
        # 13 drafted tokens for each of 64 sequences, the quantised-cache batch's heads
        _rope(name="rope_drafts_fp8", tokens=64 * 13, hq=64, form=FP8, shape=12),
        # drafted tokens at wide heads: half the head rotated, pairs side by side, weights 1 + w
        _rope(name="rope_drafts_nvfp4_d256", tokens=203, hq=8, hkv=4, d=256, rot=128,
              interleaved=True, offset=1.0, form=NVFP4, shape=13),
        # a chunk of 8192 prompt tokens on its way into the cache
        _rope(name="rope_chunk_8192", tokens=8192, shape=14),
        # one user's small tree over a short context: latency
        _tree(name="tree_b1_n8", seqs=1, lo=777, hi=777, nodes_lo=8, nodes=8, shape=21),
        # streaming decode: single tokens, the last 4096 keys and the first four
        _tree(name="step_window_sinks_b32", seqs=32, lo=4096, hi=16384, nodes=1, window=4096,
              sinks=4, shape=22),
        # a serving batch with ragged trees of 4 to 16 nodes
        _tree(name="tree_b32_n16", seqs=32, lo=1024, hi=4096, nodes_lo=4, nodes=16, shape=23),
        # two long documents, the widest trees
        _tree(name="tree_long_b2_n64", seqs=2, lo=32768, hi=32768, nodes_lo=64, nodes=64, bs=32,
              shape=24),
        # the quantised-cache batch with 5 to 13 drafted nodes
        _tree(name="tree_fp8_b64_n13", seqs=64, lo=512, hi=16384, nodes_lo=5, nodes=13, hq=64,
              form=FP8, lengths="lognormal", shape=25),
        # wide heads under a window with sinks, NVFP4 pages
        _tree(name="tree_window_d256_nvfp4", seqs=8, lo=16384, hi=16384, nodes_lo=8, nodes=24,
              hq=8, hkv=4, d=256, window=4096, sinks=16, form=NVFP4, shape=26),
        # a few layers at a time
        _compact(name="compact_b32_l4", shape=31),
        # all 32 layers of a model in one call
        _compact(name="compact_b64_l32_fp8", seqs=64, nodes=24, layers=32, form=FP8, shape=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    shape = rng.randrange(1 << 30)
    form = rng.choice([BF16, BF16, FP8, NVFP4])
    op = rng.choice(["rope", "tree", "tree", "tree", "compact"])
    if op == "rope":
        hq, hkv, d = rng.choice([(32, 8, 128), (64, 8, 128), (4, 2, 64), (8, 4, 256), (16, 2, 512),
                                 (6, 1, 64), (12, 12, 128)])
        rot = rng.choice([d, d, d // 2, 32, 48])
        tokens = min(_log(rng, 1, 8192), 8192 * 48 * 128 // ((hq + 2 * hkv) * d))
        return _rope(tokens=tokens, hq=hq, hkv=hkv, d=d, bs=rng.choice([16, 32]), form=form,
                     rot=rot, interleaved=rng.random() < 0.4, norm=rng.random() < 0.8,
                     offset=rng.choice([0.0, 1.0]), far=_log(rng, 64, 131072), shape=shape)
    if op == "tree":
        hq, hkv, d = rng.choice([(32, 8, 128), (32, 8, 128), (64, 8, 128), (4, 2, 64), (8, 4, 256),
                                 (16, 2, 512), (12, 4, 64), (16, 1, 128), (5, 5, 128)])
        nodes = _log(rng, 1, 64)
        hi = _log(rng, 64, 32768)
        lo = max(nodes, rng.randrange(1, hi + 1))
        hi = max(lo, hi)
        # no more than the largest listed case reads or computes
        most = min(400e6 / (hkv * d * 4), 60e9 / (4 * d * hq * nodes), 220000)
        seqs = max(1, min(_log(rng, 1, 64), int(most / hi)))
        window = rng.choice([0, 0, _log(rng, 8, 8192)])
        return _tree(seqs=seqs, lo=lo, hi=hi, nodes_lo=rng.randrange(1, nodes + 1), nodes=nodes,
                     hq=hq, hkv=hkv, d=d, bs=rng.choice([16, 32]), window=window,
                     sinks=rng.choice([0, 1, 4, 70]) if window else 0, form=form,
                     holes=rng.random() < 0.3, shape=shape)
    nodes = _log(rng, 2, 64)
    hkv, d = rng.choice([(8, 128), (2, 64), (4, 256), (2, 512)])
    return _compact(seqs=_log(rng, 1, 64), lo=nodes, hi=max(nodes, _log(rng, 17, 128)),
                    nodes=nodes, layers=_log(rng, 1, 32), hkv=hkv, d=d,
                    bs=rng.choice([16, 32]), form=form, shape=shape)


# ---------------------------------------------------------------------------
# what a case's sizes settle: lengths, node counts, trees, accepted paths
class _Batch:
    def __init__(self, c):
        r = np.random.RandomState(c["shape"] % (1 << 31))
        B = c["seqs"]
        if c.get("lengths") == "lognormal":
            lens = np.clip(np.round(np.exp(r.normal(math.log(2048.0), 1.0, B))), c["lo"], c["hi"])
        else:
            lens = r.randint(c["lo"], c["hi"] + 1, B)
        lens = lens.astype(np.int64)
        nodes = np.minimum(r.randint(c.get("nodes_lo", 1), c["nodes"] + 1, B), lens)
        if c.get("holes"):  # idle slots of a batch: no nodes, or nothing cached either
            nodes[1:][r.rand(B - 1) < 0.2] = 0
            idle = r.rand(B) < 0.1
            idle[0] = False
            nodes[idle] = 0
            lens[idle] = 0
        self.lens, self.nodes = lens, nodes
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int64)
        masks, self.accepted = [], np.zeros((B, c["nodes"]), np.int64)
        self.num_accepted = np.zeros(B, np.int64)
        for b in range(B):
            own_mask, parent = [], []
            for i in range(int(nodes[b])):
                # mostly the node before, else any earlier one
                p = -1 if i == 0 else (i - 1 if r.rand() < 0.5 else int(r.randint(0, i)))
                parent.append(p)
                own_mask.append((own_mask[p] if p >= 0 else 0) | (1 << i))
            if c.get("holes") and nodes[b] > 1:
                own_mask[-1] = 0  # padding node: sees the cached prefix only
            masks += own_mask
            if nodes[b]:  # the path to one node, root first, cut where the model disagreed
                path, i = [], int(r.randint(0, nodes[b]))
                while i >= 0:
                    path.append(i)
                    i = parent[i]
                path = path[::-1]
                self.accepted[b, :len(path)] = path
                self.num_accepted[b] = len(path)
        m = np.array(masks, dtype=np.uint64).astype(np.uint64)
        self.mask = m.view(np.int64) if m.size else np.zeros(0, np.int64)


def _page_bytes(form, bs, hkv, d):
    n = bs * hkv * d
    if form == BF16:
        return 2 * n
    if form == FP8:
        return n
    return (n // 2 + n // 16 + 127) // 128 * 128


def _row_bytes(form, hkv, d):
    return hkv * d * 2 if form == BF16 else hkv * d if form == FP8 else hkv * (d // 2 + d // 16)


def work(case):
    c = case
    if c["op"] == "rope":
        T, D = c["tokens"], c["d"]
        elems = T * (c["hq"] + c["hkv"]) * D
        rows = 2 * T * (c["hq"] + 2 * c["hkv"]) * D + 2 * T * c["hq"] * D
        cache = 2 * T * _row_bytes(c["form"], c["hkv"], D)
        return {"bytes": rows + cache + 8 * T + 4 * min(T, c["far"]) * c["rot"],
                "flops": elems * (8 if c["norm"] else 3)}
    s = _Batch(c)
    if c["op"] == "tree":
        W, first = c["window"], c["sinks"]
        prefix = s.lens - s.nodes
        lo = np.maximum(0, prefix + 1 - W) if W else np.zeros_like(s.lens)
        keys = np.where(s.nodes > 0, s.lens - lo + np.minimum(first, lo), 0)
        seen = np.minimum(prefix, W + first) if W else prefix
        pairs = int((s.nodes * (seen + (s.nodes + 1) // 2)).sum())
        rows = int(s.nodes.sum()) * c["hq"] * c["d"]
        return {"bytes": int(keys.sum()) * 2 * _row_bytes(c["form"], c["hkv"], c["d"]) + 4 * rows,
                "flops": 4 * c["d"] * c["hq"] * pairs}
    moved = sum(int((s.accepted[b, :s.num_accepted[b]] != np.arange(s.num_accepted[b])).sum())
                for b in range(c["seqs"]))
    return {"bytes": 4 * moved * c["layers"] * _row_bytes(c["form"], c["hkv"], c["d"]) +
            4 * c["seqs"] * (c["nodes"] + 4), "flops": 0}


# ---------------------------------------------------------------------------
# inputs
def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _i64(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int64)).to(DEV)


def _paging(lens, bs, r):
    """Block tables over a shuffled pool: (table [B, MBS] with -1 past a sequence's pages, pages)."""
    pages = (lens + bs - 1) // bs
    total = max(1, int(pages.sum()))
    perm = r.permutation(total)
    table = np.full((len(lens), max(1, int(pages.max()))), -1, np.int64)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = perm[at:at + p]
        at += p
    return table, total


def _random_cache(form, nb, bs, hkv, d, scale, g):
    """A pool whose pages hold N(0, 1) values in the cache's form (flat uint8)."""
    n = nb * bs * hkv * d
    if form == BF16:
        return torch.randn(n, generator=g, device=DEV, dtype=torch.bfloat16).view(torch.uint8)
    x = torch.randn(n, generator=g, device=DEV)
    if form == FP8:
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    packed, sc = _nvfp4_encode(x.view(nb, hkv * bs, d))
    pages = torch.zeros(nb, _page_bytes(form, bs, hkv, d), dtype=torch.uint8, device=DEV)
    data = hkv * bs * d // 2
    pages[:, :data] = packed.reshape(nb, -1)
    pages[:, data:data + hkv * bs * d // 16] = sc.reshape(nb, -1)
    return pages.view(-1)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = np.random.RandomState((seed * 2654435761 + c["shape"]) % (1 << 31))
    form, bs, hkv, d = c["form"], c["bs"], c["hkv"], c["d"]
    s = {"case": dict(c)}
    if c["op"] == "rope":
        T, hq = c["tokens"], c["hq"]
        nb = T // bs + 2
        slots = r.permutation(nb * bs)[:T].astype(np.int64)
        slots[r.rand(T) < 0.02] = -1  # padding rows of a batch: q only
        keep = np.nonzero(slots >= 0)[0]
        positions = r.randint(0, c["far"], T)
        half = c["rot"] // 2
        inv = 10000.0 ** (-np.arange(half) * 2.0 / c["rot"])
        ang = torch.arange(c["far"], dtype=torch.float64, device=DEV)[:, None] * \
            torch.from_numpy(inv).to(DEV)
        n = nb * _page_bytes(form, bs, hkv, d)
        s.update(
            qkv=torch.randn(T, (hq + 2 * hkv) * d, generator=g, device=DEV).to(torch.bfloat16),
            q_out=torch.empty(T, hq, d, dtype=torch.bfloat16, device=DEV),
            q_weight=(torch.randn(d, generator=g, device=DEV) * 0.1 + 1.0 - c["offset"]).to(torch.bfloat16),
            k_weight=(torch.randn(d, generator=g, device=DEV) * 0.1 + 1.0 - c["offset"]).to(torch.bfloat16),
            cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float().contiguous(),
            positions=_i32(positions), slots=_i32(slots), keep=_i64(keep), kept=_i64(slots[keep]),
            k_cache=torch.zeros(n, dtype=torch.uint8, device=DEV),
            v_cache=torch.zeros(n, dtype=torch.uint8, device=DEV), nb=nb,
            # scales of a calibrated cache (absmax / 448 of unit normals)
            k_scale=float(np.float32(6.0 / 448)), v_scale=float(np.float32(5.0 / 448)))
        return s
    b = _Batch(c)
    table, nb = _paging(b.lens, bs, r)
    s.update(nb=nb, tables=_i32(table), lens=_i32(b.lens), cu=_i32(b.cu))
    if c["op"] == "tree":
        T = int(b.cu[-1])
        row_seq = np.repeat(np.arange(c["seqs"]), b.nodes)
        s.update(q=torch.randn(T, c["hq"], d, generator=g, device=DEV).to(torch.bfloat16),
                 out=torch.empty(T, c["hq"], d, dtype=torch.bfloat16, device=DEV),
                 mask=_i64(b.mask) if c["nodes"] > 1 else None,
                 k_scale=float(np.float32(5.5 / 448)), v_scale=float(np.float32(5.0 / 448)),
                 rows=_i64(row_seq * max(1, c["nodes"]) + np.arange(T) - b.cu[row_seq]),
                 longest=max(1, int(b.lens.max())), most=max(1, int(b.nodes.max())))
        s["k_cache"] = _random_cache(form, nb, bs, hkv, d, s["k_scale"], g)
        s["v_cache"] = _random_cache(form, nb, bs, hkv, d, s["v_scale"], g)
        return s
    layers = c["layers"]
    n = nb * _page_bytes(form, bs, hkv, d)
    s.update(accepted=_i32(b.accepted), num_accepted=_i32(b.num_accepted),
             new_lens=torch.empty(c["seqs"], dtype=torch.int32, device=DEV),
             k_caches=torch.randint(0, 256, (layers, n), generator=g, device=DEV, dtype=torch.uint8),
             v_caches=torch.randint(0, 256, (layers, n), generator=g, device=DEV, dtype=torch.uint8))
    return s


# ---------------------------------------------------------------------------
# plain forms
def _f32(x, like):
    return torch.full((1,), x, dtype=torch.float32, device=like.device)


def _nvfp4_encode(x):
    """fp32 [..., d] -> (packed codes [..., d / 2], E4M3 scale bytes [..., d / 16])."""
    y = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    sc = (y.abs().amax(-1) / _f32(6.0, x)).clamp(max=448.0).to(torch.float8_e4m3fn)
    dec = sc.float()[..., None]
    q = torch.where(dec > 0, y / torch.where(dec > 0, dec, torch.ones_like(dec)), torch.zeros_like(y))
    a = q.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() +
            (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    code = code + torch.where(torch.signbit(q), 8, 0)
    code = torch.where(dec > 0, code, torch.zeros_like(code)).reshape(*x.shape[:-1], -1, 2)
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), sc.view(torch.uint8)


def _nvfp4_decode(packed, scales):
    """The fp32 values that packed codes [..., d / 2] and scale bytes [..., d / 16] stand for."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0,
                         -4.0, -6.0], device=packed.device)
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).int()
    return grid[code] * scales.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)


def _sum_pairs(x):
    """Sum over the last axis (a power of two) as a balanced tree over neighbours."""
    while x.shape[-1] > 1:
        x = x[..., 0::2] + x[..., 1::2]
    return x


def _norm_rotate(x, weight, s):
    """x fp32 [T, H, D]: RMS norm over each head, then the rotation; every step rounded to 32 bits."""
    c = s["case"]
    if c["norm"]:
        ms = _sum_pairs(x * x) * (1.0 / c["d"])
        inv = torch.reciprocal(torch.sqrt(ms + 1e-6))
        x = (x * inv) * (weight.float() + c["offset"])
    cs = s["cos_sin"][s["positions"].long()][:, None]
    half = c["rot"] // 2
    cos, sin = cs[..., :half], cs[..., half:]
    if c["interleaved"]:
        a, b = x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:c["rot"]]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., c["rot"]:]], -1)


def _write(cache, x, s, scale):
    """bf16 [T, Hkv, D] rows into their slots, in the cache's form."""
    c = s["case"]
    x, slot = x[s["keep"]], s["kept"]
    bs, hkv, d = c["bs"], c["hkv"], c["d"]
    if c["form"] == BF16:
        cache.view(torch.bfloat16).view(-1, hkv, d)[slot] = x
    elif c["form"] == FP8:
        q = (x.float() / _f32(scale, x)).clamp(-448, 448).to(torch.float8_e4m3fn)
        cache.view(-1, hkv, d)[slot] = q.view(torch.uint8)
    else:
        packed, sc = _nvfp4_encode(x.float())
        pages = cache.view(s["nb"], -1)
        head = torch.arange(hkv, device=x.device)
        line = head * bs + (slot % bs)[:, None]
        page = (slot // bs)[:, None, None]
        at = line[..., None] * (d // 2) + torch.arange(d // 2, device=x.device)
        pages[page, at] = packed
        at = bs * hkv * d // 2 + line[..., None] * (d // 16) + torch.arange(d // 16, device=x.device)
        pages[page, at] = sc


def _rope_plain(s):
    c = s["case"]
    x = s["qkv"].view(c["tokens"], c["hq"] + 2 * c["hkv"], c["d"])
    q, k, v = x[:, :c["hq"]], x[:, c["hq"]:c["hq"] + c["hkv"]], x[:, c["hq"] + c["hkv"]:]
    s["q_out"].copy_(_norm_rotate(q.float(), s["q_weight"], s))
    _write(s["k_cache"], _norm_rotate(k.float(), s["k_weight"], s).to(torch.bfloat16), s, s["k_scale"])
    _write(s["v_cache"], v, s, s["v_scale"])


def _gather(cache, s, scale, to=torch.float32):
    """The sequences' keys or values [B, Hkv, Lmax, D] through the block tables."""
    c = s["case"]
    bs, hkv, d = c["bs"], c["hkv"], c["d"]
    table = s["tables"][:, :(s["longest"] + bs - 1) // bs].long().clamp(min=0)
    if c["form"] == NVFP4:
        pages = cache.view(s["nb"], -1)
        n = bs * hkv * d
        vals = _nvfp4_decode(pages[:, :n // 2].reshape(s["nb"], hkv, bs, d // 2),
                             pages[:, n // 2:n // 2 + n // 16].reshape(s["nb"], hkv, bs, d // 16))
        x = vals[table].transpose(1, 2)
    elif c["form"] == FP8:
        x = cache.view(torch.float8_e4m3fn).view(s["nb"], bs, hkv, d)
        x = (x.view(torch.uint8)[table].view(torch.float8_e4m3fn).to(to) * scale).permute(0, 3, 1, 2, 4)
    else:
        x = cache.view(torch.bfloat16).view(s["nb"], bs, hkv, d)[table].to(to).permute(0, 3, 1, 2, 4)
    return x.reshape(table.shape[0], hkv, -1, d)


def _tree_visible(s, L, n):
    """[B, n, L]: which cached rows each node sees."""
    c = s["case"]
    dev = s["lens"].device
    lens, cu = s["lens"].long(), s["cu"].long()
    count = cu[1:] - cu[:-1]
    prefix = lens - count
    i = torch.arange(n, device=dev)
    bit = torch.arange(64, device=dev)
    at = (cu[:-1, None] + i).clamp(max=max(0, s["q"].shape[0] - 1))
    if s["mask"] is None:
        bits = (bit <= i[:, None]).expand(lens.shape[0], n, 64)
    else:
        bits = ((s["mask"][at][..., None] >> bit) & 1).bool()
    bits = bits & (bit < count[:, None])[:, None]
    depth = (bits.sum(-1) - 1).clamp(min=0)
    j = torch.arange(L, device=dev)
    node = j - prefix[:, None]                                   # [B, L]
    inside = (node >= 0) & (j < lens[:, None])
    node = node.clamp(0, n - 1)
    key_pos = torch.where(inside, prefix[:, None] + depth.gather(1, node), j)
    pos = prefix[:, None] + depth
    seen = torch.where(inside[:, None], bits.gather(2, node[:, None].expand(-1, n, -1)),
                       (j < prefix[:, None])[:, None])
    if c["window"]:
        near = pos[..., None] - key_pos[:, None] < c["window"]
        seen = seen & (near | (key_pos < c["sinks"])[:, None])
    return seen & (i < count[:, None])[..., None]


def _tree_plain(s):
    c = s["case"]
    B, hq, hkv, d = c["seqs"], c["hq"], c["hkv"], c["d"]
    n, grp = max(1, c["nodes"]), hq // hkv
    k = _gather(s["k_cache"], s, s["k_scale"])
    L = k.shape[2]
    q = torch.zeros(B * n, hq, d, device=k.device)
    q[s["rows"]] = s["q"].float()
    q = q.view(B, n, hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, grp * n, d)
    score = (q @ k.transpose(2, 3)).view(B, hkv, grp, n, L) * (1.0 / math.sqrt(d))
    del k
    score = score.masked_fill_(~_tree_visible(s, L, n)[:, None, None], NEG)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == NEG, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.view(B, hkv, grp * n, L) @ _gather(s["v_cache"], s, s["v_scale"])
    o = o.view(B, hkv, grp, n, d) / torch.where(total > 0, total, torch.ones_like(total))
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B * n, hq, d)[s["rows"]])


def _compact_plain(s):
    c = s["case"]
    bs, hkv, d, nb = c["bs"], c["hkv"], c["d"], s["nb"]
    lens, cu, num = s["lens"].long(), s["cu"].long(), s["num_accepted"].long()
    prefix = lens - (cu[1:] - cu[:-1])
    i = torch.arange(c["nodes"], device=lens.device)
    take = i < num[:, None]

    def slot(pos):
        return s["tables"].long().gather(1, pos // bs), pos % bs

    # entries past the accepted path leave the tree's root (always accepted) where it is
    src = torch.where(take, s["accepted"].long(), torch.zeros_like(i)) + prefix[:, None]
    dst = torch.where(take, i, torch.zeros_like(i)) + prefix[:, None]
    (sp, sr), (dp, dr) = slot(src), slot(dst)
    sp, sr, dp, dr = sp.flatten(), sr.flatten(), dp.flatten(), dr.flatten()
    pb = _page_bytes(c["form"], bs, hkv, d)
    for cache in (s["k_caches"], s["v_caches"]):
        pages = cache.view(c["layers"], nb, pb)
        if c["form"] == NVFP4:
            for start, width in ((0, d // 2), (bs * hkv * d // 2, d // 16)):
                sec = pages[:, :, start:start + bs * hkv * width].view(c["layers"], nb, hkv, bs, width)
                sec[:, dp, :, dr] = sec[:, sp, :, sr]
        else:
            rows = pages.view(c["layers"], nb, bs, -1)
            rows[:, dp, dr] = rows[:, sp, sr]
    s["new_lens"].copy_(prefix + num)


# ---------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if own:
        from paged_kv_split_gb300 import binding as pd
        geom = dict(num_kv_heads=c["hkv"], block_size=c["bs"], num_blocks=s["nb"],
                    kv_dtype=c["form"])
        if c["op"] == "rope":
            pd.pd_qk_norm_rope_cache(
                s["qkv"], s["q_out"], s["k_cache"], s["v_cache"], s["positions"], s["slots"],
                s["cos_sin"], q_weight=s["q_weight"] if c["norm"] else None,
                k_weight=s["k_weight"] if c["norm"] else None, weight_offset=c["offset"], eps=1e-6,
                interleaved=c["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"], **geom)
        elif c["op"] == "tree":
            pd.pd_decode_tree(
                s["q"], s["cu"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["out"],
                tree_mask=s["mask"], max_q_len=s["most"], scale=1.0 / math.sqrt(c["d"]),
                sliding_window=c["window"], num_sinks=c["sinks"], k_scale=s["k_scale"],
                v_scale=s["v_scale"], **geom)
        else:
            pd.pd_compact_tree(
                s["k_caches"], s["v_caches"], s["tables"], s["lens"], s["cu"], s["accepted"],
                s["num_accepted"], s["new_lens"], head_dim=c["d"], **geom)
    elif c["op"] == "rope":
        _rope_plain(s)
    elif c["op"] == "tree":
        _tree_plain(s)
    else:
        _compact_plain(s)
    if c["op"] == "rope":
        # BF16 and E4M3 caches as values; NVFP4 pages as the bytes they are: the definition
        # fixes every rounding of the norm and the rotation, so the codes have to agree
        kind = {BF16: torch.bfloat16, FP8: torch.float8_e4m3fn, NVFP4: torch.uint8}[c["form"]]
        return {"q": s["q_out"], "k_cache": s["k_cache"].view(kind),
                "v_cache": s["v_cache"].view(kind)}
    if c["op"] == "tree":
        return s["out"]
    # moved bytes, whatever they stand for
    return {"k": s["k_caches"].view(torch.int32), "v": s["v_caches"].view(torch.int32),
            "lens": s["new_lens"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written out sequence by sequence
def _exact_rope(s):
    c = s["case"]
    T, hq, hkv, d, half = c["tokens"], c["hq"], c["hkv"], c["d"], c["rot"] // 2
    x = s["qkv"].double().view(T, -1, d).clone()
    heads = hq + hkv
    if c["norm"]:
        w = torch.cat([s["q_weight"].double().expand(hq, d), s["k_weight"].double().expand(hkv, d)])
        part = x[:, :heads]
        x[:, :heads] = part / (part.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * (w + c["offset"])
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) * 2.0 / c["rot"])
    turn = torch.polar(torch.ones(T, half, dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None] * freq)[:, None]
    part = x[:, :heads, :c["rot"]]
    if c["interleaved"]:
        z = torch.view_as_real(torch.complex(part[..., 0::2].contiguous(),
                                             part[..., 1::2].contiguous()) * turn).flatten(-2)
    else:
        z = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * turn
        z = torch.cat([z.real, z.imag], -1)
    x[:, :heads, :c["rot"]] = z
    out = {"q": x[:, :hq].contiguous(), "k_cache": None, "v_cache": None}
    if c["form"] != NVFP4:
        for name, part, sc in (("k_cache", x[:, hq:heads], s["k_scale"]),
                               ("v_cache", x[:, heads:], s["v_scale"])):
            pool = torch.zeros(s["nb"] * c["bs"], hkv, d, dtype=torch.float64, device=DEV)
            part = part[s["keep"]]
            pool[s["kept"]] = part / sc if c["form"] == FP8 else part
            out[name] = pool.view(-1)
    return out


def _exact_rows(s, cache, table, length, scale):
    """One sequence's cached rows [length, Hkv, D] in 64 bits."""
    c = s["case"]
    bs, hkv, d = c["bs"], c["hkv"], c["d"]
    raw = cache.view(s["nb"], -1)[table[:(length + bs - 1) // bs].long()]
    if c["form"] == BF16:
        x = raw.view(torch.bfloat16).double().view(-1, hkv, d)
    elif c["form"] == FP8:
        x = raw.view(torch.float8_e4m3fn).double().view(-1, hkv, d) * scale
    else:
        n = bs * hkv * d
        code = raw[:, :n // 2].long()
        code = torch.stack([code % 16, code // 16], -1).view(-1, hkv, bs, d // 16, 16)
        m, e = code % 2, code // 2 % 4
        mag = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * torch.pow(2.0, (e - 1).double()))
        sc = raw[:, n // 2:n // 2 + n // 16].contiguous().view(torch.float8_e4m3fn).double()
        x = (torch.where(code >= 8, -mag, mag) * sc.view(-1, hkv, bs, d // 16, 1)).flatten(-2)
        x = x.transpose(1, 2).reshape(-1, hkv, d)
    return x[:length]


def _exact_tree(s):
    c = s["case"]
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    masks = None if s["mask"] is None else [m % (1 << 64) for m in s["mask"].tolist()]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    grp = c["hq"] // c["hkv"]
    for b in range(c["seqs"]):
        n, L = cu[b + 1] - cu[b], lens[b]
        if n == 0:
            continue
        prefix = L - n
        allowed = np.zeros((n, L), bool)
        tree = [(2 << i) - 1 if masks is None else masks[cu[b] + i] % (1 << n) for i in range(n)]
        depth = [max(0, bin(t).count("1") - 1) for t in tree]
        pos = np.concatenate([np.arange(prefix), prefix + np.array(depth)])
        for i in range(n):
            allowed[i, :prefix] = True
            allowed[i, prefix:] = [(tree[i] >> k) & 1 for k in range(n)]
            if c["window"]:
                allowed[i] &= (prefix + depth[i] - pos < c["window"]) | (pos < c["sinks"])
        keys = np.nonzero(allowed.any(0))[0]
        if not len(keys):
            continue
        ok = torch.from_numpy(allowed[:, keys]).to(DEV)
        at = _i64(keys)
        k = _exact_rows(s, s["k_cache"], s["tables"][b], L, s["k_scale"])[at]
        v = _exact_rows(s, s["v_cache"], s["tables"][b], L, s["v_scale"])[at]
        q = s["q"][cu[b]:cu[b + 1]].double()
        for h in range(c["hq"]):
            logit = (q[:, h] @ k[:, h // grp].T / math.sqrt(c["d"])).masked_fill(~ok, NEG)
            w = torch.softmax(logit, -1).nan_to_num(0.0)
            out[cu[b]:cu[b + 1], h] = w @ v[:, h // grp]
    return out


def exact(case, seed):
    if case["op"] == "compact":
        return None  # moved bytes: nothing is computed
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_tree(s)
