"""Workloads of serving from a paged cache held in INT8 with a scale per page and head.

Three operators, each in its plain form (elementary torch operations) and as
the library's call:

* append: the position rotation of new tokens' q and k heads and the append of
          K and V to the INT8 pages (``pd_rope_append_int8``): a page keeps one
          scale per kv head, and a page that gets rows larger than its scale
          reaches has its older rows' codes brought to the new scale;
* decode: single-token attention over that cache (``pd_decode_balanced`` or
          ``pd_decode``, whichever ``pd_prefer_balanced`` names for the lengths);
* prompt: attention of whole prompts over their own rotated rows, packed one
          behind the other, before or beside the cache (``pd_prefill_packed``).

An INT8 page (include/pd.h) holds [head][block][dim] signed codes, then one
fp32 scale per head; its stride is rounded up to 128 bytes.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
NEG = float("-inf")
SMALLEST, LARGEST = 2.0 ** -60, 2.0 ** 60  # a page's scale


# ---------------------------------------------------------------------------
# the cases
def _append(**kw):
    c = dict(op="append", seqs=8, lo=100, hi=1000, new_lo=1, new=1, hq=32, hkv=8, d=128, bs=16,
             rot=128, interleaved=False, keep_k=False, far=32768, shape=1)
    c.update(kw)
    return c


def _decode(**kw):
    c = dict(op="decode", seqs=1, lo=1024, hi=4096, hq=32, hkv=8, d=128, bs=16, window=0,
             holes=False, lengths="uniform", shape=1)
    c.update(kw)
    return c


def _prompt(**kw):
    c = dict(op="prompt", seqs=1, lo=64, hi=2048, hq=32, hkv=8, d=128, window=0, causal=True,
             holes=False, shape=1)
    c.update(kw)
    return c


def listed():
    return [
        # one new token for each of 8 sequences: the launch itself counts
        _append(name="append_step_b8", seqs=8, shape=11),
        # a step of the quantised-cache batch, 64 sequences of 64 / 8 heads
        _append(name="append_step_b64", seqs=64, hq=64, shape=12),
        # short chunks of 1 to 40 tokens at wide heads: half the head rotated, pairs side by side
        _append(name="append_chunks_d256", seqs=12, new=40, hq=8, hkv=4, d=256, rot=128,
                interleaved=True, shape=13),
        # four prompts of up to 4096 tokens on their way into the cache, their rotated keys kept
        # for the attention over the prompts themselves
        _append(name="append_prompts", seqs=4, lo=0, hi=0, new_lo=500, new=4000, keep_k=True,
                shape=14),
        # one user over a short context: latency
        _decode(name="decode_b1_short", seqs=1, lo=777, hi=777, shape=21),
        # a serving batch of 32 sequences, 1K to 4K keys
        _decode(name="decode_b32", seqs=32, shape=22),
        # the quantised-cache batch: 64 sequences, lengths from 512 to 16384
        _decode(name="decode_b64_lognormal", seqs=64, lo=512, hi=16384, hq=64,
                lengths="lognormal", shape=23),
        # wide heads under a window
        _decode(name="decode_window_d256", seqs=8, lo=16384, hi=16384, hq=8, hkv=4, d=256,
                window=4096, shape=24),
        # three short prompts of a chat: latency
        _prompt(name="prompt_short_b3", seqs=3, lo=17, hi=200, shape=31),
        # a prefill batch of ragged prompts
        _prompt(name="prompt_ragged_b16", seqs=16, lo=64, hi=2048, shape=32),
        # narrow heads under a window
        _prompt(name="prompt_window_d64", seqs=6, lo=1500, hi=4096, hq=8, hkv=2, d=64, window=1024,
                shape=33),
        # one long document
        _prompt(name="prompt_8192", seqs=1, lo=8192, hi=8192, shape=34),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = [(32, 8, 128), (32, 8, 128), (64, 8, 128), (4, 2, 64), (8, 4, 256), (16, 2, 512),
          (6, 1, 64), (12, 12, 128), (16, 1, 128)]


def draw(rng):
    shape = rng.randrange(1 << 30)
    op = rng.choice(["append", "decode", "prompt"])
    if op == "append":
        hq, hkv, d = rng.choice(_HEADS)
        room = 9000 * 48 * 128 // ((hq + 2 * hkv) * d)  # rows the largest listed case has
        new = rng.choice([1, _log(rng, 2, 64), min(room, _log(rng, 64, 4096))])
        seqs = max(1, min(_log(rng, 1, 64), room // new))
        lo = rng.choice([0, _log(rng, 1, 1000)])
        return _append(seqs=seqs, lo=lo, hi=lo + _log(rng, 1, 500), new_lo=rng.randrange(1, new + 1),
                       new=new, hq=hq, hkv=hkv, d=d, bs=rng.choice([16, 32]),
                       rot=rng.choice([d, d, d // 2, 32, 48]), interleaved=rng.random() < 0.4,
                       keep_k=rng.random() < 0.5, far=_log(rng, 5000, 131072), shape=shape)
    if op == "decode":
        hq, hkv, d = rng.choice(_HEADS)
        hi = _log(rng, 1, 32768)
        lo = rng.randrange(1, hi + 1)
        # no more than the largest listed case reads
        seqs = max(1, min(_log(rng, 1, 64), int(min(160e6 / (hkv * d), 220000) / hi)))
        return _decode(seqs=seqs, lo=lo, hi=hi, hq=hq, hkv=hkv, d=d, bs=rng.choice([16, 32]),
                       window=rng.choice([0, 0, _log(rng, 8, 8192)]), holes=rng.random() < 0.3,
                       lengths=rng.choice(["uniform", "lognormal"]), shape=shape)
    hq, hkv, d = rng.choice([h for h in _HEADS if h[2] <= 256])
    hi = _log(rng, 1, 8192)
    lo = rng.randrange(1, hi + 1)
    # no more products than the largest listed case, no more rows than four times its own
    causal = rng.random() < 0.8
    each = (2.0 if causal else 4.0) * d * hq
    hi = min(hi, int(math.sqrt(5e11 / each)))
    lo = min(lo, hi)
    seqs = max(1, min(_log(rng, 1, 64), int(min(5e11 / (each * hi * hi), 32768 / hi))))
    return _prompt(seqs=seqs, lo=lo, hi=hi, hq=hq, hkv=hkv, d=d,
                   window=rng.choice([0, 0, _log(rng, 8, 4096)]), causal=causal,
                   holes=rng.random() < 0.3, shape=shape)


# ---------------------------------------------------------------------------
# what a case's sizes settle: lengths and new tokens
def _lengths(c):
    """(lengths with the new tokens, new tokens) of each sequence."""
    r = np.random.RandomState(c["shape"] % (1 << 31))
    B = c["seqs"]
    if c.get("lengths") == "lognormal":
        lens = np.clip(np.round(np.exp(r.normal(math.log(2048.0), 1.0, B))), c["lo"], c["hi"])
    else:
        lens = r.randint(c["lo"], c["hi"] + 1, B)
    lens = lens.astype(np.int64)
    if c.get("holes"):  # idle slots of a batch
        lens[1:][r.rand(B - 1) < 0.15] = 0
    if c["op"] == "append":
        new = r.randint(c["new_lo"], c["new"] + 1, B).astype(np.int64)
        return lens + new, new
    return lens, lens if c["op"] == "prompt" else np.minimum(lens, 1)


def _seen(n, window, causal):
    """(query, key) pairs of a prompt of n tokens."""
    if causal:
        w = min(n, window) if window else n
        return w * (w + 1) // 2 + (n - w) * w
    return n * n if not window else n * min(n, window)


def work(case):
    c = case
    lens, new = _lengths(c)
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if c["op"] == "append":
        T = int(new.sum())
        units = int(((lens - 1) // c["bs"] - (lens - new) // c["bs"] + 1).sum())
        rows = 2 * T * (hq + 2 * hkv) * d + 2 * T * hq * d + (2 * T * hkv * d if c["keep_k"] else 0)
        return {"bytes": rows + 2 * T * hkv * d + 8 * units * hkv + 4 * units + 8 * c["seqs"] +
                4 * min(T, c["far"]) * c["rot"],
                "flops": 3 * T * (hq + hkv) * c["rot"] + 6 * T * hkv * d}
    if c["op"] == "decode":
        W = c["window"]
        keys = np.minimum(lens, W) if W else lens
        pages = int(((lens + c["bs"] - 1) // c["bs"] - (lens - keys) // c["bs"]).sum())
        return {"bytes": int(keys.sum()) * hkv * 2 * d + pages * (8 * hkv + 4) +
                4 * c["seqs"] * hq * d, "flops": 4 * d * hq * int(keys.sum())}
    T = int(lens.sum())
    pairs = sum(_seen(int(n), c["window"], c["causal"]) for n in lens)
    return {"bytes": 2 * T * (2 * hq + 2 * hkv) * d, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------
# inputs
def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _page_bytes(c):
    return (c["bs"] * c["hkv"] * c["d"] + 4 * c["hkv"] + 127) // 128 * 128


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


def _codes(cache, c):
    """The codes of a flat cache, [page][head][row][dim]."""
    hkv, bs, d = c["hkv"], c["bs"], c["d"]
    return cache.view(torch.int8).view(-1, _page_bytes(c))[:, :hkv * bs * d].unflatten(
        1, (hkv, bs, d))


def _scales(cache, c):
    """The scales of a flat cache, [page][head]."""
    n = c["hkv"] * c["bs"] * c["d"] // 4
    return cache.view(torch.float32).view(-1, _page_bytes(c) // 4)[:, n:n + c["hkv"]]


def _random_cache(c, nb, g):
    """A pool of nb pages of unit normals in the cache's form, a page's largest value at 127."""
    cache = torch.zeros(nb * _page_bytes(c), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (c["hkv"] * c["bs"] * c["d"]))
    for at in range(0, nb, step):
        n = min(step, nb - at)
        x = torch.randn(n, c["hkv"], c["bs"], c["d"], generator=g, device=DEV)
        top = x.abs().amax((2, 3))
        _codes(cache, c)[at:at + n] = torch.round(x / (top[..., None, None] / 127)).to(torch.int8)
        _scales(cache, c)[at:at + n] = top / 127
    return cache


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = np.random.RandomState((seed * 2654435761 + c["shape"]) % (1 << 31))
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    lens, new = _lengths(c)
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    s = {"case": dict(c), "cu": _i32(cu), "most": max(1, int(new.max())), "new": new.tolist()}
    if c["op"] == "prompt":
        # rows as the projections leave them: q, k and v heads of a token side by side
        qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device=DEV).to(torch.bfloat16)
        q, k, v = qkv.split([hq * d, hkv * d, hkv * d], 1)
        s.update(q=q.unflatten(1, (hq, d)), k=k.unflatten(1, (hkv, d)),
                 v=v.unflatten(1, (hkv, d)),
                 out=torch.empty(T, hq, d, dtype=torch.bfloat16, device=DEV))
        return s
    table, nb = _paging(lens, c["bs"], r)
    nb += 1  # a spare page that belongs to no sequence
    s.update(nb=nb, tables=_i32(table), lens=_i32(lens),
             k_cache=_random_cache(c, nb, g), v_cache=_random_cache(c, nb, g))
    if c["op"] == "append":
        half = c["rot"] // 2
        inv = 10000.0 ** (-np.arange(half) * 2.0 / c["rot"])
        ang = torch.arange(c["far"], dtype=torch.float64, device=DEV)[:, None] * \
            torch.from_numpy(inv).to(DEV)
        s.update(
            qkv=torch.randn(T, (hq + 2 * hkv) * d, generator=g, device=DEV).to(torch.bfloat16),
            q_out=torch.empty(T, hq, d, dtype=torch.bfloat16, device=DEV),
            k_out=torch.empty(T, hkv, d, dtype=torch.bfloat16, device=DEV) if c["keep_k"] else None,
            cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float().contiguous())
        return s
    s.update(q=torch.randn(c["seqs"], hq, d, generator=g, device=DEV).to(torch.bfloat16),
             out=torch.empty(c["seqs"], hq, d, dtype=torch.bfloat16, device=DEV),
             longest=max(1, int(lens.max())), plan=None, splits=1)
    if own:
        # the schedule of this step's lengths, which the calls of all layers share
        from paged_kv_split_gb300 import binding as pd
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        geom = dict(num_q_heads=hq, num_kv_heads=hkv, max_blocks_per_seq=table.shape[1],
                    block_size=c["bs"], head_dim=d, sliding_window=c["window"], kv_dtype="int8",
                    num_sms=sms)
        if pd.pd_prefer_balanced(lens, **geom):
            s["plan"] = pd.pd_balanced_plan(lens, **geom)
            s["plan_dev"] = s["plan"].to(DEV)
        else:
            s["splits"] = pd.pd_plan_num_splits_for_lengths(lens, **geom)
    return s


# ---------------------------------------------------------------------------
# plain forms
def _rotate(x, cs, rot, interleaved):
    """x fp32 [T, H, D] by the angles whose cosines and sines are cs [T, rot]; every operation
    rounded to 32 bits."""
    half = rot // 2
    cos, sin = cs[:, None, :half], cs[:, None, half:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _units(s):
    """The pages that get rows, [B, U] padded with the spare page: (page, a row's index in the
    batch [B, U, bs], whether the row is new, whether it is older than the new ones, fresh pages)."""
    c = s["case"]
    bs, dev = c["bs"], s["lens"].device
    lens, cu = s["lens"].long(), s["cu"].long()
    first = lens - (cu[1:] - cu[:-1])
    U = (s["most"] + bs - 2) // bs + 1
    index = (first // bs)[:, None] + torch.arange(U, device=dev)
    on = index * bs < lens[:, None]
    page = torch.where(on, s["tables"].long().gather(1, index.clamp(max=s["tables"].shape[1] - 1)),
                       torch.full_like(index, s["nb"] - 1))
    pos = index[..., None] * bs + torch.arange(bs, device=dev)
    start = first[:, None, None]
    fresh_row = (pos >= start) & (pos < lens[:, None, None]) & on[..., None]
    old_row = (pos < start) & on[..., None]
    row = (cu[:-1, None, None] + pos - start).clamp(0, max(0, s["qkv"].shape[0] - 1))
    return page, row, fresh_row, old_row, on & (index * bs >= first[:, None])


def _append_cache(cache, x, s, units):
    """x [T, Hkv, D] into the pages' codes and scales."""
    c = s["case"]
    page, row, new_row, old_row, fresh = units
    vals = x[row].float().transpose(2, 3)                       # [B, U, hkv, bs, d]
    is_new = new_row[:, :, None, :, None]
    top = torch.where(is_new, vals.abs(), torch.zeros_like(vals)).amax((3, 4))
    full = torch.full((1,), 127.0, device=x.device)
    want = (top / full).clamp(min=SMALLEST, max=LARGEST)
    codes, scales = _codes(cache, c), _scales(cache, c)
    have = scales[page]
    on = new_row.any(-1)[..., None]
    scale = torch.where(on, torch.where(fresh[..., None] | (want > have), want, have), have)
    old = codes[page]
    ratio = (have / scale)[..., None, None]
    grown = (scale > have)[..., None, None] & old_row[:, :, None, :, None]
    kept = torch.where(grown, torch.round(old.float() * ratio), old.float())
    got = torch.round(vals * (torch.ones_like(scale) / scale)[..., None, None]).clamp(-127, 127)
    codes[page] = torch.where(is_new, got, kept).to(torch.int8)
    scales[page] = scale


def _append_plain(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    T = s["qkv"].shape[0]
    x = s["qkv"].view(T, hq + 2 * hkv, d)
    lens, cu = s["lens"].long(), s["cu"].long()
    t = torch.arange(T, device=x.device)
    b = (t[:, None] >= cu[1:]).sum(1)
    cs = s["cos_sin"][t - cu[b] + lens[b] - (cu[b + 1] - cu[b])]
    s["q_out"].copy_(_rotate(x[:, :hq].float(), cs, c["rot"], c["interleaved"]))
    k = _rotate(x[:, hq:hq + hkv].float(), cs, c["rot"], c["interleaved"])
    if c["keep_k"]:
        s["k_out"].copy_(k)
    units = _units(s)
    _append_cache(s["k_cache"], k, s, units)
    _append_cache(s["v_cache"], x[:, hq + hkv:], s, units)


def _gather(cache, s):
    """The sequences' keys or values [B, Hkv, Lmax, D] through the block tables."""
    c = s["case"]
    table = s["tables"][:, :(s["longest"] + c["bs"] - 1) // c["bs"]].long().clamp(min=0)
    x = _codes(cache, c)[table].float() * _scales(cache, c)[table][..., None, None]
    return x.transpose(1, 2).reshape(table.shape[0], c["hkv"], -1, c["d"])


def _weights(score, seen):
    """exp(score - its row's maximum) where `seen`, else 0, and the rows' sums (1 for none)."""
    score = score.masked_fill_(~seen, NEG)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == NEG, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    return p, torch.where(total > 0, total, torch.ones_like(total))


def _decode_plain(s):
    c = s["case"]
    B, hq, hkv, d = c["seqs"], c["hq"], c["hkv"], c["d"]
    k = _gather(s["k_cache"], s)
    q = s["q"].float().view(B, hkv, hq // hkv, d)
    score = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    del k
    j = torch.arange(score.shape[-1], device=score.device)
    lens = s["lens"].long()[:, None]
    seen = j < lens
    if c["window"]:
        seen = seen & (j >= lens - c["window"])
    p, total = _weights(score, seen[:, None, None])
    s["out"].copy_((p @ _gather(s["v_cache"], s) / total).view(B, hq, d))


def _prompt_plain(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    at = 0
    for n in s["new"]:
        rows = slice(at, at + n)
        k = s["k"][rows].float().transpose(0, 1)[:, None]        # [hkv, 1, n, d]
        v = s["v"][rows].float().transpose(0, 1)[:, None]
        j = torch.arange(n, device=k.device)
        for i0 in range(0, n, 2048):                              # bounds the scores held at once
            i1 = min(n, i0 + 2048)
            q = s["q"][at + i0:at + i1].float().view(i1 - i0, hkv, hq // hkv, d).permute(1, 2, 0, 3)
            # the last token sees everything when the rows are not causal
            i = torch.arange(i0, i1, device=k.device)[:, None] if c["causal"] else \
                torch.full((i1 - i0, 1), n - 1, device=k.device)
            seen = j <= i
            if c["window"]:
                seen = seen & (i - j < c["window"])
            p, total = _weights((q @ k.transpose(2, 3)) * (1.0 / math.sqrt(d)), seen)
            s["out"][at + i0:at + i1] = (p @ v / total).permute(2, 0, 1, 3).reshape(i1 - i0, hq, d)
        at += n


# ---------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if own:
        from paged_kv_split_gb300 import binding as pd
        if c["op"] == "append":
            pd.pd_rope_append_int8(
                s["qkv"], s["q_out"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["cu"],
                s["cos_sin"], max_q_len=s["most"], num_kv_heads=c["hkv"], block_size=c["bs"],
                num_blocks=s["nb"], interleaved=c["interleaved"], k_out=s["k_out"])
        elif c["op"] == "prompt":
            pd.pd_prefill_packed(s["q"], s["k"], s["v"], s["cu"], s["out"], max_q_len=s["most"],
                                 scale=1.0 / math.sqrt(c["d"]), causal=c["causal"],
                                 sliding_window=c["window"])
        else:
            geom = dict(num_kv_heads=c["hkv"], block_size=c["bs"], num_blocks=s["nb"],
                        scale=1.0 / math.sqrt(c["d"]), sliding_window=c["window"],
                        kv_dtype="int8")
            if s["plan"] is not None:
                pd.pd_decode_balanced(s["q"], s["k_cache"], s["v_cache"], s["tables"],
                                      s["plan_dev"], s["plan"], s["out"], **geom)
            else:
                pd.pd_decode(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["out"],
                             num_splits=s["splits"], **geom)
    elif c["op"] == "append":
        _append_plain(s)
    elif c["op"] == "prompt":
        _prompt_plain(s)
    else:
        _decode_plain(s)
    if c["op"] != "append":
        return s["out"]
    # the definition fixes every rounding of the rotation, the scales and the codes, so the codes
    # have to agree; with the scales they are all that the cache stands for
    got = {"q": s["q_out"], "k": _codes(s["k_cache"], c), "k_scale": _scales(s["k_cache"], c),
           "v": _codes(s["v_cache"], c), "v_scale": _scales(s["v_cache"], c)}
    if c["keep_k"]:
        got["k_rows"] = s["k_out"]
    return got


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written out sequence by sequence
def _exact_append(s):
    c = s["case"]
    hq, hkv, d, bs, half = c["hq"], c["hkv"], c["d"], c["bs"], c["rot"] // 2
    T = s["qkv"].shape[0]
    lens, cu, tables = s["lens"].tolist(), s["cu"].tolist(), s["tables"].tolist()
    x = s["qkv"].double().view(T, -1, d).clone()
    pos = torch.cat([torch.arange(lens[b] - (cu[b + 1] - cu[b]), lens[b], device=DEV)
                     for b in range(c["seqs"])]).double()
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) * 2.0 / c["rot"])
    turn = torch.polar(torch.ones(T, half, dtype=torch.float64, device=DEV),
                       pos[:, None] * freq)[:, None]
    part = x[:, :hq + hkv, :c["rot"]]
    if c["interleaved"]:
        z = torch.view_as_real(torch.complex(part[..., 0::2].contiguous(),
                                             part[..., 1::2].contiguous()) * turn).flatten(-2)
    else:
        z = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * turn
        z = torch.cat([z.real, z.imag], -1)
    x[:, :hq + hkv, :c["rot"]] = z
    out = {"q": x[:, :hq].contiguous(), "k": None, "v": None}
    for name, cache, rows in (("k_scale", s["k_cache"], x[:, hq:hq + hkv]),
                              ("v_scale", s["v_cache"], x[:, hq + hkv:])):
        top = rows.abs().amax(-1) / 127
        scale = _scales(cache, c).double().clone()
        for b in range(c["seqs"]):
            p0 = lens[b] - (cu[b + 1] - cu[b])
            for i in range(p0 // bs, (lens[b] + bs - 1) // bs):
                lo, hi = max(p0, i * bs), min(lens[b], (i + 1) * bs)
                t = top[cu[b] + lo - p0:cu[b] + hi - p0].amax(0).clamp(SMALLEST, LARGEST)
                at = tables[b][i]
                scale[at] = t if lo == i * bs else torch.maximum(t, scale[at])
        out[name] = scale
    if c["keep_k"]:
        out["k_rows"] = x[:, hq:hq + hkv].contiguous()
    return out


def _exact_rows(s, cache, table, length):
    """One sequence's cached rows [length, Hkv, D] in 64 bits."""
    c = s["case"]
    at = table[:(length + c["bs"] - 1) // c["bs"]].long()
    x = _codes(cache, c)[at].double() * _scales(cache, c)[at].double()[..., None, None]
    return x.transpose(1, 2).reshape(-1, c["hkv"], c["d"])[:length]


def _exact_decode(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    grp = c["hq"] // c["hkv"]
    for b, L in enumerate(s["lens"].tolist()):
        if L == 0:
            continue
        lo = max(0, L - c["window"]) if c["window"] else 0
        k = _exact_rows(s, s["k_cache"], s["tables"][b], L)[lo:]
        v = _exact_rows(s, s["v_cache"], s["tables"][b], L)[lo:]
        q = s["q"][b].double()
        for h in range(c["hq"]):
            w = torch.softmax(k[:, h // grp] @ q[h] / math.sqrt(c["d"]), 0)
            out[b, h] = w @ v[:, h // grp]
    return out


def _exact_prompt(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    grp = c["hq"] // c["hkv"]
    at = 0
    for n in s["new"]:
        for h in range(c["hq"] if n else 0):
            q, k, v = (t[at:at + n, hh].double() for t, hh in
                       ((s["q"], h), (s["k"], h // grp), (s["v"], h // grp)))
            logit = q @ k.T / math.sqrt(c["d"])
            if c["causal"]:
                ok = torch.ones_like(logit, dtype=torch.bool).tril_()
                if c["window"]:
                    ok = ok.triu_(1 - c["window"])
                logit = logit.masked_fill_(~ok, NEG)
            elif c["window"]:
                logit[:, :max(0, n - c["window"])] = NEG
            out[at:at + n, h] = torch.softmax(logit, -1) @ v
        at += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode,
            "prompt": _exact_prompt}[case["op"]](s)
