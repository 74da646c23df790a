"""Decoding with drafted token trees, end to end over the paged cache.

A small decoder with random weights generates greedily. Each step drafts a tree
of tokens for every sequence from a bigram table, runs the model on all of them
at once, keeps the longest path that the model agrees with, and moves that
path's K/V rows to consecutive positions:

    pd_qk_norm_rope_cache_   norm and rotate q and k, write K/V   (every layer)
    pd_decode_tree_strided   attention of the trees               (every layer)
    pd_compact_tree          the accepted rows, all layers        (once a step)

Lengths, trees and accepted paths stay on the device, so that the whole step is
captured once in a CUDA graph and replayed.

    python examples/draft_and_verify.py [--kv bf16|fp8_e4m3|nvfp4] [--steps 32]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from paged_kv_split_gb300 import binding as pd  # noqa: E402

KV = {"bf16": pd.PD_KV_BF16, "fp8_e4m3": pd.PD_KV_FP8_E4M3, "nvfp4": pd.PD_KV_NVFP4}


class Model:
    """A pre-norm decoder; next-token scores lean on a fixed bigram, which is
    what makes drafting from the bigram worth while."""

    hidden, layers, hq, hkv, d, vocab = 256, 2, 8, 2, 64, 512

    def __init__(self, num_blocks, block_size=16, kv_dtype=pd.PD_KV_BF16, max_position=4096, seed=0,
                 device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def weight(*shape, gain=1.0):
            w = torch.randn(*shape, generator=g) * gain * shape[0] ** -0.5
            return w.to(device, torch.bfloat16)

        E, qkv = self.hidden, (self.hq + 2 * self.hkv) * self.d
        self.kv_dtype, self.num_blocks, self.block_size = kv_dtype, num_blocks, block_size
        self.max_position = max_position
        self.kv_scale = 6.0 / 448 if kv_dtype == pd.PD_KV_FP8_E4M3 else 1.0
        self.embed = weight(E, self.vocab, gain=E ** 0.5).t().contiguous()
        self.wqkv = [weight(E, qkv) for _ in range(self.layers)]
        self.wo = [weight(self.hq * self.d, E, gain=8) for _ in range(self.layers)]
        self.norms = [[(torch.randn(self.d, generator=g) * 0.1 + 1).to(device, torch.bfloat16)
                       for _ in range(2)] for _ in range(self.layers)]
        # a token's successor in the bigram: its embedding scores highest
        follow = torch.randperm(self.vocab, generator=g).to(device)
        self.head = torch.empty_like(self.embed)
        self.head[follow] = self.embed
        self.head = (self.head.float() * E ** -0.5).to(torch.bfloat16).t().contiguous()
        self.bigram = (self._norm(self.embed.float()) @ self.head).float().topk(2).indices
        self.cos_sin = pd.pd_rope_table(
            torch.empty(max_position, self.d, dtype=torch.float32, device=device))
        n = pd.pd_cache_bytes(kv_dtype, num_blocks, block_size, self.hkv, self.d)
        self.k = torch.zeros(self.layers, n, dtype=torch.uint8, device=device)
        self.v = torch.zeros_like(self.k)

    @staticmethod
    def _norm(h):
        return (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def shape(self):
        return dict(num_kv_heads=self.hkv, block_size=self.block_size, num_blocks=self.num_blocks,
                    kv_dtype=self.kv_dtype)

    def forward(self, tokens, positions, slots, attend):
        """Scores fp32 [T, vocab] of int64 tokens [T]; attend(layer, rows, out)
        is the attention of the rows' q heads over the layer's cache."""
        h = self.embed[tokens].float()
        att = torch.empty(tokens.shape[0], self.hq * self.d, dtype=torch.bfloat16,
                          device=tokens.device)
        for i in range(self.layers):
            rows = self._norm(h) @ self.wqkv[i]
            pd.pd_qk_norm_rope_cache_(rows, self.k[i], self.v[i], positions, slots, self.cos_sin,
                                      num_q_heads=self.hq, head_dim=self.d,
                                      q_weight=self.norms[i][0], k_weight=self.norms[i][1],
                                      k_scale=self.kv_scale, v_scale=self.kv_scale, **self.shape())
            attend(i, rows, att)
            h = h + (att @ self.wo[i]).float()
        return (self._norm(h) @ self.head).float()

    def attention(self, call, tables, lens, **kw):
        """attend() of forward through pd_prefill_strided or pd_decode_tree_strided."""
        def attend(i, rows, out):
            call(rows, kw["cu_q"], self.k[i], self.v[i], tables, lens, out, num_q_heads=self.hq,
                 head_dim=self.d, scale=self.d ** -0.5, k_scale=self.kv_scale,
                 v_scale=self.kv_scale, **self.shape(),
                 **{k: x for k, x in kw.items() if k != "cu_q"})
        return attend


def slots_of(tables, rows, seq, block_size):
    """Cache slots (int32) of rows (int64) of sequences seq, through the block tables."""
    page = tables[seq, rows // block_size].long()
    return (page * block_size + rows % block_size).int()


def rows_needed(longest, steps, depth):
    """Cached rows of a sequence that starts with `longest` and takes `steps` steps:
    each adds depth + 1 at most, and the last needs its whole tree's."""
    return longest + max(steps - 1, 0) * (depth + 1) + (1 + 2 * depth if steps > 0 else 0)


def steps_that_fit(longest, rows, depth):
    return max((rows - longest - (1 + 2 * depth)) // (depth + 1) + 1, 0)


class DraftAndVerify:
    """Sequences being decoded: `tokens` accepted last, `lens` cached rows.

    A tree is the last accepted token, then `depth` levels of the bigram's first
    choice (which goes on) and its second (which does not).

    Lengths are on the device, where a row past the block table is found by a fault
    only: so `steps_left` counts on the host what fits whatever is accepted, and a
    step beyond it is refused."""

    def __init__(self, model, prompts, tables, depth=4):
        dev = tables.device
        rows = min(tables.shape[1] * model.block_size, model.max_position)
        longest = max(len(p) for p in prompts)
        if len(prompts) != tables.shape[0] or min(len(p) for p in prompts) < 1:
            raise ValueError("one prompt of one token at least for each row of the block table")
        if longest > rows:
            raise ValueError(f"a prompt of {longest} tokens does not fit {rows} rows")
        if any(int(p.min()) < 0 or int(p.max()) >= model.vocab for p in prompts):
            raise ValueError(f"a token outside the vocabulary of {model.vocab}")
        self.steps_left = steps_that_fit(longest, rows, depth)
        self.model, self.tables, self.depth = model, tables, depth
        B, n = tables.shape[0], 1 + 2 * depth
        self.B, self.n = B, n
        parent = [-1] + [max(2 * (l - 1) - 1, 0) for l in range(1, depth + 1) for _ in range(2)]
        masks, level = [], []
        for i, p in enumerate(parent):
            masks.append((masks[p] if p >= 0 else 0) | (1 << i))
            level.append(level[p] + 1 if p >= 0 else 0)
        self.mask = torch.tensor(masks * B, dtype=torch.int64, device=dev)
        self.level = torch.tensor(level, device=dev)
        self.main = torch.tensor([0] + [2 * l - 1 for l in range(1, depth + 1)], device=dev)
        self.cu_q = torch.arange(0, (B + 1) * n, n, dtype=torch.int32, device=dev)
        self.seq = torch.arange(B, device=dev).repeat_interleave(n)
        self.lens = torch.zeros(B, dtype=torch.int32, device=dev)
        self.tokens = torch.zeros(B, dtype=torch.int64, device=dev)
        self.emitted = torch.zeros(B, depth + 2, dtype=torch.int64, device=dev)  # of the last step
        self.num_emitted = torch.zeros(B, dtype=torch.int32, device=dev)
        self._prompts(prompts)

    def _prompts(self, prompts):
        m, dev = self.model, self.tables.device
        lens = [len(p) for p in prompts]
        seq = torch.repeat_interleave(torch.arange(self.B), torch.tensor(lens)).to(dev)
        pos = torch.cat([torch.arange(x) for x in lens]).to(dev)
        cu = torch.tensor([0] + lens).cumsum(0).int().to(dev)
        self.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        scores = m.forward(torch.cat(prompts).to(dev), pos.int(),
                           slots_of(self.tables, pos, seq, m.block_size),
                           m.attention(pd.pd_prefill_strided, self.tables, self.lens, cu_q=cu,
                                       max_q_len=max(lens)))
        self.scores = scores[cu[1:].long() - 1]
        self.tokens.copy_(self.scores.argmax(-1))

    def step(self):
        """One step; nothing here waits for the device or asks it for a length."""
        self._take()
        self._step()

    def _take(self):
        if self.steps_left < 1:
            raise ValueError("no room for another step in the block table or the rotation table")
        self.steps_left -= 1

    def _step(self):
        m, B, n, depth = self.model, self.B, self.n, self.depth
        # ---- draft ----
        level = [self.tokens[:, None]]
        for _ in range(depth):
            level.append(m.bigram[level[-1][:, 0]])
        tree = torch.cat(level, 1)                                # [B, n]
        # ---- the model on every node ----
        prefix = self.lens.long()
        rows = (prefix[:, None] + torch.arange(n, device=tree.device)).view(-1)
        positions = (prefix[:, None] + self.level).view(-1).int()
        with_tree = self.lens + n
        scores = m.forward(tree.view(-1), positions, slots_of(self.tables, rows, self.seq, m.block_size),
                           m.attention(pd.pd_decode_tree_strided, self.tables, with_tree,
                                       cu_q=self.cu_q, tree_mask=self.mask, max_q_len=n))
        # ---- verify: the first choices that agree, then perhaps a second choice ----
        said = scores.argmax(-1).view(B, n)
        agree = (said[:, self.main[:-1]] == tree[:, self.main[1:]]).long().cumprod(1)
        a = agree.sum(1)                                          # accepted first choices
        last = self.main[a]
        second = (2 * a + 2).clamp(max=n - 1)
        extra = (a < depth) & (said.gather(1, last[:, None])[:, 0] ==
                               tree.gather(1, second[:, None])[:, 0])
        nodes = torch.cat([self.main, self.main[:1]]).expand(B, -1).clone()
        nodes.scatter_(1, (a + 1)[:, None], torch.where(extra, second, 0)[:, None])
        count = a + 1 + extra.long()
        # ---- keep their rows ----
        accepted, num_accepted = nodes.int(), count.int()
        new_lens = torch.empty_like(self.lens)
        pd.pd_compact_tree(m.k, m.v, self.tables, with_tree, self.cu_q, accepted, num_accepted,
                           new_lens, head_dim=m.d, **m.shape())
        final = nodes.gather(1, (count - 1)[:, None])
        self.tokens.copy_(said.gather(1, final)[:, 0])
        self.emitted.copy_(tree.gather(1, nodes))
        self.num_emitted.copy_(num_accepted)
        self.scores = scores.view(B, n, -1).gather(
            1, nodes[..., None].expand(-1, -1, scores.shape[-1]))  # of the emitted nodes
        self.lens.copy_(new_lens)

    def capture(self):
        """The step as a CUDA graph, to replay(); the state is as before the call."""
        if self.steps_left < 1:
            raise ValueError("no room for a step in the block table or the rotation table")
        keep = [x.clone() for x in (self.lens, self.tokens)]
        self._step()                                              # per-device set-up
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            self._step()
        for x, was in zip((self.lens, self.tokens), keep):
            x.copy_(was)
        return Captured(self, graph)


class Captured:
    """A captured step: replay() is step() without the host's work."""

    def __init__(self, run, graph):
        self.run, self.graph = run, graph

    def replay(self):
        self.run._take()
        self.graph.replay()


def block_tables(num_seqs, blocks_per_seq, seed=0, device="cuda"):
    """A shuffled pool: every sequence its own blocks."""
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(num_seqs * blocks_per_seq, generator=g).view(num_seqs, -1).int().to(device)


def sizes(prompt_lens, steps, depth, block_size=16):
    """(pages of a sequence, positions) for `steps` steps of these prompts."""
    rows = rows_needed(max(prompt_lens), steps, depth)
    pages = (rows + block_size - 1) // block_size
    return pages, pages * block_size


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--kv", choices=sorted(KV), default="bf16")
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--seqs", type=int, default=8)
    args = ap.parse_args(argv)
    if args.steps < 1 or args.seqs < 1:
        ap.error("--steps and --seqs are 1 at least")
    depth = 4
    prompt_lens = [20 + 7 * b for b in range(args.seqs)]
    pages, positions = sizes(prompt_lens, args.steps, depth)
    if args.seqs * pages * 16 > 2 ** 31 - 1:
        ap.error("more rows than a cache numbers")
    tables = block_tables(args.seqs, pages)
    model = Model(tables.numel(), kv_dtype=KV[args.kv], max_position=positions)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, model.vocab, (n,), generator=g) for n in prompt_lens]
    run = DraftAndVerify(model, prompts, tables, depth)
    graph = run.capture()
    total = 0
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(args.steps):
        graph.replay()
        total += run.num_emitted.sum()
    end.record()
    torch.cuda.synchronize()
    if pd.pd_device_status(reset=True):
        raise SystemExit("a kernel flagged its inputs")
    print(f"{int(total)} tokens in {args.steps} steps of {args.seqs} sequences: "
          f"{int(total) / args.steps / args.seqs:.2f} a step and sequence, "
          f"{start.elapsed_time(end) / args.steps * 1e3:.0f} us a step")


if __name__ == "__main__":
    main()
