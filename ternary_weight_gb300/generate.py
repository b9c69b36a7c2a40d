"""Prompts and a decode loop through the attention blocks of a few layers: python -m ternary_weight_gb300.generate

A batch of sequences of unlike lengths is written and attended in one call per layer; then every
sequence grows by a token a step, the step being one CUDA graph captured once: its calls read the
lengths on the device, where the loop counts them up. Weights and inputs are random (the shapes are
those of the 2B-4T layer), each layer's output is the next one's input, and a step's output is the
next step's. With --rope queries and keys are turned by their positions; with --budget the cached tokens gather
attention weight, and a cache that has grown past the budget by an eighth is cut back to it, within the captured
step; with --vocab a 4-bit head gives logits and the greatest one's token. Prints what the cache holds and the
time of both parts.
"""
from __future__ import annotations

import argparse

import torch

from . import binding, workloads
from .stack import AttentionBlock, PackedLinear, W4Linear


def make_block(cache, hidden, q_heads, seed, window=0, sinks=0, **kw):
    """An attention block with random ternary projections. kw: as ``AttentionBlock``."""
    dim = cache.head_dim
    shapes = {"q": (q_heads * dim, hidden), "k": (cache.kv_heads * dim, hidden), "v": (cache.kv_heads * dim, hidden),
              "o": (hidden, q_heads * dim)}
    made = {}
    for i, (name, (n, k)) in enumerate(shapes.items()):
        w = torch.from_numpy(workloads.ternary_weights(n, k, seed + i)).to(cache.device)
        made[name] = PackedLinear.from_ternary(name, w, workloads.weight_scale(n, k, seed + i))
    return AttentionBlock(made["q"], made["k"], made["v"], made["o"], cache, window=window, sinks=sinks, **kw)


def page_table(lengths, device):
    """A table that deals the pages of sequences of up to `lengths` tokens out in order, and their number."""
    need = [-(-n // binding.KV4_PAGE) for n in lengths]
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    return table.to(device), at


class Decoder:
    """Layers of attention blocks over one batch of sequences that may grow to `longest` tokens each.

    ``rope`` (``binding.Rope``): rotary positions. ``budget``: a sequence that has more than budget + budget / 8 tokens
    cached is cut back to budget, by the attention weight that its tokens gathered (the last 64 of a prompt vote); its last
    budget / 4 tokens and first 4 stay, and pages are held for that many tokens only (or the prompt's, if it is longer).
    ``vocab``: a 4-bit head of that many rows; `logits` and `tokens` hold what the last step gave."""

    VOTERS = 64

    def __init__(self, layers, hidden, q_heads, kv_heads, dim, prompts, longest, window=0, sinks=0, seed=0, device="cuda",
                 rope=None, budget=0, vocab=0):
        if not prompts or min(prompts) < 1 or max(prompts) > longest:
            raise ValueError("prompts must have from one to `longest` tokens")
        if budget < 0 or vocab < 0:
            raise ValueError("budget and vocab must not be negative")
        self.prompts, self.longest, self.left = list(prompts), longest, longest - max(prompts)
        self.rope, self.budget, self.limit = rope, budget, budget + budget // 8
        # tokens that are ever cached: a step appends one before it cuts
        self.most = min(longest, max(max(prompts), self.limit + 1)) if budget else longest
        self.table, pages = page_table([self.most] * len(self.prompts), device)
        self.blocks = []
        for i in range(layers):
            cache = binding.KV4Cache(pages, kv_heads, dim, device=device)
            mass = binding.kv4_mass(cache) if budget else None
            self.blocks.append(make_block(cache, hidden, q_heads, seed + 10 * i, window, sinks, rope=rope, mass=mass, voters=self.VOTERS))
        self.kv_len = torch.tensor(self.prompts, dtype=torch.int32, device=device)
        n = len(self.prompts)
        # of each sequence's last token, where a step needs them or its cache forgets them
        self.positions = self.kv_len - 1 if rope is not None or budget else None
        self.head = self.logits = self.tokens = None
        if vocab:
            w = torch.randn(vocab, hidden, generator=torch.Generator().manual_seed(seed)) * hidden ** -0.5
            self.head = W4Linear.from_weights("head", w.to(device))
            self.logits = torch.zeros((n, vocab), dtype=torch.float32, device=device)
            self.tokens = torch.zeros(n, dtype=torch.int64, device=device)
        # an int32 tensor for each batch: the calls read them when they run
        self.one = binding.KV4Batch(torch.arange(n + 1, dtype=torch.int32, device=device), self.kv_len, self.table, n, 1,
                                    self.most)
        self.x = torch.zeros((n, hidden), dtype=torch.float32, device=device)
        self.graph = None

    def _layers(self, x, batch, positions):
        for block in self.blocks:
            x = block.run(x, batch, positions=positions)
        if self.budget:  # the layers share their lengths: the last one writes the new ones
            for block in self.blocks:
                block.evict(batch, self.budget, self.limit, sinks=min(4, self.budget - self.budget // 4), recent=self.budget // 4,
                            new_len=self.kv_len if block is self.blocks[-1] else None)
        return x

    def _answer(self):
        if self.head is not None:
            self.head.run(self.x, out=self.logits)
            torch.argmax(self.logits, -1, out=self.tokens)

    def prompt(self, x):
        """x: the prompts' rows, packed. Returns each row's output; the last ones become the next step's input."""
        ends = torch.tensor([0] + self.prompts).cumsum(0)
        batch = binding.KV4Batch(ends.to(torch.int32).to(x.device), self.kv_len, self.table, int(ends[-1]),
                                 max(self.prompts), self.most)
        positions = None
        if self.rope is not None:
            positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in self.prompts]).to(x.device)
        y = self._layers(x, batch, positions)
        self.x.copy_(y[(ends[1:] - 1).to(x.device)])
        self._answer()
        return y

    def _step(self):
        self.kv_len += 1
        if self.positions is not None:
            self.positions += 1
        self.x.copy_(self._layers(self.x, self.one, self.positions if self.rope is not None else None))
        self._answer()

    def step(self):
        """One token more for every sequence: one graph launch from the second step on. Returns the tokens' outputs (overwritten by the next)."""
        if self.left == 0:
            raise ValueError("the longest sequence is full")
        self.left -= 1
        if self.graph is not None:
            self.graph.replay()
            return self.x
        # everything has to have run once before a capture: the first step is run as it is, the others are replayed
        s = torch.cuda.Stream(device=self.x.device)
        s.wait_stream(torch.cuda.current_stream(self.x.device))
        with torch.cuda.stream(s):
            self._step()
        torch.cuda.current_stream(self.x.device).wait_stream(s)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self._step()
        return self.x


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--batch", type=int, default=8, help="sequences; their prompts have from a half to all of --prompt tokens")
    p.add_argument("--prompt", type=int, default=2000)
    p.add_argument("--steps", type=int, default=64, help="tokens to decode")
    p.add_argument("--window", type=int, default=0)
    p.add_argument("--sinks", type=int, default=0)
    p.add_argument("--rope", choices=sorted(binding.ROPE_SCALINGS), help="rotary positions, base 500000, scaled by 8 from 4096 tokens")
    p.add_argument("--budget", type=int, default=0, help="tokens that a sequence's cache is cut back to")
    p.add_argument("--vocab", type=int, default=0, help="rows of the 4-bit head")
    a = p.parse_args()
    if min(a.layers, a.batch, a.prompt, a.steps) < 1:
        p.error("--layers, --batch, --prompt and --steps must be positive")
    prompts = [max(1, a.prompt - b * (a.prompt // 2) // a.batch) for b in range(a.batch)]
    hidden, q_heads, kv_heads, dim = 2560, 20, 5, 128
    if a.budget < 0 or a.vocab < 0:
        p.error("--budget and --vocab must not be negative")
    rope = binding.Rope(dim, 500000.0, scaling=a.rope, factor=8.0, original=4096) if a.rope else None
    d = Decoder(a.layers, hidden, q_heads, kv_heads, dim, prompts, a.prompt + a.steps, a.window, a.sinks, rope=rope, budget=a.budget,
                vocab=a.vocab)
    x = torch.from_numpy(workloads.activations_f32(sum(prompts), hidden, seed=1)).cuda()
    times, begun = [], min(2, a.steps)  # the first step is captured, the second brings the graph to the device
    for part in (lambda: d.prompt(x), lambda: [d.step() for _ in range(begun)], lambda: [d.step() for _ in range(a.steps - begun)]):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        part()
        end.record()
        torch.cuda.synchronize()
        times.append(begin.elapsed_time(end))
    if binding.last_device_error():
        raise SystemExit("a kernel reported a batch that breaks its bounds")
    held = sum(b.cache.pages.numel() for b in d.blocks)
    print("prompts: %d tokens x %d layers, first call %.2f ms" % (sum(prompts), a.layers, times[0]))
    print("decode: %d sequences x %d layers, %.1f us a step (captured in the first %d, %.2f ms)" % (
        a.batch, a.layers, times[2] * 1e3 / max(1, a.steps - begun), begun, times[1]))
    if a.budget:
        print("kept: %s tokens a sequence of %s" % (sorted(set(d.kv_len.tolist())), sorted(set((d.positions + 1).tolist()))))
    if a.vocab:
        print("tokens: %s" % d.tokens.tolist())
    print("cache: %.1f MB at 4 bits, %.1f MB as bf16" % (held / 1e6, held / 1e6 * 4 * dim / (dim + 8)))


if __name__ == "__main__":
    main()
