"""Prompts and a decode loop through the attention blocks of a few layers: python -m ternary_weight_gb300.generate

A batch of sequences of unlike lengths is written and attended in one call per layer; then every
sequence grows by a token a step, the step being one CUDA graph captured once: its calls read the
lengths on the device, where the loop counts them up. Weights and inputs are random (the shapes are
those of the 2B-4T layer), each layer's output is the next one's input, and a step's output is the
next step's. Prints what the cache holds and the time of both parts.
"""
from __future__ import annotations

import argparse

import torch

from . import binding, workloads
from .stack import AttentionBlock, PackedLinear


def make_block(cache, hidden, q_heads, seed, window=0, sinks=0):
    """An attention block with random ternary projections."""
    dim = cache.head_dim
    shapes = {"q": (q_heads * dim, hidden), "k": (cache.kv_heads * dim, hidden), "v": (cache.kv_heads * dim, hidden),
              "o": (hidden, q_heads * dim)}
    made = {}
    for i, (name, (n, k)) in enumerate(shapes.items()):
        w = torch.from_numpy(workloads.ternary_weights(n, k, seed + i)).to(cache.device)
        made[name] = PackedLinear.from_ternary(name, w, workloads.weight_scale(n, k, seed + i))
    return AttentionBlock(made["q"], made["k"], made["v"], made["o"], cache, window=window, sinks=sinks)


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
    """Layers of attention blocks over one batch of sequences that may grow to `longest` tokens each."""

    def __init__(self, layers, hidden, q_heads, kv_heads, dim, prompts, longest, window=0, sinks=0, seed=0, device="cuda"):
        if not prompts or min(prompts) < 1 or max(prompts) > longest:
            raise ValueError("prompts must have from one to `longest` tokens")
        self.prompts, self.longest, self.left = list(prompts), longest, longest - max(prompts)
        self.table, pages = page_table([longest] * len(self.prompts), device)
        self.blocks = [make_block(binding.KV4Cache(pages, kv_heads, dim, device=device), hidden, q_heads, seed + 10 * i,
                                  window, sinks) for i in range(layers)]
        self.kv_len = torch.tensor(self.prompts, dtype=torch.int32, device=device)
        n = len(self.prompts)
        # an int32 tensor for each batch: the calls read them when they run
        self.one = binding.KV4Batch(torch.arange(n + 1, dtype=torch.int32, device=device), self.kv_len, self.table, n, 1,
                                    longest)
        self.x = torch.zeros((n, hidden), dtype=torch.float32, device=device)
        self.graph = None

    def _layers(self, x, batch):
        for block in self.blocks:
            x = block.run(x, batch)
        return x

    def prompt(self, x):
        """x: the prompts' rows, packed. Returns each row's output; the last ones become the next step's input."""
        ends = torch.tensor([0] + self.prompts).cumsum(0)
        batch = binding.KV4Batch(ends.to(torch.int32).to(x.device), self.kv_len, self.table, int(ends[-1]),
                                 max(self.prompts), self.longest)
        y = self._layers(x, batch)
        self.x.copy_(y[(ends[1:] - 1).to(x.device)])
        return y

    def _step(self):
        self.kv_len += 1
        self.x.copy_(self._layers(self.x, self.one))

    def step(self):
        """One token more for every sequence: one graph launch. Returns the tokens' outputs (overwritten by the next)."""
        if self.left == 0:
            raise ValueError("the longest sequence is full")
        self.left -= 1
        if self.graph is None:
            # everything has to have run once before a capture: a step whose effects are taken back (the
            # places that it writes are written again by the step after it)
            keep = self.kv_len.clone(), self.x.clone()
            s = torch.cuda.Stream(device=self.x.device)
            s.wait_stream(torch.cuda.current_stream(self.x.device))
            with torch.cuda.stream(s):
                self._step()
            torch.cuda.current_stream(self.x.device).wait_stream(s)
            self.kv_len.copy_(keep[0]), self.x.copy_(keep[1])
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self._step()
        self.graph.replay()
        return self.x


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--batch", type=int, default=8, help="sequences; their prompts have from a half to all of --prompt tokens")
    p.add_argument("--prompt", type=int, default=2000)
    p.add_argument("--steps", type=int, default=64, help="tokens to decode")
    p.add_argument("--window", type=int, default=0)
    p.add_argument("--sinks", type=int, default=0)
    a = p.parse_args()
    if min(a.layers, a.batch, a.prompt, a.steps) < 1:
        p.error("--layers, --batch, --prompt and --steps must be positive")
    prompts = [max(1, a.prompt - b * (a.prompt // 2) // a.batch) for b in range(a.batch)]
    hidden, q_heads, kv_heads, dim = 2560, 20, 5, 128
    d = Decoder(a.layers, hidden, q_heads, kv_heads, dim, prompts, a.prompt + a.steps, a.window, a.sinks)
    x = torch.from_numpy(workloads.activations_f32(sum(prompts), hidden, seed=1)).cuda()
    times = []
    for part in (lambda: d.prompt(x), d.step, lambda: [d.step() for _ in range(a.steps - 1)]):
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
    print("decode: %d sequences x %d layers, %.1f us a step (captured in the first, %.2f ms)" % (
        a.batch, a.layers, times[2] * 1e3 / max(1, a.steps - 1), times[1]))
    print("cache: %.1f MB at 4 bits, %.1f MB as bf16" % (held / 1e6, held / 1e6 * 4 * dim / (dim + 8)))


if __name__ == "__main__":
    main()
