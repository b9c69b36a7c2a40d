"""The attention block of a layer (ternary projections, 4-bit cache, attention) and the decode loop.

The block has to give, bit for bit, what its calls give one by one (projections through the unfused
calls, which are held to the oracle elsewhere); the attention between them is held to the bound that
test_kv4.py works out, at the queries, keys and values that the projections gave.
"""
import subprocess
import sys
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from test_kv4 import World
from ternary_weight_gb300 import _build, binding, generate, workloads
from ternary_weight_gb300.stack import AttentionBlock, PackedLinear


def linear(n, k):
    return PackedLinear("p", torch.zeros((n, k // 4), dtype=torch.uint8), 0.02, n, k)


@pytest.mark.parametrize("q,k,v,o", [((500, 256), (128, 256), (128, 256), (256, 500)),  # not whole heads
                                     ((512, 256), (64, 256), (64, 256), (256, 512)),    # not the cache's heads
                                     ((512, 256), (128, 256), (64, 256), (256, 512)),   # values unlike keys
                                     ((320, 256), (128, 256), (128, 256), (256, 320)),  # 5 query heads on 2
                                     ((512, 256), (128, 512), (128, 256), (256, 512)),  # inputs of unlike widths
                                     ((512, 256), (128, 256), (128, 256), (256, 256))])  # o reads something else
def test_projections_that_do_not_fit_are_refused(q, k, v, o):
    cache = SimpleNamespace(head_dim=64, kv_heads=2)
    AttentionBlock(linear(512, 256), linear(128, 256), linear(128, 256), linear(256, 512), cache)
    with pytest.raises(ValueError):
        AttentionBlock(linear(*q), linear(*k), linear(*v), linear(*o), cache)


def test_page_table_deals_every_page_once():
    table, n = generate.page_table([1, 64, 65, 300], "cpu")
    assert n == 1 + 1 + 2 + 5 and table.shape == (4, 5) and table.dtype == torch.int32
    assert sorted(table[table >= 0].tolist()) == list(range(n))
    assert [(row >= 0).sum().item() for row in table] == [1, 1, 2, 5]


@pytest.mark.parametrize("prompts,longest", [([], 10), ([0], 10), ([5, 11], 10)])
def test_prompts_that_do_not_fit_are_refused(prompts, longest):
    with pytest.raises(ValueError):
        generate.Decoder(1, 256, 4, 2, 64, prompts, longest, device="cpu")


@pytest.fixture
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.fail("gpu tests need a CUDA device")
    _build.build()
    binding.lib()
    yield
    assert binding.last_device_error() == 0, "a kernel recorded a device-side error"


def rotate(q, k):
    """Stands for a rotary embedding: changes queries and keys in place, unlike each other."""
    q.mul_(1.5)
    k.copy_(k.flip(-1))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim,window,sinks", [(64, 0, 0), (128, 40, 3)])
@pytest.mark.parametrize("new,before", [([1], [70]), ([1, 1, 1], [0, 63, 64]), ([5, 130, 1], [0, 100, 9])])
def test_a_block_is_its_calls(cuda_lib, dtype, dim, window, sinks, new, before):
    kv = [n + c for n, c in zip(new, before)]
    w = World(new, kv, 2, dim, "f32", seed=dim + sum(new)).fill()
    other = binding.KV4Cache(w.n_pages, 2, dim, pages=w.cache.pages.clone())
    block = generate.make_block(w.cache, 384, 8, seed=5, window=window, sinks=sinks)
    x = torch.from_numpy(workloads.activations_f32(sum(new), 384, seed=7)).to(dtype).cuda()
    batch = w.batch(new, kv)
    got = block.run(x, batch, rotate=rotate)

    q, k, v = (binding.linear(x, l.wp, l.w_scale).view(sum(new), -1, dim) for l in block.qkv)
    rotate(q, k)
    binding.kv4_append(other, batch, k, v)
    y = binding.kv4_attention(other, batch, q, dim ** -0.5, window=window, sinks=sinks)
    want = binding.linear(y.view(sum(new), -1), block.o.wp, block.o.w_scale)
    assert got.shape == (sum(new), 384) and torch.equal(got, want)
    assert torch.equal(w.cache.pages, other.pages)
    row = 0
    for b, n in enumerate(new):
        w.k[b][before[b]:], w.v[b][before[b]:] = k[row:row + n].cpu().numpy(), v[row:row + n].cpu().numpy()
        row += n
    w.check_attention(q, y, 4, dim ** -0.5, window, sinks)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = block.run(x, batch, rotate=rotate, stream=s)
    s.synchronize()
    assert torch.equal(again, want)


@pytest.mark.gpu
def test_no_tokens(cuda_lib):
    w = World([0], [5], 2, 64).fill()
    block = generate.make_block(w.cache, 256, 4, seed=1)
    assert block.run(torch.empty(0, 256, device="cuda"), w.batch([0], [5])).shape == (0, 256)
    with pytest.raises(ValueError):
        block.run(torch.zeros(1, 256, device="cuda"), w.batch([0], [5]))


@pytest.mark.gpu
@pytest.mark.parametrize("prompts,window", [([1], 0), ([60, 7, 200], 0), ([64, 130], 50)])
def test_captured_steps_are_the_eager_ones(cuda_lib, prompts, window):
    steps, runs = 6, []
    x = torch.from_numpy(workloads.activations_f32(sum(prompts), 256, seed=3)).cuda()
    for captured in (True, False):
        d = generate.Decoder(2, 256, 4, 2, 64, prompts, max(prompts) + steps, window, 2 if window else 0, seed=40)
        runs.append([d.prompt(x).clone()])
        for _ in range(steps):
            if captured:
                d.step()
            else:
                d._step()
            runs[-1].append(d.x.clone())
        assert d.kv_len.tolist() == [n + steps for n in prompts]
        if captured:
            with pytest.raises(ValueError):
                d.step()
    assert all(torch.equal(a, b) and bool(a.isfinite().all()) for a, b in zip(*runs))
    assert not torch.equal(runs[0][1], runs[0][2])


@pytest.mark.gpu
def test_the_command(cuda_lib):
    r = subprocess.run([sys.executable, "-m", "ternary_weight_gb300.generate", "--layers", "1", "--batch", "2", "--prompt", "90",
                        "--steps", "3"], capture_output=True, text=True, timeout=300, cwd=_build.ROOT)
    assert r.returncode == 0, r.stderr
    assert "decode: 2 sequences x 1 layers" in r.stdout
