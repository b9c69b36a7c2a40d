"""The decode loop with rotary positions, eviction by gathered weight and a 4-bit head, and the attention block that
carries the first two: bit for bit what their calls give one by one."""
import subprocess
import sys
from types import SimpleNamespace

import pytest
import torch

from test_kv4 import World
from ternary_weight_gb300 import _build, binding, generate, workloads
from ternary_weight_gb300.stack import AttentionBlock, PackedLinear, W4Linear


def linear(n, k):
    return PackedLinear("p", torch.zeros((n, k // 4), dtype=torch.uint8), 0.02, n, k)


def test_blocks_that_do_not_fit_are_refused():
    cache = SimpleNamespace(head_dim=64, kv_heads=2)
    make = lambda **kw: AttentionBlock(linear(512, 256), linear(128, 256), linear(128, 256), linear(256, 512), cache, **kw)  # noqa: E731
    with pytest.raises(ValueError):
        make(rope=SimpleNamespace(dims=128))
    x, batch = torch.zeros(1, 256), SimpleNamespace(total_q=1)
    with pytest.raises(ValueError):
        make().run(x, batch, positions=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        make(rope=SimpleNamespace(dims=64)).run(x, batch)
    with pytest.raises(ValueError):
        make(rope=SimpleNamespace(dims=64)).run(x, batch, rotate=lambda q, k: None, positions=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        make().evict(batch, 10)


@pytest.mark.parametrize("kw", [dict(budget=-1), dict(vocab=-5)])
def test_bad_decoders_are_refused(kw):
    with pytest.raises(ValueError):
        generate.Decoder(1, 256, 4, 2, 64, [5], 10, device="cpu", **kw)


@pytest.fixture
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.fail("gpu tests need a CUDA device")
    _build.build()
    binding.lib()
    yield
    assert binding.last_device_error() == 0, "a kernel recorded a device-side error"


@pytest.mark.gpu
@pytest.mark.parametrize("dim,layout,window", [(64, "half", 0), (128, "interleaved", 40)])
@pytest.mark.parametrize("new,before", [([1, 1, 1], [0, 63, 64]), ([5, 130, 1], [0, 100, 9])])
def test_a_block_is_its_calls(cuda_lib, dim, layout, window, new, before):
    kv = [n + c for n, c in zip(new, before)]
    w = World(new, kv, 2, dim, "f32", seed=dim + sum(new)).fill()
    other = binding.KV4Cache(w.n_pages, 2, dim, pages=w.cache.pages.clone())
    table = binding.Rope(dim, 1e4, layout)
    mass = binding.kv4_mass(w.cache)
    apart = mass.clone()
    block = generate.make_block(w.cache, 384, 8, seed=5, window=window, sinks=2, rope=table, mass=mass, voters=3, decay=0.5)
    x = torch.from_numpy(workloads.activations_f32(sum(new), 384, seed=7)).cuda()
    positions = torch.cat([torch.arange(1000 + c, 1000 + c + n) for n, c in zip(new, before)]).to(torch.int32).cuda()
    batch = w.batch(new, kv)
    got = block.run(x, batch, positions=positions)

    q, k, v = (binding.linear(x, l.wp, l.w_scale).view(sum(new), -1, dim) for l in block.qkv)
    q, k = binding.rope(table, positions, q, k)
    binding.kv4_append(other, batch, k, v)
    binding.kv4_attention_mass(other, batch, q, dim ** -0.5, apart, decay=0.5, window=window, sinks=2, voters=3)
    y = binding.kv4_attention(other, batch, q, dim ** -0.5, window=window, sinks=2)
    assert torch.equal(got, binding.linear(y.view(sum(new), -1), block.o.wp, block.o.w_scale))
    assert torch.equal(w.cache.pages, other.pages) and torch.equal(mass, apart) and bool(mass.any())
    n = block.evict(batch, 50, 60, sinks=1, recent=5)
    assert torch.equal(n, binding.kv4_evict(other, batch, apart, 50, limit=60, sinks=1, recent=5))
    assert n.tolist() == [50 if m > 60 else m for m in kv]
    assert torch.equal(w.cache.pages, other.pages) and torch.equal(mass, apart)


@pytest.mark.gpu
@pytest.mark.parametrize("prompts,budget,steps", [([60, 7, 200], 0, 5), ([60, 7, 200], 64, 12), ([30], 24, 9)])
def test_captured_steps_are_the_eager_ones(cuda_lib, prompts, budget, steps):
    runs = []
    x = torch.from_numpy(workloads.activations_f32(sum(prompts), 256, seed=3)).cuda()
    for captured in (True, False):
        d = generate.Decoder(2, 256, 4, 2, 64, prompts, max(prompts) + steps, seed=40, budget=budget, vocab=300,
                             rope=binding.Rope(64, 1e4, scaling="by_parts", factor=4.0, original=64))
        runs.append([d.prompt(x).clone()])
        for _ in range(steps):
            if captured:
                d.step()
            else:
                d._step()
            runs[-1] += [d.x.clone(), d.logits.clone(), d.tokens.clone(), d.kv_len.clone()]
        assert (d.positions + 1).tolist() == [n + steps for n in prompts]
        limit = budget + budget // 8
        assert all(n <= limit for n in d.kv_len.tolist()) if budget else d.kv_len.tolist() == [n + steps for n in prompts]
        assert torch.equal(d.logits, d.head.run(d.x)) and torch.equal(d.tokens, d.logits.argmax(-1))
    assert all(torch.equal(a, b) and bool(a.isfinite().all()) for a, b in zip(*runs))


@pytest.mark.gpu
@pytest.mark.parametrize("budget", [1, 2, 3, 4, 5, 7, 8])
def test_small_budgets(cuda_lib, budget):
    d = generate.Decoder(1, 256, 4, 2, 64, [9, 1], 20, seed=4, budget=budget)
    d.prompt(torch.from_numpy(workloads.activations_f32(10, 256, seed=3)).cuda())
    for _ in range(11):
        assert bool(d.step().isfinite().all()) and all(n <= budget + budget // 8 for n in d.kv_len.tolist())


@pytest.mark.gpu
def test_without_eviction_the_weight_changes_nothing(cuda_lib):
    """A budget that is never reached: the same steps as without."""
    x = torch.from_numpy(workloads.activations_f32(70, 256, seed=3)).cuda()
    outs = []
    for budget in (0, 1000):
        d = generate.Decoder(1, 256, 4, 2, 64, [70], 80, seed=4, budget=budget)
        d.prompt(x)
        outs.append([d.step().clone() for _ in range(4)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.gpu
def test_a_head_is_its_calls(cuda_lib):
    w = torch.randn(130, 256, generator=torch.Generator().manual_seed(1)).cuda()
    x = torch.randn(3, 256, generator=torch.Generator().manual_seed(2)).cuda()
    for zeros in (False, True):
        head = W4Linear.from_weights("head", w, 64, zeros)
        assert (head.N, head.K) == (130, 256) and head.weight_bytes() == 130 * (128 + 4 * 2 + (4 if zeros else 0))
        assert torch.equal(head.run(x), binding.w4_matmul(x, *binding.w4_quant_weight(w, 64, zeros)))


@pytest.mark.gpu
def test_the_command(cuda_lib):
    r = subprocess.run([sys.executable, "-m", "ternary_weight_gb300.generate", "--layers", "1", "--batch", "2", "--prompt", "90", "--steps", "8",
                        "--rope", "by_wavelength", "--budget", "80", "--vocab", "1000"], capture_output=True, text=True, timeout=300, cwd=_build.ROOT)
    assert r.returncode == 0, r.stderr
    assert "kept: " in r.stdout and "tokens: " in r.stdout and "decode: 2 sequences x 1 layers" in r.stdout
