"""The decode loop without the operators around its cache: a step does nothing for them."""
import pytest
import torch

from test_decode_step import cuda_lib  # noqa: F401 (fixture)
from ternary_weight_gb300 import binding, generate, workloads


@pytest.mark.gpu
def test_plain_steps_count_no_positions(cuda_lib):  # noqa: F811
    x = torch.from_numpy(workloads.activations_f32(70, 256, seed=3)).cuda()
    d = generate.Decoder(1, 256, 4, 2, 64, [60, 10], 80, seed=4)
    d.prompt(x)
    d.step()
    assert d.positions is None and d.kv_len.tolist() == [61, 11]


@pytest.mark.gpu
@pytest.mark.parametrize("budget", [0, 2000])
def test_the_first_step_holds_no_second_cache(cuda_lib, budget):  # noqa: F811
    """Also where steps gather weight and cut: a step holds its calls' workspaces (16, 2.4 and 1 MB at most) and rows of 32 tokens (128 KB
    each at most, a dozen), not another 80 MB."""
    prompts = [2000 + i for i in range(32)]
    x = torch.zeros(sum(prompts), 256, device="cuda")
    d = generate.Decoder(2, 256, 8, 4, 128, prompts, 4000, seed=4, budget=budget)
    d.prompt(x)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    caches = sum(b.cache.pages.numel() for b in d.blocks)
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    d.step()
    cache = d.blocks[0].cache
    need = binding.kv4_attention_workspace_size(cache, d.one, 8) + binding.kv4_attention_mass_workspace_size(cache, d.one, 8, d.VOTERS)
    need += binding.kv4_evict_workspace_size(cache, d.one, 2000) + 12 * 131072
    assert torch.cuda.max_memory_allocated() - before <= need < caches / 2
    assert d.kv_len.tolist() == [n + 1 for n in prompts]
    d.step()
    assert d.kv_len.tolist() == [n + 2 for n in prompts]
