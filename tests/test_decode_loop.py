"""The decode loop without the operators around its cache: a step does nothing for them."""
import pytest
import torch

from test_decode_step import cuda_lib  # noqa: F401 (fixture)
from ternary_weight_gb300 import generate, workloads


@pytest.mark.gpu
def test_plain_steps_count_no_positions(cuda_lib):  # noqa: F811
    x = torch.from_numpy(workloads.activations_f32(70, 256, seed=3)).cuda()
    d = generate.Decoder(1, 256, 4, 2, 64, [60, 10], 80, seed=4)
    d.prompt(x)
    d.step()
    assert d.positions is None and d.kv_len.tolist() == [61, 11]
