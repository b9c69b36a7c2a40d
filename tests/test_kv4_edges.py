"""Edges of the 4-bit cache and its attention, against plain 64-bit numpy (tests/kv4_reference.py)."""
import pytest
import torch

from test_kv4 import World, attend
from ternary_weight_gb300 import _build, binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.fail("gpu tests need a CUDA device")
    _build.build()
    binding.lib()
    yield
    assert binding.last_device_error() == 0, "a kernel recorded a device-side error"


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,kv", [(256, 1), (256, 30), (512, 30), (290, 64), (256, 130)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_rows_far_before_the_first_position_are_zero(dim, new, kv, window, sinks):
    """Queries hundreds of places before position 0, in a tile with rows that see something. The cache has an
    odd number of pages, so a step has a page that does not exist, and its unused places hold NaN."""
    w = World([new], [kv], 2, dim, seed=new + kv).fill()
    q, out = attend(w, 1, window=window, sinks=sinks)
    assert not out[:new - kv].any()
