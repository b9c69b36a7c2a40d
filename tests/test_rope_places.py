"""Where the operands of rotary positions may lie."""
import ctypes
import random

import pytest
import torch

from test_rope import check, cuda_lib, frequencies, lib  # noqa: F401 (fixtures)
from ternary_weight_gb300 import binding

AT = 1 << 20


def call(lib, rows, q, qs, q_out, qos, k, ks, k_out, kos, q_heads=4, kv_heads=2):  # noqa: F811
    """bf16 heads of 128 (256 bytes). Calls whose places are allowed are refused for their table's alignment instead."""
    t = binding._RopeDesc(AT + 4, 64, 0, 1.0)
    return lib.bitnet_rope(ctypes.byref(t), AT, rows, q, q_heads, qs, q_out, qos, k, kv_heads, ks, k_out, kos, 128, 1, None)


@pytest.mark.parametrize("rows,places,want", [
    # apart; in place; slices of fused rows (512, 256 and more numbers), in place and out of the same
    (3, (AT, 512, 2 * AT, 512, 3 * AT, 256, 4 * AT, 256), -2), (3, (AT, 512, AT, 512, 2 * AT, 256, 2 * AT, 256), -2),
    (9, (AT, 1024, AT, 1024, AT + 1024, 1024, AT + 1024, 1024), -2), (9, (AT, 1536, AT + 1536, 1536, AT + 1024, 1536, AT + 2560, 1536), -2),
    # one behind the other, of unlike strides
    (5, (AT, 512, 2 * AT, 512, AT + 5120, 256, 2 * AT + 5120, 256), -2),
    # moved by 16 bytes, by a row; a row before
    (3, (AT, 512, AT + 16, 512, 3 * AT, 256, 4 * AT, 256), -1), (3, (AT, 512, AT + 1024, 512, 3 * AT, 256, 4 * AT, 256), -1),
    (3, (AT, 512, AT - 1024, 512, 3 * AT, 256, 4 * AT, 256), -1), (5, (AT, 512, AT - 5120, 512, 3 * AT, 256, 4 * AT, 256), -2),
    (5, (AT, 512, AT + 5120, 512, 3 * AT, 256, 4 * AT, 256), -2),
    # over the other operand, or its output
    (3, (AT, 512, 2 * AT, 512, 3 * AT, 256, AT, 256), -1), (3, (AT, 512, 3 * AT, 512, 3 * AT, 256, 4 * AT, 256), -1),
    (3, (AT, 512, 2 * AT, 512, 3 * AT, 256, 2 * AT, 256), -1), (3, (AT, 512, 2 * AT, 512, 3 * AT, 256, 2 * AT + 3056, 256), -1),
    # one row: strides say nothing
    (1, (AT, 512, AT + 1024, 512, AT + 2048, 256, AT + 2560, 256), -2), (1, (AT, 512, AT + 1008, 512, 3 * AT, 256, 4 * AT, 256), -1)])
def test_operands_that_overlap_are_refused(lib, rows, places, want):  # noqa: F811
    assert call(lib, rows, *places) == want


def test_rows_of_one_stride(lib):  # noqa: F811
    """Against every pair of rows, for small ones."""
    rng = random.Random(3)
    seen = set()
    for _ in range(3000):
        rows, qh, kh = rng.randint(1, 6), rng.randint(1, 3), rng.randint(1, 3)
        stride = 128 * (max(qh, kh) + rng.randint(0, 6))
        k_out = 8 * AT + 256 * rng.randint(-60, 60)
        rows_of = lambda at, heads: [(at + r * stride * 2, at + r * stride * 2 + heads * 256) for r in range(rows)]  # noqa: E731
        meet = any(a < d and c < b for a, b in rows_of(8 * AT, qh) for c, d in rows_of(k_out, kh))
        seen.add(meet)
        # q's output at 8 AT, k's near it; the inputs are apart
        assert call(lib, rows, AT, stride, 8 * AT, stride, 3 * AT, stride, k_out, stride, qh, kh) == (-1 if meet else -2)
    assert seen == {True, False}


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 5])
def test_slices_of_fused_rows(cuda_lib, rows):  # noqa: F811
    """Queries, keys and values side by side: in place, and into another fused row."""
    table, (f, m) = binding.Rope(64, 1e4), frequencies(64, 1e4)
    x = torch.randn(rows, 8 * 64, generator=torch.Generator().manual_seed(1)).cuda()
    y = torch.full((rows, 8 * 64), 7.0, device="cuda")
    part = lambda t, a, b: t[:, a * 64:b * 64].unflatten(1, (b - a, 64))  # noqa: E731
    positions = torch.arange(rows, dtype=torch.int32, device="cuda") + 100
    binding.rope(table, positions, part(x, 0, 4), part(x, 4, 6), q_out=part(y, 0, 4), k_out=part(y, 4, 6))
    check(part(y, 0, 4), part(x, 0, 4), positions, f, m, "half")
    check(part(y, 4, 6), part(x, 4, 6), positions, f, m, "half")
    q, k = part(x, 0, 4), part(x, 4, 6)
    binding.rope(table, positions, q, k, q_out=q, k_out=k)
    assert torch.equal(x[:, :384], y[:, :384]) and bool((y[:, 384:] == 7).all())
    if rows > 1:
        with pytest.raises(binding.BitnetError):
            binding.rope(table, positions[1:], x[1:, :256].unflatten(1, (4, 64)), q_out=x[:-1, :256].unflatten(1, (4, 64)))
