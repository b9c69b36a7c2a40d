"""Rotary positions against the formula in 64 bits.

The bound, for a pair (a, b): the angle is off by pi (2^-25 + 2^-32) from its rounding to fp32 half turns and
by 2^-52 of itself from the table, sine and cosine by 2^-23 each (two units in the last place, twice what CUDA states), the
magnitude's product by 2^-24 of each, the turn by 2^-24 of a product and 2^-24 of the result: in all less
than 2^-21 (|a| + |b|) magnitude; then the output's rounding, half a step of its type.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from ternary_weight_gb300 import _build, binding

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.lib()


def frequencies(dims, base, scaling="none", factor=1.0, original=0.0, low=1.0, high=32.0):
    i = np.arange(dims // 2)
    if scaling == "ntk":
        base = base * factor ** (dims / (dims - 2))
    f = base ** (-2.0 * i / dims)
    if scaling == "linear":
        f = f / factor
    if scaling == "by_parts":
        d = [dims / 2 * math.log(original / (2 * math.pi * n)) / math.log(base) for n in (high, low)]
        a, b = max(math.floor(d[0]), 0), min(math.ceil(d[1]), dims - 1)
        r = np.clip((i - a) / max(b - a, 0.001), 0, 1)
        return f * (1 - r) + f / factor * r, 0.1 * math.log(factor) + 1
    if scaling == "by_wavelength":
        t = np.clip((original * f / (2 * math.pi) - low) / (high - low), 0, 1)
        f = f * (t + (1 - t) / factor)
    return f, 1.0


SCALED = [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=2.5)),
          ("by_parts", dict(factor=16.0, original=4096)), ("by_parts", dict(factor=2.0, original=100, low=0.5, high=8.0)),
          ("by_wavelength", dict(factor=8.0, original=8192))]


@pytest.mark.parametrize("dims,base", [(2, 1e4), (8, 1e4), (20, 5e5), (128, 5e5), (1024, 1e6)])
@pytest.mark.parametrize("scaling,kw", SCALED)
def test_turns_are_the_frequencies(lib, dims, base, scaling, kw):
    if scaling == "ntk" and dims == 2:
        with pytest.raises(binding.BitnetError):
            binding.rope_turns(dims, base, scaling, **kw)
        return
    turns, magnitude = binding.rope_turns(dims, base, scaling, **kw)
    ends = dict(high=4.0) if scaling == "by_wavelength" else {}
    f, m = frequencies(dims, base, scaling, **{**ends, **kw})
    assert len(turns) == dims // 2 and all(0 <= t < 1 << 62 for t in turns)
    got = np.array(turns, dtype=np.float64) / 2.0 ** 64 * 2 * math.pi
    assert np.allclose(got, f, rtol=1e-13, atol=2.0 ** -62) and math.isclose(magnitude, m, rel_tol=1e-7)


@pytest.mark.parametrize("kw", [dict(dims=0), dict(dims=7), dict(dims=1026), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
                                dict(scaling=5), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=1, factor=float("nan")),
                                dict(scaling=3, factor=2.0, original=0.0), dict(scaling=3, factor=2.0, low=2.0, high=2.0),
                                dict(scaling=4, factor=2.0, low=0.0), dict(scaling=4, factor=2.0, high=float("inf")),
                                dict(turns=None), dict(magnitude=None), dict(scaling=2, factor=1e308)])
def test_bad_frequencies_are_refused(lib, kw):
    out, m = (ctypes.c_uint64 * 512)(), ctypes.c_float()
    a = {**dict(dims=8, base=1e4, scaling=0, factor=1.0, original=100.0, low=1.0, high=4.0, turns=ctypes.cast(out, ctypes.c_void_p),
                magnitude=ctypes.byref(m)), **kw}
    assert lib.bitnet_rope_turns(*a.values()) == -1


def call(lib, **kw):
    t = binding._RopeDesc(**{**dict(turns=FAKE, dims=64, layout=0, magnitude=1.0), **{k: v for k, v in kw.items() if k in ("turns", "dims", "layout", "magnitude")}})
    a = dict(positions=FAKE, rows=3, q=FAKE, q_heads=4, qs=512, q_out=2 * FAKE, qos=512, k=3 * FAKE, kv_heads=2, ks=256, k_out=4 * FAKE,
             kos=256, head_dim=128, dtype=1)
    a.update({k: v for k, v in kw.items() if k in a})
    return lib.bitnet_rope(None if kw.get("table", 1) is None else ctypes.byref(t), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(table=None), -1), (dict(turns=None), -1), (dict(dims=4), -1), (dict(dims=136), -1), (dict(dims=60), -1), (dict(layout=2), -1),
    (dict(magnitude=float("inf")), -1), (dict(positions=None), -1), (dict(rows=-1), -1), (dict(rows=1 << 31), -1), (dict(q=None), -1),
    (dict(q_out=None), -1), (dict(k=None), -1), (dict(k_out=None), -1), (dict(q_heads=0), -1), (dict(kv_heads=-1), -1),
    (dict(q_heads=(1 << 17) + 1, qs=1 << 25), -1), (dict(head_dim=132), -1), (dict(head_dim=1032, qs=1 << 20, ks=1 << 20), -1),
    (dict(head_dim=0), -1), (dict(dtype=2), -1), (dict(qs=511), -1), (dict(kos=255), -1), (dict(ks=(1 << 26) + 8), -1), (dict(qs=516), -2),
    (dict(q=FAKE + 8), -2), (dict(k_out=FAKE + 4), -2), (dict(positions=FAKE + 2), -2), (dict(turns=FAKE + 4), -2),
    (dict(q_out=FAKE, qos=1024), -1),  # in place, but with another stride
    (dict(rows=0), 0), (dict(rows=0, kv_heads=0, k=None, k_out=None), 0), (dict(rows=0, q_out=FAKE), 0)])
def test_bad_calls_are_refused(lib, kw, want):
    assert call(lib, **kw) == want


@pytest.mark.parametrize("kw", [dict(dims=4), dict(dims=12), dict(dims=0), dict(layout="both"), dict(scaling="more")])
def test_bad_tables_are_refused(lib, kw):
    with pytest.raises(ValueError):
        binding.Rope(**{**dict(dims=64, device="cpu"), **kw})


# ------------------------------------------------------------------- on the GPU
@pytest.fixture
def cuda_lib(lib):
    if not torch.cuda.is_available():
        pytest.fail("gpu tests need a CUDA device")
    yield
    assert binding.last_device_error() == 0


def turned(x, positions, f, magnitude, layout):
    """The formula, and the bound's |a| + |b|, in 64 bits."""
    dims = 2 * len(f)
    x = x.double().cpu().numpy()
    angle = positions.cpu().numpy().astype(np.float64)[:, None, None] * f
    cos, sin = np.cos(angle) * magnitude, np.sin(angle) * magnitude
    a, b = (slice(0, dims // 2), slice(dims // 2, dims)) if layout == "half" else (slice(0, dims, 2), slice(1, dims, 2))
    y, size = x.copy(), np.zeros_like(x)
    y[..., a], y[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., b] * cos + x[..., a] * sin
    size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * magnitude
    return y, size


def check(got, x, positions, f, magnitude, layout):
    y, size = turned(x, positions, f, magnitude, layout)
    got64 = got.double().cpu().numpy()
    half = torch.finfo(got.dtype).eps / 2
    bound = 2.0 ** -21 * size + (half if got.dtype != torch.float32 else 0) * (np.abs(y) + 2.0 ** -21 * size) + 1e-40
    # the table's fp64 frequency, over far positions
    bound += 2.0 ** -52 * 2 * np.abs(positions.cpu().numpy().astype(np.float64))[:, None, None] * size
    dims = 2 * len(f)
    assert np.array_equal(got64[..., dims:], y[..., dims:])
    err = np.abs(got64 - y)
    assert (err <= bound).all(), "worst %.3g of the bound" % (err / bound).max()


def rows_of(rows, heads, dim, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, heads * dim + pad, generator=g).to(dtype).cuda()
    return x[:, :heads * dim].unflatten(1, (heads, dim)) if pad else x.view(rows, heads, dim)


POSITIONS = [0, 1, 77, 131071, 2 ** 24 + 1, 2 ** 31 - 1, -1, -131071, -2 ** 31]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,dims,heads", [(8, 8, (1, 1)), (64, 64, (4, 2)), (128, 128, (20, 5)), (128, 40, (3, 3)), (80, 80, (7, 1)),
                                            (96, 24, (2, 0)), (256, 128, (9, 4)), (1024, 1024, (1, 1))])
def test_positions_far_and_near(cuda_lib, dtype, layout, dim, dims, heads):
    table = binding.Rope(dims, 1e4, layout)
    f, m = frequencies(dims, 1e4)
    positions = torch.tensor(POSITIONS, dtype=torch.int32, device="cuda")
    q = rows_of(len(POSITIONS), heads[0], dim, dtype, dim)
    k = rows_of(len(POSITIONS), heads[1], dim, dtype, dim + 1) if heads[1] else None
    got = binding.rope(table, positions, q, k)
    for x, y in zip((q, k), got if heads[1] else (got,)):
        assert y.dtype == dtype and y.shape == x.shape
        check(y, x, positions, f, m, layout)


@pytest.mark.gpu
@pytest.mark.parametrize("scaling,kw", SCALED)
def test_scaled_tables(cuda_lib, scaling, kw):
    table = binding.Rope(128, 5e5, scaling=scaling, **kw)
    f, m = frequencies(128, 5e5, scaling, **{**(dict(high=4.0) if scaling == "by_wavelength" else {}), **kw})
    positions = torch.arange(131000, 131040, dtype=torch.int32, device="cuda")
    q = rows_of(40, 4, 128, torch.float32, 3)
    check(binding.rope(table, positions, q), q, positions, f, m, "half")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 2, 33, 1000, 4099])
def test_row_counts_strides_and_places(cuda_lib, rows, dtype):
    """Rows from one to many (the heads that share angles change with them), slices of wider rows, in place, into given outputs."""
    table = binding.Rope(64, 1e4, "half")
    f, m = frequencies(64, 1e4)
    g = torch.Generator().manual_seed(rows)
    positions = torch.randint(0, 1 << 20, (rows,), generator=g, dtype=torch.int32).cuda()
    q, k = rows_of(rows, 12, 96, dtype, 1, pad=48), rows_of(rows, 3, 96, dtype, 2, pad=16)
    a, b = binding.rope(table, positions, q, k)
    check(a, q, positions, f, m, "half")
    check(b, k, positions, f, m, "half")
    qo, ko = torch.full_like(a, 7.0), torch.full((rows, 3, 96 + 32), 7.0, device="cuda", dtype=dtype)[:, :, :96]
    if rows > 1:
        with pytest.raises(ValueError):
            binding.rope(table, positions, q, k, q_out=qo, k_out=ko)  # heads apart
    wide = torch.full((rows, 3 * 96 + 64), 7.0, device="cuda", dtype=dtype)
    ko = wide[:, :288].unflatten(1, (3, 96))
    binding.rope(table, positions, q, k, q_out=qo, k_out=ko)
    assert torch.equal(qo, a) and torch.equal(ko, b) and bool((wide[:, 288:] == 7).all())
    binding.rope(table, positions, q, k, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b)


@pytest.mark.gpu
def test_turning_back_and_the_gradient(cuda_lib):
    """The gradient of sum(turned * w) is w turned by the negative positions: held to the formula's own bound, and to
    differences of the loss in 64 bits."""
    table = binding.Rope(32, 1e4, "interleaved", scaling="by_parts", factor=4.0, original=256)
    f, m = frequencies(32, 1e4, "by_parts", factor=4.0, original=256)
    positions = torch.tensor([3, 1000, 0], dtype=torch.int32, device="cuda")
    q, w = rows_of(3, 2, 48, torch.float32, 5), rows_of(3, 2, 48, torch.float32, 6)
    grad = binding.rope(table, -positions, w).double().cpu().numpy()
    loss = lambda x: (turned(x, positions, f, m, "interleaved")[0] * w.double().cpu().numpy()).sum()  # noqa: E731
    for at in ((0, 0, 0), (0, 1, 31), (1, 0, 5), (1, 1, 47), (2, 0, 16)):
        e = torch.zeros(3, 2, 48, dtype=torch.float64)
        e[at] = 0.5
        # the loss is linear: the difference is the gradient but for fp64 and the bound above
        assert abs((loss(q.double().cpu() + e) - loss(q.double().cpu() - e)) - grad[at]) < 1e-5
    check(torch.tensor(grad).float(), w, -positions.cpu(), f, m, "interleaved")


@pytest.mark.gpu
def test_infinities_and_nan_stay_in_their_pair(cuda_lib):
    table = binding.Rope(16, 1e4, "half")
    q = torch.ones(1, 2, 24, device="cuda")
    q[0, 0, 3], q[0, 1, 20] = float("nan"), float("inf")
    got = binding.rope(table, torch.tensor([5], dtype=torch.int32, device="cuda"), q)
    bad = torch.zeros(1, 2, 24, dtype=torch.bool)
    bad[0, 0, 3] = bad[0, 0, 11] = bad[0, 1, 20] = True
    assert torch.equal(~got.isfinite().cpu(), bad) and float(got[0, 1, 20]) == float("inf")


@pytest.mark.gpu
def test_captured_with_positions_that_move_on(cuda_lib):
    table = binding.Rope(64, 1e4)
    positions = torch.tensor([5, 900], dtype=torch.int32, device="cuda")
    q, k = rows_of(2, 4, 64, torch.bfloat16, 8), rows_of(2, 2, 64, torch.bfloat16, 9)
    binding.rope(table, positions, q, k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = binding.rope(table, positions, q, k)
    for _ in range(3):
        positions += 1
        graph.replay()
        c, d = binding.rope(table, positions, q, k)
        assert torch.equal(a, c) and torch.equal(b, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    e, _ = binding.rope(table, positions, q, k, stream=s)
    s.synchronize()
    assert torch.equal(e, a)


@pytest.mark.gpu
def test_refusals_of_the_binding(cuda_lib):
    table, p = binding.Rope(64), torch.zeros(2, dtype=torch.int32, device="cuda")
    q, k = rows_of(2, 4, 64, torch.float32, 8), rows_of(2, 2, 64, torch.float32, 9)
    for args, kw in (((table, p.long(), q), {}), ((table, p[:1], q), {}), ((table, p.cpu(), q), {}), ((table, p, q.cpu()), {}),
                     ((table, p, q, k.bfloat16()), {}), ((table, p, q.half()), {}), ((table, p, q[0]), {}), ((table, p, q, k[:1]), {}),
                     ((table, p, q), dict(k_out=k)), ((table, p, q), dict(q_out=q.bfloat16())), ((table, p, q), dict(q_out=q[:, :2])),
                     ((table, p, q.transpose(1, 2)), {}), ((table, torch.zeros(4, dtype=torch.int32, device="cuda")[::2], q), {})):
        with pytest.raises(ValueError):
            binding.rope(*args, **kw)
    with pytest.raises(binding.BitnetError):
        binding.rope(binding.Rope(128), p, q)  # more than the head
    assert binding.rope(table, p[:0], q[:0]).shape == (0, 4, 64)
