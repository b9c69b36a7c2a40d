"""4-bit weights with group scales against plain 64-bit arithmetic.

Codes, scales and zero points match bit for bit (fp32 divisions, each rounded once). The bound of a product, with W = sum |w| |x| and X the
row's largest number:
  - fp32 rows enter as two fp16 parts: 2^-11 of 2^-11 of each number, 2^-22 W; what lies below fp16's least step
    (2^-25 where X is at least 2^14): 2^-39 X sum |w|, of bf16 rows too
  - sums in fp32 of exact products: within a group at most G + 8 additions, over the groups K / G + 8 more, each off by 2^-23 of
    the sum of sizes at most (the matrix unit may cut, not round): (G + K / G + 16) 2^-23 W
"""
import ctypes

import numpy as np
import pytest
import torch

from ternary_weight_gb300 import _build, binding

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.lib()


def product(lib, **kw):
    a = {**dict(x=FAKE, dtype=0, M=2, K=256, codes=FAKE, scales=FAKE, zeros=FAKE, N=5, group=64, out=FAKE), **kw}
    return lib.bitnet_w4_matmul(*a.values(), None)


def quant(lib, **kw):
    a = {**dict(w=FAKE, dtype=0, N=5, K=256, group=64, codes=FAKE, scales=FAKE, zeros=FAKE), **kw}
    return lib.bitnet_w4_quant_weight(*a.values(), None)


BOTH = [(dict(codes=None), -1), (dict(scales=None), -1), (dict(N=0), -1), (dict(N=1 << 31), -1), (dict(K=0), -1), (dict(K=192), -1),
        (dict(K=32896), -1), (dict(group=16), -1), (dict(group=256), -1), (dict(group=0), -1), (dict(dtype=2), -1), (dict(codes=FAKE + 8), -2),
        (dict(scales=FAKE + 2), -2), (dict(zeros=FAKE + 4), -2)]


@pytest.mark.parametrize("kw,want", BOTH + [(dict(x=None), -1), (dict(out=None), -1), (dict(M=0), -1), (dict(M=1 << 31), -1),
                                            (dict(x=FAKE + 4), -2), (dict(out=FAKE + 2), -2)])
def test_bad_products_are_refused(lib, kw, want):
    assert product(lib, **kw) == want


@pytest.mark.parametrize("kw,want", BOTH + [(dict(w=None), -1), (dict(w=FAKE + 8), -2)])
def test_bad_weights_are_refused(lib, kw, want):
    assert quant(lib, **kw) == want


@pytest.mark.parametrize("bad", [dict(x=(2, 128)), dict(x=(256,)), dict(scales=(5, 3)), dict(scales=(4, 4)), dict(scales=(5, 0)), dict(zeros=(5, 2)),
                                 dict(out=(2, 4)), dict(codes_dtype=torch.int8), dict(scales_dtype=torch.float32), dict(out_dtype=torch.float16),
                                 dict(zeros_dtype=torch.int32), {}])
def test_tensors_that_do_not_fit_are_refused(lib, bad):
    """On the CPU: also what fits, since no tensor is on a GPU."""
    make = lambda name, shape, dtype: torch.zeros(bad.get(name, shape), dtype=bad.get(name + "_dtype", dtype))  # noqa: E731
    with pytest.raises(ValueError):
        binding.w4_matmul(make("x", (2, 256), torch.float32), make("codes", (5, 128), torch.uint8), make("scales", (5, 4), torch.float16),
                          zeros=make("zeros", (5, 4), torch.uint8), out=make("out", (2, 5), torch.float32))


# ------------------------------------------------------------------- on the GPU
@pytest.fixture
def cuda_lib(lib):
    if not torch.cuda.is_available():
        pytest.fail("gpu tests need a CUDA device")
    yield
    assert binding.last_device_error() == 0


def quantised(w, group, zeros):
    """codes (N x K), scales, zero points of fp32 weights, in numpy."""
    w = w.reshape(w.shape[0], -1, group)
    lo, hi = np.minimum(w.min(-1), 0), np.maximum(w.max(-1), 0)
    size = hi - lo if zeros else np.maximum(hi, -lo)
    scale = (size / np.float32(15 if zeros else 7)).astype(np.float16)
    s = scale.astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        zero = np.where(s > 0, np.clip(np.rint(-lo / s), 0, 15), 0) if zeros else np.full(s.shape, 8.0)
        code = np.where(s[..., None] > 0, np.clip(np.rint(w / s[..., None]) + zero[..., None], 0, 15), zero[..., None])
    return code.reshape(code.shape[0], -1).astype(np.uint8), scale, zero.astype(np.uint8)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,k", [(1, 128), (7, 384), (300, 1024)])
def test_codes_bit_for_bit(cuda_lib, group, zeros, dtype, n, k):
    rng = np.random.default_rng(n + group)
    w = rng.normal(size=(n, k)) * rng.choice([1e-6, 0.02, 30.0], size=(n, k // 32)).repeat(32, 1)
    w[0, :32] = 0
    w[-1, 64:128] = np.abs(w[-1, 64:128])
    w = torch.tensor(w).to(dtype)
    codes, scales, z = binding.w4_quant_weight(w.cuda(), group, zeros)
    c, s, zz = quantised(w.float().numpy(), group, zeros)
    assert np.array_equal(scales.cpu().numpy().view(np.uint16), s.view(np.uint16))
    assert np.array_equal(codes.cpu().numpy(), c[:, 0::2] | c[:, 1::2] << 4)
    assert (z is None) != zeros and (not zeros or np.array_equal(z.cpu().numpy(), zz))


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 1e30])
def test_weights_out_of_range_are_reported(cuda_lib, value):
    w = torch.ones(3, 256, device="cuda")
    w[1, 200] = value
    binding.w4_quant_weight(w)
    assert binding.last_device_error() == binding.BITNET_ERANGE


def weights(n, k, group, zeros, seed):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, size=(n, k), dtype=np.uint8)
    scales = (rng.random((n, k // group)) * 0.02 + 0.001).astype(np.float16)
    scales[rng.random(scales.shape) < 0.02] = 0
    z = rng.integers(0, 16, size=scales.shape, dtype=np.uint8) if zeros else None
    return codes, scales, z


def check(got, x, codes, scales, z, group):
    x64 = x.double().cpu().numpy()
    s = scales.astype(np.float64).repeat(group, 1)
    zero = (z.astype(np.float64) if z is not None else np.full(scales.shape, 8.0)).repeat(group, 1)
    w = s * (codes - zero)
    want, k = x64 @ w.T, codes.shape[1]
    wide = np.abs(x64) @ np.abs(w).T
    bound = (group + k / group + 16) * 2.0 ** -23 * wide + 2.0 ** -39 * np.abs(x64).max(1, keepdims=True) * np.abs(w).sum(1) + 1e-44
    if x.dtype == torch.float32:
        bound += 2.0 ** -22 * wide
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= bound).all(), "worst %.3g of the bound at %s" % ((err / bound).max(), np.argwhere(err > bound)[0])


def run(x, codes, scales, z, **kw):
    packed = torch.from_numpy(codes[:, 0::2] | codes[:, 1::2] << 4).cuda()
    return binding.w4_matmul(x, packed, torch.from_numpy(scales).cuda(), zeros=None if z is None else torch.from_numpy(z).cuda(), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (128, False), (64, True), (32, False)])
@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (1, 2560, 6912), (3, 17, 1152), (5, 640, 2560), (9, 33, 384), (17, 1000, 256), (33, 130, 1280),
                                   (70, 50, 640), (1, 5000, 128)])
def test_products(cuda_lib, dtype, group, zeros, m, n, k):
    codes, scales, z = weights(n, k, group, zeros, m + n + k)
    g = torch.Generator().manual_seed(k)
    x = (torch.randn(m, k, generator=g) * (0.5 + torch.randn(1, k, generator=g).abs() ** 3)).to(dtype).cuda()
    got = run(x, codes, scales, z)
    check(got, x, codes, scales, z, group)
    assert torch.equal(got, run(x, codes, scales, z))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k,dtype", [(4, 40, 32768, torch.float32), (12, 24, 32768, torch.bfloat16), (1, 100003, 256, torch.float32),
                                         (16, 20011, 512, torch.bfloat16)])
def test_products_of_large_sizes(cuda_lib, m, n, k, dtype):
    codes, scales, z = weights(n, k, 64, True, 9)
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    check(run(x, codes, scales, z), x, codes, scales, z, 64)


@pytest.mark.gpu
def test_rows_of_every_size(cuda_lib):
    """Rows of very large, tiny, subnormal and zero numbers, and one great number among small ones."""
    codes, scales, z = weights(50, 256, 32, True, 4)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(8, 256, generator=g)
    x *= torch.tensor([1e30, 1e-30, 1e-42, 0.0, 1.0, 3e4, 1e-7, 1.0])[:, None]
    x[4, 7], x[7, 8] = 1e6, -1e8
    for dtype in (torch.float32, torch.bfloat16):
        t = x.to(dtype).cuda()
        got = run(t, codes, scales, z)
        check(got, t, codes, scales, z, 32)
        assert bool((got[3] == 0).all())


@pytest.mark.gpu
def test_rows_with_no_number_leave_the_others_alone(cuda_lib):
    codes, scales, z = weights(40, 256, 128, False, 4)
    x = torch.randn(3, 256, generator=torch.Generator().manual_seed(3)).cuda()
    want = run(x, codes, scales, z)
    x[1, 5] = float("nan")
    x[2, 9] = float("inf")
    got = run(x, codes, scales, z)
    assert torch.equal(got[0], want[0]) and not bool(got[1:][:, torch.from_numpy(scales[:, 0] != 0).cuda()].isfinite().any())


@pytest.mark.gpu
def test_captured_on_a_stream_and_into_a_given_output(cuda_lib):
    codes, scales, z = weights(300, 512, 64, True, 4)
    packed, s, zz = torch.from_numpy(codes[:, 0::2] | codes[:, 1::2] << 4).cuda(), torch.from_numpy(scales).cuda(), torch.from_numpy(z).cuda()
    x, out = torch.randn(2, 512, device="cuda"), torch.full((2, 300), 7.0, device="cuda")
    assert binding.w4_matmul(x, packed, s, zz, out=out) is out
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = binding.w4_matmul(x, packed, s, zz)
    x.mul_(-2.0)
    graph.replay()
    assert torch.equal(y, out * -2.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = binding.w4_matmul(x, packed, s, zz, stream=side)
    side.synchronize()
    assert torch.equal(again, y)
    assert binding.w4_matmul(x[:0], packed, s, zz).shape == (0, 300)
    with pytest.raises(ValueError):
        binding.w4_matmul(x.t().contiguous().t(), packed, s, zz)
    with pytest.raises(ValueError):
        binding.w4_matmul(x.half(), packed, s, zz)


@pytest.mark.gpu
def test_quantised_weights_multiply(cuda_lib):
    """The two calls together: what the codes stand for is what is multiplied."""
    w = torch.randn(200, 640, generator=torch.Generator().manual_seed(1)).cuda() * 0.03
    x = torch.randn(2, 640, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    for zeros in (False, True):
        codes, scales, z = binding.w4_quant_weight(w, 32, zeros)
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).cpu().numpy()
        zz = None if z is None else z.cpu().numpy()
        got = binding.w4_matmul(x, codes, scales, z)
        check(got, x, c, scales.cpu().numpy(), zz, 32)
        # A weight is off by half a step; what the scale's own rounding (2^-11 of up to 15 steps) moves a code beyond the last
        # is less than 15 2^-11 of one. The product adds its own roundings: (32 + 640 / 32 + 17) 2^-23 of the numbers met.
        s, xx = scales.double().repeat_interleave(32, 1), x.double()
        off = xx.abs() @ (s * (0.5 + 15 * 2.0 ** -11)).T + 2.0 ** -16 * (xx.abs() @ (w.double().abs() + s).T)
        assert bool(((got.double() - xx @ w.double().T).abs() <= off).all())


@pytest.mark.gpu
def test_quantisation_refuses_places_of_another_group(cuda_lib):
    w = torch.randn(6, 256, device="cuda")
    codes, scales, z = binding.w4_quant_weight(w, 64, True)
    for group in (32, 128):
        with pytest.raises(ValueError):
            binding.w4_quant_weight(w, group, codes=codes, scales=scales)
        with pytest.raises(ValueError):
            binding.w4_quant_weight(w, group, codes=codes, scales=scales, zeros=z)
    with pytest.raises(ValueError):
        binding.w4_quant_weight(w, 64, codes=codes[:5], scales=scales)
    again = binding.w4_quant_weight(w, 64, codes=torch.zeros_like(codes), scales=torch.zeros_like(scales), zeros=torch.zeros_like(z))
    assert all(torch.equal(a, b) for a, b in zip(again, (codes, scales, z)))
