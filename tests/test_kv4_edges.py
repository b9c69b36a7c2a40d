"""Edges of the 4-bit cache and its attention, against plain 64-bit numpy (tests/kv4_reference.py)."""
import numpy as np
import pytest
import torch

import kv4_reference as ref
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


@pytest.mark.parametrize("dim", [64, 128])
def test_numbers_beyond_the_clamp_take_its_code(dim):
    """Vectors that begin just below 61440 and end beyond it: it is the clamped number that is rounded."""
    rows = []
    for low in (61425.0, 61430.0, 61439.99, 61440.0, 61408.0, 61000.0):
        for high in (61440.0, 61441.0, 65000.0, 1e30, np.inf):
            x = np.full(dim, low, np.float32)
            x[dim // 2:] = high
            x[1] = (low + min(high, 61440.0)) / 2
            rows += [x, -x, np.roll(x, 5)]
    x = np.stack(rows)[:, None]
    w = World([len(x)], [len(x)], 1, dim, "f32", seed=1)
    w.k, w.v = [x], [x[::-1].copy()]
    w.fill()
    assert np.array_equal(w.cache.pages.cpu().numpy().reshape(w.n_pages, 1, -1), w.expected_pages())
    k, v = binding.kv4_read(w.cache, w.batch(w.kv, w.kv), torch.float32)
    for got, parts in ((k, w.k), (v, w.v)):
        assert np.array_equal(got.cpu().numpy(), w.values(parts)[0].astype(np.float32))


def directed(new, kv, dim, share, at, nats, rng, dtype, spread=0.1):
    """Queries near one direction for each key/value head, and keys among which token `at` stands `nats`
    above (below, if negative) the others, whose scores are small. Returns q (new, heads * share, dim) and k."""
    heads = 2
    r = rng.normal(size=(heads, dim))
    q = np.repeat(r, share, 0)[None] * (1 + 0.02 * rng.random((new, heads * share, 1)))
    k = rng.normal(size=(kv, heads, dim)) * spread
    k[at] = r * nats / ((r * r).sum(-1, keepdims=True) * dim ** -0.5)
    return torch.tensor(q).to(dtype).cuda(), torch.tensor(k).to(dtype).float().numpy()


SHAPES = [(64, 1, 4, 64), (128, 1, 4, 64), (128, 1, 4, 700), (64, 1, 8, 6000), (128, 5, 4, 700), (128, 3, 4, 6000), (64, 100, 4, 700)]


@pytest.mark.parametrize("dim,new,share,kv", SHAPES)
@pytest.mark.parametrize("ratio", [2.0 ** 14, 2.0 ** 17, 2.0 ** 20])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_a_value_without_weight_costs_the_others_nothing(dim, new, share, kv, ratio, where):
    """One token with a weight of e^-60 and values many times the others': the result is that of the others, to
    the roundings of weights and values (fp16), queries and keys (fp16: 2^-10 of what they add to a score, fp32
    sums within 2^-16), and the result (bf16). A weight times its step is off by 2^-32 of a row's largest at
    least, a code or (where base and code go together) a number of up to 79 steps."""
    w = World([new], [kv], 2, dim, "f32", seed=kv)
    at = {"first": 0, "middle": (kv - new) // 2, "last": kv - new}[where]
    q, w.k[0] = directed(new, kv, dim, share, at, -60.0, w.rng, torch.float32)
    v = w.rng.normal(size=(kv, 2, dim)) + w.rng.normal(size=(1, 2, dim))
    v *= 2.0 ** -8
    v[at] *= ratio
    w.v[0] = v.astype(np.float32)
    w.fill()
    got = binding.kv4_attention(w.cache, w.batch([new], [kv]), q, dim ** -0.5).float().cpu().numpy()
    kk, vv = (np.delete(w.values(x)[0], at, 0) for x in (w.k, w.v))
    o, av, size = ref.attention(q.cpu().numpy(), kk, vv, np.arange(kv - new, kv) - 1, dim ** -0.5, 0, 0)
    d = dim ** -0.5 * size * (2.0 ** -10 + 2.0 ** -16)
    low = 2.0 ** -32 * 79 / 15 * kv * 2 * np.abs(vv).max()
    bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + np.expm1(2 * d)[..., None]) * av * 1.01 + low
    err = np.abs(got - o)
    assert (err <= bound).all(), "worst %.3g times the bound" % (err / bound).max()


@pytest.mark.parametrize("dim,new,share,kv", SHAPES)
@pytest.mark.parametrize("nats", [9.0, 13.0, 16.0])
@pytest.mark.parametrize("first", ["zero", "constant", "small"])
def test_small_weights_beside_a_large_one(dim, new, share, kv, nats, first):
    """The first token takes nearly all of the weight and has values of nothing, or next to it: what the others
    give, each e^-nats of it, has to come out. The bound is that of the roundings: weights enter the
    product with 11 bits and, relative to the row's largest, 2^-32 at least; values as fp16, keys as
    fp16 (2^-11 of what they add to a score); fp32 sums within 2^-16 of them; the result as bf16."""
    w = World([new], [kv], 2, dim, "bf16", seed=kv)
    q, w.k[0] = directed(new, kv, dim, share, 0, nats, w.rng, torch.bfloat16)
    v = 1 + w.rng.normal(size=(kv, 2, dim))
    v[0] = {"zero": 0 * v[0], "constant": 0 * v[0] + 1e-6, "small": v[0] * 1e-6}[first]
    w.v[0] = torch.tensor(v).bfloat16().float().numpy()
    w.fill()
    got = binding.kv4_attention(w.cache, w.batch([new], [kv]), q, dim ** -0.5).float().cpu().numpy()
    kk, vv = w.values(w.k)[0], w.values(w.v)[0]
    pos = np.arange(kv - new, kv)
    o, av, size = ref.attention(q.float().cpu().numpy(), kk, vv, pos, dim ** -0.5, 0, 0)
    d = dim ** -0.5 * size * (2.0 ** -11 + 2.0 ** -16)
    # sum |v| over the sum of weights relative to the largest (at least 1)
    low = 2.0 ** -32 * np.repeat(np.abs(vv).sum(0), share, 0)[None]
    bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + np.expm1(2 * d)[..., None]) * av * 1.01 + low
    err = np.abs(got - o)
    assert (err <= bound).all(), "worst %.3g times the bound" % (err / bound).max()


@pytest.mark.parametrize("dim,new,share,kv", SHAPES)
@pytest.mark.parametrize("kind", ["zeros", "constants", "offset"])
def test_values_without_spread(dim, new, share, kv, kind):
    """Value vectors of one number each (their step is 0), all zeros, and numbers that stand thousands of steps
    from 0: held to the roundings of the weights and of the result."""
    w = World([new], [kv], 2, dim, "f32", seed=kv)
    shape = (kv, 2, 1 if kind == "constants" else dim)
    v = {"zeros": np.zeros(shape), "constants": w.rng.normal(size=shape), "offset": 1000 + 0.01 * w.rng.normal(size=shape)}[kind]
    w.v[0] = np.broadcast_to(v, (kv, 2, dim)).astype(np.float32)
    w.fill()
    q, out = attend(w, share)
    assert bool(out.any()) == (kind != "zeros")


@pytest.mark.parametrize("dim,new,share,kv", [(64, 1, 4, 200), (128, 1, 4, 200), (128, 1, 2, 5000), (128, 5, 4, 700), (64, 130, 2, 700), (128, 300, 1, 700)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("log2", [16, 22, 26, 30, 34, 40, 60, 100, 115, 120, 126])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_large_scores_choose_their_token(dim, new, share, kv, dtype, log2, sign):
    """Scores from thousands to the largest of fp32, all of either sign, with one token far above the others:
    its value is the result, to the roundings of values (fp16) and of the result (bf16)."""
    w = World([new], [kv], 2, dim, "f32" if dtype == torch.float32 else "bf16", seed=log2)
    at = (kv - new) // 2
    r = w.rng.choice([-1.0, 1.0], size=(2, dim))
    q = torch.tensor(np.repeat(r, share, 0)[None].repeat(new, 0) * 2.0 ** log2).to(dtype).cuda()
    size = 1.0 + w.rng.random((kv, 2, 1)) if sign > 0 else 3.0 + w.rng.random((kv, 2, 1))
    size[at] = 3.0 if sign > 0 else 1.0
    w.k[0] = torch.tensor(r[None] * size * (1 + 0.05 * w.rng.random((kv, 2, dim)))).to(w.dtype).float().numpy()
    w.fill()
    got = binding.kv4_attention(w.cache, w.batch([new], [kv]), q, sign * dim ** -0.5).float().cpu().numpy()
    want = np.repeat(w.values(w.v)[0][at], share, 0)[None]
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(want) * 1.01 + 2.0 ** -10 * np.abs(want).max(-1, keepdims=True)).all()


@pytest.mark.parametrize("share,new", [(16, 2), (10, 2), (10, 3), (9, 3)])
@pytest.mark.parametrize("dim", [64, 128])
def test_few_rows_go_one_way_whatever_stands_beside_them(share, new, dim):
    """A sequence of 17 to 32 rows a head, alone and beside a prompt: the same kernel, so the same bits."""
    w = World([new, 150], [300, 150], 2, dim, seed=share).fill()
    q = torch.randn(new + 150, 2 * share, dim, dtype=torch.bfloat16, device="cuda")
    both = binding.kv4_attention(w.cache, w.batch(w.new, w.kv), q, dim ** -0.5)
    w.check_attention(q, both, share, dim ** -0.5)
    alone = binding.kv4_attention(w.cache, w.batch([new, 0], w.kv), q[:new], dim ** -0.5)
    assert torch.equal(both[:new], alone)
