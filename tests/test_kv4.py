"""The 4-bit key/value cache on the GPU against plain 64-bit numpy (tests/kv4_reference.py).

Pages must match byte for byte (the rounding is exact), values read back bit for bit. Attention is
held to a bound worked out from its roundings (u16 = 2^-11 for fp16, u8 = 2^-8 for bf16), with
A = sum p |v| and S = scale * max sum |q| |k| over the positions seen:
  - softmax weights and values enter the product as fp16:       2 u16 A, and 2^-24 A for weights below the normal range
  - keys as fp16, fp32 queries as fp16: scores off by (1 or 2) u16 S, and by fp32 sums, 2^-16 S at most;
    a score error of d changes a weight by a factor within exp(+-2 d): (exp(2 d) - 1) A
  - the result as bf16:                                          u8 |out|
"""
import numpy as np
import pytest
import torch

import kv4_reference as ref
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class World:
    """A cache with some sequences in it, and the same in numpy."""

    def __init__(self, new, kv, heads=2, dim=128, dtype="bf16", seed=0, extra_pages=2, garbage=255):
        self.new, self.kv, self.heads, self.dim = new, kv, heads, dim
        rng = self.rng = np.random.default_rng(seed)
        self.dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        need = [-(-n // 64) for n in kv]
        self.n_pages = sum(need) + extra_pages
        ids = rng.permutation(self.n_pages)[:sum(need)]
        self.wide = max(1, max(need))
        table = np.full((len(kv), self.wide), -7, np.int32)  # entries past the end are never read
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        self.table = table
        pages = torch.full((binding.kv4_cache_bytes(self.n_pages, heads, dim),), garbage, dtype=torch.uint8, device="cuda")
        self.cache = binding.KV4Cache(self.n_pages, heads, dim, pages=pages)
        self.k = [self.numbers(n) for n in kv]
        self.v = [self.numbers(n) for n in kv]

    def numbers(self, n):
        x = self.rng.normal(size=(n, self.heads, self.dim)) * (0.3 + self.rng.random((n, self.heads, 1)) * 2)
        x += self.rng.normal(size=(1, self.heads, self.dim))
        return torch.tensor(x).to(self.dtype).float().numpy()

    def batch(self, new, kv, **kw):
        cu = np.concatenate([[0], np.cumsum(new)])
        return binding.KV4Batch(i32(cu), i32(kv), torch.tensor(self.table, device="cuda"), int(cu[-1]), max(1, max(new)),
                                kw.get("max_kv", self.wide * 64))

    def packed(self, parts):
        return torch.tensor(np.concatenate(parts)).to(self.dtype).cuda()

    def fill(self):
        """Everything cached, in one call."""
        binding.kv4_append(self.cache, self.batch(self.kv, self.kv), self.packed(self.k), self.packed(self.v))
        return self

    def expected_pages(self, garbage=255):
        blk = 64 * self.dim + 512
        pages = np.full((self.n_pages, self.heads, blk), garbage, np.uint8)
        for b, n in enumerate(self.kv):
            for j in range(n):
                for h in range(self.heads):
                    ref.write_token(pages[self.table[b, j // 64], h], j % 64, self.k[b][j, h], self.v[b][j, h])
        return pages

    def values(self, x):
        return [ref.stands_for(*ref.quantise(a)) for a in x]

    def check_attention(self, q, out, share, scale, window=0, sinks=0):
        q, out = q.float().cpu().numpy(), out.float().cpu().numpy()
        row = 0
        for b, n in enumerate(self.new):
            pos = np.arange(self.kv[b] - n, self.kv[b])
            mine = slice(row, row + n)
            o, av, size = ref.attention(q[mine], self.values(self.k)[b], self.values(self.v)[b], pos, scale, window, sinks)
            u16, d = 2.0 ** -11, abs(scale) * size
            d = d * (u16 * (1 if self.dtype == torch.bfloat16 else 2) + 2.0 ** -16)
            bound = 2.0 ** -8 * np.abs(o) + (2 * u16 + 2.0 ** -24 + np.expm1(2 * d)[..., None]) * av * 1.01 + 1e-30
            got = out[mine]
            assert np.array_equal(np.isnan(got), np.isnan(o)), "NaN in the wrong rows of sequence %d" % b
            err = np.where(np.isnan(o), 0, np.abs(got - o))
            bad = err > np.where(np.isnan(o), 1, bound)
            assert not bad.any(), "sequence %d: %d of %d off, worst %.3g times the bound, first %s" % (
                b, bad.sum(), bad.size, (err / bound)[bad].max(), np.argwhere(bad)[0])
            row += n


# ------------------------------------------------------------------- the cache
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv", [(1, [1]), (3, [0, 65, 1, 64]), (5, [130, 7])])
def test_pages_byte_for_byte_and_read_back(dim, dtype, heads, kv):
    w = World(kv, kv, heads, dim, dtype, seed=len(kv) + dim).fill()
    got = w.cache.pages.cpu().numpy().reshape(w.n_pages, heads, -1)
    assert np.array_equal(got, w.expected_pages())
    for t in (torch.float32, torch.bfloat16):
        k, v = binding.kv4_read(w.cache, w.batch(kv, kv), t)
        for x, parts in ((k, w.k), (v, w.v)):
            want = torch.tensor(np.concatenate(w.values(parts))).float().to(t)
            assert torch.equal(x.cpu(), want)


def test_token_by_token_equals_all_at_once():
    kv = [70, 3]
    a, b = World(kv, kv, seed=5), World(kv, kv, seed=5)
    a.fill()
    for j in range(70):
        new = [1, 1 if j < 3 else 0]
        now = [j + 1, min(j + 1, 3)]
        parts = [[x[s][now[s] - new[s]:now[s]] for s in range(2)] for x in (b.k, b.v)]
        binding.kv4_append(b.cache, b.batch(new, now), b.packed(parts[0]), b.packed(parts[1]))
    assert torch.equal(a.cache.pages, b.cache.pages)


@pytest.mark.parametrize("dim", [64, 128])
def test_quantisation_next_to_borders(dim):
    """fp32 values on, one ulp below and one ulp above the borders between codes, over steps and bases
    of very unlike sizes; constant vectors, tiny ranges, and values beyond the format's."""
    rng = np.random.default_rng(dim)
    rows = []
    for _ in range(400):
        base = np.float32(np.float16(rng.choice([0, 1, -3, 1000, -3e4, 1e-3, 7e-6]) * (1 + rng.random())))
        step = np.float32(np.float16(2.0 ** rng.integers(-20, 12) * (1 + rng.random())))
        x = (base.astype(np.float64) + step * (rng.integers(0, 15, dim) + 0.5)).astype(np.float32)
        x = np.where(rng.random(dim) < 0.3, np.nextafter(x, np.float32(-np.inf)), x)
        x = np.where(rng.random(dim) < 0.3, np.nextafter(x, np.float32(np.inf)), x).astype(np.float32)
        x[0], x[1] = base, np.float32(base.astype(np.float64) + 15 * step.astype(np.float64))
        rows.append(x)
    rows += [np.full(dim, 7.77, np.float32), np.zeros(dim, np.float32), np.linspace(0, 1e-6, dim, dtype=np.float32),
             np.linspace(-1e6, 1e6, dim, dtype=np.float32), np.linspace(61000, 65504, dim, dtype=np.float32),
             np.linspace(-np.float32(1e30), 0, dim, dtype=np.float32), np.full(dim, -1e38, np.float32)]
    inf = np.linspace(-1, 1, dim, dtype=np.float32)
    inf[3], inf[5] = np.inf, -np.inf
    rows.append(inf)
    nan = inf.copy()
    nan[9] = np.nan
    rows.append(nan)
    x = np.stack(rows)[:, None]
    w = World([len(x)], [len(x)], 1, dim, "f32", seed=1)
    w.k, w.v = [x], [x[::-1].copy()]
    w.fill()
    k, v = binding.kv4_read(w.cache, w.batch(w.kv, w.kv), torch.float32)
    for got, parts in ((k, w.k), (v, w.v)):
        want = w.values(parts)[0].astype(np.float32)
        assert np.array_equal(got.cpu().numpy(), want, equal_nan=True)


def test_strided_rows():
    """k and v as slices of one fused row; read back into strided rows too."""
    w = World([33], [33], 2, 64, seed=3)
    fused = torch.zeros(33, 4 * 128, dtype=torch.bfloat16, device="cuda")
    kk, vv = fused[:, 256:384].unflatten(1, (2, 64)), fused[:, 384:].unflatten(1, (2, 64))
    kk.copy_(w.packed(w.k)), vv.copy_(w.packed(w.v))
    binding.kv4_append(w.cache, w.batch([33], [33]), kk, vv)
    assert np.array_equal(w.cache.pages.cpu().numpy().reshape(w.n_pages, 2, -1), w.expected_pages())
    back = torch.full((33, 512), 9.0, dtype=torch.bfloat16, device="cuda")
    binding.kv4_read(w.cache, w.batch([33], [33]), k=back[:, :128].unflatten(1, (2, 64)), v=back[:, 256:384].unflatten(1, (2, 64)))
    assert torch.equal(back[:, :128].cpu().double(), torch.tensor(w.values(w.k)[0]).bfloat16().flatten(1).double())
    assert bool((back[:, 128:256] == 9).all()) and bool((back[:, 384:] == 9).all())


def test_append_leaves_other_tokens_alone():
    w = World([3], [100], 2, 128, seed=8)
    before = w.cache.pages.clone()
    binding.kv4_append(w.cache, w.batch([3], [100]), w.packed([w.k[0][97:]]), w.packed([w.v[0][97:]]))
    want = before.cpu().numpy().reshape(w.n_pages, 2, -1)
    for j in range(97, 100):
        for h in range(2):
            ref.write_token(want[w.table[0, j // 64], h], j % 64, w.k[0][j, h], w.v[0][j, h])
    assert np.array_equal(w.cache.pages.cpu().numpy().reshape(want.shape), want)


# ------------------------------------------------------------------- attention
def attend(w, share, dtype=None, scale=None, window=0, sinks=0, size=1.0, **kw):
    hq = w.heads * share
    q = torch.tensor(w.rng.normal(size=(sum(w.new), hq, w.dim)) * size).to(dtype or w.dtype).cuda()
    scale = scale if scale is not None else w.dim ** -0.5
    out = binding.kv4_attention(w.cache, w.batch(w.new, w.kv, **kw), q, scale, window=window, sinks=sinks)
    assert out.dtype == torch.bfloat16 and out.shape == q.shape
    w.check_attention(q, out, share, scale, window, sinks)
    return q, out


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("share", [1, 4, 7])
@pytest.mark.parametrize("kv", [[1], [2, 63, 64, 65], [700, 1, 129], [3000]])
def test_single_tokens(dim, dtype, share, kv):
    attend(World([1] * len(kv), kv, 2, dim, dtype, seed=share).fill(), share)


@pytest.mark.parametrize("dim,share", [(128, 4), (64, 3), (128, 8), (64, 1), (128, 16), (64, 40)])
@pytest.mark.parametrize("new,kv", [([2], [2]), ([5, 1, 0, 3], [5, 300, 40, 67]), ([8, 8], [129, 1000])])
def test_a_few_tokens(dim, share, new, kv):
    attend(World(new, kv, 2, dim, seed=dim + share).fill(), share)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("share,new,kv", [(4, [33], [33]), (4, [64], [64]), (1, [128], [128]), (4, [129], [200]),
                                          (5, [257, 1, 0, 40], [257, 500, 9, 1000]), (1, [300], [300]),
                                          (7, [100, 77], [100, 2000])])
def test_prompts(dim, dtype, share, new, kv):
    attend(World(new, kv, 2, dim, dtype, seed=share).fill(), share)


@pytest.mark.parametrize("new,kv", [([1, 1, 1], [1000, 64, 5]), ([6, 1], [700, 300]), ([200], [200]), ([150, 90], [900, 91])])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (100, 0), (100, 70), (5000, 3), (130, 128), (7, 900)])
def test_windows_and_sinks(new, kv, window, sinks):
    attend(World(new, kv, 1, 64, seed=window).fill(), 4, window=window, sinks=sinks)


@pytest.mark.parametrize("new,kv", [([1, 1], [0, 5]), ([7], [3]), ([4], [0]), ([60, 20], [20, 0]), ([1, 40], [0, 90])])
def test_rows_that_see_nothing_are_zero(new, kv):
    """More queries than cached tokens: the first ones stand before position 0."""
    w = World(new, kv, 2, 64, seed=2)
    w.fill()
    q, out = attend(w, 4)
    row = 0
    for n, length in zip(new, kv):
        assert not out[row:row + max(0, n - length)].any()
        row += n


@pytest.mark.parametrize("new", [1, 3, 50])
def test_nan_reaches_only_the_rows_that_see_it(new):
    """NaN keys and values past the queries, inside a window's gap, and in the pages' unused places."""
    kv = 400
    for window, sinks, where in ((0, 0, kv - 1), (0, 0, kv - 2), (100, 4, 200), (100, 4, 3), (100, 4, 5)):
        for kind in "kv":
            w = World([new], [kv], 1, 128, seed=new)
            getattr(w, kind)[0][where] = np.nan
            w.fill()
            attend(w, 4, window=window, sinks=sinks)


@pytest.mark.parametrize("new", [1, 40])
def test_infinite_and_huge_queries_stay_in_their_rows(new):
    w = World([new], [130], 1, 64, "f32", seed=4).fill()
    q = torch.randn(new, 4, 64, device="cuda")
    clean = binding.kv4_attention(w.cache, w.batch([new], [130]), q, 0.1)
    dirty = q.clone()
    dirty[0, 1, 7] = float("inf")
    dirty[0, 2, 7] = float("nan")
    out = binding.kv4_attention(w.cache, w.batch([new], [130]), dirty, 0.1)
    assert bool(out[0, 2].isnan().all())
    keep = torch.ones(new, 4, dtype=torch.bool)
    keep[0, 1] = keep[0, 2] = False
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("new,kv", [([1], [500]), ([70], [70])])
@pytest.mark.parametrize("size,scale", [(1e4, 1e-4), (1e-6, 1e5), (30.0, 0.2), (1.0, 0.0), (1.0, -0.3), (1e30, 1e-31)])
def test_scales(new, kv, size, scale):
    for dtype in (torch.float32, torch.bfloat16):
        w = World(new, kv, 2, 64, "f32" if dtype == torch.float32 else "bf16", seed=9).fill()
        attend(w, 4, dtype=dtype, size=size, scale=scale)


@pytest.mark.parametrize("new", [1, 80])
def test_values_of_unlike_sizes(new):
    """Values from 1e-4 to 1e4 in one sequence: each token has a step of its own."""
    w = World([new], [300], 1, 128, "f32", seed=6)
    w.v[0] *= (10.0 ** w.rng.integers(-4, 5, (300, 1, 1))).astype(np.float32)
    attend(w.fill(), 4)


def test_strided_queries_and_output():
    w = World([5, 40], [70, 90], 2, 64, seed=7).fill()
    fused = torch.randn(45, 1024, dtype=torch.bfloat16, device="cuda")
    q = fused[:, 256:768].unflatten(1, (8, 64))
    out = torch.full((45, 800), 3.0, dtype=torch.bfloat16, device="cuda")
    got = binding.kv4_attention(w.cache, w.batch(w.new, w.kv), q, 0.125, out=out[:, 8:520].unflatten(1, (8, 64)))
    w.check_attention(q, got, 4, 0.125)
    assert bool((out[:, :8] == 3).all()) and bool((out[:, 520:] == 3).all())
    assert torch.equal(got, binding.kv4_attention(w.cache, w.batch(w.new, w.kv), q.contiguous(), 0.125))


@pytest.mark.parametrize("new,kv", [([1] * 3, [9000, 40, 2500]), ([9], [7000]), ([300, 1], [5000, 77])])
def test_same_bits_each_time(new, kv):
    w = World(new, kv, 2, 128, seed=11).fill()
    q = torch.randn(sum(new), 8, 128, dtype=torch.bfloat16, device="cuda")
    b = w.batch(new, kv)
    first = binding.kv4_attention(w.cache, b, q, 0.09)
    for _ in range(5):
        ws = torch.full((max(256, binding.kv4_attention_workspace_size(w.cache, b, 8)),), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(first, binding.kv4_attention(w.cache, b, q, 0.09, workspace=ws))


def test_loose_bounds_change_nothing():
    """max_q, max_kv and the table's width above what the sequences have."""
    new, kv = [1, 3], [500, 66]
    w = World(new, kv, 2, 128, seed=12).fill()
    q = torch.randn(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    cu, lens = i32([0, 1, 4]), i32(kv)
    wide = torch.full((2, 4000), -1, dtype=torch.int32, device="cuda")
    wide[:, :w.wide] = torch.tensor(w.table, device="cuda")
    for max_q, max_kv in ((3, 512), (7, 4000 * 64), (300, 5000)):
        b = binding.KV4Batch(cu, lens, wide, 4, max_q, max_kv)
        w.check_attention(q, binding.kv4_attention(w.cache, b, q, 0.09), 4, 0.09)


def test_a_long_cache():
    """131 072 tokens: the values of a few far positions decide the result."""
    n = 131072
    w = World([1], [n], 1, 64, seed=13)
    w.fill()
    attend(w, 8)


def test_pages_past_4_gb():
    """Page offsets beyond 32 bits."""
    heads, dim, n_pages = 8, 128, 65000  # 8 * 8704 * 65000 = 4.5e9 bytes
    cache = binding.KV4Cache(n_pages, heads, dim)
    w = World([70], [130], heads, dim, seed=14)
    w.cache, w.table = cache, np.array([[n_pages - 1, 3, n_pages - 2]], np.int32)
    w.fill()
    k, v = binding.kv4_read(cache, w.batch([130], [130]), torch.float32)
    assert np.array_equal(k.cpu().numpy(), w.values(w.k)[0].astype(np.float32))
    assert np.array_equal(v.cpu().numpy(), w.values(w.v)[0].astype(np.float32))
    attend(w, 1)
    w.new = [1]
    attend(w, 4)


def test_on_another_stream():
    w = World([1, 40], [900, 90], 2, 128, seed=15).fill()
    q = torch.randn(41, 8, 128, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    want = binding.kv4_attention(w.cache, w.batch(w.new, w.kv), q, 0.09)
    s = torch.cuda.Stream()
    out = binding.kv4_attention(w.cache, w.batch(w.new, w.kv), q, 0.09, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_captured_decode_step():
    """Append and attention in one graph, replayed as the sequences grow: lengths are read when it runs."""
    w = World([1, 1], [200, 65], 2, 128, seed=16).fill()
    lens = i32([150, 30])
    b = binding.KV4Batch(i32([0, 1, 2]), lens, torch.tensor(w.table, device="cuda"), 2, 1, 256)
    k, v = (torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.randn(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(256, binding.kv4_attention_workspace_size(w.cache, b, 8)), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def step():
        binding.kv4_append(w.cache, b, k, v)
        binding.kv4_attention(w.cache, b, q, 0.09, out=out, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        k.copy_(w.packed([w.k[0][149:150], w.k[1][29:30]])), v.copy_(w.packed([w.v[0][149:150], w.v[1][29:30]]))
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for a, c in ((151, 31), (192, 64), (193, 65), (200, 1)):
        lens.copy_(i32([a, c]))
        k.copy_(w.packed([w.k[0][a - 1:a], w.k[1][c - 1:c]])), v.copy_(w.packed([w.v[0][a - 1:a], w.v[1][c - 1:c]]))
        g.replay()
        torch.cuda.synchronize()
        w.kv, keep = [a, c], (w.kv, w.k, w.v)
        w.k, w.v = [x[:n] for x, n in zip(w.k, w.kv)], [x[:n] for x, n in zip(w.v, w.kv)]
        w.check_attention(q, out, 4, 0.09)
        w.kv, w.k, w.v = keep


@pytest.mark.parametrize("new,breaks", [
    (1, "page"), (40, "page"), (1, "len"), (1, "negative"), (40, "len"), (1, "cu"), (40, "cu"), (2, "max_q"), (40, "max_q")])
def test_batches_that_break_their_bounds_are_reported(new, breaks):
    """Every call keeps inside its arrays and reports; the other sequence's rows are right. (A sequence
    that cu_q counts twice, as a falling cu_q makes it, is not looked at here.)"""
    kv = [130, 200]
    w = World([new, new], kv, 2, 128, seed=17).fill()
    table, lens, cu = w.table.copy(), list(kv), [0, new, 2 * new]
    max_q = new
    if breaks == "page":
        table[1, 0] = w.n_pages
    elif breaks == "len":
        lens[1] = w.wide * 64 + 1
    elif breaks == "negative":
        lens[1] = -5
    elif breaks == "cu":
        cu[2] = 2 * new + 3
    else:
        max_q, cu = new - 1, [0, new - 1, 2 * new]
    rows = cu[1]
    b = binding.KV4Batch(i32(cu), i32(lens), torch.tensor(table, device="cuda"), 2 * new, max_q, w.wide * 64)
    q = torch.randn(2 * new, 8, 128, dtype=torch.bfloat16, device="cuda")
    assert binding.last_device_error() == 0
    out = binding.kv4_attention(w.cache, b, q, 0.09)
    assert binding.last_device_error() == binding.BITNET_ERANGE
    w.new, w.kv = [rows], [130]
    w.check_attention(q[:rows], out[:rows], 4, 0.09)
    k = torch.zeros(2 * new, 2, 128, dtype=torch.bfloat16, device="cuda")
    k[:rows], v = w.packed([w.k[0][130 - rows:]]), k.clone()
    v[:rows] = w.packed([w.v[0][130 - rows:]])
    if breaks != "page" or new > 1:  # the bad page holds none of a single new token
        binding.kv4_read(w.cache, b)
        if breaks != "page":
            assert binding.last_device_error() == binding.BITNET_ERANGE
    binding.last_device_error()
    binding.kv4_append(w.cache, b, k, v)
    if breaks != "page":
        assert binding.last_device_error() == binding.BITNET_ERANGE
    assert binding.last_device_error() == 0


# ------------------------------------------------------------------- wider shapes
@pytest.mark.parametrize("heads,share,dim", [(70, 1, 64), (66, 2, 128), (1, 128, 64), (2, 100, 128), (3, 33, 64), (1, 17, 128)])
@pytest.mark.parametrize("new,kv", [([1, 1], [129, 64]), ([2, 1], [70, 3]), ([40], [100])])
def test_many_heads_and_wide_groups(heads, share, dim, new, kv):
    attend(World(new, kv, heads, dim, seed=heads + share).fill(), share)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,kv,share", [([1, 600, 1, 5, 33, 0], [5000, 900, 1, 2000, 33, 700], 4),  # all kinds in one call
                                          ([8, 9, 8, 2], [4000, 4100, 10, 300], 4),                   # 32 and 36 rows a head
                                          ([16, 17, 1], [3000, 3000, 40], 1),                         # 16 and 17
                                          ([128, 1], [6000, 6000], 1), ([32, 20], [9000, 65], 4)])     # long caches, few rows
def test_unlike_sequences_in_one_call(dim, new, kv, share):
    attend(World(new, kv, 2, dim, seed=sum(new)).fill(), share)


@pytest.mark.parametrize("window,sinks", [(300, 0), (1000, 4), (3000, 130), (65, 1)])
@pytest.mark.parametrize("new", [[1] * 4, [4, 1, 7, 2], [30, 12, 1, 3]])
def test_windows_far_into_long_caches(new, window, sinks):
    """Few and many pages inside the window, in caches that are far longer."""
    attend(World(new, [9000, 4097, 8000, 2500], 2, 128, seed=window).fill(), 4, window=window, sinks=sinks)


@pytest.mark.parametrize("seed", range(6))
def test_ragged_batches(seed):
    rng = np.random.default_rng(100 + seed)
    n = int(rng.integers(2, 20))
    top = int(rng.choice([1, 8, 60, 300]))
    new = rng.integers(0, top + 1, n).tolist()
    kv = [a + int(c) for a, c in zip(new, rng.integers(0, 1500, n))]
    dim, heads, share = int(rng.choice([64, 128])), int(rng.integers(1, 4)), int(rng.integers(1, 9))
    window, sinks = (int(rng.integers(1, 600)), int(rng.integers(0, 80))) if seed % 2 else (0, 0)
    w = World(new, kv, heads, dim, "f32" if seed % 3 == 0 else "bf16", seed=seed).fill()
    if sum(new):
        attend(w, share, window=window, sinks=sinks)


def test_calls_on_several_streams_at_once():
    """Each with an output and a workspace of its own."""
    kinds = [([1] * 5, [3000] * 5), ([300], [2000]), ([6], [4000]), ([1], [40])]
    worlds = [World(new, kv, 2, 128, seed=i).fill() for i, (new, kv) in enumerate(kinds)]
    qs = [torch.randn(sum(w.new), 8, 128, dtype=torch.bfloat16, device="cuda") for w in worlds]
    batches = [w.batch(w.new, w.kv) for w in worlds]
    want = [binding.kv4_attention(w.cache, b, q, 0.09) for w, b, q in zip(worlds, batches, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in worlds]
    got = [[binding.kv4_attention(w.cache, b, q, 0.09, stream=s) for w, b, q, s in zip(worlds, batches, qs, streams)]
           for _ in range(10)]
    torch.cuda.synchronize()
    for outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
