"""Eviction by gathered weight against plain numpy: every byte of the pages and every bit of the masses, also of what the
call must leave alone."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_reference as ref
from test_kv4 import World, i32
from ternary_weight_gb300 import _build, binding

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.lib()


@pytest.fixture
def cuda_lib(lib):
    if not torch.cuda.is_available():
        pytest.fail("gpu tests need a CUDA device")
    yield
    assert binding.last_device_error() == 0, "a kernel recorded a device-side error"


# ------------------------------------------------------------------- without a GPU
def call(lib, c=None, b=None, **kw):
    c = binding._KV4CacheDesc(**{**dict(pages=FAKE, n_pages=4, kv_heads=2, head_dim=128), **(c or {})})
    b = binding._KV4BatchDesc(**{**dict(cu_q=FAKE, kv_len=FAKE, page_table=FAKE, batch=2, max_pages=2, total_q=0, max_q=1, max_kv=128), **(b or {})})
    a = {**dict(mass=FAKE, budget=50, limit=60, sinks=4, recent=10, into=None, into_pages=0, new_len=FAKE, ws=FAKE, ws_bytes=1 << 40), **kw}
    return lib.bitnet_kv4_evict(ctypes.byref(c), ctypes.byref(b), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(mass=None), -1), (dict(budget=0), -1), (dict(limit=49), -1), (dict(limit=1 << 31), -1), (dict(sinks=-1), -1), (dict(sinks=51), -1),
    (dict(recent=-1), -1), (dict(recent=47), -1), (dict(into=FAKE, into_pages=0), -1), (dict(into=FAKE, into_pages=(1 << 24) + 1), -1),
    (dict(into=FAKE, into_pages=1, budget=65, limit=65), -1), (dict(ws=None), -1), (dict(ws_bytes=100), -1), (dict(mass=FAKE + 4), -2), (dict(ws=FAKE + 16), -2),
    (dict(into=FAKE + 2, into_pages=2), -2), (dict(new_len=FAKE + 1), -2), (dict(c=dict(pages=None)), -1), (dict(c=dict(head_dim=32)), -1),
    (dict(b=dict(kv_len=None)), -1), (dict(b=dict(max_kv=129)), -1), (dict(b=dict(batch=0)), -1)])
def test_bad_calls_are_refused(lib, kw, want):
    assert call(lib, **kw) == want


def test_workspace_size(lib):
    c, b = binding._KV4CacheDesc(FAKE, 4, 2, 128), binding._KV4BatchDesc(FAKE, FAKE, FAKE, 2, 2, 0, 1, 128)
    size = lambda n: lib.bitnet_kv4_evict_workspace_size(ctypes.byref(c), ctypes.byref(b), n)  # noqa: E731
    assert size(0) == -1 and size(1 << 31) == -1 and 0 < size(1) <= size(128) == size(2 ** 31 - 1)


# ------------------------------------------------------------------- on the GPU
class Evict(World):
    def masses(self, kind):
        n = (self.n_pages, self.heads, 64)
        m = self.rng.random(n)
        if kind == "equal":
            m = np.ones(n)
        elif kind == "few values":
            m = self.rng.integers(0, 4, size=n) * 0.25
        elif kind == "odd":
            m = self.rng.choice([0.0, -0.0, 1e-45, -1e-45, 3.0, -3.0, np.inf, -np.inf, np.nan, 1e30], size=n)
        elif kind == "rising":  # the last tokens have most: nearly all moves
            m = m + np.arange(64)
        elif kind == "wide":
            m = np.exp(20 * self.rng.normal(size=n))
        return m.astype(np.float32)

    def own(self, b, n):
        return [self.table[b, j // 64] for j in range(n)], [j % 64 for j in range(n)]

    def expect(self, pages, mass, budget, limit, sinks, recent, into=None):
        """What the call makes of pages (n_pages x heads x bytes) and masses, and the new lengths."""
        d, new_pages, new_mass, lens = self.dim, pages.copy(), mass.copy(), []
        at = 64 * d // 2
        for b, n in enumerate(self.kv):
            cut = n > limit
            lens.append(budget if cut else n)
            if not cut and into is None:
                continue
            for h in range(self.heads):
                keep = list(range(n))
                if cut:
                    middle = np.arange(sinks, n - recent)
                    m = np.array([mass[self.table[b, j // 64], h, j % 64] for j in middle])
                    key = np.where(np.isnan(m), np.inf, m) + 0.0
                    # NaN above infinity, then greater masses, then earlier tokens
                    order = sorted(range(len(middle)), key=lambda i: (not np.isnan(m[i]), -key[i], i))
                    keep = sorted(list(range(sinks)) + list(range(n - recent, n)) + [int(middle[i]) for i in order[:budget - sinks - recent]])
                for r, j in enumerate(keep):
                    p0, t0, t1 = self.table[b, j // 64], j % 64, r % 64
                    p1 = (self.table if into is None else into)[b, r // 64]
                    row = lambda x, t: slice(x + t * d // 2, x + (t + 1) * d // 2)  # noqa: E731
                    new_pages[p1, h, row(0, ref.rho(t1))] = pages[p0, h, row(0, ref.rho(t0))]
                    v = pages[p0, h, row(at, t0)]
                    new_pages[p1, h, row(at, t1)] = np.roll(v, d // 4) if d == 128 and (t0 ^ t1) & 2 else v
                    par = lambda t: slice(2 * at + 8 * ref.rho(t), 2 * at + 8 * ref.rho(t) + 8)  # noqa: E731
                    new_pages[p1, h, par(t1)] = pages[p0, h, par(t0)]
                    new_mass[p1, h, t1] = mass[p0, h, t0]
        return new_pages, new_mass, lens

    def check(self, mass, budget, limit, sinks, recent, into=None, **kw):
        pages = self.cache.pages.cpu().numpy().reshape(self.n_pages, self.heads, -1).copy()
        want = self.expect(pages, mass, budget, limit, sinks, recent, into)
        m = torch.tensor(mass).cuda()
        got = binding.kv4_evict(self.cache, self.batch([0] * len(self.kv), self.kv), m, budget, limit=limit, sinks=sinks, recent=recent,
                                into=None if into is None else torch.tensor(into, device="cuda"), **kw)
        assert got.tolist() == want[2]
        assert np.array_equal(m.cpu().numpy().view(np.uint32), want[1].view(np.uint32)), "masses"
        assert np.array_equal(self.cache.pages.cpu().numpy().reshape(pages.shape), want[0]), "pages"


KINDS = ["any", "equal", "few values", "odd", "rising", "wide"]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,heads,kv", [(64, 2, [200]), (128, 3, [130, 64, 65, 0, 1, 700])])
@pytest.mark.parametrize("budget,limit,sinks,recent", [(64, 64, 0, 0), (100, 129, 4, 20), (65, 65, 65, 0), (33, 64, 0, 33), (50, 50, 3, 46), (1, 1, 0, 0),
                                                       (128, 199, 1, 0)])
def test_in_place(cuda_lib, kind, dim, heads, kv, budget, limit, sinks, recent):
    w = Evict([0] * len(kv), kv, heads, dim, seed=budget + dim).fill()
    w.check(w.masses(kind), budget, limit, sinks, recent)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,heads,kv", [(128, 2, [200, 63]), (64, 3, [130, 64, 65, 0, 1, 700])])
@pytest.mark.parametrize("budget,limit,sinks,recent", [(64, 64, 0, 0), (100, 129, 4, 20), (33, 64, 0, 33), (1, 700, 0, 0)])
def test_into_other_pages(cuda_lib, kind, dim, heads, kv, budget, limit, sinks, recent):
    keeps = [n if n <= limit else budget for n in kv]
    spare = sum(-(-n // 64) for n in keeps)
    w = Evict([0] * len(kv), kv, heads, dim, seed=budget + dim, extra_pages=2 + spare).fill()
    free = sorted(set(range(w.n_pages)) - {int(w.table[b, p]) for b, n in enumerate(kv) for p in range(-(-n // 64))})
    wide = -(-min(limit, w.wide * 64) // 64)
    into = np.full((len(kv), wide), -5, np.int32)
    for b, n in enumerate(keeps):
        for p in range(-(-n // 64)):
            into[b, p] = free.pop(w.rng.integers(len(free)))
    w.check(w.masses(kind), budget, limit, sinks, recent, into)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["any", "few values", "rising", "equal"])
@pytest.mark.parametrize("kv,budget,sinks,recent", [([9000, 100], 2100, 4, 256), ([5000], 4999, 0, 0), ([70000], 70, 2, 5), ([2500, 2600], 2049, 1000, 1000)])
def test_long_sequences(cuda_lib, kind, kv, budget, sinks, recent):
    w = Evict([0] * len(kv), kv, 1, 64, seed=budget)
    # pages of any bytes: the call does not look at them
    w.cache.pages.copy_(torch.tensor(w.rng.integers(0, 256, size=w.cache.pages.numel(), dtype=np.uint8)))
    w.check(w.masses(kind), budget, budget, sinks, recent)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["any", "few values"])
@pytest.mark.parametrize("heads,kv,budget,sinks,recent", [(2, [50000, 49999, 7], 20000, 4, 256), (5, [60001], 1030, 0, 1000), (1, [330000], 2000, 4, 64)])
def test_very_long_sequences(cuda_lib, kind, heads, kv, budget, sinks, recent):
    """Clusters of sixteen blocks; at last runs too long for their blocks' shared memory."""
    w = Evict([0] * len(kv), kv, heads, 64, seed=budget)
    w.cache.pages.copy_(torch.tensor(w.rng.integers(0, 256, size=w.cache.pages.numel(), dtype=np.uint8)))
    w.check(w.masses(kind), budget, budget, sinks, recent)


@pytest.mark.gpu
def test_lengths_in_place_for_the_last_layer(cuda_lib):
    """Layers that share their lengths: each is cut by the old ones, the last call writes the new ones over them."""
    kv, n = [300, 90, 131], 100
    layers = [Evict([0] * 3, kv, 2, 64, seed=9).fill() for _ in range(2)]
    mass = layers[0].masses("any")
    want = [w.expect(w.cache.pages.cpu().numpy().reshape(w.n_pages, 2, -1), mass, n, n, 2, 10) for w in layers]
    b, got = layers[0].batch([0] * 3, kv), [torch.tensor(mass).cuda() for _ in layers]
    cu_q = torch.full((4,), 1 << 30, dtype=torch.int32, device="cuda")  # not looked at
    b = binding.KV4Batch(cu_q, b.kv_len, b.page_table, 3, 1, b.max_kv)
    for i, w in enumerate(layers):
        r = binding.kv4_evict(w.cache, b, got[i], n, sinks=2, recent=10, new_len=b.kv_len if i else None)
        assert r.tolist() == [100, 90, 100]
        assert np.array_equal(w.cache.pages.cpu().numpy().reshape(w.n_pages, 2, -1), want[i][0]) and np.array_equal(got[i].cpu().numpy(), want[i][1])
    assert b.kv_len.tolist() == [100, 90, 100]


@pytest.mark.gpu
def test_captured_and_on_a_stream(cuda_lib):
    kv = [500, 64]
    w = Evict([0, 0], kv, 2, 128, seed=4).fill()
    start, mass = w.cache.pages.clone(), w.masses("any")
    m, b = torch.tensor(mass).cuda(), w.batch([0, 0], kv)
    w.check(mass, 90, 100, 4, 16)
    done, length = w.cache.pages.clone(), torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.empty(binding.kv4_evict_workspace_size(w.cache, b, 90), dtype=torch.uint8, device="cuda").fill_(255)
    binding.kv4_evict(w.cache, b, m, 90, limit=100, sinks=4, recent=16, new_len=length, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.kv4_evict(w.cache, b, m, 90, limit=100, sinks=4, recent=16, new_len=length, workspace=ws)
    w.cache.pages.copy_(start), m.copy_(torch.tensor(mass)), length.zero_()
    graph.replay()
    assert torch.equal(w.cache.pages, done) and length.tolist() == [90, 64]
    # once it has been cut, nothing is left to do
    b.kv_len.copy_(length)
    graph.replay()
    assert torch.equal(w.cache.pages, done) and length.tolist() == [90, 64]
    w.cache.pages.copy_(start), m.copy_(torch.tensor(mass)), b.kv_len.copy_(i32(kv))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = binding.kv4_evict(w.cache, b, m, 90, limit=100, sinks=4, recent=16, stream=s)
    s.synchronize()
    assert torch.equal(w.cache.pages, done) and r.tolist() == [90, 64]


@pytest.mark.gpu
@pytest.mark.parametrize("kv,entry", [([10 ** 6, 100], None), ([-1, 100], None), ([300, 100], 10 ** 6), ([300, 100], -2)])
def test_bad_batches_are_reported_and_stay_inside(cuda_lib, kv, entry):
    w = Evict([0, 0], [300, 100], 2, 64, seed=4).fill()
    mass = w.masses("any")
    pages = w.cache.pages.cpu().numpy().reshape(w.n_pages, 2, -1).copy()
    want = w.expect(pages, mass, 80, 80, 0, 0)
    mine = [int(p) for p in w.table[0]]
    if entry is not None:
        w.table[0, 2] = entry
    m, b = torch.tensor(mass).cuda(), w.batch([0, 0], kv)
    got = binding.kv4_evict(w.cache, b, m, 80)
    assert binding.last_device_error() == binding.BITNET_ERANGE
    other = np.ones(w.n_pages, bool)
    other[mine] = False
    assert np.array_equal(w.cache.pages.cpu().numpy().reshape(pages.shape)[other], want[0][other])
    assert np.array_equal(m.cpu().numpy()[other], want[1][other]) and got.tolist() == [kv[0] if entry is None else 80, 80]


@pytest.mark.gpu
def test_bad_pages_to_write_to_are_left_out(cuda_lib):
    w = Evict([0], [100], 2, 64, seed=4, extra_pages=3).fill()
    mass, pages = w.masses("any"), w.cache.pages.clone()
    m = torch.tensor(mass).cuda()
    binding.kv4_evict(w.cache, w.batch([0], [100]), m, 80, into=i32([[w.n_pages, -1]]))
    assert binding.last_device_error() == binding.BITNET_ERANGE
    assert torch.equal(w.cache.pages, pages) and np.array_equal(m.cpu().numpy(), mass)


@pytest.mark.gpu
def test_shorter_sequences_that_do_not_fit_are_reported(cuda_lib):
    """`into` has room for those that are cut; one that keeps all its tokens has more."""
    w = Evict([0, 0], [300, 150], 2, 64, seed=4, extra_pages=6).fill()
    free = sorted(set(range(w.n_pages)) - set(w.table[w.table >= 0].tolist()))
    into = np.array([free[:2], free[2:4]], np.int32)
    mass, pages = w.masses("any"), w.cache.pages.cpu().numpy().reshape(w.n_pages, 2, -1).copy()
    m = torch.tensor(mass).cuda()
    got = binding.kv4_evict(w.cache, w.batch([0, 0], w.kv), m, 80, limit=200, into=torch.tensor(into, device="cuda"))
    assert binding.last_device_error() == binding.BITNET_ERANGE
    w.kv[1] = 0  # as if it were not there
    want = w.expect(pages, mass, 80, 200, 0, 0, into)
    assert np.array_equal(w.cache.pages.cpu().numpy().reshape(pages.shape), want[0]) and np.array_equal(m.cpu().numpy(), want[1])
    assert got.tolist() == [80, 150]


@pytest.mark.gpu
def test_refusals_of_the_binding(cuda_lib):
    w = Evict([0], [100], 2, 64, seed=4).fill()
    m, b = torch.tensor(w.masses("any")).cuda(), w.batch([0], [100])
    for kw in (dict(into=i32([1, 2])), dict(into=i32([[1, 2]]).long()), dict(into=i32([[1, 2], [1, 2]])), dict(new_len=i32([1, 2])),
               dict(new_len=i32([1]).cpu()), dict(workspace=torch.empty(1 << 16, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            binding.kv4_evict(w.cache, b, m, 80, **kw)
    for args, kw in (((0,), {}), ((80,), dict(limit=79)), ((80,), dict(sinks=81)), ((80,), dict(into=i32([[1]]))), ((65,), dict(into=i32([[1]]))),
                     ((80,), dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(binding.BitnetError):
            binding.kv4_evict(w.cache, b, m, *args, **kw)
    with pytest.raises(ValueError):
        binding.kv4_evict(w.cache, b, m[:1], 80)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
def test_steps_of_gathering_and_cutting(cuda_lib, dim):
    """As they are used: append, gather, cut, attend. What is attended to is what the cut cache reads back as."""
    rng = np.random.default_rng(dim)
    kv, heads, share = [200, 90], 2, 4
    w = Evict([0, 0], kv, heads, dim, seed=dim).fill()
    mass, length = binding.kv4_mass(w.cache), i32(kv)
    table, cu = torch.tensor(w.table, device="cuda"), i32([0, 1, 2])
    tokens = lambda h: torch.tensor(rng.normal(size=(2, h, dim))).bfloat16().cuda()  # noqa: E731
    one = binding.KV4Batch(cu, length, table, 2, 1, w.wide * 64)
    for step in range(12):
        length += 1
        binding.kv4_append(w.cache, one, tokens(heads), tokens(heads))
        q = tokens(heads * share)
        binding.kv4_attention_mass(w.cache, one, q, dim ** -0.5, mass, decay=0.95)
        before = length.tolist()
        binding.kv4_evict(w.cache, one, mass, 80, limit=95, sinks=2, recent=8, new_len=length)
        now = length.tolist()
        assert now == [80 if n > 95 else n for n in before]
        k, v = binding.kv4_read(w.cache, binding.KV4Batch(i32(np.cumsum([0] + now)), length, table, sum(now), max(now)), torch.float32)
        got = binding.kv4_attention(w.cache, one, q, dim ** -0.5).double().cpu().numpy()
        at = 0
        for b, n in enumerate(now):
            o, av, size = ref.attention(q[b:b + 1].float().cpu().numpy(), k[at:at + n].double().cpu().numpy(), v[at:at + n].double().cpu().numpy(),
                                        np.array([n - 1]), dim ** -0.5, 0, 0)
            d = dim ** -0.5 * size * (2.0 ** -11 + 2.0 ** -16)
            bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2.0 ** -24 + np.expm1(2 * d)[..., None]) * av * 1.01 + 1e-30
            assert (np.abs(got[b:b + 1] - o) <= bound).all()
            at += n
    gained = [float(mass[torch.tensor(w.table[b]).cuda().long()[torch.arange(n, device="cuda") // 64], 0, torch.arange(n, device="cuda") % 64].sum())
              for b, n in enumerate(length.tolist())]
    assert all(0 < g < 12 * share + 1 for g in gained)
