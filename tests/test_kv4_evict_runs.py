"""Eviction of sequences whose runs are longer than what a block keeps in shared memory, and by clusters into other pages:
byte for byte against plain numpy, also where a table names pages that are not in the pool."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_reference as ref
from ternary_weight_gb300 import _build, binding


@pytest.mark.parametrize("to,want", [(0, -2), (4 * 8, -2), (-4 * 8, -2), (4, -1), (-4, -1), (4 * 7, -1), (-4 * 7, -1)])
def test_new_lengths_over_those_of_other_sequences_are_refused(to, want):
    """Over the old lengths themselves, or apart from them. (Calls that pass this check are refused for their masses' alignment.)"""
    _build.build()
    at = 1 << 20
    c, b = binding._KV4CacheDesc(at, 4, 2, 128), binding._KV4BatchDesc(at, at, at, 8, 2, 0, 1, 128)
    assert binding.lib().bitnet_kv4_evict(ctypes.byref(c), ctypes.byref(b), at + 4, 50, 60, 4, 10, None, 0, at + to, at, 1 << 40, None) == want


@pytest.fixture
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.fail("gpu tests need a CUDA device")
    _build.build()
    binding.lib()
    yield
    assert binding.last_device_error() == 0, "a kernel recorded a device-side error"


class Pool:
    """Sequences of these lengths in pages of any bytes (the call does not look at them), with masses."""

    def __init__(self, kv, heads, dim, seed, spare=0, kind="any"):
        rng = self.rng = np.random.default_rng(seed)
        self.kv, self.heads, self.dim = kv, heads, dim
        need = [-(-n // 64) for n in kv]
        self.n_pages = sum(need) + spare + 1
        ids = rng.permutation(self.n_pages)
        self.table = np.full((len(kv), max(need)), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.free = ids[at:].tolist()
        g = torch.Generator(device="cuda").manual_seed(seed)
        size = binding.kv4_cache_bytes(self.n_pages, heads, dim)
        self.pages = torch.randint(0, 256, (size,), generator=g, dtype=torch.uint8, device="cuda")
        self.cache = binding.KV4Cache(self.n_pages, heads, dim, pages=self.pages)
        m = rng.random((self.n_pages, heads, 64))
        if kind == "equal":
            m = np.ones(m.shape)
        elif kind == "few values":
            m = np.floor(m * 4) * 0.25
        self.mass = m.astype(np.float32)

    def into(self, pages):
        return np.array([[self.free.pop() for _ in range(pages)] for _ in self.kv], np.int32)

    def expect(self, budget, sinks, recent, into=None, table=None):
        """(pages, masses, lengths) as the call leaves them; table: where the kept tokens are looked up (default: the sequences')."""
        d, half = self.dim, np.arange(self.dim // 2)
        old = self.pages.cpu().numpy().reshape(self.n_pages, self.heads, -1)
        new, mass, lens = old.copy(), self.mass.copy(), []
        for b, n in enumerate(self.kv):
            lens.append(min(n, budget))
            if n <= budget and into is None:
                continue
            for h in range(self.heads):
                j = np.arange(n)
                if n > budget:
                    mid = j[sinks:n - recent]
                    m = self.mass[self.table[b, mid // 64], h, mid % 64]
                    best = mid[np.lexsort((mid, -m))[:budget - sinks - recent]]
                    j = np.sort(np.concatenate([j[:sinks], best, j[n - recent:]]))
                r = np.arange(len(j))
                p0, t0, p1, t1 = self.table[b, j // 64], j % 64, (self.table if into is None else into)[b, r // 64], r % 64
                cols = lambda at, row, width: at + row[:, None] * width + np.arange(width)  # noqa: E731
                new[p1[:, None], h, cols(0, ref.rho(t1), d // 2)] = old[p0[:, None], h, cols(0, ref.rho(t0), d // 2)]
                turn = ((t0 ^ t1) & 2 > 0) & (d == 128)  # the halves of a wide value row
                v = old[p0[:, None], h, 32 * d + t0[:, None] * (d // 2) + (half + np.where(turn, d // 4, 0)[:, None]) % (d // 2)]
                new[p1[:, None], h, cols(32 * d, t1, d // 2)] = v
                new[p1[:, None], h, cols(64 * d, ref.rho(t1), 8)] = old[p0[:, None], h, cols(64 * d, ref.rho(t0), 8)]
                mass[p1, h, t1] = self.mass[p0, h, t0]
        return new, mass, lens

    def call(self, budget, sinks, recent, into=None, table=None):
        """The call's (pages, masses, lengths)."""
        t = torch.tensor(self.table if table is None else table, device="cuda")
        n = torch.tensor(self.kv, dtype=torch.int32, device="cuda")
        b = binding.KV4Batch(torch.zeros(len(self.kv) + 1, dtype=torch.int32, device="cuda"), n, t, 0, 1, 64 * self.table.shape[1])
        m = torch.tensor(self.mass).cuda()
        # what a workspace held before is no token
        ws = torch.empty(binding.kv4_evict_workspace_size(self.cache, b, budget), dtype=torch.uint8, device="cuda").fill_(0x7f)
        got = binding.kv4_evict(self.cache, b, m, budget, sinks=sinks, recent=recent, into=None if into is None else torch.tensor(into, device="cuda"),
                                workspace=ws)
        return self.pages.cpu().numpy().reshape(self.n_pages, self.heads, -1), m.cpu().numpy(), got.tolist()


# more than 152 units: a block each, whose runs of 21 thousand tokens keep no ranks, and of 33 thousand no ballots either
LONG = [33000, 40001, 21000] + [40 + 9 * i for i in range(28)]


@pytest.mark.gpu
def test_bad_pages_in_long_runs_stay_inside(cuda_lib):
    """A page outside the pool has tokens without any mass; it is reported, and the other sequences are what they would have been."""
    w = Pool(LONG, 5, 64, seed=5)
    want = w.expect(300, 4, 60)
    table = w.table.copy()
    table[0, 100:400] = w.rng.choice([-1, w.n_pages, 1 << 30], size=300)
    got = w.call(300, 4, 60, table=table)
    assert binding.last_device_error() == binding.BITNET_ERANGE
    mine = np.zeros(w.n_pages, bool)
    mine[w.table[0]] = True
    assert got[2] == want[2] and np.array_equal(got[0][~mine], want[0][~mine]) and np.array_equal(got[1][~mine], want[1][~mine])


def check(w, *args):
    want = w.expect(*args)
    got = w.call(*args)
    assert got[2] == want[2] and np.array_equal(got[1].view(np.uint32), want[1].view(np.uint32)) and np.array_equal(got[0], want[0])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["any", "equal", "few values"])
@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("budget,sinks,recent", [(300, 4, 60), (20900, 0, 20000)])
def test_runs_longer_than_shared_memory(cuda_lib, kind, other, budget, sinks, recent):
    w = Pool(LONG, 5, 64, seed=budget, kind=kind, spare=len(LONG) * -(-budget // 64) if other else 0)
    check(w, budget, sinks, recent, w.into(-(-budget // 64)) if other else None)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["any", "equal"])
@pytest.mark.parametrize("dim,heads,kv,budget,sinks,recent", [(128, 2, [9000, 100], 2100, 4, 256), (64, 1, [70000], 70, 2, 5), (64, 5, [131007, 4], 4096, 4, 1024),
                                                              (128, 1, [5000, 2600], 2500, 0, 0), (64, 1, [60001], 60000, 1, 1)])
def test_clusters_into_other_pages(cuda_lib, kind, dim, heads, kv, budget, sinks, recent):
    w = Pool(kv, heads, dim, seed=budget, kind=kind, spare=len(kv) * -(-budget // 64))
    check(w, budget, sinks, recent, w.into(-(-budget // 64)))
