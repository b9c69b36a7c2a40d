"""The attention weight that cached tokens gather, against plain 64-bit numpy.

The bound of a token's votes v (a sum over R rows and heads, of softmax weights over at most n positions). A score's fp32
sums and its query's two fp16 parts (fp32 queries) leave e = scale (D + 16) 2^-23 max_j (step sum code |q| + |base| sum |q|); a weight is
then off by a factor within exp(+-2 e); exponentials by 2^-21, the sum of a row's exponentials by n 2^-24 at most, the
sum of the votes by R 2^-24:  v (expm1(2 e) + (n + R + 32) 2^-23). The last multiply-add rounds once more. Weights below
fp32's normal range may be lost: R 2^-125.
"""
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
def cache(**kw):
    return binding._KV4CacheDesc(**{**dict(pages=FAKE, n_pages=4, kv_heads=2, head_dim=128), **kw})


def batch(**kw):
    return binding._KV4BatchDesc(**{**dict(cu_q=FAKE, kv_len=FAKE, page_table=FAKE, batch=2, max_pages=2, total_q=0, max_q=2, max_kv=128), **kw})


def call(lib, c=None, b=None, **kw):
    a = {**dict(q=FAKE, dtype=1, heads=8, qs=1024, scale=0.1, window=0, sinks=0, voters=0, decay=1.0, mass=FAKE, out=FAKE, ws=FAKE, ws_bytes=1 << 40), **kw}
    return lib.bitnet_kv4_attention_mass(ctypes.byref(c or cache()), ctypes.byref(b or batch()), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    ({}, 0), (dict(q=None), -1), (dict(dtype=2), -1), (dict(heads=7), -1), (dict(heads=0), -1), (dict(heads=258), -1), (dict(qs=1023), -1), (dict(qs=1028), -2),
    (dict(scale=float("nan")), -1), (dict(window=-1), -1), (dict(window=1 << 31), -1), (dict(sinks=-1), -1), (dict(voters=-1), -1),
    (dict(voters=1 << 31), -1), (dict(decay=float("inf")), -1), (dict(mass=None), -1), (dict(out=None), -1), (dict(ws=None), -1), (dict(ws_bytes=0), -1),
    (dict(mass=FAKE + 4, out=FAKE + 4), -2), (dict(out=FAKE + 4 * 2 * 256 + 8), -2),
    (dict(out=FAKE + 16), -1), (dict(out=FAKE - 16), -1), (dict(out=FAKE + 4 * 2 * 256 - 16), -1), (dict(ws=FAKE + 128), -2), (dict(q=FAKE + 8), -2)])
def test_bad_calls_are_refused(lib, kw, want):
    b = batch(total_q=3, max_pages=1 << 16, max_kv=1 << 22) if want else batch()  # long enough for a workspace
    assert call(lib, b=b, **kw) == want


@pytest.mark.parametrize("c,b,want", [(dict(pages=None), {}, -1), (dict(head_dim=96), {}, -1), (dict(pages=FAKE + 8), {}, -2), ({}, dict(cu_q=None), -1),
                                      ({}, dict(max_kv=129), -1), ({}, dict(batch=0), -1), ({}, dict(kv_len=FAKE + 1), -2)])
def test_bad_caches_and_batches_are_refused(lib, c, b, want):
    assert call(lib, cache(**c), batch(**b)) == want
    assert lib.bitnet_kv4_attention_mass_workspace_size(ctypes.byref(cache(**c)), ctypes.byref(batch(**b)), 8, 0) == want


def test_sizes(lib):
    assert lib.bitnet_kv4_mass_bytes(3, 5) == 3 * 5 * 256 and lib.bitnet_kv4_mass_bytes(0, 5) == -1 and lib.bitnet_kv4_mass_bytes(1, 1025) == -1
    size = lambda heads, voters: lib.bitnet_kv4_attention_mass_workspace_size(ctypes.byref(cache()), ctypes.byref(batch(total_q=3)), heads, voters)  # noqa: E731
    large = batch(total_q=(1 << 30) - 64, max_q=(1 << 30) - 64)
    assert lib.bitnet_kv4_attention_mass_workspace_size(ctypes.byref(cache()), ctypes.byref(large), 4, 1) == -1
    assert call(lib, b=large, heads=4) == -1
    assert size(8, 0) >= 0 and size(8, 5) >= 0 and size(7, 0) == -1 and size(8, -1) == -1


# ------------------------------------------------------------------- on the GPU
class Mass(World):
    """A cache with masses beside it: what is not a cached token's has NaN, and so have the call's own tokens."""

    def start(self):
        self.mass = np.full((self.n_pages, self.heads, 64), np.nan, np.float32)
        for b in range(len(self.kv)):
            for j in range(self.kv[b] - self.new[b]):
                self.mass[self.table[b, j // 64], :, j % 64] = self.rng.random(self.heads) * 0.1
        return torch.tensor(self.mass).cuda()

    def queries(self, share, size=1.5, pad=0):
        n = sum(self.new)
        x = torch.tensor(self.rng.normal(size=(n, self.heads * share * self.dim + pad)) * size).to(self.dtype).cuda()
        return x[:, :self.heads * share * self.dim].unflatten(1, (self.heads * share, self.dim))

    def check(self, got, q, share, scale, decay=1.0, window=0, sinks=0, voters=0):
        decay = float(np.float32(decay))  # the call takes it as fp32
        got, q64, row = got.double().cpu().numpy(), q.double().cpu().numpy(), 0
        want, bound = self.mass.astype(np.float64), np.zeros(self.mass.shape)
        for b, n in enumerate(self.new):
            row += n
            if n == 0:
                continue
            length, votes = self.kv[b], min(n, voters) if voters else n
            pos, j = np.arange(length - votes, length), np.arange(length)
            sees = j[None] <= pos[:, None]
            if window:
                sees &= (j[None] > pos[:, None] - window) | (j[None] < sinks)
            code, step, base = ref.quantise(self.k[b])
            step, base = step.astype(np.float64)[..., None], base.astype(np.float64)[..., None]
            for h in range(self.heads):
                total, off = np.zeros(length), np.zeros(length)
                for a in range(h * share, (h + 1) * share):
                    x = q64[row - votes:row, a]
                    s = np.where(sees, scale * x @ (step[:, h] * code[:, h] + base[:, h]).T, -np.inf)
                    some = sees.any(1)
                    p = np.zeros(s.shape)
                    with np.errstate(invalid="ignore"):
                        p[some] = np.exp(s[some] - s[some].max(1, keepdims=True))
                        p[some] /= p[some].sum(1, keepdims=True)
                    size = (np.abs(x) @ (step[:, h] * code[:, h]).T + np.abs(x).sum(1, keepdims=True) * np.abs(base[:, h]).T) * sees
                    e = abs(scale) * (self.dim + 16) * 2.0 ** -23 * size.max(1, keepdims=True)
                    total += p.sum(0)
                    off += (p * (np.expm1(2 * e) + (sees.sum(1, keepdims=True) + votes * share + 32) * 2.0 ** -23)).sum(0)
                old = np.where(j < length - n, decay * self.mass[self.table[b][j // 64], h, j % 64].astype(np.float64), 0.0)
                want[self.table[b][j // 64], h, j % 64] = old + total
                bound[self.table[b][j // 64], h, j % 64] = off + 2.0 ** -24 * np.abs(old + total) + votes * share * 2.0 ** -125
        assert np.array_equal(np.isnan(got), np.isnan(want)), "NaN in the wrong places"
        err = np.abs(got - want)
        bad = ~np.isnan(want) & (err > bound)
        assert not bad.any(), "%d of %d off, worst %.3g of the bound, first %s" % (bad.sum(), bad.size, np.nanmax(err[bad] / bound[bad].clip(1e-60)), np.argwhere(bad)[0])


def gather(w, q, mass, **kw):
    return binding.kv4_attention_mass(w.cache, w.batch(w.new, w.kv), q, w.dim ** -0.5, mass, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("share", [1, 4, 5, 8])
@pytest.mark.parametrize("new,kv", [([1], [1]), ([1], [77]), ([1, 1, 1], [64, 65, 1000]), ([0, 1], [30, 129]), ([3, 7, 2], [3, 300, 66])])
def test_a_few_rows(cuda_lib, dim, dtype, share, new, kv):
    w = Mass(new, kv, 2, dim, dtype, seed=dim + sum(kv) + share).fill()
    mass, q = w.start(), w.queries(share)
    before = w.cache.pages.clone()
    got = gather(w, q, mass, decay=0.9)
    assert got is mass
    w.check(got, q, share, dim ** -0.5, 0.9)
    assert torch.equal(w.cache.pages, before)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,dtype,share", [(128, "bf16", 4), (64, "f32", 3), (128, "f32", 1), (64, "bf16", 16)])
@pytest.mark.parametrize("new,kv,voters", [([200], [200], 0), ([130, 1, 33], [400, 70, 33], 0), ([300, 20], [300, 520], 64), ([65, 129], [1500, 129], 1),
                                           ([257, 0, 5], [300, 10, 64], 17)])
def test_many_rows(cuda_lib, dim, dtype, share, new, kv, voters):
    w = Mass(new, kv, 2, dim, dtype, seed=dim + sum(kv) + share).fill()
    mass, q = w.start(), w.queries(share, pad=16)
    w.check(gather(w, q, mass, voters=voters), q, share, dim ** -0.5, voters=voters)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 0), (100, 4), (63, 70), (5000, 1), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("new,kv,dtype", [([1, 1], [500, 40], "bf16"), ([90, 5], [300, 700], "f32"), ([150], [1000], "bf16")])
def test_windows_and_first_tokens(cuda_lib, window, sinks, new, kv, dtype):
    w = Mass(new, kv, 1, 128, dtype, seed=window % 1000 + sum(kv)).fill()
    mass, q = w.start(), w.queries(4)
    w.check(gather(w, q, mass, decay=0.5, window=window, sinks=sinks), q, 4, 128 ** -0.5, 0.5, window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,share,dim", [(1, 128, 64), (5, 4, 128), (12, 1, 64), (1, 20, 128)])
@pytest.mark.parametrize("n,kv", [(1, 3000), (2, 190), (40, 200)])
def test_head_layouts(cuda_lib, heads, share, dim, n, kv):
    w = Mass([n], [kv], heads, dim, "bf16", seed=heads + n).fill()
    mass, q = w.start(), w.queries(share)
    w.check(gather(w, q, mass), q, share, dim ** -0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "f32")])
@pytest.mark.parametrize("share,n,kv,most_q,most_kv,window,sinks", [(32, 200, 200, 200, 80000, 0, 0), (32, 200, 260, 200, 80000, 90, 7), (32, 3, 4500, 64, 160000, 0, 0),
                                                                    (32, 4, 9000, 64, 160000, 4200, 130), (16, 8, 5000, 128, 160000, 64, 0)])
def test_batches_made_for_far_more(cuda_lib, dim, dtype, share, n, kv, most_q, most_kv, window, sinks):
    """Sizes of a batch are upper bounds: work is cut by them, and a block goes through more than 32 tiles or blocks of rows."""
    w = Mass([n], [kv], 1, dim, dtype, seed=kv + n).fill()
    mass, q = w.start(), w.queries(share)
    table = torch.full((1, -(-most_kv // 64)), -7, dtype=torch.int32, device="cuda")
    table[:, :w.wide] = torch.tensor(w.table)
    q_all = torch.cat([q, q.new_zeros((most_q - n, *q.shape[1:]))])
    b = binding.KV4Batch(i32([0, n]), i32([kv]), table, most_q, most_q, most_kv)
    got = binding.kv4_attention_mass(w.cache, b, q_all, dim ** -0.5, mass, window=window, sinks=sinks)
    w.check(got, q, share, dim ** -0.5, window=window, sinks=sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,dtype,share,longest", [(64, "bf16", 16, 1100), (64, "f32", 8, 9000), (128, "bf16", 16, 4500), (128, "bf16", 4, 300)])
def test_many_sequences(cuda_lib, dim, dtype, share, longest):
    """More units than fill the GPU, some of them long: clusters of one to eight blocks."""
    kv = [longest, 0, 1] + [1 + 37 * i % 200 for i in range(117)]
    w = Mass([int(n > 0) for n in kv], kv, 2, dim, dtype, seed=longest).fill()
    mass, q = w.start(), w.queries(share)
    w.check(gather(w, q, mass, decay=0.3), q, share, dim ** -0.5, 0.3)


@pytest.mark.gpu
def test_two_calls_at_once(cuda_lib):
    """Calls on two streams, and graphs of theirs replayed side by side: nothing of the calls is shared."""
    worlds = [Mass([n] * 3, [kv, 70, kv // 2], 2, 64, "bf16", seed=n).fill() for n, kv in ((1, 5000), (60, 3000), (1, 300), (9, 900))]
    starts = [(w.start(), w.queries(4)) for w in worlds]
    want = [gather(w, q, mass.clone()) for w, (mass, q) in zip(worlds, starts)]
    batches = [w.batch(w.new, w.kv) for w in worlds]
    outs, graphs, streams = [mass.clone() for mass, _ in starts], [], [torch.cuda.Stream() for _ in worlds]
    for w, (mass, q), b, out in zip(worlds, starts, batches, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            binding.kv4_attention_mass(w.cache, b, q, 64 ** -0.5, mass, out=out)
    for _ in range(3):
        for out, (mass, _) in zip(outs, starts):
            out.copy_(mass)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.nan_to_num(9.0), b.nan_to_num(9.0)) for a, b in zip(outs, want))


@pytest.mark.gpu
@pytest.mark.parametrize("size", [0.0, 60.0, 4000.0])
def test_scores_of_every_size(cuda_lib, size):
    """Zero queries vote evenly; great ones for one token alone (the bound then says little about the others, and they vote 0 or so)."""
    w = Mass([1, 40], [700, 300], 2, 64, "bf16", seed=3).fill()
    mass, q = w.start(), w.queries(2, size)
    got = gather(w, q, mass)
    w.check(got, q, 2, 64 ** -0.5)
    total = got.double().cpu().numpy()
    for b, votes in ((0, 1), (1, 40)):  # every row gives away one vote in all
        j = np.arange(w.kv[b])
        old = np.nan_to_num(w.mass[w.table[b][j // 64], :, j % 64].astype(np.float64)).sum(0)
        gained = total[w.table[b][j // 64], :, j % 64].sum(0) - old
        # both passes use the same scores: only the exponentials', the sums' and the last addition's roundings are left
        assert (np.abs(gained - votes * 2) <= votes * 2 * (w.kv[b] + votes * 2 + 32) * 2.0 ** -23 + 2.0 ** -24 * (old + votes * 2)).all()


@pytest.mark.gpu
def test_nan_reaches_what_its_row_sees(cuda_lib):
    w = Mass([1, 1, 70], [100, 90, 90], 2, 64, "f32", seed=5)
    w.k[1][3, 0, 5] = np.nan  # a key of sequence 1, head 0
    w.fill()
    mass, q = w.start(), w.queries(2)
    q[2 + 10, 3, 7] = float("nan")  # a query of sequence 2 at position 30, head 1
    got = gather(w, q, mass).cpu().numpy()
    for b in range(3):
        j = np.arange(w.kv[b])
        nan = np.isnan(got[w.table[b][j // 64], :, j % 64])
        want = np.zeros((w.kv[b], 2), bool)
        if b == 1:
            want[:, 0] = True
        if b == 2:
            want[:31, 1] = True
        assert np.array_equal(nan, want)


@pytest.mark.gpu
def test_more_new_tokens_than_cached_ones(cuda_lib):
    """Rows at negative positions see nothing and vote for nothing."""
    w = Mass([5], [3], 2, 64, "f32", seed=5).fill()
    w.new = [3]
    mass = w.start()
    w.new = [5]
    q = w.queries(2)
    got = gather(w, q, mass)
    w.new = [3]
    w.check(got, q[2:], 2, 64 ** -0.5)


@pytest.mark.gpu
def test_out_of_place_strided_captured_and_again(cuda_lib):
    w = Mass([1, 1], [300, 65], 5, 128, "bf16", seed=11).fill()
    mass, q = w.start(), w.queries(4, pad=64)
    keep = mass.clone()
    out = torch.full_like(mass, 3.0)
    got = gather(w, q, mass, decay=0.7, out=out)
    assert got is out and torch.equal(mass.nan_to_num(9.0), keep.nan_to_num(9.0))
    kept = out.clone()
    written = torch.zeros_like(out, dtype=torch.bool)
    for b in range(2):
        j = torch.arange(w.kv[b])
        written[torch.tensor(w.table[b])[j // 64].long().cuda(), :, (j % 64).cuda()] = True
    assert bool((out[~written] == 3.0).all())
    w.check(torch.where(written, out, torch.tensor(w.mass).cuda()), q, 4, 128 ** -0.5, 0.7)
    batch_ = w.batch(w.new, w.kv)
    ws = torch.empty(max(1, binding.kv4_attention_mass_workspace_size(w.cache, batch_, 20)), dtype=torch.uint8, device="cuda").fill_(255)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.kv4_attention_mass(w.cache, batch_, q, 128 ** -0.5, mass, decay=0.7, out=out, workspace=ws)
    for _ in range(2):
        out.fill_(3.0)
        graph.replay()
        assert torch.equal(out, kept)
    # as the sequences grow, the captured call reads the lengths anew
    batch_.kv_len -= 30
    graph.replay()
    w2 = Mass([1, 1], [270, 35], 5, 128, "bf16")
    w2.table, w2.k, w2.mass, w2.n_pages = w.table, [x[:n] for x, n in zip(w.k, w2.kv)], w.mass, w.n_pages
    first = torch.zeros_like(written)
    for b in range(2):
        j = torch.arange(w2.kv[b])
        first[torch.tensor(w.table[b])[j // 64].long().cuda(), :, (j % 64).cuda()] = True
    w2.check(torch.where(first, out, torch.tensor(w.mass).cuda()), q, 4, 128 ** -0.5, 0.7)


@pytest.mark.gpu
def test_on_a_stream(cuda_lib):
    w = Mass([1, 40], [300, 65], 2, 64, "bf16", seed=11).fill()
    mass, q = w.start(), w.queries(4)
    a, b = torch.zeros_like(mass), torch.zeros_like(mass)
    gather(w, q, mass, out=a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gather(w, q, mass, out=b, stream=s)
    s.synchronize()
    assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("kv,table", [([999999, 50], None), ([-4, 50], None), ([100, 50], 1 << 20), ([100, 50], -3)])
def test_bad_batches_are_reported_and_stay_inside(cuda_lib, kv, table):
    w = Mass([1, 1], [100, 50], 2, 64, "bf16", seed=11).fill()
    mass, q = w.start(), w.queries(2)
    want = gather(w, q, mass.clone())
    if table is not None:
        w.table[0, 1] = table
    got = binding.kv4_attention_mass(w.cache, w.batch([1, 1], kv), q, 64 ** -0.5, mass.clone())
    assert binding.last_device_error() == binding.BITNET_ERANGE
    # the other sequence, and the pages of none, are right
    mine = torch.ones(w.n_pages, dtype=torch.bool)
    own = [p for p in Mass([1, 1], [100, 50], 2, 64, "bf16", seed=11).table[0].tolist() if p >= 0]
    mine[own] = False
    assert torch.equal(got[mine].nan_to_num(9.0), want[mine].nan_to_num(9.0))


@pytest.mark.gpu
def test_refusals_of_the_binding(cuda_lib):
    w = Mass([1], [70], 2, 64, "bf16").fill()
    mass, q, b = w.start(), w.queries(2), w.batch([1], [70])
    call = lambda *a, **kw: binding.kv4_attention_mass(w.cache, b, *a, **kw)  # noqa: E731
    for bad in (mass[:1], mass.double(), mass.cpu(), mass.transpose(0, 2)):
        with pytest.raises(ValueError):
            call(q, 0.1, bad)
        with pytest.raises(ValueError):
            call(q, 0.1, mass, out=bad)
    for bad in (q.half(), q[0], q.cpu(), q[:, :, :32]):
        with pytest.raises(ValueError):
            call(bad, 0.1, mass)
    with pytest.raises(binding.BitnetError):
        call(q[:, :3].contiguous(), 0.1, mass)
    with pytest.raises(binding.BitnetError):
        call(q, 0.1, mass, voters=-1)
    assert binding.kv4_mass(w.cache).shape == mass.shape and not bool(binding.kv4_mass(w.cache).any())
    e = binding.KV4Batch(i32([0, 0]), i32([70]), torch.tensor(w.table, device="cuda"), 0, 1)
    assert binding.kv4_attention_mass(w.cache, e, q[:0], 0.1, mass) is mass
