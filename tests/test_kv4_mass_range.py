"""The attention weight that cached tokens gather, at the ends of the numbers' ranges, in every form that the call takes: a
cluster a sequence and head (up to 16 columns), two kernels (the same, longer), two that make the scores twice (the same, of
batches with room for very many tokens), blocks of 64 columns (up to 96 rows), blocks of 128 rows."""
import numpy as np
import pytest
import torch

import kv4_reference as ref
from test_kv4_mass import Mass, cuda_lib, lib  # noqa: F401 (fixtures)
from ternary_weight_gb300 import binding

# new tokens and cached ones of each sequence: query heads that share a key/value head are two
ROOM = 1 << 25
FORMS = {"cluster": ([1, 3], [77, 130]), "two kernels": ([1, 3], [900, 1500]), "scores twice": ([1, 3], [900, 1501]), "64 columns": ([20, 33], [77, 1500]), "128 rows": ([70, 130], [90, 1500])}


def batch_of(w, form):
    if form != "scores twice":
        return w.batch(w.new, w.kv)
    table = torch.full((len(w.kv), ROOM // 64), -7, dtype=torch.int32, device="cuda")
    table[:, :w.wide] = torch.tensor(w.table)
    b = w.batch(w.new, w.kv)
    return binding.KV4Batch(b.cu_q, b.kv_len, table, sum(w.new), max(w.new), ROOM)


def gather(w, form, q, mass, scale=None, **kw):
    return binding.kv4_attention_mass(w.cache, batch_of(w, form), q, w.dim ** -0.5 if scale is None else scale, mass, **kw)


def seen_by(w, b, row):
    """Tokens that the row-th new token of sequence b sees."""
    return w.kv[b] - w.new[b] + row + 1


@pytest.mark.gpu
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (64, "f32"), (128, "bf16"), (128, "f32")])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
def test_a_query_that_is_not_finite(cuda_lib, dim, dtype, form, what):
    """It reaches the tokens that its row sees, of its head alone. Keys are above 0 with a code above 0 at the query's place, so
    that -inf makes every score -inf."""
    new, kv = FORMS[form]
    w = Mass(new, kv, 2, dim, dtype, seed=dim)
    for k in w.k:
        k[:] = np.abs(k) + 0.5
        k[:, :, 5] = k.max() + 1.0
    w.fill()
    mass, q = w.start(), w.queries(2)
    row = new[1] - 2  # of sequence 1
    q[new[0] + row, 3, 5] = what
    got = gather(w, form, q, mass).cpu().numpy()
    for b in range(2):
        j = np.arange(kv[b])
        want = np.zeros((kv[b], 2), bool)
        if b == 1:
            want[:seen_by(w, 1, row), 1] = True
        assert np.array_equal(np.isnan(got[w.table[b][j // 64], :, j % 64]), want)


def check_winners(w, q, share, scale, got):
    """Scores so far apart that a row's vote goes to one token. Scores of the call are off by
    e = scale (D + 16) 2^-23 max_j (step sum code |q| + |base| sum |q|) at most; a token whose score is 2 e + 64 below the greatest one
    has less than exp(-64). Where only one is not, the row's whole vote is its; where more are, any of them may have it.
    got: of a call with decay 0."""
    got, q64, row = got.double().cpu().numpy(), q.double().cpu().numpy(), 0
    sure_rows = 0
    for b, n in enumerate(w.new):
        j = np.arange(w.kv[b])
        code, step, base = (x.astype(np.float64) for x in ref.quantise(w.k[b]))
        step, base = step[..., None], base[..., None]
        for h in range(w.heads):
            least, most = np.zeros(w.kv[b]), np.zeros(w.kv[b])
            for a in range(h * share, (h + 1) * share):
                x = q64[row:row + n, a]
                sees = j[None] <= np.arange(w.kv[b] - n, w.kv[b])[:, None]
                s = np.where(sees, scale * x @ (step[:, h] * code[:, h] + base[:, h]).T, -np.inf)
                size = (np.abs(x) @ (step[:, h] * code[:, h]).T + np.abs(x).sum(1, keepdims=True) * np.abs(base[:, h]).T) * sees
                e = abs(scale) * (w.dim + 16) * 2.0 ** -23 * size.max(1, keepdims=True)
                near = s >= s.max(1, keepdims=True) - 2 * e - 64
                most += near.sum(0)
                least += (near & (near.sum(1, keepdims=True) == 1)).sum(0)
            have = got[w.table[b][j // 64], h, j % 64]
            slack = n * share * ((w.kv[b] + n * share + 32) * 2.0 ** -23 + np.exp(-64.0))
            assert (have >= least - slack).all() and (have <= most + slack).all()
            assert abs(have.sum() - n * share) <= slack * 2  # its own sum over the tokens is off by their rounding too
            sure_rows += least.sum()
        row += n
    assert sure_rows > sum(w.new) * w.heads * share / 2  # else the check says little


@pytest.mark.gpu
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (64, "f32"), (128, "bf16"), (128, "f32")])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("power,above", [(60, False), (118, False), (124, True), (125, False)])
def test_queries_up_to_the_greatest_numbers(cuda_lib, dim, dtype, form, power, above):
    """above: all numbers of a query above 0, so that their sum passes the range."""
    new, kv = FORMS[form]
    w = Mass(new, kv, 2, dim, dtype, seed=dim + power).fill()
    mass, q = w.start(), w.queries(2, 1.0)
    q = (q.abs() if above else q) * 2.0 ** power
    assert bool(q.isfinite().all())
    check_winners(w, q, 2, dim ** -0.5, gather(w, form, q, mass, decay=0.0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("scale,power", [(3e38, 0), (-3e38, 0), (-1e10, 3), (1e38, 30)])
def test_the_greatest_scales(cuda_lib, dtype, form, scale, power):
    new, kv = FORMS[form]
    w = Mass(new, kv, 2, 64, dtype, seed=power + 5).fill()
    mass, q = w.start(), w.queries(2, 2.0 ** power)
    scale = float(np.float32(scale))
    got = gather(w, form, q, mass, scale, decay=0.0)
    check_winners(w, q, 2, scale, got)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("scale,power", [(-64 ** -0.5, 0), (0.0, 0), (-0.0, 0), (1e-38, 0), (2.0 ** 120, -122), (-2.0 ** 120, -122), (2.0 ** -122, 118), (1e-40, 0)])
def test_scales_of_every_size_and_sign(cuda_lib, dtype, form, scale, power):
    """With queries of such a size that many tokens have weight."""
    new, kv = FORMS[form]
    w = Mass(new, kv, 2, 64, dtype, seed=7).fill()
    mass, q = w.start(), w.queries(2, 1.5 * 2.0 ** power)
    scale = float(np.float32(scale))
    got = gather(w, form, q, mass, scale, decay=0.5)
    w.check(got, q, 2, scale, 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (64, "f32"), (128, "bf16"), (128, "f32")])
@pytest.mark.parametrize("new,kv", [([140, 60], [3000, 5000]), ([400], [400]), ([49], [9001])])
@pytest.mark.parametrize("size", [0.0, 1.5, 60.0, 4000.0, 1e6, 1e20])
def test_many_rows_give_one_vote_each(cuda_lib, dim, dtype, new, kv, size):
    """Blocks of 128 rows: rows are the product's rows where maxima and sums are found, and its columns where votes are added up. Both
    have to make the same scores: a difference in the last place of great ones would show as votes lost or won. What is left are
    the roundings of exponentials and sums."""
    w = Mass(new, kv, 2, dim, dtype, seed=dim + int(min(size, 1e6))).fill()
    mass, q = w.start(), w.queries(2, size)
    got = gather(w, "128 rows", q, mass, decay=0.0).double().cpu().numpy()
    for b, n in enumerate(new):
        j = np.arange(kv[b])
        votes = got[w.table[b][j // 64], :, j % 64].sum(0)
        assert (np.abs(votes - 2 * n) <= 2 * n * (kv[b] + 2 * n + 32) * 2.0 ** -23).all()
