"""The attention weight that cached tokens gather, at the ends of the numbers' ranges, in every form that the call takes: a
cluster a sequence and head (up to 16 columns), two kernels (the same, longer), blocks of 64 columns (up to 96 rows), blocks of
128 rows."""
import numpy as np
import pytest
import torch

from test_kv4_mass import Mass, cuda_lib, gather, lib  # noqa: F401 (fixtures)
from ternary_weight_gb300 import binding

# new tokens and cached ones of each sequence: query heads that share a key/value head are two
FORMS = {"cluster": ([1, 3], [77, 130]), "two kernels": ([1, 3], [900, 1500]), "64 columns": ([20, 33], [77, 1500]), "128 rows": ([70, 130], [90, 1500])}


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
    got = gather(w, q, mass).cpu().numpy()
    for b in range(2):
        j = np.arange(kv[b])
        want = np.zeros((kv[b], 2), bool)
        if b == 1:
            want[:seen_by(w, 1, row), 1] = True
        assert np.array_equal(np.isnan(got[w.table[b][j // 64], :, j % 64]), want)
