"""The workspace of the attention weight that cached tokens gather: its size, and the forms of the call that it decides over."""
import ctypes

import numpy as np
import pytest
import torch

from test_kv4_mass import Mass, cuda_lib, lib  # noqa: F401 (fixtures)
from ternary_weight_gb300 import binding

MB = 1 << 20


def size_of(lib, sequences, total_q, max_q, max_kv, share, kv_heads=5, dim=128, voters=0):  # noqa: F811
    at = 1 << 20
    c = binding._KV4CacheDesc(at, 1 << 20, kv_heads, dim)
    b = binding._KV4BatchDesc(at, at, at, sequences, max_kv // 64, total_q, max_q, max_kv)
    return lib.bitnet_kv4_attention_mass_workspace_size(ctypes.byref(c), ctypes.byref(b), share * kv_heads, voters)


@pytest.mark.parametrize("n,share", [(1, 1), (1, 4), (2, 4), (4, 4), (1, 16), (8, 1)])
@pytest.mark.parametrize("sequences", [1, 64, 500, 4096])
def test_steps_of_many_long_caches(lib, n, share, sequences):  # noqa: F811
    """A decode step's scores are kept up to 256 MB. Else it has 32 KB at most for 64 columns of a sequence and head: their queries and
    constants, and their (M, L) of each chunk of tokens. (fp32 queries are two columns a row.)"""
    blocks = -(-2 * n * share // 64)
    assert 0 <= size_of(lib, sequences, n * sequences, n, 131072, share) <= 256 * MB + sequences * 5 * blocks * 32768


@pytest.mark.parametrize("n,share", [(4, 8), (10, 4), (20, 4), (2, 40)])
def test_many_columns_of_long_caches(lib, n, share):  # noqa: F811
    """17 columns to 96 rows: the shares of the votes lie in the workspace where there are several, which is where units are few."""
    blocks = -(-2 * n * share // 64)
    for sequences in (1, 8, 64, 500):
        assert 0 <= size_of(lib, sequences, n * sequences, n, 131072, share) <= 32 * MB + sequences * 5 * blocks * 32768


@pytest.mark.parametrize("prompts,share,voters", [([2048], 4, 0), ([9000, 3], 4, 0), ([500] * 4, 8, 0), ([9000, 700], 4, 64), ([31], 4, 0)])
@pytest.mark.parametrize("steps", [0, 63, 1000])
def test_prompts_beside_single_tokens(lib, prompts, share, voters, steps):  # noqa: F811
    """More than 96 rows of the longest: every sequence and head has blocks of 128 rows for its own rows, each of 67 KB (3 KB of them
    constants) with 1 KB for each 2048 cached tokens. Votes that are shared out over blocks are few."""
    new = prompts + [1] * steps
    blocks = min(sum(new) * share // 128 + len(new), len(new) * -(-min(max(new), voters or max(new)) * share // 128))
    assert 0 < size_of(lib, len(new), sum(new), max(new), 8192 if max(new) < 8192 else 9024, share, voters=voters) <= 5 * blocks * 72 * 1024 + 8 * MB


def with_room(w, room):
    b = w.batch(w.new, w.kv)
    table = torch.full((len(w.kv), room // 64), -7, dtype=torch.int32, device="cuda")
    table[:, :w.wide] = torch.tensor(w.table)
    return binding.KV4Batch(b.cu_q, b.kv_len, table, sum(w.new), max(w.new), room)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (64, "f32"), (128, "bf16"), (128, "f32")])
@pytest.mark.parametrize("share,new,kv", [(4, [1], [1]), (4, [1, 1, 1], [64, 65, 5000]), (1, [3, 0, 8], [3, 40, 3001]), (16, [1, 1], [9000, 31]),
                                          (8, [1, 1], [20000, 33]), (2, [5, 4], [3, 900])])
@pytest.mark.parametrize("window,sinks,decay", [(0, 0, 0.9), (0, 0, 1.0), (70, 4, 1.0), (600, 0, 0.5)])
def test_scores_made_twice(cuda_lib, dim, dtype, share, new, kv, window, sinks, decay):  # noqa: F811
    """Batches with room for so many tokens that their scores are not kept. (5 new tokens of 3 cached: two see nothing.)"""
    w = Mass([min(n, k) for n, k in zip(new, kv)], kv, 2, dim, dtype, seed=sum(kv) + share).fill()
    mass, w.new = w.start(), list(new)
    q, b = w.queries(share), with_room(w, 1 << 25)
    assert binding.kv4_attention_mass_workspace_size(w.cache, b, 2 * share) < 16 * MB
    out = mass.clone()
    got = binding.kv4_attention_mass(w.cache, b, q, dim ** -0.5, mass, decay=decay, window=window, sinks=sinks)
    apart = binding.kv4_attention_mass(w.cache, b, q, dim ** -0.5, out, decay=decay, window=window, sinks=sinks, out=torch.full_like(out, 7.0))
    written = apart != 7.0
    assert torch.equal(apart[written].nan_to_num(9.0), got[written].nan_to_num(9.0))
    rows = np.concatenate([np.arange(e - min(n, k), e) for e, n, k in zip(np.cumsum(new), new, kv)]).astype(int)
    w.new = [min(n, k) for n, k in zip(new, kv)]
    w.check(got, q[torch.tensor(rows, device="cuda")], share, dim ** -0.5, decay, window, sinks)


@pytest.mark.gpu
def test_scores_made_twice_captured(cuda_lib):  # noqa: F811
    w = Mass([1, 1], [3000, 65], 5, 128, "bf16", seed=11).fill()
    mass, q, b = w.start(), w.queries(4), with_room(w, 1 << 24)
    want = binding.kv4_attention_mass(w.cache, b, q, 128 ** -0.5, mass, decay=0.7, out=torch.full_like(mass, 3.0))
    out = torch.full_like(mass, 3.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.kv4_attention_mass(w.cache, b, q, 128 ** -0.5, mass, decay=0.7, out=out)
    for _ in range(3):
        out.fill_(3.0)
        graph.replay()
        assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("entry", [1 << 20, -3])
def test_scores_made_twice_of_bad_pages(cuda_lib, entry):  # noqa: F811
    """Reported, and the other sequence is what it would have been."""
    w = Mass([1, 1], [100, 50], 2, 64, "bf16", seed=11).fill()
    mass, q = w.start(), w.queries(2)
    call = lambda: binding.kv4_attention_mass(w.cache, with_room(w, 1 << 26), q, 64 ** -0.5, mass.clone())  # noqa: E731
    want, own = call(), [int(p) for p in w.table[0] if p >= 0]
    w.table[0, 1] = entry
    got = call()
    assert binding.last_device_error() == binding.BITNET_ERANGE
    mine = torch.ones(w.n_pages, dtype=torch.bool)
    mine[own] = False
    assert torch.equal(got[mine].nan_to_num(9.0), want[mine].nan_to_num(9.0))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,dtype,share", [(128, "bf16", 4), (128, "f32", 4), (64, "bf16", 3), (64, "f32", 32)])
@pytest.mark.parametrize("new,kv,voters", [([300] + [1] * 12 + [0, 130, 7], [300] + [40 * i + 1 for i in range(12)] + [20, 2500, 600], 0),
                                           ([1] * 9 + [700], [64 * i + 9 for i in range(9)] + [900], 0),
                                           ([0, 1, 400, 0, 350, 1, 0, 1, 1, 1], [5, 1, 3000, 70, 350, 90, 0, 64, 65, 2], 200)])
def test_sequences_of_unlike_rows(cuda_lib, dim, dtype, share, new, kv, voters):  # noqa: F811
    """Their blocks lie one behind another in the workspace; what it held before is not looked at."""
    w = Mass(new, kv, 2, dim, dtype, seed=sum(kv)).fill()
    mass, q, b = w.start(), w.queries(share), w.batch(new, kv)
    ws = torch.empty(binding.kv4_attention_mass_workspace_size(w.cache, b, 2 * share, voters), dtype=torch.uint8, device="cuda").fill_(255)
    got = binding.kv4_attention_mass(w.cache, b, q, dim ** -0.5, mass, decay=0.5, window=0, voters=voters, workspace=ws)
    w.check(got, q, share, dim ** -0.5, 0.5, voters=voters)


@pytest.mark.gpu
def test_a_batch_whose_rows_fall_is_reported(cuda_lib):  # noqa: F811
    """Nothing outside the cached tokens' masses is written."""
    w = Mass([300, 1, 1, 1, 100], [300, 60, 60, 60, 200], 2, 64, "bf16", seed=3).fill()
    mass, q, b = w.start(), w.queries(4), w.batch(w.new, w.kv)
    b.cu_q.copy_(torch.tensor([0, 300, 120, 500, -9, 403], dtype=torch.int32))
    got = binding.kv4_attention_mass(w.cache, b, q, 0.125, mass.clone())
    assert binding.last_device_error() == binding.BITNET_ERANGE
    used = torch.zeros_like(mass, dtype=torch.bool)
    for s, n in enumerate(w.kv):
        j = torch.arange(n)
        used[torch.tensor(w.table[s])[j // 64].long().cuda(), :, (j % 64).cuda()] = True
    assert torch.equal(got[~used].nan_to_num(9.0), mass[~used].nan_to_num(9.0))
