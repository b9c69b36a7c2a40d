"""The 4-bit key/value cache's entry points without a GPU: sizes, and refusals of bad arguments on
the host before any CUDA call. No kernel is launched here."""
import ctypes

import numpy as np
import pytest

import kv4_reference as ref
from ternary_weight_gb300 import _build, binding

FAKE = 1 << 20  # 256-byte aligned, non-null; never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.lib()


def cache(**kw):
    return binding._KV4CacheDesc(**{**dict(pages=FAKE, n_pages=4, kv_heads=2, head_dim=128), **kw})


def batch(**kw):
    return binding._KV4BatchDesc(**{**dict(cu_q=FAKE, kv_len=FAKE, page_table=FAKE, batch=2, max_pages=2, total_q=3,
                                           max_q=2, max_kv=128), **kw})


def append(lib, c, b, k=FAKE, v=FAKE, dtype=1, ks=256, vs=256, entry="bitnet_kv4_append"):
    return getattr(lib, entry)(ctypes.byref(c) if c else None, ctypes.byref(b) if b else None, k, v, dtype, ks, vs, None)


def attention(lib, c, b, q=FAKE, dtype=1, heads=8, qs=1024, scale=0.1, window=0, sinks=0, out=FAKE, os=1024, ws=FAKE,
              ws_bytes=1 << 40):
    return lib.bitnet_kv4_attention(ctypes.byref(c), ctypes.byref(b), q, dtype, heads, qs, scale, window, sinks, out, os,
                                    ws, ws_bytes, None)


@pytest.mark.parametrize("args,want", [((1, 1, 64), 64 * 64 + 512), ((3, 5, 128), 15 * 8704), ((0, 1, 64), -1),
                                       ((1, 0, 64), -1), ((1, 1025, 64), -1), ((1, 1, 96), -1), ((1 << 31, 1, 64), -1),
                                       ((2 ** 31 - 1, 1024, 128), (2 ** 31 - 1) * 1024 * 8704)])
def test_cache_bytes(lib, args, want):
    assert lib.bitnet_kv4_cache_bytes(*args) == want


CACHES = [(dict(pages=None), -1), (dict(n_pages=0), -1), (dict(n_pages=1 << 31), -1), (dict(kv_heads=0), -1),
          (dict(kv_heads=-2), -1), (dict(head_dim=32), -1), (dict(head_dim=256), -1), (dict(pages=FAKE + 8), -2)]
BATCHES = [(dict(cu_q=None), -1), (dict(kv_len=None), -1), (dict(page_table=None), -1), (dict(batch=0), -1),
           (dict(batch=65536), -1), (dict(max_pages=0), -1), (dict(max_pages=(1 << 24) + 1), -1), (dict(total_q=-1), -1),
           (dict(total_q=1 << 31), -1), (dict(max_q=0), -1), (dict(max_kv=-1), -1), (dict(max_kv=129), -1),
           (dict(cu_q=FAKE + 2), -2), (dict(kv_len=FAKE + 1), -2), (dict(page_table=FAKE + 3), -2)]


@pytest.mark.parametrize("kw,status", CACHES)
def test_bad_caches_are_refused(lib, kw, status):
    c, b = cache(**kw), batch()
    assert append(lib, c, b) == status
    assert append(lib, c, b, entry="bitnet_kv4_read") == status
    assert attention(lib, c, b) == status
    assert lib.bitnet_kv4_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), 8) == status


@pytest.mark.parametrize("kw,status", BATCHES)
def test_bad_batches_are_refused(lib, kw, status):
    c, b = cache(), batch(**kw)
    assert append(lib, c, b) == status
    assert append(lib, c, b, entry="bitnet_kv4_read") == status
    assert attention(lib, c, b) == status
    assert lib.bitnet_kv4_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), 8) == status


def test_null_descriptors_are_refused(lib):
    assert append(lib, None, batch()) == -1 and append(lib, cache(), None) == -1
    assert lib.bitnet_kv4_attention_workspace_size(None, ctypes.byref(batch()), 8) == -1


@pytest.mark.parametrize("entry", ["bitnet_kv4_append", "bitnet_kv4_read"])
@pytest.mark.parametrize("kw,status", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(dtype=2), -1), (dict(dtype=-1), -1), (dict(ks=255), -1),
    (dict(vs=0), -1), (dict(vs=-256), -1), (dict(ks=260), -2), (dict(dtype=0, vs=258), -2), (dict(k=FAKE + 8), -2),
    (dict(v=FAKE + 2), -2)])
def test_append_and_read_refuse(lib, entry, kw, status):
    assert append(lib, cache(), batch(), entry=entry, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(dtype=3), -1), (dict(heads=0), -1), (dict(heads=3), -1),
    (dict(heads=1), -1), (dict(heads=258, qs=1 << 16, os=1 << 16), -1), (dict(qs=1023), -1), (dict(os=512), -1),
    (dict(qs=1028), -2), (dict(os=1025), -2), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(window=-1), -1), (dict(window=1 << 31), -1), (dict(sinks=-1), -1), (dict(sinks=1 << 31), -1),
    (dict(q=FAKE + 8), -2), (dict(out=FAKE + 2), -2), (dict(ws=FAKE + 128), -2)])
def test_attention_refuses(lib, kw, status):
    assert attention(lib, cache(), batch(), **kw) == status


def test_short_workspace_is_refused(lib):
    c, b = cache(n_pages=5000), batch(batch=1, max_pages=4096, total_q=1, max_q=1, max_kv=200000)
    need = lib.bitnet_kv4_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), 8)
    assert need >= 0
    if need:
        assert attention(lib, c, b, ws_bytes=need - 1) == -1
        assert attention(lib, c, b, ws=None, ws_bytes=need) == -1


def test_empty_batch_does_nothing(lib):
    b = batch(total_q=0)
    assert append(lib, cache(), b) == 0
    assert append(lib, cache(), b, entry="bitnet_kv4_read") == 0
    assert attention(lib, cache(), b) == 0


def test_descriptor_layout_matches_header():
    c, b = binding._KV4CacheDesc, binding._KV4BatchDesc
    assert ctypes.sizeof(c) == 24 and c.kv_heads.offset == 16 and c.head_dim.offset == 20
    assert ctypes.sizeof(b) == 64 and b.batch.offset == 24 and b.max_kv.offset == 56


def test_binding_refuses_tensors_it_cannot_pass():
    torch = pytest.importorskip("torch")
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # host tensors
        binding.KV4Batch(i, i[:1], torch.zeros(1, 4, dtype=torch.int32), 1, 1)
    with pytest.raises(ValueError):  # wrong dtype
        binding.KV4Batch(i.long(), i[:1], torch.zeros(1, 4, dtype=torch.int32), 1, 1)
    with pytest.raises(ValueError):  # shapes that do not belong together
        binding.KV4Batch(i, i, torch.zeros(1, 4, dtype=torch.int32), 1, 1)
    with pytest.raises(ValueError):
        binding.KV4Cache(1, 1, 64, pages=torch.zeros(17, dtype=torch.uint8))


def test_reference_pins():
    """The reference itself, on values worked out by hand."""
    code, step, base = ref.quantise(np.arange(64, dtype=np.float32)[None] / 63 * 15)
    assert step[0] == 1 and base[0] == 0 and code[0, 0] == 0 and code[0, -1] == 15
    assert code[0, 21] == 5 and code[0, 32] == 8  # 5.0; 7.619
    code, step, base = ref.quantise(np.array([[0, 15, 0.5, 1.5, 2.5] + [3.0] * 59], np.float32))
    assert list(code[0, :5]) == [0, 15, 0, 2, 2]  # ties to even
    code, step, base = ref.quantise(np.full((1, 64), 7.0, np.float32))
    assert step[0] == 0 and base[0] == 7 and not code.any()
    assert [ref.rho(t) for t in range(9)] == [0, 2, 4, 6, 1, 3, 5, 7, 8]
    w = ref.words_of(np.arange(64) % 16)
    assert w[0] == sum(((8 * n) % 16) << (4 * n) for n in range(8)) and w[3] & 15 == 3
    block = np.zeros(64 * 128 + 512, np.uint8)
    x = np.zeros(128, np.float32)
    x[1] = 15  # dimension 1: word 1, nibble 0
    ref.write_token(block, 2, x, x)
    assert block[4 * 64 + 4] == 15  # key row rho(2) = 4, word 1
    assert block[64 * 64 + 2 * 64 + 32 + 4] == 15  # value row 2 with its halves exchanged
    assert list(block[64 * 128 + 8 * 4:].view(np.float16)[:4]) == [1, 0, 1, 0]
