"""The 4-bit key/value cache and its attention in plain 64-bit numpy, from the definitions in
include/bitnet.h: what the tests compare the kernels with. Shares no code with the library."""
import numpy as np

PAGE = 64


def quantise(x):
    """x (..., D) fp32 -> codes (uint8), step and base (fp16, without the last axis)."""
    x = np.asarray(x, np.float32)
    nan = np.isnan(x).any(-1)
    c = np.clip(np.where(np.isnan(x), np.float32(0), x), np.float32(-61440), np.float32(61440))
    lo, hi = c.min(-1), c.max(-1)
    base = np.where(nan, np.float16(np.nan), lo.astype(np.float16))
    step = np.where(nan, np.float16(np.nan), ((hi - lo) / np.float32(15)).astype(np.float16))
    s64 = step.astype(np.float64)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.rint((c.astype(np.float64) - base.astype(np.float64)[..., None]) / s64)
    code = np.where(s64 > 0, np.clip(t, 0, 15), 0)  # a NaN step compares false
    return code.astype(np.uint8), step, base


def stands_for(code, step, base):
    return step.astype(np.float64)[..., None] * code + base.astype(np.float64)[..., None]


def rho(t):
    return (t & ~7) | ((t & 3) << 1) | ((t >> 2) & 1)


def words_of(code):
    """codes of one vector -> its W 32-bit words."""
    d = len(code)
    w = d // 8
    return np.array([sum(int(code[i + w * n]) << (4 * n) for n in range(8)) for i in range(w)], np.uint32)


def write_token(block, t, k, v):
    """Writes one token's key and value (D fp32 each) into a page's block of one head (bytes)."""
    d = len(k)
    w = d // 8
    rows = block[:PAGE * d].view(np.uint32).reshape(2, PAGE, w)
    par = block[PAGE * d:].view(np.float16).reshape(PAGE, 4)
    (kc, ks, kb), (vc, vs, vb) = quantise(k), quantise(v)
    rows[0, rho(t)] = words_of(kc)
    vw = words_of(vc)
    rows[1, t] = np.roll(vw, w // 2) if d == 128 and t & 2 else vw
    par[rho(t)] = ks, kb, vs, vb


def attention(q, k, v, pos, scale, window, sinks):
    """q (n, Hq, D), k and v (L, H, D) as the values they stand for, pos (n) positions -> the exact
    output (n, Hq, D) and what the tests' bounds need: sum p |v| and, for each row and head, the
    largest sum |q| |k| over the positions seen."""
    n, hq, d = q.shape
    length, h, _ = k.shape
    q = q.astype(np.float64)
    j = np.arange(length)
    sees = j[None] <= pos[:, None]
    if window:
        sees &= (j[None] > pos[:, None] - window) | (j[None] < sinks)
    out, av, size = np.zeros((n, hq, d)), np.zeros((n, hq, d)), np.zeros((n, hq))
    for a in range(hq):
        kk, vv = k[:, a // (hq // h)], v[:, a // (hq // h)]
        for i in range(n):
            m = sees[i]
            if not m.any():
                continue
            with np.errstate(invalid="ignore"):
                s = scale * (kk[m] @ q[i, a])
                p = np.exp(s - s.max())
                p /= p.sum()
                out[i, a] = p @ vv[m]
                av[i, a] = p @ np.abs(vv[m])
                size[i, a] = (np.abs(kk[m]) @ np.abs(q[i, a])).max()
            if np.isnan(vv[m]).any():  # a NaN value vector: NaN in every dimension
                out[i, a] = np.nan
    return out, av, size
