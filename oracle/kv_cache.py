"""fp64 restatement of the paged key/value cache operators: quantisation of appended rows, reading back,
and the attention of new tokens over a cache. Sequences are plain arrays here; pages are the product's."""
from __future__ import annotations

import numpy as np

EXP_MIN, EXP_MAX = -64, 15


def e4m3_grid() -> np.ndarray:
    """The 127 non-negative finite e4m3 numbers, ascending (4 exponent bits of bias 7, 3 mantissa bits)."""
    sub = [m * 2.0 ** -9 for m in range(8)]
    normal = [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array(sub + normal[:-1])            # the last code is NaN


_GRID = e4m3_grid()


def round_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 number, ties to the one with the even code, magnitudes above 448 to 448."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    hi = np.clip(np.searchsorted(_GRID, a), 0, len(_GRID) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.copysign(_GRID[pick], x)


def quantise(x: np.ndarray):
    """Rows x [..., 64] -> (values on the e4m3 grid, exponents e). e: the smallest with max|x| <= 448 2^e,
    within [EXP_MIN, EXP_MAX]; the row stands for values * 2^e. Non-finite rows: NaN values."""
    x = np.asarray(x, dtype=np.float64)
    top = np.abs(x).max(-1)
    e = np.full(top.shape, EXP_MIN)
    for k in range(EXP_MIN, EXP_MAX):
        e = np.where(top > 448.0 * 2.0 ** k, k + 1, e)
    finite = np.isfinite(x).all(-1)
    vals = round_e4m3(np.where(np.isfinite(x), x, 0.0) / 2.0 ** e[..., None])
    return np.where(finite[..., None], vals, np.nan), e


def dequantise(vals: np.ndarray, e: np.ndarray) -> np.ndarray:
    return vals * 2.0 ** np.asarray(e, dtype=np.float64)[..., None]


def seen(length: int, n: int, unit: int = 0, window: int = 0, sink: int = 0) -> np.ndarray:
    """[n, length] truth values: what each of the last n tokens of a sequence sees."""
    out = np.zeros((n, length), dtype=bool)
    for i in range(n):
        p = length - n + i
        for j in range(length):
            ok = True
            if unit:
                ok = j // unit <= p // unit
                if window:
                    ok = ok and (j // unit > p // unit - window or j < sink)
            out[i, j] = ok
    return out


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, see: np.ndarray):
    """q [n, H, d], k, v [L, Hk, d], see [n, L] -> out [n, H, d], lse [H, n] in fp64. Keys that a row does
    not see are left out of its sums altogether; rows that see nothing give 0 and -inf."""
    n, H, d = q.shape
    G = H // k.shape[1]
    out = np.zeros((n, H, d))
    lse = np.full((H, n), -np.inf)
    for i in range(n):
        at = np.flatnonzero(see[i])
        if not len(at):
            continue
        for h in range(H):
            s = k[at, h // G].astype(np.float64) @ q[i, h].astype(np.float64) / np.sqrt(d)
            m = s.max()
            w = np.exp(s - m)
            out[i, h] = w @ v[at, h // G].astype(np.float64) / w.sum()
            lse[h, i] = m + np.log(w.sum())
    return out, lse
