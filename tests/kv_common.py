"""Shared helpers of the paged key/value cache tests: a cache filled from plain per-sequence arrays, the
oracle's results for it, and the error bound that the kernels' roundings allow."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from oracle import kv_cache as okv

D = 64


@dataclass
class Case:
    name: str
    new: tuple             # new tokens per sequence
    lens: tuple            # cached tokens per sequence, the new ones included
    heads: int = 2
    kv_heads: int = 2
    page: int = 16
    fmt: str = "bf16"
    unit: int = 0
    window: int = 0
    sink: int = 0
    evict: tuple = ()      # (sequence, page index) pairs without a page
    scale: float = 1.0     # of the queries: larger = more peaked

    def __str__(self):
        return self.name


def bf16(x: np.ndarray) -> np.ndarray:
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).double().numpy()


def tensors(c: Case, seed: int = 0, stale=float("nan"), device="cuda"):
    """The case's device tensors (pools filled through the oracle's quantisation, every unused place of the
    pools holding `stale`) and its host arrays."""
    import torch
    rng = np.random.default_rng(seed)
    S, Hk, P = len(c.new), c.kv_heads, c.page
    need = [-(-m // P) for m in c.lens]
    pages, width = sum(need) + 2, max(need + [1]) + 1
    order = rng.permutation(pages)
    table = np.full((S, width), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    x = {}
    host = {"k": [], "v": [], "q": []}
    pool = {n: np.full((pages, Hk, P, D), np.nan) for n in "kv"}
    expo = {n: np.zeros((pages, Hk, P), dtype=np.int64) for n in "kv"}
    used = np.zeros((pages, Hk, P), dtype=bool)
    for s, m in enumerate(c.lens):
        host["q"].append(bf16(c.scale * rng.standard_normal((c.new[s], c.heads, D))))
        pos = np.arange(m)
        pg, slot = table[s, pos // P], pos % P
        for n in "kv":
            rows = bf16(rng.standard_normal((m, Hk, D)))
            if c.fmt == "e4m3":
                vals, e = okv.quantise(rows)
                expo[n][pg, :, slot] = e
                pool[n][pg, :, slot] = vals
                rows = okv.dequantise(vals, e)
            else:
                pool[n][pg, :, slot] = rows
            host[n].append(rows)
        used[pg, :, slot] = True
    gone = [np.zeros(m, dtype=bool) for m in c.lens]
    for s, t in c.evict:
        table[s, t] = -1
        gone[s][t * P:(t + 1) * P] = True
    for n in "kv":
        if c.fmt == "e4m3":
            t = torch.from_numpy(np.nan_to_num(pool[n])).to(torch.float8_e4m3fn)
            b = torch.from_numpy((expo[n] + 127).astype(np.uint8))
            codes = t.view(torch.uint8)
            codes[torch.from_numpy(~used)] = 0x7f              # stale: NaN codes under NaN scales
            b[torch.from_numpy(~used)] = 255
            x[n + "_pool"], x[n + "_scale"] = t.to(device), b.view(torch.float8_e8m0fnu).to(device)
        else:
            x[n + "_pool"] = torch.from_numpy(np.where(used[..., None], pool[n], stale)).to(torch.bfloat16).to(device)
            x[n + "_scale"] = None
    cu = np.concatenate([[0], np.cumsum(c.new)]).astype(np.int32)
    x["table"], x["kv_len"] = (torch.from_numpy(a).to(device) for a in (table, np.array(c.lens, dtype=np.int32)))
    x["cu"] = torch.from_numpy(cu).to(device)
    q = np.concatenate(host["q"]) if cu[-1] else np.zeros((0, c.heads, D))
    x["q"] = torch.from_numpy(q).to(torch.bfloat16).to(device)
    x["rows"], x["max_new"] = int(cu[-1]), max(c.new)
    host["gone"], host["cu"] = gone, cu
    return x, host


def cache_over(c: Case, x):
    from view_transformers_b200.cache import KVCache
    return KVCache.over(x["k_pool"], x["v_pool"], x["table"], x["kv_len"], c.heads, x["k_scale"], x["v_scale"])


def attention_oracle(c: Case, host):
    """Packed out, lse, and the bounds of their errors.

    With p the exact weights: a score is a 64-term fp32 sum of exact products, scaled: off by at most
    d = 70 2^-24 sum|q k| / 8 (plus 2^-21 for the subtraction and the exponential at |x| < 64 log2 units, and
    2^-22 |x| of x itself), so each weight is off by that factor, and so is their sum. P is rounded to bf16
    (2^-8), the result once more (2^-8). The fp32 sums over L keys add L 2^-24 (all terms positive for l; for
    P.V relative to sum p|v|)."""
    outs, lses, bo, bl = [], [], [], []
    for s, (n, m) in enumerate(zip(c.new, c.lens)):
        if n == 0:
            continue
        q, k, v = host["q"][s], host["k"][s], host["v"][s]
        see = okv.seen(m, n, c.unit, c.window, c.sink) & ~host["gone"][s][None, :]
        o, lse = okv.attention(q, k, v, see)
        a, _ = okv.attention(q, k, np.abs(v), see)
        G = c.heads // c.kv_heads
        dots = np.einsum("nhd,lhd->hnl", np.abs(q), np.repeat(np.abs(k), G, axis=1)) / 8
        d = np.where(see[None], dots, 0).max(-1, initial=0) * (70 * 2.0 ** -24 + 2.0 ** -22) + 2.0 ** -21 + m * 2.0 ** -24
        outs.append(o)
        lses.append(lse)
        bo.append(2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * d.T[..., None]) * 1.01 * a + 1e-30)
        bl.append(2 * d + 2.0 ** -21 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0))))
    if not outs:
        return np.zeros((0, c.heads, D)), np.zeros((c.heads, 0)), np.ones(0), np.ones(0)
    return np.concatenate(outs), np.concatenate(lses, 1), np.concatenate(bo), np.concatenate(bl, 1)


def check_attention(got, lse, want):
    o, l, bo, bl = want
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    assert got.shape == o.shape and lse.shape == l.shape
    assert np.array_equal(np.isneginf(lse), np.isneginf(l))
    fin = np.isfinite(l)
    assert np.isfinite(got).all() and np.isfinite(lse[fin]).all()
    if o.size:
        assert np.max(np.abs(got - o) / bo) <= 1.0, np.max(np.abs(got - o) / bo)
    if fin.any():
        assert np.max(np.abs(lse[fin] - l[fin]) / bl[fin]) <= 1.0, np.max(np.abs(lse[fin] - l[fin]) / bl[fin])
