"""What the paged key/value cache operators are measured on: appending a chunk of new tokens to the
cache (bf16 as it is, or quantised to e4m3 with a power-of-two scale per token and head), reading
cached tokens back, and the attention of a chunk of new tokens over the cache.

`run` computes them in elementary fp32 torch operations, or with `own` set by the library's calls.
The cache is paged and head-major: a pool [pages, kv_heads, page_tokens, 64] for K and for V, a page
table [seqs, max_pages] (-1: no page) and the lengths kv_len [seqs], which count the new tokens.

  append   position kv_len[s] - n_s + i of sequence s takes new token i. e4m3: per row of 64 values,
           e = the smallest exponent with max|x| <= 448 2^e, kept within [-64, 15]; code = x 2^-e
           rounded to e4m3; scale = 2^e.
  read     row i of sequence s = the value of position first[s] + i (code * scale), 0 without a page.
  attend   token at position p sees position j if j < kv_len, its page exists and, with unit > 0,
           j < (p // unit + 1) unit and, with window > 0, also j >= (p // unit - window + 1) unit or
           j < sink; out = softmax(q.k / 8) v over those, lse = ln sum exp; 0 and -inf for none.
"""
import math
import random

import torch

own = False
D = 64

# One 294x518 frame has 782 tokens, one 518x518 frame 1374, 5 of them camera and register tokens;
# 16 heads of 64: the repository's own layer shapes. Grouped heads and token-wise causal masks are the
# generic forms.
_LISTED = [
    # one token against 10 frames: the latency of the single-token form
    dict(name="decode_one", op="attend", fmt="bf16", seqs=1, heads=16, kv_heads=16, page=64, new=1, len=7820),
    # 32 streams, one token each, ragged lengths, grouped heads, quantised cache
    dict(name="decode_batch_e4m3", op="attend", fmt="e4m3", seqs=32, heads=32, kv_heads=8, page=64, new=1, len=32768,
         ragged=True, unit=1),
    # the 5 camera and register tokens of a frame against 100 frames
    dict(name="special_tokens_e4m3", op="attend", fmt="e4m3", seqs=1, heads=16, kv_heads=16, page=128, new=5,
         len=78200),
    # a new frame against 100 frames: the streaming step's attention
    dict(name="frame_chunk_bf16", op="attend", fmt="bf16", seqs=1, heads=16, kv_heads=16, page=64, new=782, len=78200,
         unit=782),
    # a new 518x518 frame over the first frame and the last 32 of 60
    dict(name="frame_window_e4m3", op="attend", fmt="e4m3", seqs=1, heads=16, kv_heads=16, page=64, new=1374,
         len=82440, unit=1374, window=32, sink=1374),
    # ragged chunks of several streams, token-wise causal, grouped heads, small pages
    dict(name="ragged_chunks_bf16", op="attend", fmt="bf16", seqs=6, heads=32, kv_heads=8, page=16, new=600, len=9000,
         ragged=True, unit=1),
    # the first 10 frames at once, frame-wise causal: nothing cached before
    dict(name="first_frames_e4m3", op="attend", fmt="e4m3", seqs=1, heads=16, kv_heads=16, page=64, new=7820,
         len=7820, unit=782),
    # one frame written, quantised
    dict(name="append_frame_e4m3", op="append", fmt="e4m3", seqs=1, heads=16, kv_heads=16, page=64, new=782,
         len=7820),
    # a whole scene of 100 frames written
    dict(name="append_scene_bf16", op="append", fmt="bf16", seqs=1, heads=16, kv_heads=16, page=64, new=78200,
         len=78200),
    # the scene read back, e.g. for a global layer over all of it
    dict(name="read_scene_e4m3", op="read", fmt="e4m3", seqs=1, heads=16, kv_heads=16, page=64, new=78200, len=78200),
    # ragged pieces of several streams read back
    dict(name="read_ragged_bf16", op="read", fmt="bf16", seqs=8, heads=16, kv_heads=16, page=32, new=1500, len=9000,
         ragged=True),
    # one streaming step: the frame appended, then its attention over 40 frames
    dict(name="step_e4m3", op="step", fmt="e4m3", seqs=1, heads=16, kv_heads=16, page=64, new=782, len=31280,
         unit=782),
]
_DEFAULTS = dict(ragged=False, unit=0, window=0, sink=0, evict=0)


def _full(c):
    return {**_DEFAULTS, **c}


def listed():
    return [_full(c) for c in _LISTED]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "read", "step"])
    fmt = rng.choice(["bf16", "e4m3"])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([g for g in (1, 1, 2, 4, 8) if kv_heads * g <= 32])
    seqs = _log_uniform(rng, 1, 32)
    page = rng.choice([16, 32, 64, 128])
    new = 1 if op in ("attend", "step") and rng.random() < 0.3 else _log_uniform(rng, 1, 1374)
    if op in ("append", "read"):
        new = min(78200, new * rng.choice([1, 1, 50]))
        new = max(1, min(new, 78200 * 16 // (seqs * kv_heads)))
    length = _log_uniform(rng, new, max(new, 78200))
    while op in ("attend", "step") and seqs * heads * new * length > 782 * 16 * 78200 * 9 // 10 and length > new:
        length = max(new, length // 2)
    while op in ("attend", "step") and seqs > 1 and seqs * heads * new * length > 782 * 16 * 78200 * 9 // 10:
        seqs //= 2
    while seqs * kv_heads * length > 78200 * 32 and length > new:
        length = max(new, length // 2)
    unit = rng.choice([0, 1, 1, 97, 782]) if op in ("attend", "step") else 0
    window = rng.choice([0, 0, max(1, length // (3 * unit))]) if unit else 0
    sink = rng.choice([0, 5, 782]) if window else 0
    evict = rng.choice([0, 0, 3]) if op in ("attend", "read") else 0
    return dict(op=op, fmt=fmt, seqs=seqs, heads=heads, kv_heads=kv_heads, page=page, new=new, len=length,
                ragged=seqs > 1 and rng.random() < 0.7, unit=unit, window=window, sink=sink, evict=evict)


def _lengths(c):
    """New (or read) tokens and cache length of each sequence: part of the case, not of the seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    if not c["ragged"]:
        return [c["new"]] * c["seqs"], [c["len"]] * c["seqs"]
    new = [rng.randint(1, c["new"]) for _ in range(c["seqs"])]
    return new, [rng.randint(max(n, c["len"] // 8), c["len"]) for n in new]


def _visible(c, n, length):
    """(visible keys summed over the chunk's tokens, visible keys of the whole chunk) without evicted pages."""
    pairs, low, high = 0, length, 0
    u, w = c["unit"], c["window"]
    for p in range(length - n, length) if u else (length - 1,):
        hi = min(length, (p // u + 1) * u) if u else length
        lo = max(0, (p // u - w + 1) * u) if w else 0
        pairs += (hi - lo + min(c["sink"], lo)) * (1 if u else n)
        low, high = min(low, lo), max(high, hi)
    return pairs, high - low + min(c["sink"], low)


def work(case):
    c = _full(case)
    new, lens = _lengths(c)
    row = 2 * D if c["fmt"] == "bf16" else D + 1          # bytes of one cached row of K or V
    rows = sum(new)
    if c["op"] in ("append", "read"):
        return {"bytes": 2 * rows * c["kv_heads"] * (2 * D + row), "flops": 0}
    pairs, keys = (sum(x) for x in zip(*(_visible(c, n, m) for n, m in zip(new, lens))))
    flops = 4 * D * c["heads"] * pairs
    nbytes = 2 * keys * c["kv_heads"] * row + rows * c["heads"] * (4 * D + 4)
    if c["op"] == "step":
        nbytes += 2 * rows * c["kv_heads"] * (2 * D + row)
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------------- inputs

def _quantise(x):
    """x [..., 64] -> e4m3 codes and the scale 2^e (float8_e8m0fnu) of each row."""
    x = x.float()
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)                                 # top = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    e = torch.where(top > 0, e - 9 + (m > 0.875), -64).clamp(-64, 15).to(torch.int32)
    codes = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def prepare(case, seed):
    c = _full(case)
    new, lens = _lengths(c)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    S, H, Hk, P = c["seqs"], c["heads"], c["kv_heads"], c["page"]
    need = [-(-m // P) for m in lens]
    max_pages, pages = max(need) + 1, sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=dev, dtype=torch.int64).to(torch.int32)
    table = torch.full((S, max_pages), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = order[at:at + k]
        at += k
        if c["evict"] and k > c["evict"] + 4:               # pages given back from inside the sequence
            table[s, 2:2 + c["evict"]] = -1

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)

    st = {"case": c, "page_table": table, "kv_len": torch.tensor(lens, dtype=torch.int32, device=dev),
          "k_scale": None, "v_scale": None, "rows": sum(new), "max_new": max(new)}
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st["cu_new"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    st["first"] = torch.tensor([m - n for n, m in zip(new, lens)], dtype=torch.int32, device=dev)
    if c["op"] in ("attend", "step"):
        st["q"] = randn(sum(new), H, D)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((H, sum(new)), dtype=torch.float32, device=dev)
    for name in ("k", "v"):
        pool = randn(pages, Hk, P, D)
        if name == "k" and "q" in st:
            # planted correspondences, as in the repository's synthetic layers: 5% of the cached keys
            # are three times a query of the chunk plus noise
            n = max(1, pages * P // 20)
            at = torch.randperm(pages * P, generator=gen, device=dev)[:n]
            src = st["q"][torch.randint(0, sum(new), (n,), generator=gen, device=dev)][:, :: H // Hk]
            pool[at // P, :, at % P] = 3 * (src + 0.1 * randn(n, Hk, D))
        if c["fmt"] == "e4m3":
            st[name + "_pool"], st[name + "_scale"] = _quantise(pool)
        else:
            st[name + "_pool"] = pool
        if c["op"] in ("append", "step"):
            st[name] = randn(sum(new), Hk, D)
    if c["op"] == "read":
        st["k"], st["v"] = (torch.empty((sum(new), Hk, D), dtype=torch.bfloat16, device=dev) for _ in range(2))
    return st


# ---------------------------------------------------------------------------------- one pass

def _pools(st):
    return {n: st[n] for n in ("k_pool", "v_pool", "k_scale", "v_scale") if st[n] is not None}


def _places(st):
    """Sequence, page and slot of each row of the chunk."""
    cu, P = st["cu_new"].long(), st["case"]["page"]
    row = torch.arange(st["rows"], device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = st["first"].long()[seq] + row - cu[seq]
    return st["page_table"].long()[seq, pos // P], pos % P


def _plain_append(st):
    page, slot = _places(st)
    for n in ("k", "v"):
        if st["case"]["fmt"] == "e4m3":
            codes, scale = _quantise(st[n])
            st[n + "_pool"].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            st[n + "_scale"].view(torch.uint8)[page, :, slot] = scale.view(torch.uint8)
        else:
            st[n + "_pool"][page, :, slot] = st[n]


def _values(st, n):
    """The pool's values in fp32."""
    x = st[n + "_pool"].float()
    return x if st[n + "_scale"] is None else x * st[n + "_scale"].float()[..., None]


def _plain_read(st):
    page, slot = _places(st)
    got = [_values(st, n)[page.clamp(min=0), :, slot].masked_fill_((page < 0)[:, None, None], 0) for n in ("k", "v")]
    return [x.to(torch.bfloat16) for x in got]


def _plain_attend(st):
    c = st["case"]
    Hk, G, u = c["kv_heads"], c["heads"] // c["kv_heads"], c["unit"]
    table, length = st["page_table"].long(), st["kv_len"].long()
    S, L = len(length), table.shape[1] * c["page"]
    dev = table.device
    j = torch.arange(L, device=dev)
    there = (table >= 0).repeat_interleave(c["page"], 1) & (j < length[:, None])                  # [S, L]
    K, V = (_values(st, n)[table.clamp(min=0)].transpose(1, 2).reshape(S, Hk, L, D) for n in ("k", "v"))
    V = V.masked_fill_(~there[:, None, :, None], 0)
    cu = st["cu_new"].long()
    i = torch.arange(st["max_new"], device=dev)
    row = cu[:-1, None] + i
    used = row < cu[1:, None]                                                                     # [S, n]
    q = st["q"].float()[row.clamp(max=st["rows"] - 1)].reshape(S, len(i), Hk, G, D).permute(0, 2, 3, 1, 4)
    s = (q.reshape(S, Hk, -1, D) @ K.transpose(2, 3)).reshape(S, Hk, G, len(i), L) * D ** -0.5
    p = (st["first"].long()[:, None] + i)[:, :, None]                                             # [S, n, 1]
    see = there[:, None, :].expand(S, len(i), L)
    if u:
        see = see & (j < (p // u + 1) * u)
    if c["window"]:
        see = see & ((j >= (p // u - c["window"] + 1) * u) | (j < c["sink"]))
    s = s.masked_fill_(~see[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0)
    e = torch.exp(s.sub_(m))
    total = e.sum(-1, keepdim=True)
    o = (e.reshape(S, Hk, -1, L) @ V).reshape(S, Hk, G, len(i), D) / torch.where(total > 0, total, 1)
    lse = (m + torch.log(total))[..., 0]
    out = o.permute(0, 3, 1, 2, 4).reshape(S, len(i), c["heads"], D)[used].to(torch.bfloat16)
    return out, lse.permute(1, 2, 0, 3).reshape(c["heads"], S, len(i))[:, used].contiguous()


def _handle(st):
    """The cache over the program's own tensors, made once per state as such a program makes it."""
    if "cache" not in st:
        from view_transformers_b200.cache import KVCache
        st["cache"] = KVCache.over(st["k_pool"], st["v_pool"], st["page_table"], st["kv_len"],
                                   heads=st["case"]["heads"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    return st["cache"]


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        cache = _handle(state)
        if op in ("append", "step"):
            cache.append(state["k"], state["v"], state["cu_new"])
        if op == "read":
            return cache.read(state["cu_new"], state["first"], out=(state["k"], state["v"]))
        if op != "append":
            out = cache.attend(state["q"], state["cu_new"], state["max_new"], unit=c["unit"], window=c["window"],
                               sink=c["sink"], out=state["out"], lse=state["lse"])
            lse = state["lse"]
    else:
        if op in ("append", "step"):
            _plain_append(state)
        if op == "read":
            return tuple(_plain_read(state))
        if op != "append":
            out, lse = _plain_attend(state)
    if op == "append":
        return _pools(state)
    return {"out": out, "lse": lse, **(_pools(state) if op == "step" else {})}


# ---------------------------------------------------------------------------------- in 64 bits

def _grid(x):
    """x rounded to the nearest e4m3 number, ties to the even one: 4 significant bits, steps of 2^-9 at least."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448)


def _exact_scale(x):
    """2^e, the smallest power with max|x| <= 448 2^e within [2^-64, 2^15], by trying the neighbours."""
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -80) / 448)).clamp(-64, 15)
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    return torch.exp2(torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e).clamp(-64, 15))


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    new, lens = _lengths(c)
    pool, scale = {}, {}
    for n in ("k", "v"):
        pool[n] = st[n + "_pool"].double()
        scale[n] = torch.ones(pool[n].shape[:3], dtype=torch.float64, device="cuda") if st[n + "_scale"] is None \
            else st[n + "_scale"].float().double()
    table = st["page_table"].cpu()
    slots = []                                              # flat page and slot of every position
    for s, m in enumerate(lens):
        pos = torch.arange(m)
        slots.append((table[s].long()[pos // c["page"]].cuda(), (pos % c["page"]).cuda()))
    cu = st["cu_new"].tolist()
    if c["op"] in ("append", "step"):
        for s, n_s in enumerate(new):
            page, slot = (x[lens[s] - n_s:] for x in slots[s])
            for n in ("k", "v"):
                x = st[n][cu[s]:cu[s + 1]].double()
                if c["fmt"] == "e4m3":
                    f = _exact_scale(x)
                    scale[n][page, :, slot] = f
                    x = _grid(x / f[..., None])
                pool[n][page, :, slot] = x
    pools = {n + "_pool": pool[n] for n in ("k", "v")}
    if c["fmt"] == "e4m3":
        pools.update({n + "_scale": scale[n] for n in ("k", "v")})
    if c["op"] == "append":
        return pools
    if c["op"] == "read":
        got = {"k": [], "v": []}
        for s, n_s in enumerate(new):
            page, slot = (x[lens[s] - n_s:] for x in slots[s])
            for n in ("k", "v"):
                x = pool[n][page, :, slot] * scale[n][page, :, slot][..., None]
                got[n].append(torch.where((page >= 0)[:, None, None], x, torch.zeros_like(x)))
        return tuple(torch.cat(got[n]) for n in ("k", "v"))
    H, Hk = c["heads"], c["kv_heads"]
    out = torch.zeros((sum(new), H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((H, sum(new)), -math.inf, dtype=torch.float64, device="cuda")
    for s, n_s in enumerate(new):
        page, slot = slots[s]
        keys = torch.nonzero(page >= 0)[:, 0]
        if not len(keys):
            continue
        p = torch.arange(lens[s] - n_s, lens[s], device="cuda")[:, None]
        see = torch.ones((n_s, len(keys)), dtype=torch.bool, device="cuda")
        if c["unit"]:
            frame, of_key = p // c["unit"], keys // c["unit"]
            see = of_key <= frame
            if c["window"]:
                see &= (of_key > frame - c["window"]) | (keys < c["sink"])
        some = see.any(1)
        for h in range(H):
            g = h // (H // Hk)
            k, v = (pool[n][page[keys], g, slot[keys]] * scale[n][page[keys], g, slot[keys]][:, None] for n in ("k", "v"))
            a = st["q"][cu[s]:cu[s + 1], h].double() @ k.T / 8
            a = torch.where(see, a, -math.inf)
            z = torch.logsumexp(a, 1)
            w = torch.exp(a - torch.where(some, z, torch.zeros_like(z))[:, None])
            out[cu[s]:cu[s + 1], h] = w @ v
            lse[h, cu[s]:cu[s + 1]] = z
    return {"out": out, "lse": lse, **(pools if c["op"] == "step" else {})}
