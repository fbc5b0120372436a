"""The paged key/value cache on a B200 against the fp64 oracle (oracle/kv_cache.py): appending and reading
back bit for bit, the attention within the bound of its roundings (tests/kv_common.py), the masks that leave
rows empty, stale and non-finite memory, bad tables, strides, streams, captured calls, and a stream of frames
through AttentionBlock."""
import numpy as np
import pytest

from kv_common import D, Case, attention_oracle, bf16, cache_over, check_attention, tensors
from oracle import kv_cache as okv
from oracle import layer_io
from view_transformers_b200 import _lib

pytestmark = pytest.mark.gpu


def _attend(c, x, cache=None, **kw):
    import torch
    cache = cache or cache_over(c, x)
    out = torch.full((x["rows"], c.heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.heads, x["rows"]), 7.0, dtype=torch.float32, device="cuda")
    cache.attend(x["q"], x["cu"], kw.pop("max_new", x["max_new"]), unit=c.unit, window=c.window, sink=c.sink, out=out,
                 lse=lse, **kw)
    return cache, out, lse


ATTEND = [
    # single tokens
    Case("one_key", (1,), (1,)),
    Case("one_15", (1,), (15,), heads=1, kv_heads=1),
    Case("one_16", (1,), (16,), page=32),
    Case("one_129_e4m3", (1,), (129,), page=64, fmt="e4m3"),
    Case("one_long", (1,), (5001,), heads=3, kv_heads=3, page=64, scale=3.0),
    Case("one_long_e4m3", (1,), (4999,), heads=2, kv_heads=1, page=128, fmt="e4m3", scale=3.0),
    Case("one_256_page", (1,), (700,), page=256, unit=1),
    # grouped heads: 4, 8 (one 8-row tile), 12 and 16 rows
    Case("group4", (1, 1), (300, 33), heads=8, kv_heads=2, unit=1),
    Case("group8_e4m3", (1,), (257,), heads=8, kv_heads=1, fmt="e4m3", page=32),
    Case("rows12", (3,), (200,), heads=8, kv_heads=2, unit=1, page=32),
    Case("rows15_e4m3", (5,), (333,), heads=6, kv_heads=2, unit=1, page=64, fmt="e4m3"),
    # chunks
    Case("chunk17", (17,), (17,), unit=1),
    Case("chunk33_e4m3", (33,), (400,), unit=1, page=64, fmt="e4m3", scale=2.0),
    Case("chunk128", (128,), (128,), unit=0, page=128),
    Case("chunk129", (129,), (515,), heads=4, kv_heads=2, unit=1, page=64),
    Case("chunk130_e4m3", (130,), (1000,), heads=1, kv_heads=1, unit=69, page=32, fmt="e4m3"),
    Case("frame_782", (300,), (1111,), heads=1, kv_heads=1, unit=150, page=64),
    Case("group3_chunk", (100,), (260,), heads=6, kv_heads=2, unit=1, page=16),
    Case("group8_chunk_e4m3", (37,), (600,), heads=8, kv_heads=1, unit=1, page=16, fmt="e4m3"),
    # windows and sinks
    Case("window", (70,), (900,), unit=50, window=3, page=16),
    Case("window_sink", (70,), (900,), unit=50, window=2, sink=21, page=64),
    Case("window_sink_e4m3", (5,), (900,), unit=7, window=2, sink=130, page=16, fmt="e4m3"),
    Case("window_one_token", (40,), (500,), unit=1, window=1, page=32),
    Case("window_tiles", (200,), (1500,), heads=1, kv_heads=1, unit=1, window=300, sink=140, page=64),
    Case("window_beyond", (9,), (100,), unit=10, window=50, sink=1000),
    # several sequences, some without new tokens, some without anything
    Case("ragged", (3, 0, 40, 1), (50, 20, 300, 1), heads=4, kv_heads=2, unit=1),
    Case("empty_seq", (0, 2, 0), (0, 2, 0), unit=1),
    Case("many", tuple([1] * 70), tuple(range(1, 211, 3)), heads=2, kv_heads=1, fmt="e4m3"),
    Case("many_mixed", tuple([i % 5 for i in range(33)]), tuple([7 * i % 200 + 5 for i in range(33)]), unit=1),
    Case("long_and_short", (140, 1, 1), (900, 2000, 3), heads=2, kv_heads=2, unit=1, page=64),
    # evicted pages; the last case leaves every row empty
    Case("evicted", (20,), (400,), unit=1, evict=((0, 0), (0, 3), (0, 4), (0, 9))),
    Case("evicted_e4m3", (1, 2), (400, 90), page=32, fmt="e4m3", evict=((0, 0), (1, 1))),
    Case("evicted_chunk", (200,), (600,), unit=1, page=64, evict=((0, 1), (0, 7))),
    Case("all_evicted", (2,), (40,), evict=((0, 0), (0, 1), (0, 2))),
    Case("all_evicted_chunk", (150,), (300,), page=64, evict=tuple((0, i) for i in range(5))),
    Case("window_evicted", (150,), (600,), unit=10, window=2, page=16, evict=tuple((0, i) for i in range(29, 34))),
]


@pytest.mark.parametrize("c", ATTEND, ids=str)
def test_attention_against_the_oracle(c):
    import torch
    x, host = tensors(c)
    cache, out, lse = _attend(c, x)
    assert cache.check_status() == 0
    want = attention_oracle(c, host)
    check_attention(out, lse, want)
    # the same bits again, and whatever kernel max_new picks (each within the bound)
    _, out2, lse2 = _attend(c, x, cache)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for mx in (1, 2000):
        _, out3, lse3 = _attend(c, x, cache, max_new=mx)
        check_attention(out3, lse3, want)
    assert cache.check_status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 24, 200])
def test_many_ranges_of_lengths(n, fmt):
    """Lengths around the borders of steps (16), units (128) and pages."""
    for m in (1, 2, 15, 16, 17, 31, 127, 128, 129, 255, 256, 257, 383, 385, 640):
        if m < n:
            continue
        c = Case(f"len{m}", (n,), (m,), heads=1, kv_heads=1, page=32, fmt=fmt, unit=1)
        x, host = tensors(c, seed=m)
        cache, out, lse = _attend(c, x)
        check_attention(out, lse, attention_oracle(c, host))
        assert cache.check_status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [3, 150])
def test_nan_of_a_later_token_stays_with_those_that_see_it(fmt, n):
    import torch
    c = Case("nan", (n,), (n + 50,), heads=1, kv_heads=1, page=16, fmt=fmt, unit=1)
    x, host = tensors(c)
    pos = n + 50 - 2                                         # the last token but one
    page, slot = int(x["table"][0, pos // 16]), pos % 16
    if fmt == "bf16":
        x["v_pool"][page, 0, slot, 5] = float("nan")
        x["v_pool"][page, 0, slot, 40] = float("inf")
    else:
        x["v_scale"].view(torch.uint8)[page, 0, slot] = 255  # the row stands for NaN
    cache, out, lse = _attend(c, x)
    o, l, bo, bl = attention_oracle(c, host)
    k = n - 2                                                # rows before do not see it
    check_attention(out[:k], lse[:, :k], (o[:k], l[:, :k], bo[:k], bl[:, :k]))
    bad = ~torch.isfinite(out[k:, 0].float())
    assert bool((bad[:, 5] & bad[:, 40]).all()) if fmt == "bf16" else bool(bad.all())
    if fmt == "bf16":
        assert not bool(bad[:, [0, 4, 6, 39, 41, 63]].any())
    # and a key that is NaN spoils the rows that see it, no other
    x, host = tensors(c)
    if fmt == "bf16":
        x["k_pool"][page, 0, slot, 5] = float("nan")
    else:
        x["k_scale"].view(torch.uint8)[page, 0, slot] = 255
    _, out, lse = _attend(c, x)
    check_attention(out[:k], lse[:, :k], (o[:k], l[:, :k], bo[:k], bl[:, :k]))
    assert bool(torch.isnan(out[k:].float()).all())


@pytest.mark.parametrize("n", [1, 12, 150])
def test_scores_far_below_zero(n):
    """Finite scores of -1e31 are scores like any others; a row whose scores are all -inf counts as one that sees
    nothing. Keys are equal here, so the weights are 1 / keys and the values' mean is the result (a bf16 P of
    1, each product exact; the sum of up to 512 of them off by 512 2^-24, the quotient and the result by 2^-8)."""
    import torch
    m = 512
    c = Case("low", (n,), (m,), heads=1, kv_heads=1, page=64)
    for key, finite in ((-2.0 ** 50, True), (-float("inf"), False)):
        x, host = tensors(c)
        x["q"].fill_(2.0 ** 50)
        x["k_pool"].fill_(0.0)
        x["k_pool"][..., 0] = key
        if finite:
            x["k_pool"][...] = key
        cache, out, lse = _attend(c, x)
        if finite:
            want = torch.from_numpy(host["v"][0].mean(0)).cuda()
            bound = (2.0 ** -8 + 512 * 2.0 ** -24) * torch.from_numpy(np.abs(host["v"][0]).mean(0)).cuda()
            assert bool(((out.double() - want).abs() <= bound).all())
            score = -64 * 2.0 ** 100 / 8                                   # + ln 512, far below its last place
            assert bool(((lse.double() / score - 1).abs() <= 2.0 ** -21).all())
        else:
            assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
        assert cache.check_status() == 0


@pytest.mark.parametrize("n", [1, 12, 150])
def test_small_values_beside_a_large_one_in_e4m3(n):
    """One large element sets a row's scale and leaves the others among the subnormal codes."""
    import torch
    c = Case("small", (n,), (n + 300,), page=32, fmt="e4m3", unit=1)
    x, host = tensors(c)
    rng = np.random.default_rng(7)
    table, P = x["table"].cpu().numpy(), c.page
    for name in "kv":
        rows = rng.uniform(-2.0 ** -6, 2.0 ** -6, host[name][0].shape)
        rows[..., 11] = rng.choice([-400.0, 448.0], rows.shape[:-1])
        if name == "k":
            rows[..., 11] = 0.0
            rows[..., 12] = 448.0
        rows = bf16(rows * 2.0 ** rng.integers(-9, 2, rows.shape[:-1])[..., None])
        vals, e = okv.quantise(rows)
        host[name][0] = okv.dequantise(vals, e)
        pos = np.arange(n + 300)
        pg, slot = (torch.from_numpy(a).cuda() for a in (table[0, pos // P].astype(np.int64), pos % P))
        x[name + "_pool"].view(torch.uint8)[pg, :, slot] = torch.from_numpy(vals).cuda().to(torch.float8_e4m3fn).view(torch.uint8)
        x[name + "_scale"].view(torch.uint8)[pg, :, slot] = torch.from_numpy((e + 127).astype(np.uint8)).cuda()
    x["q"][:, :, 12] = 0                                 # the large key element does not decide the scores
    host["q"][0][:, :, 12] = 0
    cache, out, lse = _attend(c, x)
    assert cache.check_status() == 0
    check_attention(out, lse, attention_oracle(c, host))


def _fresh(c, device="cuda"):
    """A cache with its tables set, empty pools of a sentinel, and the new tokens."""
    import torch
    x, host = tensors(c)
    for n in ("k_pool", "v_pool"):
        x[n].view(torch.uint8).fill_(0x55)
        if c.fmt == "e4m3":
            x[n[0] + "_scale"].view(torch.uint8).fill_(0x55)
    return x, host


APPEND = [
    Case("a_one", (1,), (1,), fmt="e4m3"), Case("a_one_bf16", (1,), (33,)),
    Case("a_frame", (69,), (200,), heads=3, kv_heads=3, page=32, fmt="e4m3"),
    Case("a_ragged", (5, 0, 37, 1), (5, 9, 64, 300), heads=4, kv_heads=2, page=64),
    Case("a_ragged_e4m3", (5, 0, 37, 1), (5, 9, 64, 300), heads=4, kv_heads=2, page=64, fmt="e4m3"),
    Case("a_many", tuple([i % 3 for i in range(200)]), tuple([20 + i % 7 for i in range(200)]), fmt="e4m3"),
    Case("a_long", (3000,), (3001,), heads=4, kv_heads=4, page=128, fmt="e4m3"),
]


@pytest.mark.parametrize("strided", [False, True], ids=["packed", "strided"])
@pytest.mark.parametrize("c", APPEND, ids=str)
def test_append_and_read_back(c, strided):
    import torch
    x, _ = _fresh(c)
    rng = np.random.default_rng(5)
    rows, Hk, P = x["rows"], c.kv_heads, c.page
    kv = rng.standard_normal((2, rows, Hk, D)) * 2.0 ** rng.integers(-70, 13, (2, rows, Hk, 1))
    kv[:, ::7] = 0.0
    kv[0, ::5, :, 3] = 448 * 2.0 ** rng.integers(-20, 5)                  # a largest element on the border
    kv = bf16(kv)
    dev = torch.from_numpy(kv).to(torch.bfloat16).cuda()
    if strided:                                                           # rows inside a wider tensor
        wide = torch.full((2, rows + 1, Hk + 3, D), 9.0, dtype=torch.bfloat16, device="cuda")
        wide[:, :rows, 1:Hk + 1] = dev
        dev = wide[:, :rows, 1:Hk + 1]
    cache = cache_over(c, x)
    cache.append(dev[0], dev[1], x["cu"])
    assert cache.check_status() == 0
    table, cu = x["table"].cpu().numpy(), x["cu"].cpu().numpy()
    for which, n in enumerate("kv"):
        pool = x[n + "_pool"].float().cpu().double().numpy()
        raw = x[n + "_pool"].view(torch.uint8).cpu().numpy()
        touched = np.zeros(pool.shape[:3], dtype=bool)
        for s, (m, k) in enumerate(zip(c.lens, c.new)):
            for i in range(k):
                pos = m - k + i
                pg, slot = table[s, pos // P], pos % P
                touched[pg, :, slot] = True
                row = kv[which, cu[s] + i]
                if c.fmt == "e4m3":
                    vals, e = okv.quantise(row)
                    assert np.array_equal(pool[pg, :, slot], vals)
                    assert np.array_equal(x[n + "_scale"].view(torch.uint8)[pg, :, slot].cpu().numpy(), e + 127)
                else:
                    assert np.array_equal(pool[pg, :, slot], row)
        assert (raw[~touched] == 0x55).all()                              # nothing else was written
    # read back: exactly what the cache holds, into a strided destination too
    first = torch.tensor([m - k for m, k in zip(c.lens, c.new)], dtype=torch.int32, device="cuda")
    wide = torch.full((2, rows + 2, Hk + 1, D), 3.0, dtype=torch.bfloat16, device="cuda")
    got = (wide[0, :rows, :Hk], wide[1, :rows, :Hk]) if strided else None
    got = cache.read(x["cu"], first, rows=rows, out=got)
    assert cache.check_status() == 0
    for which in range(2):
        want = kv[which]
        if c.fmt == "e4m3":
            want = okv.dequantise(*okv.quantise(want))
        assert np.array_equal(got[which].double().cpu().numpy(), want)
    if strided:
        assert bool((wide[:, rows:] == 3).all()) and bool((wide[:, :, Hk:] == 3).all())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_append_reports_what_the_format_cannot_hold(fmt):
    import torch
    c = Case("r", (4,), (4,), heads=1, kv_heads=1, fmt=fmt)
    ok = torch.ones((4, 1, D), dtype=torch.bfloat16, device="cuda")
    for where, value, code in ((0, float("nan"), 6), (1, float("-inf"), 6), (0, 1.5e7, 6 if fmt == "e4m3" else 0),
                               (1, 14680064.0, 0), (0, 3e38, 6 if fmt == "e4m3" else 0)):
        x, _ = _fresh(c)
        cache = cache_over(c, x)
        kv = [ok.clone(), ok.clone()]
        kv[where][2, 0, 17] = value
        cache.append(kv[0], kv[1], x["cu"])
        assert cache.check_status() == code, (value, fmt)
        got = cache.read(x["cu"], torch.zeros(1, dtype=torch.int32, device="cuda"), rows=4)[where].float()
        if not np.isfinite(value):
            if fmt == "e4m3":
                assert bool(torch.isnan(got[2]).all())                   # the whole row
            else:
                assert torch.equal(got[2, 0, 17].isnan(), torch.tensor(value).isnan().cuda())
        elif fmt == "e4m3" and code:
            assert float(got[2, 0, 17]) == 14680064.0                    # saturated
        keep = [0, 1, 3]
        assert bool((got[keep] == 1).all())


def test_read_of_missing_tokens():
    import torch
    c = Case("m", (1, 1), (50, 20), page=16, evict=((0, 1),))
    x, host = tensors(c)
    cache = cache_over(c, x)
    cu = torch.tensor([0, 40, 60], dtype=torch.int32, device="cuda")
    k, v = cache.read(cu, torch.tensor([10, 0], dtype=torch.int32, device="cuda"), rows=60)
    assert cache.check_status() == 0                                     # a missing page is no error
    want = np.concatenate([np.where(host["gone"][0][10:50, None, None], 0, host["k"][0][10:50]), host["k"][1]])
    assert np.array_equal(k.double().cpu().numpy(), want)
    # past the end, before the start: zeros, reported
    for first in ([11, 0], [-1, 0]):
        k, v = cache.read(cu, torch.tensor(first, dtype=torch.int32, device="cuda"), rows=60)
        assert cache.check_status() == _lib.BSA_ERR_DEVICE_BOUNDS
        assert bool((v[39 if first[0] > 0 else 0] == 0).all())


@pytest.mark.parametrize("n", [2, 40, 200])
def test_rows_behind_the_last_sequence_stay(n):
    import torch
    c = Case("behind", (n,), (n + 60,), unit=1)
    x, host = tensors(c)
    q = torch.cat([x["q"], torch.full((9, c.heads, D), float("nan"), dtype=torch.bfloat16, device="cuda")])
    x2 = {**x, "q": q, "rows": n + 9}
    cache, out, lse = _attend(c, x2)
    assert cache.check_status() == 0
    assert bool((out[n:] == 7).all()) and bool((lse[:, n:] == 7).all())
    check_attention(out[:n], lse[:, :n].contiguous(), attention_oracle(c, host))
    # appending and reading with more rows than the offsets name
    before = x["k_pool"].view(torch.int16).clone()
    kv = torch.full((n + 9, c.kv_heads, D), 2.0, dtype=torch.bfloat16, device="cuda")
    cache.append(kv, kv, x["cu"])
    assert int((x["k_pool"].view(torch.int16) != before).sum()) <= n * c.kv_heads * D
    k = torch.full_like(kv, 5.0)
    cache.read(x["cu"], x["kv_len"] - n, out=(k, k.clone()))
    assert bool((k[n:] == 5).all()) and bool((k[:n] == 2).all()) and cache.check_status() == 0


@pytest.mark.parametrize("n", [1, 150])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_bad_tables_are_reported_and_skipped(n, fmt):
    """Every entry is bounds-checked on the device before it is used."""
    import torch
    c = Case("bad", (n, n), (n + 100, n + 30), page=16, unit=1, fmt=fmt)
    kv = torch.zeros((2 * n, 2, D), dtype=torch.bfloat16, device="cuda")
    two = lambda a, b: torch.tensor([a, b], dtype=torch.int32, device="cuda")
    for what in ("page", "len", "neg_len", "cu", "cu_neg", "short"):
        x, host = tensors(c)
        if what == "page":
            x["table"][0, 2] = x["k_pool"].shape[0]
        elif what == "len":
            x["kv_len"][0] = 1 << 30
        elif what == "neg_len":
            x["kv_len"][0] = -5
        elif what == "cu":
            x["cu"][1] = 5 * n
        elif what == "cu_neg":
            x["cu"][0] = -3
        else:
            x["kv_len"][0] = n - 1                         # fewer cached than new
        cache, out, lse = _attend(c, x)
        assert cache.check_status() == _lib.BSA_ERR_DEVICE_BOUNDS, what
        if what in ("page", "len", "neg_len", "short"):    # the other sequence is not touched by it
            o, l, bo, bl = attention_oracle(c, host)
            check_attention(out[n:], lse[:, n:].contiguous(), (o[n:], l[:, n:], bo[n:], bl[:, n:]))
        cache.append(kv, kv, x["cu"])
        if what == "page":                                 # no new token lies on that page
            cache.check_status()
        else:
            assert cache.check_status() == _lib.BSA_ERR_DEVICE_BOUNDS, what
        cache.read(x["cu"], two(0, 0), rows=2 * n)
        cache.check_status()
    x, _ = tensors(c)
    x["table"][1] = -1                                     # a new token without a page
    cache = cache_over(c, x)
    cache.append(kv, kv, x["cu"])
    assert cache.check_status() == _lib.BSA_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [3, 140])
def test_strided_queries_and_outputs_on_another_stream(n, fmt):
    import torch
    c = Case("strided", (n,), (n + 333,), heads=4, kv_heads=2, page=32, unit=1, fmt=fmt)
    x, host = tensors(c)
    side = torch.cuda.Stream()
    wide = torch.full((n, 7, D), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:5] = x["q"]
    out = torch.full((n, 6, D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((4, n), dtype=torch.float32, device="cuda")
    cache = cache_over(c, x)
    side.wait_stream(torch.cuda.current_stream())
    cache.attend(wide[:, 1:5], x["cu"], n, unit=1, out=out[:, 1:5], lse=lse, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    check_attention(out[:, 1:5], lse, attention_oracle(c, host))
    assert bool((out[:, [0, 5]] == 5).all())
    got = cache.attend(x["q"], x["cu"], n, unit=1)                        # own output, no lse
    assert torch.equal(got, out[:, 1:5]) and cache.check_status(side.cuda_stream) == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_captured_calls_follow_the_tables(fmt):
    """A captured append + attend replays for the next tokens after the tables moved on; two graphs that share
    the cache's workspace replay one after the other."""
    import torch
    from view_transformers_b200.cache import KVCache
    H, P = 2, 16
    cache = KVCache(1, H, H, pages=16, page_tokens=P, max_pages=16, fmt=fmt)
    rng = np.random.default_rng(3)
    total, chunk = 180, 6
    host = {n: bf16(rng.standard_normal((total, H, D))) for n in "qkv"}
    dev = {n: torch.from_numpy(host[n]).to(torch.bfloat16).cuda() for n in "qkv"}
    buf = {n: torch.zeros((chunk, H, D), dtype=torch.bfloat16, device="cuda") for n in "qkv"}
    out, one = (torch.zeros((chunk, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.zeros((H, chunk), dtype=torch.float32, device="cuda")
    cu = torch.tensor([0, chunk], dtype=torch.int32, device="cuda")
    cache.append(buf["k"], buf["v"], cu)                                  # warm-up: kv_len 0, reported and dropped
    cache.attend(buf["q"], cu, chunk, unit=1, out=out, lse=lse)
    assert cache.check_status() == _lib.BSA_ERR_DEVICE_BOUNDS
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        cache.append(buf["k"], buf["v"], cu)
        cache.attend(buf["q"], cu, chunk, unit=1, out=out, lse=lse)
    with torch.cuda.graph(g2):
        cache.attend(buf["q"], cu, 200, unit=1, out=one)                  # the form for many rows
    for at in range(0, total, chunk):
        cache.extend([chunk])
        for n in "qkv":
            buf[n].copy_(dev[n][at:at + chunk])
        g1.replay()
        g2.replay()
        if at in (0, 6, 60, 126, 132, 174):
            m = at + chunk
            c = Case("g", (chunk,), (m,), heads=H, kv_heads=H, unit=1, fmt=fmt)
            k, v = (okv.dequantise(*okv.quantise(host[n][:m])) if fmt == "e4m3" else host[n][:m] for n in "kv")
            want = attention_oracle(c, {"q": [host["q"][at:m]], "k": [k], "v": [v], "gone": [np.zeros(m, bool)]})
            check_attention(out, lse, want)
            check_attention(one, lse, want)
    assert cache.check_status() == 0
    K, V = cache.read_all(0)
    assert np.array_equal(K.double().cpu().numpy(), okv.dequantise(*okv.quantise(host["k"])) if fmt == "e4m3" else host["k"])


def test_two_caches_over_one_pool_on_two_streams():
    import torch
    cs = [Case("a", (1,), (3000,), page=64), Case("a", (1,), (3000,), page=64, unit=1)]
    x, host = tensors(cs[0])
    caches = [cache_over(c, x) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for c, cache, st in zip(cs, caches, streams):
            with torch.cuda.stream(st):
                outs.append(cache.attend(x["q"], x["cu"], 1, unit=c.unit))
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("n,fmt", [(1, "bf16"), (9, "e4m3"), (150, "bf16"), (150, "e4m3")])
def test_no_writes_outside_the_buffers(n, fmt):
    import torch
    from test_gpu_canary import Guarded
    c = Case("canary", (n, 3), (n + 200, 40), heads=4, kv_heads=2, page=16, unit=1, fmt=fmt)
    x, host = tensors(c)
    cache = cache_over(c, x)
    rows = x["rows"]
    g = {"out": Guarded(torch, rows * 4 * D * 2), "lse": Guarded(torch, rows * 4 * 4),
         "ws": Guarded(torch, cache.ws_bytes), "k": Guarded(torch, rows * 2 * D * 2), "v": Guarded(torch, rows * 2 * D * 2)}
    st = torch.cuda.current_stream().cuda_stream
    first = torch.zeros(2, dtype=torch.int32, device="cuda")
    sp = cache.status.data_ptr()
    _lib.bsa_kv_attention(cache.c, rows, n, 1, 0, 0, x["cu"].data_ptr(), x["q"].data_ptr(), 4 * D, g["out"].ptr, 4 * D,
                          g["lse"].ptr, g["ws"].ptr, cache.ws_bytes, sp, st)
    _lib.bsa_kv_read(cache.c, rows, x["cu"].data_ptr(), first.data_ptr(), g["k"].ptr, g["v"].ptr, 2 * D, sp, st)
    torch.cuda.synchronize()
    assert not [k for k, b in g.items() if not b.intact()] and cache.check_status() == 0
    got = g["out"].raw[g["out"].off:g["out"].off + rows * 4 * D * 2].view(torch.bfloat16).view(rows, 4, D)
    lse = g["lse"].raw[g["lse"].off:g["lse"].off + rows * 16].view(torch.float32).view(4, rows)
    check_attention(got, lse, attention_oracle(c, host))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_stream_of_frames_through_the_attention_block(fmt):
    """Frames arrive one by one: projection, append, attention over the first frame and the last two,
    output projection, each step against the oracle on the device's own tensors; then the cached scene is read
    back and taken by the block-sparse layer."""
    import torch
    from oracle.compare import rel_l2
    import oracle
    from view_transformers_b200 import configs, layer, synth
    from view_transformers_b200.cache import KVCache
    T, H, frames = 133, 2, 5
    w = configs.VGGT518.with_(name="kv_stream", frames=frames, heads=H, patch_per_frame=T - 5, tau=0.0)
    bi = synth.make_block_inputs(w)
    dev = lambda a: torch.from_numpy(a).cuda() if a.dtype == np.float32 else layer.to_device(a, "bf16")
    x, wq, bq, wo, bo = (dev(a) for a in (bi.x, bi.w_qkv, bi.b_qkv, bi.w_o, bi.b_o))
    cache = KVCache(1, H, H, pages=48, page_tokens=16, max_pages=48, fmt=fmt)
    blk = layer.AttentionBlock(1, T, 5, H, D, wq, bq, wo, bo, cache=cache, window=2, anchor=1)
    K, V = [], []
    for f in range(frames):
        y = blk.forward(x[f * T:(f + 1) * T].contiguous())
        assert blk.check_status() == 0
        q, k, v, o = (t.double().cpu().numpy() for t in (blk.q, blk.k, blk.v, blk.o))
        for acc, t in ((K, k), (V, v)):
            acc.append(okv.dequantise(*okv.quantise(t)) if fmt == "e4m3" else t)
        m = (f + 1) * T
        c = Case("s", (T,), (m,), heads=H, kv_heads=H, unit=T, window=2, sink=T, fmt=fmt)
        ro, _, bnd, _ = attention_oracle(c, {"q": [q], "k": [np.concatenate(K)], "v": [np.concatenate(V)],
                                             "gone": [np.zeros(m, bool)]})
        assert np.max(np.abs(o - ro) / bnd) <= 1.0
        ref = layer_io.out_project(o, synth.bf16_bits_to_f32(bi.w_o).astype(np.float64), bi.b_o)
        assert rel_l2(y.double().cpu().numpy(), ref) <= 2e-3
    assert cache.lengths == [frames * T]
    k, v = cache.read_all(0)
    assert np.array_equal(k.double().cpu().numpy(), np.concatenate(K))
    assert np.array_equal(v.double().cpu().numpy(), np.concatenate(V))
    L = layer.BlockSparseLayer.for_workload(w)
    q = torch.randn_like(k)
    out = L.forward(q, k, v).double().cpu().numpy()
    assert L.check_status() == 0
    lay = oracle.Layout(frames, T, 5, H, D, w.block)
    want = oracle.layer_forward(q.double().cpu().numpy(), np.concatenate(K), np.concatenate(V), lay, L.selected())
    assert rel_l2(out, want) <= 2e-3


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [1, 3])
def test_pieces_of_every_size_beside_one_another(fmt, group):
    """Chunks around the borders of query tiles (128 / group tokens) and pairs of them, in one call; sequences that
    end inside a page; windows and a sink; the same call under three bounds max_new."""
    import torch
    t = 128 // group
    new = (1, t - 1, 0, t, t + 1, 2 * t - 1, 2 * t, 2 * t + 1, 300, 5)
    lens = tuple(n + e for n, e in zip(new, (0, 130, 40, 1, 517, 0, 127, 256, 700, 1200)))
    for unit, window, sink in ((0, 0, 0), (1, 0, 0), (31, 4, 70)):
        c = Case("pieces", new, lens, heads=2 * group, kv_heads=2, page=32, fmt=fmt, unit=unit, window=window, sink=sink,
                 evict=((1, 2), (6, 0), (8, 11)))
        x, host = tensors(c, seed=unit)
        want = attention_oracle(c, host)
        for mx in (300, 17, 5000):
            cache, out, lse = _attend(c, x, max_new=mx)
            check_attention(out, lse, want)
        assert cache.check_status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,back", [(40, 20), (300, 150), (300, 40), (300, 299)])
def test_nan_values_inside_a_chunk(fmt, n, back):
    """The rows from the NaN on are spoiled, in every query tile that holds some; those before are not."""
    import torch
    c = Case("nan", (n,), (n + 70,), heads=1, kv_heads=1, page=64, fmt=fmt, unit=1)
    x, host = tensors(c)
    pos = n + 70 - back                                       # seen by the chunk's last `back` rows
    page, slot = int(x["table"][0, pos // 64]), pos % 64
    if fmt == "bf16":
        x["v_pool"][page, 0, slot, 33] = float("nan")
    else:
        x["v_scale"].view(torch.uint8)[page, 0, slot] = 255
    _, out, lse = _attend(c, x)
    o, l, bo, bl = attention_oracle(c, host)
    k = n - back
    check_attention(out[:k], lse[:, :k], (o[:k], l[:, :k], bo[:k], bl[:, :k]))
    bad = torch.isnan(out[k:, 0].float())
    assert bool(bad[:, 33].all())
    if fmt == "bf16":
        keep = [c for c in range(D) if c != 33]
        assert not bool(bad[:, keep].any())
        check_attention(out[k:][..., keep], lse[:, k:], (o[k:][..., keep], l[:, k:], bo[k:][..., keep], bl[:, k:]))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 12, 40, 200])
def test_a_nan_key_spoils_a_row_however_its_keys_are_split(n, fmt):
    import torch
    for m in (300, 2000, 6000):
        c = Case("nan", (n,), (m,), heads=2, kv_heads=2, page=64, fmt=fmt, unit=0)
        for pos in (0, m // 3, m - 1):
            x, _ = tensors(c)
            page, slot = int(x["table"][0, pos // 64]), pos % 64
            if fmt == "bf16":
                x["k_pool"][page, 1, slot, 9] = float("nan")
            else:
                x["k_scale"].view(torch.uint8)[page, 1, slot] = 255
            _, out, lse = _attend(c, x)
            assert bool(torch.isnan(out[:, 1]).all()) and bool(torch.isnan(lse[1]).all()), (m, pos)
            assert bool(torch.isfinite(out[:, 0]).all()) and bool(torch.isfinite(lse[0]).all())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_many_sequences(fmt):
    """More sequences than a warp has lanes, with few rows each and with many; the most there may be."""
    for new, lens, unit in ((tuple(i * 7 % 90 for i in range(45)), tuple(i * 7 % 90 + i * 31 % 300 for i in range(45)), 1),
                            (tuple(int(i % 9 == 0) for i in range(1024)), tuple(1 + i * 13 % 40 for i in range(1024)), 0)):
        c = Case("many", new, lens, heads=2, kv_heads=1, page=16, fmt=fmt, unit=unit)
        x, host = tensors(c)
        cache, out, lse = _attend(c, x)
        check_attention(out, lse, attention_oracle(c, host))
        assert cache.check_status() == 0


@pytest.mark.parametrize("n", [1, 100])
def test_sequences_that_share_pages(n):
    """A common prefix: the first pages of two sequences are the same pages."""
    import torch
    c = Case("prefix", (n, n), (n + 64, n + 64), heads=2, kv_heads=2, page=16, unit=1)
    x, host = tensors(c)
    x["table"][1, :4] = x["table"][0, :4]                     # 64 positions
    for kv in "kv":
        host[kv][1][:64] = host[kv][0][:64]
    cache, out, lse = _attend(c, x)
    check_attention(out, lse, attention_oracle(c, host))
    assert cache.check_status() == 0


def test_calls_without_rows():
    import torch
    c = Case("none", (0, 0), (5, 0))
    x, _ = tensors(c)
    cache = cache_over(c, x)
    empty = torch.empty((0, 2, D), dtype=torch.bfloat16, device="cuda")
    assert cache.attend(empty, x["cu"], 0).shape == (0, 2, D)
    cache.append(empty, empty, x["cu"])
    k, v = cache.read(x["cu"], torch.zeros(2, dtype=torch.int32, device="cuda"), rows=0)
    assert k.shape == v.shape == (0, 2, D) and cache.check_status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_pools_beyond_32_bit_offsets(fmt):
    """Pages whose bytes lie past 2^32: written, read back and attended over."""
    import torch
    from view_transformers_b200.cache import KVCache
    P, n, m = 256, 140, 700
    pages = (1 << 32) // (P * 64 * (2 if fmt == "bf16" else 1)) + 8
    dtype = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    pools = [torch.empty((pages, 1, P, D), dtype=dtype, device="cuda") for _ in range(2)]
    scales = [torch.empty((pages, 1, P), dtype=torch.uint8, device="cuda") for _ in range(2)] if fmt == "e4m3" else (None, None)
    table = torch.tensor([[pages - 1, pages - 4, pages - 2]], dtype=torch.int32, device="cuda")
    length = torch.tensor([m], dtype=torch.int32, device="cuda")
    cache = KVCache.over(*pools, table, length, 1, *scales)
    rng = np.random.default_rng(11)
    host = {s: bf16(rng.standard_normal((m, 1, D))) for s in "qkv"}
    dev = {s: torch.from_numpy(host[s]).to(torch.bfloat16).cuda() for s in "qkv"}
    cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    cache.append(dev["k"], dev["v"], cu)
    back = cache.read(cu, torch.zeros(1, dtype=torch.int32, device="cuda"), rows=m)
    for got, s in zip(back, "kv"):
        want = okv.dequantise(*okv.quantise(host[s])) if fmt == "e4m3" else host[s]
        assert np.array_equal(got.double().cpu().numpy(), want)
        host[s] = want
    for k in (1, n):
        c = Case("far", (k,), (m,), heads=1, kv_heads=1, fmt=fmt, unit=1)
        want = attention_oracle(c, {"q": [host["q"][:k]], "k": [host["k"]], "v": [host["v"]], "gone": [np.zeros(m, bool)]})
        lse = torch.empty((1, k), dtype=torch.float32, device="cuda")
        out = cache.attend(dev["q"][:k], torch.tensor([0, k], dtype=torch.int32, device="cuda"), k, unit=1, lse=lse)
        check_attention(out, lse, want)
    assert cache.check_status() == 0


@pytest.mark.parametrize("unit", [0, 1])
@pytest.mark.parametrize("max_new", [1, 1 << 20])
def test_work_beyond_the_limit_is_refused(max_new, unit):
    """2^20 new tokens over 2^30 positions (without pages): their products pass 2^32, and the call says so."""
    import torch
    from view_transformers_b200.cache import KVCache
    n, P = 1 << 20, 256
    pool = torch.zeros((1, 1, P, D), dtype=torch.bfloat16, device="cuda")
    table = torch.full((1, (1 << 30) // P), -1, dtype=torch.int32, device="cuda")
    cache = KVCache.over(pool, pool.clone(), table, torch.tensor([1 << 30], dtype=torch.int32, device="cuda"), 1)
    q = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    cache.attend(q, torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_new, unit=unit, out=out)
    assert cache.check_status() == _lib.BSA_ERR_UNSUPPORTED
    assert bool((out == 7).all())
    # one token over as many positions is no more than it can do
    one = cache.attend(q[:1], torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1, unit=unit)
    assert cache.check_status() == 0 and bool((one == 0).all())


def _held_up():
    """Work queued on the current stream that lasts about a tenth of a second."""
    import torch
    torch.cuda._sleep(200_000_000)


def _filled(n, H=2, pages=24, P=16, fmt="bf16", stream=None):
    """A cache of its own with n tokens, made and filled on the current stream or on `stream`, and what it then
    answers for one query: (cache, q, cu_new, out, k, v), computed on one stream with a wait before and after."""
    import torch
    from view_transformers_b200.cache import KVCache
    rng = np.random.default_rng(n)
    k, v, q = (torch.from_numpy(bf16(rng.standard_normal((n, H, D)))).to(torch.bfloat16).cuda() for _ in range(3))
    cache = KVCache(1, H, H, pages=pages, page_tokens=P, max_pages=pages, fmt=fmt)
    chunk = cache.extend([n])
    cache.append(k, v, chunk.cu_new)
    out = cache.attend(q, chunk.cu_new, n, unit=1)
    back = cache.read_all(0)
    torch.cuda.synchronize()
    assert cache.check_status() == 0
    return cache, q, chunk.cu_new, out, *back


@pytest.mark.parametrize("n", [3, 200])
def test_results_on_another_stream_are_not_touched_by_the_current_one(n):
    """The current stream still has work queued that writes blocks which Python has dropped; the results of calls on
    another stream, which does not wait for it, take other memory."""
    import torch
    cache, q, cu, out, k, v = _filled(n)
    side = torch.cuda.Stream()
    first = torch.zeros(1, dtype=torch.int32, device="cuda")
    calls = (lambda: (cache.attend(q, cu, n, unit=1, stream=side.cuda_stream),),
             lambda: cache.read(cu, first, rows=n, stream=side.cuda_stream),
             lambda: cache.read_all(0, stream=side.cuda_stream))
    for call, want in zip(calls, ((out,), (k, v), (k, v))):
        dropped = [torch.empty_like(w) for w in want]
        torch.cuda.synchronize()
        _held_up()
        for x in dropped:
            x.fill_(float("nan"))
        del dropped, x
        got = call()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
    assert cache.check_status() == 0


@pytest.mark.parametrize("n", [3, 200])
def test_a_cache_dropped_while_another_stream_works_on_it(n):
    """Its memory is given out again only when that stream is done. (What takes it here is as large as the pools; the
    workspace is of another size class.)"""
    import torch
    cache, q, cu, want, k, v = _filled(n)
    side = torch.cuda.Stream()
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _held_up()
    cache.attend(q, cu, n, unit=1, out=out, stream=side.cuda_stream)
    shape = cache.k.shape
    del cache
    takers = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del takers


@pytest.mark.parametrize("own", [True, False], ids=["its_tables", "callers_tables"])
def test_a_cache_made_behind_queued_work_and_used_on_another_stream(own):
    """The zeros that it begins with are written before the other stream's first call."""
    import torch
    from view_transformers_b200.cache import KVCache
    n, H = 40, 2
    _, q, cu, want, k, v = _filled(n)
    side = torch.cuda.Stream()
    st = side.cuda_stream
    pool = torch.zeros((3, H, 16, D), dtype=torch.bfloat16, device="cuda")
    args = (pool, pool.clone(), torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda"),
            torch.tensor([n], dtype=torch.int32, device="cuda"), H)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    _held_up()
    if own:
        cache = KVCache(1, H, H, pages=24, page_tokens=16, max_pages=24)
        cu = cache.extend([n], stream=st).cu_new
    else:
        cache = KVCache.over(*args)
    cache.append(k, v, cu, stream=st)
    cache.attend(q, cu, n, unit=1, out=out, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and cache.check_status() == 0


def test_a_cache_first_used_or_made_inside_a_capture():
    import torch
    from view_transformers_b200.cache import KVCache
    n, H = 40, 2
    _, q, cu, want, k, v = _filled(n)
    pool = torch.zeros((3, H, 16, D), dtype=torch.bfloat16, device="cuda")
    args = (pool, pool.clone(), torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda"),
            torch.tensor([n], dtype=torch.int32, device="cuda"), H)
    out = torch.empty_like(q)
    caches = [KVCache.over(*args)]
    for made_inside in (False, True):
        out.fill_(7.0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if made_inside:
                caches.append(KVCache.over(*args))
            caches[-1].append(k, v, cu)
            caches[-1].attend(q, cu, n, unit=1, out=out)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and caches[-1].check_status() == 0
        assert torch.equal(caches[-1].attend(q, cu, n, unit=1), want)      # and outside of it
        del g


def test_a_capture_goes_on_after_refused_changes_of_the_tables():
    """AttentionBlock(cache=) in a capture too: the refusal comes before the cache counts the frame."""
    import torch
    from view_transformers_b200 import layer
    n, H = 40, 2
    cache, q, cu, want, *_ = _filled(n)
    w = torch.zeros((3 * H * D, H * D), dtype=torch.bfloat16, device="cuda")
    blk = layer.AttentionBlock(1, 20, 5, H, D, w, None, w[:H * D].contiguous(), None, cache=cache)
    x = torch.zeros((20, H * D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    free = len(cache._free)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in (lambda: cache.extend([1]), lambda: cache.forget(0, 0, n), lambda: cache.release(0),
                     lambda: cache.read_all(0), lambda: blk.forward(x)):
            with pytest.raises(RuntimeError, match="captur"):
                call()
        cache.attend(q, cu, n, unit=1, out=out)
    assert cache.lengths == [n] and len(cache._free) == free
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and cache.check_status() == 0
    blk.forward(x)
    assert cache.lengths == [n + 20] and blk.check_status() == 0


GROUPS = [Case(f"group{g}_{fmt}", (1, n, 0, 3), (90, n + 150, 7, 300), heads=g * h, kv_heads=h, page=32, fmt=fmt, unit=1)
          for fmt in ("bf16", "e4m3")
          for g, h, n in ((5, 2, 60), (7, 2, 40), (12, 3, 25), (16, 1, 20), (33, 1, 9), (100, 1, 5), (128, 1, 5))]
PAGES = [Case(f"page256_{fmt}", (n,), (1100,), page=256, fmt=fmt, unit=unit, window=w, sink=s, evict=((0, 1),))
         for fmt in ("bf16", "e4m3") for n, unit, w, s in ((300, 1, 0, 0), (140, 70, 3, 600))]


@pytest.mark.parametrize("c", GROUPS + PAGES, ids=str)
def test_head_groups_and_long_pages_against_the_oracle(c):
    """Groups that do not divide a query tile, or leave it one token; pages of two key tiles."""
    x, host = tensors(c)
    want = attention_oracle(c, host)
    for mx in (x["max_new"], 1, 2000):
        cache, out, lse = _attend(c, x, max_new=mx)
        check_attention(out, lse, want)
        assert cache.check_status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,more,unit,window,sink", [
    (tuple(500 - 9 * i if i % 8 == 3 else i % 3 for i in range(40)), lambda i: i * 37 % 200, 1, 0, 0),
    (tuple(500 - 9 * i if i % 8 == 3 else i % 3 for i in range(40)), lambda i: i * 37 % 200, 60, 2, 21),
    ((190,) * 34, lambda i: i, 1, 0, 0),
], ids=["mixed", "mixed_window", "alike"])
def test_long_chunks_of_more_sequences_than_a_warp_has_lanes(fmt, new, more, unit, window, sink):
    """Chunks of many row groups (of 8, 128 or 256 rows, by max_new) between short and empty ones."""
    lens = tuple(n + more(i) for i, n in enumerate(new))
    c = Case("long", new, lens, heads=4, kv_heads=1, page=64, fmt=fmt, unit=unit, window=window, sink=sink)
    x, host = tensors(c)
    want = attention_oracle(c, host)
    for mx in (x["max_new"], 1, 5000):
        cache, out, lse = _attend(c, x, max_new=mx)
        check_attention(out, lse, want)
        assert cache.check_status() == 0


@pytest.mark.parametrize("max_new", [1, 1 << 20])
@pytest.mark.parametrize("unit", [0, 1])
@pytest.mark.parametrize("what", ["one", "sum"])
def test_work_of_many_sequences_beyond_the_limits_is_refused(what, unit, max_new):
    """2^25 units (of a query tile and 128 keys) in one sequence, 2^30 in all; positions without pages."""
    import torch
    from view_transformers_b200.cache import KVCache
    S, P, far = 40, 256, 1 << 30
    # sum: four tiles of 8, 128 rows each in every sequence: 2^25 a sequence, 40 of them
    n = [1] * S if what == "one" else [4 * (8 if max_new == 1 else 128)] * S
    if what == "one":
        n[17] = 1 << 20
    lens = [far] * S if what == "sum" else [n[i] if i != 17 else far for i in range(S)]
    pool = torch.zeros((1, 1, P, D), dtype=torch.bfloat16, device="cuda")
    table = torch.full((S, far // P), -1, dtype=torch.int32, device="cuda")
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache = KVCache.over(pool, pool.clone(), table, length, 1)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
    q = torch.zeros((sum(n), 1, D), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    cache.attend(q, cu, max_new, unit=unit, out=out)
    assert cache.check_status() == _lib.BSA_ERR_UNSUPPORTED
    assert bool((out == 7).all())
    one = torch.arange(S + 1, dtype=torch.int32, device="cuda")           # one token each over 1,000 positions
    length.fill_(1000)
    assert bool((cache.attend(q[:S], one, 1, unit=unit) == 0).all()) and cache.check_status() == 0
