"""Paged key/value cache without a GPU: the oracle's pins, the host-side refusals of the C ABI, and the page
bookkeeping of KVCache."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv_cache as okv
from view_transformers_b200 import _lib, build
from view_transformers_b200.cache import KVCache

E = _lib
A = 0x10000   # aligned fake device address (never dereferenced: validation fails first)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


# ------------------------------------------------------------------ oracle pins

def test_e4m3_grid_is_torchs():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(okv.e4m3_grid(), codes)


def test_round_e4m3_matches_torch_conversion():
    """Within +-448 torch's conversion is round to nearest even too; ties and subnormals included."""
    g = okv.e4m3_grid()
    mid = (g[1:] + g[:-1]) / 2
    x = np.concatenate([g, mid, np.nextafter(mid, 0), np.nextafter(mid, 999), np.random.default_rng(0).normal(0, 50, 4000)])
    x = x[np.abs(x) <= 448]
    x = np.concatenate([x, -x]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(okv.round_e4m3(x.astype(np.float64)), want)
    assert okv.round_e4m3(np.array([449.0, 1e9, -460.0])).tolist() == [448.0, 448.0, -448.0]


def test_quantise_exponent_is_the_smallest_that_fits():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 64)) * 2.0 ** rng.integers(-60, 12, (200, 1))
    vals, e = okv.quantise(x)
    top = np.abs(x).max(-1)
    assert (top <= 448 * 2.0 ** e).all() and ((top > 448 * 2.0 ** (e - 1)) | (e == -64)).all()
    assert np.abs(okv.dequantise(vals, e) - x).max(-1).max() <= (2.0 ** -4 * top).max()
    # borders: exactly 448 2^k fits, the next bf16 number does not; zero rows and saturation
    for v, want in ((448.0, 0), (450.0, 1), (224.0, -1), (0.0, -64), (448.0 * 2 ** 15, 15), (1e9, 15)):
        assert okv.quantise(np.full((1, 64), v))[1][0] == want
    assert np.isnan(okv.quantise(np.array([[np.inf] + [0.0] * 63]))[0]).all()


def test_seen_closed_forms():
    assert okv.seen(5, 2).all()
    assert okv.seen(4, 4, unit=1).tolist() == np.tril(np.ones((4, 4), bool)).tolist()
    # frames of 2: tokens 2, 3 see frames 0 and 1; token 4 starts frame 2
    assert okv.seen(5, 3, unit=2).tolist() == [[1, 1, 1, 1, 0], [1, 1, 1, 1, 0], [1, 1, 1, 1, 1]]
    assert okv.seen(6, 2, unit=2, window=1).tolist() == [[0, 0, 0, 0, 1, 1]] * 2
    assert okv.seen(6, 1, unit=2, window=1, sink=1).tolist() == [[1, 0, 0, 0, 1, 1]]


def test_attention_matches_torch_softmax():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 4, 64)), rng.standard_normal((9, 2, 64)), rng.standard_normal((9, 2, 64))
    see = okv.seen(9, 3, unit=1)
    out, lse = okv.attention(q, k, v, see)
    s = torch.einsum("nhd,lhd->hnl", torch.from_numpy(q), torch.from_numpy(k).repeat_interleave(2, 1)) / 8
    s = s.masked_fill(~torch.from_numpy(see), -float("inf"))
    want = torch.einsum("hnl,lhd->nhd", s.softmax(-1), torch.from_numpy(v).repeat_interleave(2, 1))
    assert np.allclose(out, want.numpy(), rtol=0, atol=1e-13) and np.allclose(lse, s.logsumexp(-1).numpy(), atol=1e-13)
    out, lse = okv.attention(q, k, v, np.zeros((3, 9), bool))
    assert (out == 0).all() and np.isneginf(lse).all()


# ------------------------------------------------------------------ refusals (nothing is launched)

def _cache(**kw):
    base = dict(seqs=2, heads=4, kv_heads=2, head_dim=64, page_tokens=16, pages=8, max_pages=4, format=E.BSA_KV_E4M3,
                k=A, v=A, k_scale=A, v_scale=A, page_table=A, kv_len=A)
    base.update(kw)
    return ctypes.byref(_lib.bsa_kv_cache(**base))


BAD_SIZES = [
    (dict(seqs=0), E.BSA_ERR_INVALID_ARG), (dict(heads=0), E.BSA_ERR_INVALID_ARG),
    (dict(heads=3), E.BSA_ERR_INVALID_ARG), (dict(kv_heads=0), E.BSA_ERR_INVALID_ARG),
    (dict(pages=0), E.BSA_ERR_INVALID_ARG), (dict(max_pages=0), E.BSA_ERR_INVALID_ARG),
    (dict(format=7), E.BSA_ERR_INVALID_ARG), (dict(page_tokens=0), E.BSA_ERR_INVALID_ARG),
    (dict(head_dim=128), E.BSA_ERR_UNSUPPORTED), (dict(page_tokens=8), E.BSA_ERR_UNSUPPORTED),
    (dict(page_tokens=48), E.BSA_ERR_UNSUPPORTED), (dict(page_tokens=512), E.BSA_ERR_UNSUPPORTED),
    (dict(seqs=1025), E.BSA_ERR_UNSUPPORTED), (dict(heads=130), E.BSA_ERR_UNSUPPORTED),
    (dict(pages=1 << 27), E.BSA_ERR_UNSUPPORTED), (dict(max_pages=1 << 28), E.BSA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_SIZES, ids=lambda x: str(x))
def test_bad_sizes_are_refused_by_every_call(lib, kw, code):
    n = ctypes.c_size_t()
    assert lib.bsa_kv_workspace_size(_cache(**kw), ctypes.byref(n)) == code
    assert lib.bsa_kv_append(_cache(**kw), 1, A, A, A, 128, None, None) == code
    assert lib.bsa_kv_read(_cache(**kw), 1, A, A, A, A, 128, None, None) == code
    assert lib.bsa_kv_attention(_cache(**kw), 1, 1, 0, 0, 0, A, A, 256, A, 256, None, A, 1 << 40, None, None) == code


def test_bad_arguments_are_refused(lib):
    I, U = E.BSA_ERR_INVALID_ARG, E.BSA_ERR_UNSUPPORTED
    n = ctypes.c_size_t()
    assert lib.bsa_kv_workspace_size(_cache(), ctypes.byref(n)) == E.BSA_OK and n.value > 0
    assert lib.bsa_kv_workspace_size(_cache(), None) == I
    assert lib.bsa_kv_workspace_size(None, ctypes.byref(n)) == I
    for kw in (dict(k=None), dict(v=A + 8), dict(k_scale=None), dict(v_scale=A + 4), dict(page_table=None),
               dict(kv_len=A + 2)):
        assert lib.bsa_kv_append(_cache(**kw), 1, A, A, A, 128, None, None) == I, kw
    assert lib.bsa_kv_append(_cache(), -1, A, A, A, 128, None, None) == I
    assert lib.bsa_kv_append(_cache(), 1, None, A, A, 128, None, None) == I
    assert lib.bsa_kv_append(_cache(), 1, A, None, A, 128, None, None) == I
    assert lib.bsa_kv_append(_cache(), 1, A, A, A + 8, 128, None, None) == I
    assert lib.bsa_kv_append(_cache(), 1, A, A, A, 120, None, None) == I          # rows overlap
    assert lib.bsa_kv_append(_cache(), 1, A, A, A, 132, None, None) == I          # not a multiple of 8
    assert lib.bsa_kv_append(_cache(), 1 << 30, A, A, A, 128, None, None) == U    # rows * heads
    assert lib.bsa_kv_append(_cache(), 0, A, None, None, 128, None, None) == E.BSA_OK
    assert lib.bsa_kv_read(_cache(), 1, A, None, A, A, 128, None, None) == I
    assert lib.bsa_kv_read(_cache(), 1, A, A, A, None, 128, None, None) == I
    att = lambda **kw: lib.bsa_kv_attention(*[{**dict(c=_cache(), rows=1, mx=1, unit=0, win=0, sink=0, cu=A, q=A, qs=256,
                                              o=A, os=256, lse=None, ws=A, wb=n.value, st=None, stream=None), **kw}[x]
                                              for x in "c rows mx unit win sink cu q qs o os lse ws wb st stream".split()])
    for kw in (dict(rows=-1), dict(mx=-1), dict(unit=-1), dict(win=-1, unit=1), dict(win=1), dict(sink=1, unit=1),
               dict(sink=-1, unit=1, win=1), dict(cu=None), dict(q=None), dict(q=A + 8), dict(o=None), dict(qs=248),
               dict(os=252), dict(lse=A + 2), dict(ws=None), dict(ws=A + 8), dict(wb=n.value - 1), dict(st=A + 1)):
        assert att(**kw) == I, kw
    assert att(rows=0, q=None, o=None, ws=None) == E.BSA_OK


# ------------------------------------------------------------------ page bookkeeping

def _own(**kw):
    base = dict(seqs=2, heads=4, kv_heads=2, pages=6, page_tokens=16, max_pages=5, fmt="e4m3", device="cpu")
    base.update(kw)
    return KVCache(**base)


def test_extend_takes_pages_and_counts(lib):
    c = _own()
    ch = c.extend([17, 0])
    assert ch.cu_new.tolist() == [0, 17, 17] and (ch.max_new, ch.rows) == (17, 17)
    assert c.kv_len.tolist() == [17, 0] and (c.page_table[0] >= 0).sum() == 2 and (c.page_table[1] < 0).all()
    ch = c.extend([15, 33])
    assert ch.cu_new.tolist() == [0, 15, 48] and c.kv_len.tolist() == [32, 33]
    used = c.page_table[c.page_table >= 0].tolist()
    assert sorted(used) == sorted(set(used)) and len(used) == 5     # no page given twice
    before = c.page_table.clone(), list(c.lengths)
    with pytest.raises(RuntimeError, match="free"):
        c.extend([32, 0])
    with pytest.raises(RuntimeError, match="max_pages"):
        c.extend([0, 60])
    assert torch.equal(c.page_table, before[0]) and c.lengths == before[1]
    with pytest.raises(ValueError):
        c.extend([1])
    with pytest.raises(ValueError):
        c.extend([1, -1])


def test_forget_and_release_return_pages(lib):
    c = _own()
    c.extend([40, 16])
    c.forget(0, 5, 40)                                              # only page 1 lies wholly inside [5, 40)
    assert (c.page_table[0] >= 0).tolist() == [True, False, True, False, False]
    c.extend([0, 48])                                               # 3 pages: the forgotten one and the 2 free ones
    assert (c.page_table[1] >= 0).sum() == 4
    c.release(0)
    assert c.kv_len.tolist() == [0, 64] and (c.page_table[0] < 0).all()
    c.extend([32, 0])
    live = c.page_table[c.page_table >= 0].tolist()
    assert len(live) == len(set(live)) == 6


def test_wrapped_tensors_are_checked(lib):
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    t, n = torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    c = KVCache.over(k, k.clone(), t, n, heads=4)
    assert c.fmt == "bf16"
    for call in (lambda: c.extend([1]), lambda: c.release(0), lambda: c.read_all(0)):
        with pytest.raises(RuntimeError):
            call()
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    bad = [lambda: KVCache.over(k, k[:3], t, n, 4), lambda: KVCache.over(k.float(), k.float(), t, n, 4),
           lambda: KVCache.over(k, k, t.long(), n, 4), lambda: KVCache.over(k, k, t, t[0], 4),
           lambda: KVCache.over(k.transpose(1, 2), k.transpose(1, 2), t, n, 4),
           lambda: KVCache.over(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn), t, n, 4),
           lambda: c.attend(q.float(), cu, 1), lambda: c.attend(q[:, :2], cu, 1), lambda: c.attend(q, cu.long(), 1),
           lambda: c.attend(q, cu[:1], 1), lambda: c.attend(q, cu, 1, out=q[:2]),
           lambda: c.attend(q, cu, 1, out=q, lse=torch.zeros(4, 2)), lambda: c.append(q[:, :2], q[:2, :2], cu),
           lambda: c.append(q[:, ::2], q[:, ::2], cu), lambda: c.read(cu, cu), lambda: c.read(cu, cu, rows=3)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"case {i} was accepted")
    with pytest.raises(_lib.BsaError):
        KVCache.over(k, k, t, n, heads=3)
    with pytest.raises(ValueError):
        _own(fmt="int8")


def test_attention_block_checks_its_cache_arguments(lib):
    from view_transformers_b200.layer import AttentionBlock
    w = torch.zeros((1, 1), dtype=torch.bfloat16)
    block = lambda heads=4, **kw: AttentionBlock(1, 20, 5, heads, 64, w, None, w, None, device="cpu", **kw)
    own = _own(seqs=1, kv_heads=4)
    assert block(own.heads, cache=own, window=2, anchor=1).sink == 20
    for kw in (dict(window=1), dict(anchor=1), dict(cache=own, window=-1), dict(cache=own, anchor=-1),
               dict(cache=own, layer=object())):
        with pytest.raises(ValueError):
            block(own.heads, **kw)
    with pytest.raises(ValueError):
        block(own.heads * 2, cache=own)


# ------------------------------------------------------------------ streams

def test_results_come_from_the_memory_of_the_stream_that_writes_them(lib, monkeypatch):
    """A block of the current stream's memory may still be in use by work queued there; a call on another stream
    does not wait for that work."""
    import contextlib
    c = _own()
    c.extend([20, 3])
    inside, taken, kept = [], [], []

    @contextlib.contextmanager
    def on(stream):
        inside.append(stream)
        yield
        inside.pop()

    empty = torch.empty
    monkeypatch.setattr(c, "_torch_stream", on)
    monkeypatch.setattr(c, "_call", lambda *a: None)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (taken.append(inside[-1:]), empty(*a, **k))[1])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: h)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda x, s: kept.append(s))
    q = torch.zeros((23, 4, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 20, 23], dtype=torch.int32)
    first = torch.zeros(2, dtype=torch.int32)
    for call, n in ((lambda s: c.attend(q, cu, 20, stream=s), 1), (lambda s: c.read(cu, first, rows=23, stream=s), 2),
                    (lambda s: c.read_all(0, stream=s), 2)):
        for stream in (77, None):
            taken.clear()
            kept.clear()
            call(stream)
            assert taken == [[stream]] * n
            assert kept == (["current"] * n if stream else [])


def _on_a_device(c, monkeypatch, current=5):
    """The cache believes to be on device 0, whose current stream is `current`; streams are their handles."""
    from view_transformers_b200 import cache
    c.device, c._index = torch.device("cuda", 0), 0
    monkeypatch.setattr(cache, "_raw_stream", lambda index: current)
    monkeypatch.setattr(cache, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: h)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_caches_tensors_are_kept_for_every_stream_that_works_on_them(lib, monkeypatch, fmt):
    c = _own(fmt=fmt)
    _on_a_device(c, monkeypatch)
    own = {t.data_ptr() for t in (c.k, c.v, c.k_scale, c.v_scale, c.page_table, c.kv_len, c.workspace, c.status)
           if t is not None}
    kept = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda x, s: kept.append((s, x.data_ptr())))
    used = []
    for stream in (77, 77, None, 78, None, 77):
        c._call("call", lambda ref, *a: used.append(a) or 0, stream, "argument")
    assert used == [("argument", s) for s in (77, 77, 5, 78, 5, 77)]
    assert sorted(kept) == sorted((s, p) for s in (77, 5, 78) for p in own)


def test_a_stream_waits_once_until_the_caches_tensors_are_made(lib, monkeypatch):
    class Stream(int):
        def wait_event(self, event):
            waits.append((int(self), event))

    c = _own()
    _on_a_device(c, monkeypatch)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: Stream(h))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda x, s: None)
    monkeypatch.setattr(c, "_capturing", lambda stream: stream == 79)
    c._made, waits = "made", []
    for stream in (77, 77, None, 79, 79, 78):
        c._call("call", lambda ref, *a: 0, stream)
    assert waits == [(77, "made"), (5, "made"), (78, "made")]


def test_what_changes_the_tables_is_refused_in_a_capture_before_any_change(lib, monkeypatch):
    def fails(*a):
        raise RuntimeError("operation not permitted when stream is capturing")

    c = _own()
    c.extend([40, 7])
    before = list(c.lengths), c._table.clone(), list(c._free)
    _on_a_device(c, monkeypatch)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: 5)
    monkeypatch.setattr(c, "_capturing", lambda stream: True)
    monkeypatch.setattr(c, "_upload", fails)               # what a copy from host memory does there
    for call in (lambda: c.extend([1, 1]), lambda: c.extend([1, 1], stream=77), lambda: c.forget(0, 0, 16),
                 lambda: c.release(0), lambda: c.read_all(0)):
        with pytest.raises(RuntimeError, match="captur"):
            call()
        assert c.lengths == before[0] and torch.equal(c._table, before[1]) and c._free == before[2]


def test_sequences_counted_from_the_end(lib, monkeypatch):
    """read_all(-1) reads the last sequence: its offsets hold all of the result's rows."""
    c = _own()
    c.extend([20, 33])
    got = []
    monkeypatch.setattr(c, "read", lambda cu, first, rows, stream: got.append((cu.tolist(), rows)))
    for seq in (-1, 1, 0, -2):
        c.read_all(seq)
    assert got == [([0, 0, 33], 33), ([0, 0, 33], 33), ([0, 20, 20], 20), ([0, 20, 20], 20)]
    for call in (c.read_all, c.release, lambda s: c.forget(s, 0, 20)):
        for seq in (2, -3):
            with pytest.raises(IndexError):
                call(seq)
    assert c.lengths == [20, 33] and len(c._free) == 1
    c.forget(-1, 0, 16)
    c.release(-2)
    assert c.lengths == [0, 33] and c.page_table[1].tolist()[0] == -1 and len(c._free) == 4


def test_numbers_beyond_32_bits_are_refused(lib, monkeypatch):
    """Cut to 32 bits, a window of 2^32 + 1 units would be one of 1."""
    c = _own()
    calls = []
    monkeypatch.setattr(c, "_call", lambda name, fn, stream, *a: calls.append(a[1:5]))
    q, cu = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for name in ("max_new", "unit", "window", "sink"):
        for n in (2 ** 31, 2 ** 32 + 1, -2 ** 32 + 1):
            with pytest.raises(ValueError, match=name):
                c.attend(q, cu, **{**dict(max_new=3, unit=1, window=1, sink=1), name: n})
    most = 2 ** 31 - 1
    c.attend(q, cu, most, unit=most, window=most, sink=most)
    assert calls == [(most,) * 4]
    for name in ("seqs", "heads", "kv_heads", "head_dim", "page_tokens", "pages", "max_pages"):
        good = dict(seqs=2, heads=4, kv_heads=2, head_dim=64, page_tokens=16, pages=6, max_pages=5)[name]
        with pytest.raises(ValueError, match=name):
            _own(**{name: 2 ** 32 + good})
    with pytest.raises(ValueError, match="heads"):
        KVCache.over(c.k, c.v, c.page_table, c.kv_len, 2 ** 32 + 4, c.k_scale, c.v_scale)


def test_attention_block_refuses_a_cache_that_its_steps_cannot_fill(lib):
    """When the block is made: a step counts its tokens in the cache before it appends them."""
    from view_transformers_b200.layer import AttentionBlock
    w = torch.zeros((1, 1), dtype=torch.bfloat16)
    own = _own(seqs=1, kv_heads=4)
    over = KVCache.over(own.k, own.v, own.page_table, own.kv_len, 4, own.k_scale, own.v_scale)
    block = lambda head_dim=64, device="cpu", **kw: AttentionBlock(1, 20, 5, 4, head_dim, w, None, w, None, device=device, **kw)
    block(cache=own, window=3, anchor=1)
    for kw, why in ((dict(cache=own, device="meta"), "on cpu"), (dict(cache=own, head_dim=32), "64 elements"),
                    (dict(cache=over), "own tables"), (dict(cache=own, window=2 ** 31), "32 bits"),
                    (dict(cache=own, window=1, anchor=2 ** 31 // 20 + 1), "32 bits")):
        with pytest.raises(ValueError, match=why):
            block(**kw)


def test_attention_block_clears_every_status_that_it_checks(lib, monkeypatch):
    """An error of the cache beside one of the block's own belongs to this check, not to the next."""
    from view_transformers_b200 import layer
    w = torch.zeros((1, 1), dtype=torch.bfloat16)
    own = _own(seqs=1, kv_heads=4)
    blk = layer.AttentionBlock(1, 20, 5, 4, 64, w, None, w, None, device="cpu", cache=own)
    status = {blk.status.data_ptr(): 0, "cache": 0}

    def check(key):
        code, status[key] = status[key], 0
        return code

    monkeypatch.setattr(_lib, "bsa_check_status", lambda p, stream: check(p))
    monkeypatch.setattr(own, "check_status", lambda stream: check("cache"))
    for mine, cache, want in ((0, 0, 0), (5, 0, 5), (0, 6, 6), (5, 6, 5)):
        status.update({blk.status.data_ptr(): mine, "cache": cache})
        assert blk.check_status(stream=77) == want
        assert blk.check_status(stream=77) == 0
