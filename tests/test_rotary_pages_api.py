"""Refusals of the rotary and page-keeping entry points before anything is launched, and the rotary
frequencies (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def kv():
    import kv_cache_eviction_split_gb300 as kv
    kv.build()
    kv.load()
    return kv


def _cache(kv, R=2, L=3, H=2, Hq=8, d=128, page=64, **kw):
    import torch
    return kv.PagedCache.allocate(R, L, H, Hq, d, 100, page, torch.bfloat16, True, device="cpu", **kw)


F = 1 << 20   # a device address that is never used: the checks fail first


def _each(fn, good, bad):
    for i, value, code in bad:
        a = list(good)
        a[i] = value
        assert fn(*a) == code, (i, value)


def test_rotary_argument_checks(kv):
    lib, INV, UNS = kv.load(), kv.KV_ERR_INVALID_ARG, kv.KV_ERR_UNSUPPORTED

    def rot(dims=64, factor=1.0, freq=F):
        return ctypes.byref(kv._KvRotation(dims, 0, factor, freq))

    good = [rot(), F, 10, 4, 128, 0, F, 512, 128, 2 * F, 512, 128, 0, None]
    _each(lib.kv_rotary, good, [
        (0, None, INV), (0, rot(-16), INV), (0, rot(144), INV), (0, rot(24), UNS), (0, rot(freq=None), INV),
        (0, rot(factor=math.inf), INV), (0, rot(factor=math.nan), INV), (0, rot(freq=F + 2), INV),
        (1, None, INV), (1, F + 2, INV),
        (2, -1, INV), (2, 1 << 40, UNS), (3, 0, INV), (3, 1 << 24, UNS), (4, 96, UNS), (5, 2, INV), (6, None, INV),
        (6, F + 8, INV), (7, -8, INV), (7, 12, INV), (8, 4, INV), (9, None, INV), (9, F + 2, INV),
        (10, 120, INV), (11, 64, INV)])
    inplace = list(good)
    inplace[9] = F
    inplace[7] = 1024
    assert lib.kv_rotary(*inplace) == INV                       # other strides than the input's
    # rows of out on one another: 4 heads 128 apart with tokens 128 .. 504 apart, 10 tokens 512 apart
    # with heads less than 10 * 512 - 384 apart
    for strides in ((128, 128), (384, 128), (504, 128), (512, 256), (512, 4728), (1 << 62, 1 << 62)):
        _each(lib.kv_rotary, [*good[:10], *strides, *good[12:]], [(2, 10, INV)])
    none = list(good)
    none[2] = 0
    assert lib.kv_rotary(*none) == kv.KV_OK


def test_append_rotary_argument_checks(kv):
    lib, INV, UNS = kv.load(), kv.KV_ERR_INVALID_ARG, kv.KV_ERR_UNSUPPORTED
    c, t = _cache(kv), kv.Chunk([1, 5], device="cpu")
    rot = kv._KvRotation(64, 0, 1.0, F)
    good = [c.c, t.c, 0, ctypes.byref(rot), F, None, F, 1024, 2 * F, 1024, F, 256, F, 256, None]
    _each(lib.kv_paged_append_rotary, good, [
        (0, None, INV), (1, None, INV), (2, 3, INV), (2, -1, INV), (3, None, INV), (4, None, INV),
        (4, F + 1, INV), (5, F + 4, INV), (6, F + 4, INV), (7, 1016, INV),
        (7, 1028, INV), (8, None, INV), (8, F + 8, INV), (9, 1000, INV),
        (10, None, INV), (11, 248, INV), (12, F + 2, INV), (13, 260, INV)])
    rot.dims = 144
    assert lib.kv_paged_append_rotary(*good) == INV
    rot.dims = 40
    assert lib.kv_paged_append_rotary(*good) == UNS
    rot.dims = 64
    good[8], good[9] = good[6], 2048
    assert lib.kv_paged_append_rotary(*good) == INV             # in place with another stride
    none = kv.Chunk([0, 0], device="cpu")
    assert lib.kv_paged_append_rotary(c.c, none.c, 0, ctypes.byref(rot), None, None, None, 0, None, 0, None, 0,
                                      None, 0, None) == kv.KV_OK


def test_page_keeping_argument_checks(kv):
    lib, INV = kv.load(), kv.KV_ERR_INVALID_ARG
    c, t = _cache(kv), kv.Chunk([1, 5], device="cpu")
    ws = kv.kv_paged_reserve_workspace_size(c)
    _each(lib.kv_paged_reserve, [c.c, t.c, F, None, F, ws, None],
          [(0, None, INV), (1, None, INV), (2, None, INV), (2, F + 4, INV), (3, F + 4, INV), (4, None, INV),
           (4, F + 8, INV), (5, ws - 1, kv.KV_ERR_WORKSPACE)])
    ws = kv.kv_paged_compact_workspace_size(c)
    _each(lib.kv_paged_compact, [c.c, F, None, None, F, ws, None],
          [(0, None, INV), (1, None, INV), (1, F + 4, INV), (2, F + 4, INV), (3, F + 2, INV), (4, None, INV),
           (5, ws - 1, kv.KV_ERR_WORKSPACE)])
    _each(lib.kv_paged_fork, [c.c, F, F, None], [(0, None, INV), (1, None, INV), (1, F + 4, INV), (2, None, INV),
                                                  (2, F + 2, INV)])
    _each(lib.kv_paged_count_refs, [c.c, F, None], [(0, None, INV), (1, None, INV), (1, F + 4, INV)])
    d = _cache(kv)
    _each(lib.kv_paged_place_positions, [c.c, F, d.c, 2 * F, F, 50, None, None],
          [(0, None, INV), (1, None, INV), (2, None, INV), (2, _cache(kv, H=4).c, INV), (3, F, INV), (4, None, INV),
           (5, -1, INV), (1, F + 4, INV), (3, 2 * F + 4, INV), (4, F + 2, INV), (6, F + 4, INV)])
    assert lib.kv_paged_place_positions(c.c, F, None, None, None, 0, F, None) == INV
    for name in ("kv_paged_reserve_workspace_size", "kv_paged_compact_workspace_size"):
        assert getattr(lib, name)(None, ctypes.byref(ctypes.c_size_t())) == INV
        assert getattr(lib, name)(c.c, None) == INV
    # more tokens than the pool has rows
    big = kv.Chunk([1 << 20, 0], device="cpu")
    assert lib.kv_paged_reserve(c.c, big.c, F, None, F, 1 << 40, None) == kv.KV_ERR_BUDGET
    c._c.num_requests = 16385
    assert lib.kv_paged_fork(c.c, F, F, None) == kv.KV_ERR_UNSUPPORTED


def test_scored_attention_argument_checks(kv):
    lib, INV, UNS = kv.load(), kv.KV_ERR_INVALID_ARG, kv.KV_ERR_UNSUPPORTED
    c, t = _cache(kv), kv.Chunk([1, 5], device="cpu")
    assert not any([kv._KvScoring().softcap, kv._KvScoring().slopes])

    def form(softcap=30.0, window=0, sinks=0, slopes=F, pos=None, first=None, last=None):
        return ctypes.byref(kv._KvScoring(softcap, window, sinks, slopes, pos, first, last))

    size = kv.kv_paged_attention_scored_workspace_size(c, t)
    good = [c.c, t.c, 0, form(), 0.1, F, 1024, 2 * F, 1024, None, 0, 3 * F, size, None]
    _each(lib.kv_paged_attention_scored, good, [
        (0, None, INV), (1, None, INV), (2, -1, INV), (2, 3, INV), (3, None, INV), (3, form(-1.0), INV),
        (3, form(math.nan), INV), (3, form(math.inf), INV), (3, form(window=-1), INV), (3, form(sinks=-1), INV),
        (3, form(slopes=F + 2), INV), (3, form(first=F + 1), INV), (3, form(last=F + 2), INV),
        (3, form(pos=F + 4), INV), (4, 0.0, INV), (4, -0.1, INV), (4, math.nan, INV), (4, math.inf, INV),
        (4, 1e-40, INV), (5, None, INV), (5, F + 8, INV), (6, 1016, INV), (6, 1028, INV), (7, None, INV),
        (7, 2 * F + 2, INV), (8, 512, INV), (9, F + 4, INV), (11, None, INV), (11, F + 8, INV),
        (12, size - 1, kv.KV_ERR_WORKSPACE)])
    few = kv.Chunk([4, 1], device="cpu")                        # 16 query rows a head: weights are added
    assert kv.kv_paged_attention_scored_workspace_size(c, few, True) > 0
    _each(lib.kv_paged_attention_scored, good, [(10, 1, UNS)])
    with pytest.raises(kv.KvError) as e:
        kv.kv_paged_attention_scored_workspace_size(c, t, True)
    assert e.value.code == UNS
    bare = kv.PagedCache.allocate(2, 3, 2, 8, 128, 100, 64, c.k_pages.dtype, False, device="cpu")
    with pytest.raises(kv.KvError) as e:                        # no weights to add to
        kv.kv_paged_attention_scored_workspace_size(bare, few, True)
    assert e.value.code == INV
    none = list(good)
    none[1] = kv.Chunk([0, 0], device="cpu").c
    none[5] = none[7] = none[11] = None
    assert lib.kv_paged_attention_scored(*none) == kv.KV_OK
    null = ctypes.POINTER(ctypes.c_size_t)()
    assert lib.kv_paged_attention_scored_workspace_size(c.c, t.c, 0, null) == INV


def test_scored_attention_binding_refusals(kv):
    import torch
    c, t = _cache(kv, positions=True), kv.Chunk([1, 5], device="cpu")
    size = kv.kv_paged_attention_scored_workspace_size(c, t)
    q = torch.zeros((6, 8, 128), dtype=torch.bfloat16)
    good = dict(cache=c, chunk=t, layer=0, q=q, out=q.clone(), workspace=torch.zeros(size, dtype=torch.uint8))
    i6 = torch.zeros(6, dtype=torch.int32)
    for name, value in [
            ("q", q[:5]), ("q", q.half()), ("out", q[:, :4]), ("lse", torch.zeros((6, 7))),
            ("lse", torch.zeros((6, 8), dtype=torch.float64)), ("slopes", torch.zeros(7)),
            ("slopes", torch.zeros(8, dtype=torch.bfloat16)), ("slopes", torch.zeros(16)[::2]),
            ("first", i6[:5]), ("first", i6.long()), ("last", torch.zeros(12, dtype=torch.int32)[::2]),
            ("last", i6.float()), ("layer", 1 << 32), ("layer", -(1 << 40)), ("window", 1 << 31),
            ("num_sinks", -(1 << 33)), ("workspace", torch.zeros((size, 2), dtype=torch.uint8)[:, 0]),
            ("chunk", kv.Chunk([1], device="cpu"))]:
        with pytest.raises((ValueError, kv.KvError)) as e:
            kv.kv_paged_attention_scored(**{**good, name: value})
        assert "CUDA device" not in str(e.value), name
    with pytest.raises(ValueError, match="CUDA device"):
        kv.kv_paged_attention_scored(**good)


def test_no_requests_is_a_no_op(kv):
    lib, c, t = kv.load(), _cache(kv, R=0), kv.Chunk([], device="cpu")
    assert lib.kv_paged_reserve(c.c, t.c, None, None, None, 0, None) == kv.KV_OK
    assert lib.kv_paged_fork(c.c, None, None, None) == kv.KV_OK
    assert lib.kv_paged_compact(c.c, None, None, None, None, 0, None) == kv.KV_OK
    assert lib.kv_paged_count_refs(c.c, None, None) == kv.KV_OK
    assert lib.kv_paged_place_positions(c.c, None, None, None, None, 0, None, None) == kv.KV_OK


def test_binding_refuses_other_shapes_types_and_devices(kv):
    import torch
    c, t = _cache(kv, positions=True, refs=True), kv.Chunk([1, 5], device="cpu")
    rot = kv.Rotary.make(64, device="cpu")
    pos = torch.zeros(6, dtype=torch.int32)
    q, k = (torch.zeros((6, h, 128), dtype=torch.bfloat16) for h in (8, 2))
    for bad in (dict(pos=pos.long()), dict(pos=pos[:5]), dict(q=q.half()), dict(q=q[:, :4]), dict(k=k[:5]),
                dict(out=q.float()), dict(k=k.half())):
        a = {"pos": pos, "q": q, "out": torch.empty_like(q), "k": k, **bad}
        with pytest.raises(ValueError, match="positions|q|k_new"):
            kv.kv_paged_append_rotary(c, t, 0, rot, a["pos"], a["q"], a["out"], a["k"], k)
    for bad in (dict(x=q.float()), dict(x=q[0]), dict(out=q[:5]), dict(x=q.transpose(1, 2)), dict(pos=pos[:5])):
        a = {"x": q, "out": torch.empty_like(q), "pos": pos, **bad}
        with pytest.raises(ValueError):
            kv.kv_rotary(rot, a["pos"], a["x"], a["out"])
    for freq in (torch.zeros(4, dtype=torch.float64), torch.zeros((2, 4)), torch.zeros(8)[::2]):
        with pytest.raises(ValueError, match="inv_freq"):
            kv.Rotary(freq)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    parents = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: kv.kv_rotary(rot, pos, q, torch.empty_like(q)),
                 lambda: kv.kv_paged_append_rotary(c, t, 0, rot, pos, None, None, k, k),
                 lambda: kv.kv_paged_reserve(c, t, ws), lambda: kv.kv_paged_fork(c, parents),
                 lambda: kv.kv_paged_compact(c, ws), lambda: kv.kv_paged_count_refs(c),
                 lambda: kv.kv_paged_place_positions(c)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    plain = _cache(kv)
    for call in (lambda: kv.kv_paged_reserve(plain, t, ws), lambda: kv.kv_paged_fork(plain, parents),
                 lambda: kv.kv_paged_compact(plain, ws), lambda: kv.kv_paged_count_refs(plain)):
        with pytest.raises(ValueError, match="refs"):
            call()
    with pytest.raises(ValueError, match="positions"):
        kv.kv_paged_place_positions(plain)
    index = torch.zeros((12, 5), dtype=torch.int32)
    for kw in (dict(index=index.long()), dict(index=index[:5]), dict(offsets=torch.zeros(13).long()),
               dict(index=index, offsets=torch.zeros(12).long()), dict(source=c), dict(index=index, source=plain)):
        with pytest.raises(ValueError):
            kv.kv_paged_place_positions(c, **kw)
    for bad in (parents.long(), parents[:1], torch.zeros(4, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="parents"):
            kv.kv_paged_fork(c, bad)
    for bad in (torch.zeros(2, dtype=torch.int32), torch.zeros(1)):
        with pytest.raises(ValueError, match="live"):
            kv.kv_paged_compact(c, ws, live=bad)
    for call in (lambda: kv.kv_paged_reserve(c, t, ws[::2]), lambda: kv.kv_paged_compact(c, ws[::2])):
        with pytest.raises(ValueError, match="workspace"):
            call()
    with pytest.raises(ValueError, match="requests"):
        kv.kv_paged_reserve(c, kv.Chunk([1], device="cpu"), ws)
    with pytest.raises(kv.KvError):
        kv.kv_paged_append_rotary(c, t, 1 << 32, rot, pos, None, None, k, k)
    a = (c.k_pages, c.v_pages, c.page_table, c.lens, 8)
    for kw in (dict(positions=c.positions.long()), dict(positions=c.positions[:-1]), dict(refs=c.refs[:-1]),
               dict(refs=c.refs.float())):
        with pytest.raises(ValueError):
            kv.PagedCache(*a, **kw)


def test_rotary_frequencies(kv):
    w, f = kv.kv_rotary_frequencies(128, 10000.0)
    plain = 10000.0 ** (-np.arange(64) / 64)
    assert f == 1.0
    np.testing.assert_allclose(w, plain, rtol=2.0 ** -24)
    w, f = kv.kv_rotary_frequencies(128, 10000.0, "linear", 4.0)
    assert f == 1.0
    np.testing.assert_allclose(w, plain / 4, rtol=2.0 ** -24)
    # a larger base: the first frequency stays, the last is divided by scale
    w, f = kv.kv_rotary_frequencies(64, 10000.0, "base", 8.0)
    last = 10000.0 ** (-62 / 64)
    assert f == 1.0 and w[0] == 1.0
    np.testing.assert_allclose(w[-1], last / 8, rtol=2.0 ** -23)
    # by parts: frequencies of 32 turns and more in 4096 positions kept, of 1 and fewer divided
    w, f = kv.kv_rotary_frequencies(128, 10000.0, "parts", 8.0, 4096)
    turns = 4096 * plain / (2 * math.pi)
    np.testing.assert_allclose(w[turns >= 32], plain[turns >= 32], rtol=2.0 ** -24)
    np.testing.assert_allclose(w[turns <= 1], plain[turns <= 1] / 8, rtol=2.0 ** -24)
    assert (np.diff(w) < 0).all() and abs(f - (0.1 * math.log(8.0) + 1)) < 1e-7
    assert kv.kv_rotary_frequencies(128, 10000.0, "parts", 1.0, 4096)[1] == 1.0
    for bad in (dict(dims=0), dict(dims=3), dict(base=0.0), dict(base=math.inf), dict(scaling="linear", scale=0.5),
                dict(scaling="parts", scale=2.0), dict(scaling="parts", scale=2.0, context=4096.0, slow=8, fast=8),
                dict(scaling="base", scale=math.nan), dict(dims=2 ** 33)):
        with pytest.raises(kv.KvError):
            kv.kv_rotary_frequencies(**{"dims": 64, **bad})
    with pytest.raises(ValueError, match="scaling"):
        kv.kv_rotary_frequencies(64, scaling="other")
