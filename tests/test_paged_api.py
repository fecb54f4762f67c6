"""Refusals of the paged-cache entry points before anything is launched (no GPU needed)."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def kv():
    import kv_cache_eviction_split_gb300 as kv
    kv.build()
    kv.load()
    return kv


def _cache(kv, R=2, L=3, H=2, Hq=8, d=128, page=64, mass=True, **kw):
    import torch
    return kv.PagedCache.allocate(R, L, H, Hq, d, 100, page, kw.get("dtype", torch.bfloat16), mass,
                                  device="cpu")


F = 1 << 20   # a device address that is never used: the checks fail first


def test_workspace_sizes_and_shape_checks(kv):
    import torch
    c, t = _cache(kv), kv.Chunk([1, 5], device="cpu")
    assert kv.kv_paged_attention_workspace_size(c, t) >= 256
    assert kv.kv_paged_attention_workspace_size(c, t, True) >= 256
    assert kv.kv_paged_evict_workspace_size(c) >= 256
    for field, value, code in [("head_dim", 96, kv.KV_ERR_UNSUPPORTED),
                               ("page_size", 48, kv.KV_ERR_UNSUPPORTED),
                               ("page_size", 0, kv.KV_ERR_UNSUPPORTED),
                               ("num_q_heads", 7, kv.KV_ERR_INVALID_ARG),
                               ("num_q_heads", 1, kv.KV_ERR_INVALID_ARG),
                               ("num_layers", 0, kv.KV_ERR_INVALID_ARG),
                               ("num_requests", -1, kv.KV_ERR_INVALID_ARG),
                               ("max_pages", 0, kv.KV_ERR_INVALID_ARG),
                               ("num_pages", 0, kv.KV_ERR_INVALID_ARG),
                               ("dtype", 2, kv.KV_ERR_INVALID_ARG),
                               # 2^31 pool rows or cache rows: 32-bit row coordinates
                               ("num_pages", 1 << 25, kv.KV_ERR_UNSUPPORTED),
                               ("max_pages", 1 << 25, kv.KV_ERR_UNSUPPORTED),
                               ("k_pages", None, kv.KV_ERR_INVALID_ARG),
                               ("lens", c.lens.data_ptr() + 4, kv.KV_ERR_INVALID_ARG),
                               ("status", None, kv.KV_ERR_INVALID_ARG)]:
        old = getattr(c._c, field)
        setattr(c._c, field, value)
        for call in (lambda: kv.kv_paged_attention_workspace_size(c, t),
                     lambda: kv.kv_paged_evict_workspace_size(c)):
            with pytest.raises(kv.KvError) as e:
                call()
            assert e.value.code == code, field
        setattr(c._c, field, old)
    with pytest.raises(kv.KvError):      # weights asked for, none kept
        kv.kv_paged_attention_workspace_size(_cache(kv, mass=False), t, True)
    bad = kv.Chunk([1, 5], device="cpu")
    for host in ([1, 2, 7], [0, 3, 2]):
        bad.cu_host[:] = host
        with pytest.raises(kv.KvError):
            kv.kv_paged_attention_workspace_size(c, bad)
    assert torch.equal(c.lens, torch.zeros_like(c.lens))


def test_attention_argument_checks(kv):
    lib, c, t = kv.load(), _cache(kv), kv.Chunk([1, 5], device="cpu")
    ws = kv.kv_paged_attention_workspace_size(c, t, True)
    good = [c.c, t.c, 1, 0, 0, 0.1, F, 1024, F, 1024, F, 1, F, ws, None]

    def call(i, value):
        a = list(good)
        a[i] = value
        return lib.kv_paged_attention(*a)

    for i, value in [(2, -1), (2, 3), (3, -1), (4, -1), (5, 0.0), (5, float("nan")), (5, float("inf")),
                     (6, None), (6, F + 8), (7, 1016), (7, 1028), (8, None), (8, F + 2), (9, 8),
                     (10, F + 4), (12, None), (12, F + 64 + 1)]:
        assert call(i, value) == kv.KV_ERR_INVALID_ARG, (i, value)
    assert call(13, ws - 1) == kv.KV_ERR_WORKSPACE
    none = kv.Chunk([0, 0], device="cpu")
    assert lib.kv_paged_attention(c.c, none.c, 1, 0, 0, 0.1, None, 0, None, 0, None, 0, None, 0,
                                  None) == kv.KV_OK


def test_attention_refuses_more_tiles_than_it_counts(kv):
    lib, c = kv.load(), _cache(kv)
    t = kv.Chunk([1, 1 << 21], device="cpu")
    c._c.max_pages = 1 << 15                                    # tables of 2^21 rows
    args = [c.c, t.c, 1, 0, 0, 0.1, F, 1024, F, 1024, F, 0, F, 1 << 62, None]
    # 2 heads x 2^23 / 256 row blocks x 2^21 / 128 key tiles: 2^30
    t.cu_host[2] = 1 << 22                                      # twice that, and the items' costs
    assert lib.kv_paged_attention(*args) == kv.KV_ERR_UNSUPPORTED
    args[11] = 1
    t.cu_host[2] = 1 << 22
    args[3] = 4096                                # a window: few tiles, but the weights' count
    assert lib.kv_paged_attention(*args) == kv.KV_ERR_UNSUPPORTED


def test_binding_refuses_tensors_the_gpu_cannot_take(kv):
    import torch
    c, t = _cache(kv), kv.Chunk([1, 5], device="cpu")
    ws = torch.empty(1 << 24, dtype=torch.uint8)
    q, k = (torch.zeros((6, h, 128), dtype=torch.bfloat16) for h in (8, 2))
    rows, off = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros(c.num_units + 1).long()
    kept = torch.zeros((c.num_units, 50), dtype=torch.int32)
    for call in (lambda: kv.kv_paged_attention(c, t, 0, q, torch.empty_like(q), ws),
                 lambda: kv.kv_paged_append(c, t, 0, k, k),
                 lambda: kv.kv_paged_load(c, rows, rows, off, 4),
                 lambda: kv.kv_paged_evict(c, _cache(kv), kept[:, 0].contiguous(), 4, 16, kept, ws)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    # views that lie apart
    with pytest.raises(ValueError, match="workspace"):
        kv.kv_paged_attention(c, t, 0, q, torch.empty_like(q), ws[::2])
    with pytest.raises(ValueError, match="workspace"):
        kv.kv_paged_evict(c, _cache(kv), kept[:, 0].contiguous(), 4, 16, kept, ws[::2])
    with pytest.raises(ValueError, match="offsets"):
        kv.kv_paged_load(c, rows, rows, torch.zeros(2 * c.num_units + 2).long()[::2], 4)


def test_append_load_evict_argument_checks(kv):
    lib, c, t = kv.load(), _cache(kv), kv.Chunk([1, 5], device="cpu")
    good = [c.c, t.c, 0, F, 256, F, 256, None]
    for i, value in [(2, 3), (2, -1), (3, None), (3, F + 4), (4, 248), (4, 260), (5, None), (6, 0)]:
        a = list(good)
        a[i] = value
        assert lib.kv_paged_append(*a) == kv.KV_ERR_INVALID_ARG, (i, value)
    good = [c.c, F, F, F, F, 10, None]
    for i, value in [(1, None), (2, F + 8), (3, F + 4), (4, None), (5, -1),
                     (5, c.num_pages * c.page_size + 1)]:
        a = list(good)
        a[i] = value
        assert lib.kv_paged_load(*a) == kv.KV_ERR_INVALID_ARG, (i, value)
    d = _cache(kv)
    good = [c.c, d.c, F, 4, 16, F, 50, F, 256, None]
    for i, value in [(1, c.c), (2, None), (3, -1), (4, -1), (5, None), (6, 0), (7, None),
                     (1, _cache(kv, H=4).c), (1, _cache(kv, d=64).c),
                     (0, _cache(kv, mass=False).c)]:
        a = list(good)
        a[i] = value
        assert lib.kv_paged_evict(*a) == kv.KV_ERR_INVALID_ARG, (i, value)
    good[8] = 255
    assert lib.kv_paged_evict(*good) == kv.KV_ERR_WORKSPACE


def test_no_requests_is_a_no_op(kv):
    lib, c, t = kv.load(), _cache(kv, R=0), kv.Chunk([], device="cpu")
    assert lib.kv_paged_append(c.c, t.c, 0, None, 0, None, 0, None) == kv.KV_OK
    assert lib.kv_paged_load(c.c, None, None, None, None, 0, None) == kv.KV_OK
    assert lib.kv_paged_attention(c.c, t.c, 0, 0, 0, 1.0, None, 0, None, 0, None, 0, None, 0,
                                  None) == kv.KV_OK
    assert lib.kv_paged_evict(c.c, _cache(kv, R=0).c, None, 0, 0, None, 0, None, 0,
                              None) == kv.KV_OK


def test_binding_refuses_other_shapes_and_types(kv):
    import torch
    c, t = _cache(kv), kv.Chunk([1, 5], device="cpu")
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    q = torch.zeros((6, 8, 128), dtype=torch.bfloat16)
    lse = torch.zeros((6, 8))
    for bad in (dict(q=q.half()), dict(q=q[:5]), dict(q=q.transpose(0, 1).reshape(8, 6, 128)),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(out=q[:, :4]),
                dict(lse=lse[:5]), dict(lse=lse.double())):
        args = {"q": q, "out": torch.empty_like(q), "lse": lse, **bad}
        with pytest.raises(ValueError):
            kv.kv_paged_attention(c, t, 0, args["q"], args["out"], ws, lse=args["lse"])
    with pytest.raises(ValueError):
        kv.kv_paged_append(c, kv.Chunk([6], device="cpu"), 0, q[:, :2], q[:, :2])
    with pytest.raises(ValueError):
        kv.kv_paged_append(c, t, 0, q[:, :2], q[:, :2].float())
    rows = torch.zeros((10, 128), dtype=torch.bfloat16)
    off = torch.zeros(c.num_units + 1, dtype=torch.int64)
    for bad in (dict(k=rows[:9]), dict(off=off[:-1]), dict(off=off.int()),
                dict(mass=torch.zeros(9)), dict(k=rows.half())):
        args = {"k": rows, "off": off, "mass": None, **bad}
        with pytest.raises(ValueError):
            kv.kv_paged_load(c, args["k"], rows, args["off"], 10, mass_rows=args["mass"])
    k, v, tab, lens = c.k_pages, c.v_pages, c.page_table, c.lens
    for a in ((k.float(), v.float(), tab, lens), (k, v[:-1], tab, lens), (k, v, tab.long(), lens),
              (k, v, tab, lens[:1]), (k, v, tab.transpose(0, 1), lens.transpose(0, 1)),
              (k, v.half(), tab, lens)):
        with pytest.raises(ValueError):
            kv.PagedCache(*a, 8)
    with pytest.raises(ValueError):
        kv.PagedCache(k, v, tab, lens, 8, mass=c.mass[:-1])
    kept = torch.zeros((c.num_units, 50), dtype=torch.int32)
    for budgets, kp in ((torch.zeros(3, dtype=torch.int32), kept),
                        (torch.zeros(c.num_units), kept),
                        (torch.zeros(c.num_units, dtype=torch.int32), kept[:3])):
        with pytest.raises(ValueError):
            kv.kv_paged_evict(c, _cache(kv), budgets, 4, 16, kp, ws)


def test_advance_raises_every_units_length(kv):
    c = _cache(kv)
    c.lens[0, 1, 1] = 7
    c.advance(kv.Chunk([1, 5], device="cpu"))
    assert c.lens[0].tolist() == [[1, 1], [1, 8], [1, 1]] and c.lens[1].eq(5).all()
    assert np.array_equal(kv.Chunk([1, 0, 5], device="cpu").cu_host, [0, 1, 1, 6])
    assert ctypes.sizeof(kv._KvPaged) == 88


def test_a_chunk_of_other_requests_is_refused(kv):
    """The library reads an offset per request of the cache: a shorter chunk has fewer."""
    c = _cache(kv)
    for counts in ([], [5], [1, 2, 3]):
        bad = kv.Chunk(counts, device="cpu")
        with pytest.raises(ValueError, match="requests"):
            kv.kv_paged_attention_workspace_size(c, bad)
        with pytest.raises(ValueError, match="requests"):
            c.advance(bad)
    assert c.lens.eq(0).all()


@pytest.mark.parametrize("big", [2 ** 32, 2 ** 32 + 1, -2 ** 32, 2 ** 31, 2 ** 63, 2 ** 70])
def test_integers_past_32_bits_are_refused(kv, monkeypatch, big):
    """ctypes would keep their low 32 bits: layer 2^32 is not layer 0."""
    import torch
    c, t = _cache(kv), kv.Chunk([1, 5], device="cpu")
    # as if the tensors were on the GPU, and nothing that could be called there
    monkeypatch.setattr(kv, "_on_current_device", lambda *tensors: None)
    monkeypatch.setattr(kv, "_stream", lambda stream: None)
    calls, real = [], kv.load()

    class Lib:
        kv_status_string = real.kv_status_string

        def __getattr__(self, name):
            return lambda *args: calls.append((name, args)) or 0

    monkeypatch.setattr(kv, "_lib", Lib())
    monkeypatch.setattr(kv, "load", lambda: kv._lib)
    q, k = (torch.zeros((6, h, 128), dtype=torch.bfloat16) for h in (8, 2))
    ws = torch.empty(1 << 10, dtype=torch.uint8)
    kept = torch.zeros((c.num_units, 50), dtype=torch.int32)
    budgets = torch.zeros(c.num_units, dtype=torch.int32)

    def attend(layer=0, **kw):
        kv.kv_paged_attention(c, t, layer, q, torch.empty_like(q), ws, **kw)

    def evict(sinks=4, recent=16):
        kv.kv_paged_evict(c, _cache(kv), budgets, sinks, recent, kept, ws)

    attend()
    evict()
    kv.kv_paged_append(c, t, 0, k, k)
    assert len(calls) == 3
    for call in (lambda: attend(layer=big), lambda: attend(window=big), lambda: attend(num_sinks=big),
                 lambda: kv.kv_paged_append(c, t, big, k, k), lambda: evict(sinks=big),
                 lambda: evict(recent=big)):
        with pytest.raises(kv.KvError) as e:
            call()
        assert e.value.code == kv.KV_ERR_INVALID_ARG
    assert len(calls) == 3
    with pytest.raises(kv.KvError):
        kv.PagedCache(c.k_pages, c.v_pages, c.page_table, c.lens, big)


def test_attention_refuses_tiles_that_only_just_fit_32_bits(kv):
    """The kernels round the count of tiles up to equal runs, 304 at most: that has to fit too."""
    lib, c, t = kv.load(), _cache(kv, R=32), kv.Chunk([1] * 32, device="cpu")
    c._c.max_pages = (1 << 25) - 6           # 64 units of 2^25 - 6 tiles and 5 more each: 2^31 - 64
    args = [c.c, t.c, 1, 0, 0, 0.1, F, 1024, F, 1024, F, 0, F, 1 << 62, None]
    assert lib.kv_paged_attention(*args) == kv.KV_ERR_UNSUPPORTED


@pytest.mark.parametrize("counts,G,rows", [([1] * 64, 4, 4), ([1] * 64, 1, 1), ([1] * 64, 16, 16),
                                           ([3] * 64, 4, 12), ([1] * 63 + [500], 4, 4)])
def test_attention_workspace_holds_the_logits_of_the_rows_there_are(kv, counts, G, rows):
    c = _cache(kv, R=64, L=1, H=8, Hq=8 * G)
    c._c.max_pages = 131072 // 64
    t = kv.Chunk(counts, device="cpu")
    more = kv.kv_paged_attention_workspace_size(c, t, True) - kv.kv_paged_attention_workspace_size(c, t)
    logits = 64 * 8 * 131072 * rows * 4
    # beside them the rows' sums and, for a request with more rows, the packed queries
    beside = t.tokens * 8 * G * (4 + (128 * 2 if max(counts) == 500 else 0))
    assert logits <= more <= logits + beside + 1024
