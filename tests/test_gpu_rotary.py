"""Rotary positions against the formula in 64 bits: rows turned alone, in place and backward, and on
their way into the pages of a cache."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _turn64(x, positions, freq, factor, interleaved, sign=1.0):
    """x [tokens][heads][d] double; returns the turned rows and, per element, factor (|x1| + |x2|)."""
    import torch
    m = 2 * freq.numel()
    y, mag = x.clone(), torch.zeros_like(x)
    a = positions.double()[:, None] * freq.double()
    cos, sin = (a.cos() * factor)[:, None], (sign * a.sin() * factor)[:, None]
    i, j = (slice(0, m, 2), slice(1, m, 2)) if interleaved else (slice(0, m // 2), slice(m // 2, m))
    one, two = x[..., i], x[..., j]
    y[..., i], y[..., j] = one * cos - two * sin, one * sin + two * cos
    mag[..., i] = mag[..., j] = abs(factor) * (one.abs() + two.abs())
    return y, mag


def _bound(want, mag, positions, freq, dtype):
    """An angle p w: w / 2 pi in 53 bits twice (2^-52 p w), 64 bits after the point, half turns in 24
    bits (pi 2^-25).  Its sine and cosine within 2 ulp, their product with the factor and with the
    row, the sum: 6 x 2^-24 in all.  One rounding to the type."""
    import torch
    pw = float(positions.abs().max()) * float(freq.abs().max()) if freq.numel() else 0.0
    p = float(positions.abs().max()) if positions.numel() else 0.0
    angle = 2.0 ** -52 * pw + 2 * math.pi * p * 2.0 ** -64 + math.pi * 2.0 ** -25
    half = torch.finfo(dtype).eps / 2
    least = torch.finfo(dtype).smallest_normal * half
    err = (angle + 6 * 2.0 ** -24) * mag
    return half * want.abs() + (1 + half) * err + least


# (tokens, heads, d, dims, interleaved, dtype, scaling, first position, strided)
CASES = {
    "one_row": (1, 1, 64, 64, False, "bf16", "none", 0, False),
    "one_token": (1, 40, 128, 128, False, "bf16", "none", 131071, False),
    "part": (37, 7, 128, 64, False, "fp16", "linear", 900000, True),
    "part_interleaved": (37, 7, 128, 48, True, "bf16", "parts", 5, True),
    "least": (9, 3, 64, 16, True, "fp16", "base", 77, False),
    "none": (9, 3, 64, 0, False, "bf16", "none", 77, False),
    "odd_part": (300, 5, 128, 112, False, "bf16", "parts", 1 << 20, False),
    "many_heads": (3, 700, 64, 64, True, "bf16", "none", 1000, False),
    "far": (33, 2, 128, 128, False, "fp16", "none", (1 << 31) - 33, False),
    "negative": (33, 2, 128, 128, True, "fp16", "none", -20, False),
    "many_tokens": (5003, 1, 64, 32, False, "bf16", "none", 3, True),
    "group_ends": (1217, 3, 128, 128, False, "bf16", "parts", 4000, False),
}


def _frequencies(kv, dims, scaling):
    import torch
    if dims == 0:
        return torch.zeros(0, device="cuda"), 1.25
    w, factor = kv.kv_rotary_frequencies(dims, 10000.0, scaling, 1.0 if scaling == "none" else 8.0, 4096.0)
    return torch.from_numpy(w).cuda(), factor


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_rows_against_the_formula(cuda_lib, name, backward):
    import torch
    from tests import paged
    kv = cuda_lib
    tokens, heads, d, dims, inter, dtype, scaling, first, strided = CASES[name]
    dt = paged.DTYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(len(name))
    wide = torch.randn((tokens, heads * d + (40 if strided else 0)), generator=g, device="cuda").to(dt)
    x = wide[:, (16 if strided else 0):][:, :heads * d].view(tokens, heads, d)
    freq, factor = _frequencies(kv, dims, scaling)
    rot = kv.Rotary(freq, factor, inter)
    pos = torch.arange(tokens, device="cuda")
    pos = (first + (pos * 7919 % tokens if first >= 0 and first < 1 << 30 else pos)).to(torch.int32)
    out = torch.full((tokens, heads * d + 8), -3.0, device="cuda", dtype=dt)
    y = out[:, :heads * d].view(tokens, heads, d)
    kv.kv_rotary(rot, pos, x, y, backward=backward)
    want, mag = _turn64(x.double(), pos, freq, factor, inter, -1.0 if backward else 1.0)
    assert ((y.double() - want).abs() <= _bound(want, mag, pos, freq, dt)).all()
    assert torch.equal(y[..., dims:], x[..., dims:])
    assert (out[:, heads * d:] == -3.0).all()
    # in place
    z = x.clone()
    kv.kv_rotary(rot, pos, z, z, backward=backward)
    assert torch.equal(z, y)


def test_backward_is_the_gradient(cuda_lib):
    """sum(g * turn(x)) changes with x as backward(g) says: the turn is linear, so <g, turn(x)> =
    <backward(g), x>, up to the two roundings."""
    import torch
    kv = cuda_lib
    g0 = torch.Generator(device="cuda").manual_seed(1)
    freq, factor = _frequencies(kv, 96, "parts")
    for inter in (False, True):
        rot = kv.Rotary(freq, factor, inter)
        x, g = (torch.randn((65, 3, 128), generator=g0, device="cuda").half() for _ in range(2))
        pos = torch.arange(1000, 1065, device="cuda", dtype=torch.int32)
        y, gx = torch.empty_like(x), torch.empty_like(g)
        kv.kv_rotary(rot, pos, x, y)
        kv.kv_rotary(rot, pos, g, gx, backward=True)
        a = (g.double() * y.double()).sum((1, 2))
        b = (gx.double() * x.double()).sum((1, 2))
        # each element rounded once to 2^-11 of itself, and 2^-20 for angles and products
        tol = (2.0 ** -11 + 2.0 ** -20) * ((g.double() * y.double()).abs().sum((1, 2)) +
                                           (gx.double() * x.double()).abs().sum((1, 2))) \
            + 2.0 ** -20 * 4 * (g.double().norm(dim=(1, 2)) * x.double().norm(dim=(1, 2)))
        assert ((a - b).abs() <= tol).all()
        # differences of the rounded function, an element at a time: a step of 1 in x changes y by
        # the column of the turn, which backward applies to unit gradients
        for e in (0, 1, 47, 48, 95, 96, 127):
            step = torch.zeros_like(x)
            step[..., e] = 1
            col, row = torch.empty_like(x), torch.empty_like(x)
            kv.kv_rotary(rot, pos, step, col)
            for f in (e, (e + 48) % 96 if e < 96 else e, e ^ 1):
                one = torch.zeros_like(x)
                one[..., f] = 1
                kv.kv_rotary(rot, pos, one, row, backward=True)
                assert torch.equal(col[..., f], row[..., e])


def test_keys_in_their_own_layout(cuda_lib):
    """[L][H][N][d] keys as N tokens of L * H heads, and queries of a window as w tokens."""
    import torch
    kv = cuda_lib
    L, H, N, d = 2, 3, 70, 128
    k = torch.randn((L, H, N, d), device="cuda").bfloat16()
    freq, factor = _frequencies(kv, 128, "none")
    rot = kv.Rotary(freq, factor)
    pos = torch.arange(N, device="cuda", dtype=torch.int32)
    rows = k.view(L * H, N, d).transpose(0, 1)
    out = torch.empty_like(k)
    kv.kv_rotary(rot, pos, rows, out.view(L * H, N, d).transpose(0, 1))
    want, mag = _turn64(rows.double(), pos, freq, factor, False)
    got = out.view(L * H, N, d).transpose(0, 1).double()
    assert ((got - want).abs() <= _bound(want, mag, pos, freq, k.dtype)).all()


# (KV heads, query heads, d, page, dtype, dims, interleaved, counts, shortest, longest, queries)
APPENDS = {
    "one_token": (1, 1, 64, 16, "bf16", 64, False, [1], 1, 1, True),
    "decode": (8, 32, 128, 64, "bf16", 128, False, [1] * 5, 40, 90, True),
    "no_queries": (4, 28, 128, 32, "fp16", 64, True, [1, 3], 10, 90, False),
    "ragged": (3, 3, 64, 128, "fp16", 32, False, [5, 0, 17, 1], 17, 300, True),
    "longer_than_units": (2, 4, 128, 16, "bf16", 96, True, [40], 20, 30, True),
    "many_requests": (1, 4, 64, 64, "bf16", 64, False, [1, 2, 0] * 300, 2, 9, True),
    "prompt": (8, 32, 128, 64, "bf16", 128, False, [1500, 700], 1500, 1600, True),
    "wide": (70, 700, 64, 16, "bf16", 16, True, [2], 3, 40, True),
}


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("name", APPENDS)
def test_appended_rows_against_the_formula(cuda_lib, name, strided):
    import torch
    from tests import paged
    from tests.test_gpu_paged_cache import _bits, _spread
    kv = cuda_lib
    H, Hq, d, page, dtype, dims, inter, counts, lo, hi, queries = APPENDS[name]
    L, layer, tok = 2, 1, sum(counts)
    made = paged.Made(kv, _spread(len(counts), L, H, lo, hi), Hq, d, page, dtype, mass=True, seed=3)
    c = made.cache
    c.positions = torch.full(c.mass.shape, -9, dtype=torch.int32, device="cuda")
    freq, factor = _frequencies(kv, dims, "parts")
    rot = kv.Rotary(freq, factor, inter)
    g = torch.Generator(device="cuda").manual_seed(4)
    pos = torch.randint(0, 1 << 20, (tok,), generator=g, device="cuda").int()
    new = torch.randn((tok, (Hq + 2 * H) * d + (24 if strided else 0)), generator=g,
                      device="cuda").to(made.dtype)
    q, k, v = (new[:, a * d:b * d].view(tok, b - a, d)
               for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    before = [t.clone() for t in (c.k_pages, c.v_pages, c.mass, c.positions)]
    q_out = torch.empty((tok, Hq, d), dtype=made.dtype, device="cuda") if queries else None
    kv.kv_paged_append_rotary(c, kv.Chunk(counts), layer, rot, pos, q if queries else None, q_out, k, v)
    assert kv.kv_check_status(c.status) == 0
    if queries:
        want, mag = _turn64(q.double(), pos, freq, factor, inter)
        assert ((q_out.double() - want).abs() <= _bound(want, mag, pos, freq, made.dtype)).all()
    want, mag = _turn64(k.double(), pos, freq, factor, inter)
    bound = _bound(want, mag, pos, freq, made.dtype)
    rows, heads, toks = [], [], []
    t0 = 0
    for r, count in enumerate(counts):
        for h in range(H):
            n = int(made.lens_host[r, layer, h])
            mine = made.rows(r, layer, h).tolist()
            for i in range(count):
                if n - count + i >= 0:
                    rows.append(mine[n - count + i])
                    heads.append(h)
                    toks.append(t0 + i)
        t0 += count
    rows, heads, toks = (torch.tensor(x, device="cuda", dtype=torch.long) for x in (rows, heads, toks))
    got = c.k_pages.view(-1, d)[rows].double()
    assert ((got - want[toks, heads]).abs() <= bound[toks, heads]).all()
    assert torch.equal(_bits(c.v_pages.view(-1, d)[rows]), _bits(v[toks, heads]))
    assert (c.mass.view(-1)[rows] == 0).all()
    assert torch.equal(c.positions.view(-1)[rows], pos[toks])
    # nothing else has changed
    for t, old in zip((c.k_pages, c.v_pages, c.mass, c.positions), before):
        t, old = t.view(c.num_pages * page, -1), old.view(c.num_pages * page, -1)
        rest = torch.ones(t.shape[0], dtype=torch.bool, device="cuda")
        rest[rows] = False
        assert torch.equal(_bits(t[rest]) if t.is_floating_point() else t[rest],
                           _bits(old[rest]) if t.is_floating_point() else old[rest])


def test_append_is_append_of_turned_rows_and_follows_replays(cuda_lib):
    """The same bits as kv_rotary then kv_paged_append; captured once, replayed with other inputs and
    lengths; queries turned in place; pages that do not exist are skipped."""
    import torch
    from tests import paged
    from tests.test_gpu_paged_cache import _bits, _spread
    kv = cuda_lib
    counts, H, Hq, d = [3, 1], 2, 8, 128
    a = paged.Made(kv, _spread(2, 1, H, 30, 80), Hq, d, 16, seed=5, max_rows=100)
    b = paged.Made(kv, _spread(2, 1, H, 30, 80), Hq, d, 16, seed=5, max_rows=100)
    rot = kv.Rotary.make(128)
    pos = torch.tensor([70, 71, 72, 900], dtype=torch.int32, device="cuda")
    q = torch.randn((4, Hq, d), device="cuda").bfloat16()
    k, v = (torch.randn((4, H, d), device="cuda").bfloat16() for _ in range(2))
    q0 = q.clone()
    chunk = kv.Chunk(counts)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        kv.kv_paged_append_rotary(a.cache, chunk, 0, rot, pos, q, q, k, v)
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for t in (q, k, v):
            t.normal_(generator=gen)
        pos.add_(1000)
        a.cache.lens.fill_(40 + seed)
        b.cache.lens.fill_(40 + seed)
        table = torch.randperm(a.cache.num_pages, device="cuda")[:a.cache.page_table.numel()].int()
        table = table.view(a.cache.page_table.shape)
        a.cache.page_table.copy_(table)
        b.cache.page_table.copy_(table)
        q0.copy_(q)
        kt, qt = torch.empty_like(k), torch.empty_like(q)
        kv.kv_rotary(rot, pos, k, kt)
        kv.kv_rotary(rot, pos, q0, qt)
        kv.kv_paged_append(b.cache, chunk, 0, kt, v)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, qt)
        assert torch.equal(_bits(a.cache.k_pages), _bits(b.cache.k_pages))
        assert torch.equal(_bits(a.cache.v_pages), _bits(b.cache.v_pages))
        assert kv.kv_check_status(a.cache.status) == 0
    a.cache.page_table[0, 0, 1] = a.cache.num_pages
    a.cache.lens[1, 0, 0] = -1
    before = a.cache.k_pages.clone()
    kv.kv_paged_append_rotary(a.cache, chunk, 0, rot, pos, None, None, k, v)
    assert kv.kv_check_status(a.cache.status) == kv.KV_ERR_INVALID_ARG
    bad = (_bits(before) != _bits(a.cache.k_pages)).any(-1).nonzero().shape[0]
    assert bad <= 4                               # 3 rows of one head, 1 of another


def test_positions_follow_loads_and_evictions(cuda_lib):
    import torch
    kv = cuda_lib
    R, L, H, d = 2, 1, 2, 64
    kept = [[3, 5, 9, 10], [0, 1], [2, 4, 6, 8, 11], []]
    offsets = torch.tensor(np.concatenate([[0], np.cumsum([len(x) for x in kept])]), device="cuda")
    index = torch.tensor(sum(kept, []), dtype=torch.int32, device="cuda")
    c = kv.PagedCache.allocate(R, L, H, 2, d, 20, 16, positions=True, mass=True)
    rows = torch.randn((index.numel(), d), device="cuda").bfloat16()
    kv.kv_paged_load(c, rows, rows, offsets, index.numel())
    kv.kv_paged_place_positions(c, index, offsets)
    flat = c.positions.view(4, -1)                # pages in order, 2 a unit
    for u, x in enumerate(kept):
        assert flat[u, :len(x)].tolist() == x
    # an eviction's rows keep theirs
    c.mass.copy_(torch.rand(c.mass.shape, device="cuda"))
    small = kv.PagedCache.allocate(R, L, H, 2, d, 20, 32, positions=True, mass=True)
    small.positions.fill_(-7)
    out = torch.full((4, 5), -1, dtype=torch.int32, device="cuda")
    ws = torch.empty(kv.kv_paged_evict_workspace_size(c), dtype=torch.uint8, device="cuda")
    budgets = torch.full((4,), 3, dtype=torch.int32, device="cuda")
    kv.kv_paged_evict(c, small, budgets, 1, 1, out, ws)
    kv.kv_paged_place_positions(small, out, source=c)
    assert kv.kv_check_status(small.status) == 0
    for u, x in enumerate(kept):
        n = min(3, len(x))
        assert small.positions.view(4, -1)[u, :n].tolist() == [x[i] for i in out[u, :n].tolist()]
        assert (small.positions.view(4, -1)[u, n:] == -7).all()
    kv.kv_paged_place_positions(small)
    assert small.positions.view(4, -1)[2, :3].tolist() == [0, 1, 2]
    # a row that the source does not have
    out[0, 0] = 1 << 20
    kv.kv_paged_place_positions(small, out, source=c)
    assert kv.kv_check_status(small.status) == kv.KV_ERR_INVALID_ARG


def test_positions_of_units_with_more_rows_than_their_lists(cuda_lib):
    """Only what the lists name is read and written."""
    import torch
    kv = cuda_lib
    for offsets in (None, torch.tensor([0, 3, 6], device="cuda")):
        c = kv.PagedCache.allocate(1, 1, 2, 2, 64, 20, 16, positions=True)
        c.lens.copy_(torch.tensor([2, 9], dtype=torch.int32).view(1, 1, 2))
        c.positions.fill_(-7)
        index = torch.arange(10, 16, dtype=torch.int32, device="cuda")
        kv.kv_paged_place_positions(c, index.view(2, 3) if offsets is None else index, offsets)
        assert kv.kv_check_status(c.status) == kv.KV_ERR_INVALID_ARG
        flat = c.positions.view(2, -1)
        assert flat[0, :2].tolist() == [10, 11] and flat[1, :3].tolist() == [13, 14, 15]
        assert (flat[0, 2:] == -7).all() and (flat[1, 3:] == -7).all()
