"""Attention of new tokens over the paged cache against the formula in 64 bits, at the sizes and
masks where it can go wrong; unused memory is poison everywhere (tests/paged.py)."""
import math

import pytest

pytestmark = pytest.mark.gpu


def _spread(R, L, H, lo, hi):
    return [[[lo + int((hi - lo + 1) * ((0.618 * (r * H + h) + 0.99) % 1)) for h in range(H)]
             for _ in range(L)] for r in range(R)]


def _chunk_inputs(made, counts, Hq, strided, seed, device="cuda"):
    import torch
    g = torch.Generator(device=device).manual_seed(seed + 1000)
    tok, d = sum(counts), made.d
    if strided:   # queries inside a wider row, as a fused projection leaves them
        wide = torch.randn((tok, Hq * d + 24), generator=g, device=device).to(made.dtype)
        q = wide[:, 16:16 + Hq * d].view(tok, Hq, d)
        out = torch.full((tok, Hq * d + 8), -3.0, device=device,
                         dtype=made.dtype)[:, :Hq * d].view(tok, Hq, d)
    else:
        q = torch.randn((tok, Hq, d), generator=g, device=device).to(made.dtype)
        out = torch.full_like(q, -3.0)
    return q, out


def _run(kv, made, counts, q, out, layer=0, window=0, sinks=0, mass=False, scale=None, stream=None):
    import torch
    chunk = kv.Chunk(counts)
    c = made.cache
    lse = torch.full((q.shape[0], c.num_q_heads), 7.0, device="cuda")
    ws = torch.full((kv.kv_paged_attention_workspace_size(c, chunk, mass),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    kv.kv_paged_attention(c, chunk, layer, q, out, ws, window=window, num_sinks=sinks, lse=lse,
                          add_mass=mass, softmax_scale=scale, stream=stream)
    return lse, kv.kv_check_status(c.status, stream)


def _check(made, counts, q, out, lse, layer=0, window=0, sinks=0, mass=False, scale=None):
    import torch
    from tests import paged
    c = made.cache
    G, d = c.num_q_heads // c.num_kv_heads, made.d
    scale = scale or 1 / math.sqrt(d)
    want_mass = made.mass0.double().clone().view(-1)
    tol_mass = torch.zeros_like(want_mass)
    t0 = 0
    for r, count in enumerate(counts):
        for h in range(c.num_kv_heads):
            n = max(int(made.lens_host[r, layer, h]), 0)
            qs = q[t0:t0 + count, h * G:(h + 1) * G].double()
            K, V = made.K[r, layer, h], made.V[r, layer, h]
            o, z, w, absv, logit = paged.attend_unit(qs, K, V, window, sinks, scale)
            got = out[t0:t0 + count, h * G:(h + 1) * G].double()
            bound = paged.out_bound(o, absv, made.dtype, d, n, logit, 1)
            assert torch.isfinite(got).all()
            bad = (got - o).abs() > bound
            assert not bad.any(), (r, h, float(((got - o).abs() / bound).max()))
            gz = lse[t0:t0 + count, h * G:(h + 1) * G].double()
            empty = torch.isinf(z)
            assert torch.equal(torch.isinf(gz) & (gz < 0), empty)
            assert ((gz - z).abs()[~empty] <= paged.lse_bound(z, d, n, logit)[~empty]).all()
            if mass and n:
                rows = made.rows(r, layer, h)
                tol_mass[rows] = paged.mass_bound(w, want_mass[rows], d, n, logit, count * G)
                want_mass[rows] += w
        t0 += count
    if mass:
        assert ((c.mass.double().view(-1) - want_mass).abs() <= tol_mass).all()


# (KV heads, query heads, d, page, dtype, counts, shortest, longest, window, sinks, mass, strided)
CASES = {
    "one_row": (1, 1, 64, 16, "bf16", [1], 1, 1, 0, 0, True, False),
    "decode_short": (2, 8, 128, 16, "bf16", [1, 1, 1], 1, 70, 0, 0, False, True),
    "decode_g7": (2, 14, 128, 64, "bf16", [1, 1], 900, 1300, 0, 0, True, False),
    "decode_g1": (3, 3, 64, 32, "fp16", [1] * 5, 63, 129, 0, 0, True, False),
    "decode_g16": (1, 16, 128, 32, "bf16", [1, 1], 100, 500, 0, 0, True, True),
    "decode_g9": (2, 18, 64, 128, "fp16", [1, 1], 100, 700, 0, 0, True, False),
    "decode_page128": (2, 8, 128, 128, "fp16", [1, 1], 127, 2050, 0, 0, False, False),
    "decode_window": (2, 8, 128, 16, "bf16", [1, 1, 1], 400, 3000, 130, 4, True, False),
    "decode_window_1": (1, 4, 64, 64, "bf16", [1], 513, 513, 1, 0, True, False),
    "decode_window_no_sinks": (1, 4, 128, 32, "bf16", [1, 1], 77, 900, 100, 0, True, True),
    "decode_many_sinks": (1, 4, 128, 64, "bf16", [1, 1], 300, 1000, 65, 200, True, False),
    "few_tokens": (2, 4, 128, 64, "bf16", [3, 0, 5, 1], 8, 400, 0, 0, True, True),
    "few_tokens_window": (2, 4, 64, 16, "fp16", [8, 2], 40, 900, 33, 3, True, False),
    "empty_rows": (2, 4, 128, 16, "bf16", [4, 3], 0, 5, 0, 0, True, False),
    "all_empty": (1, 4, 64, 16, "bf16", [1, 2], 0, 0, 0, 0, True, False),
    "chunk_33": (2, 8, 128, 64, "bf16", [33], 33, 50, 0, 0, True, False),
    "chunk_ragged": (2, 8, 128, 32, "bf16", [200, 1, 0, 37], 211, 700, 0, 0, True, True),
    "chunk_d64": (2, 6, 64, 16, "fp16", [100, 131], 131, 500, 0, 0, True, False),
    "chunk_g7": (1, 7, 128, 64, "bf16", [150], 1000, 1000, 0, 0, True, False),
    "chunk_g1": (2, 2, 128, 128, "fp16", [300], 400, 900, 0, 0, True, True),
    "chunk_window": (2, 8, 128, 64, "bf16", [257, 64], 500, 1500, 100, 4, True, False),
    "chunk_window_small": (1, 4, 64, 16, "bf16", [200], 900, 900, 5, 2, True, False),
    "chunk_window_wide": (1, 4, 128, 32, "bf16", [130], 300, 300, 5000, 4, True, False),
    "chunk_sinks_in_window": (1, 4, 128, 64, "bf16", [140], 140, 140, 64, 100, True, False),
    # sinks that end behind the windows' begin, in a tile that only some rows' windows reach
    "chunk_sinks_past_window": (1, 1, 128, 64, "bf16", [700], 1500, 1500, 200, 1000, True, False),
    "chunk_sinks_past_window_g4": (2, 8, 64, 32, "fp16", [150], 900, 1300, 40, 777, True, False),
    "decode_sinks_past_window": (1, 4, 128, 64, "bf16", [3], 700, 700, 40, 690, True, False),
    "chunk_window_largest": (1, 4, 128, 64, "bf16", [150], 600, 600, 2 ** 31 - 1, 2 ** 31 - 1, True,
                             False),
    "decode_window_largest": (1, 4, 128, 64, "bf16", [1, 3], 500, 9000, 2 ** 31 - 1, 4, True, False),
    "chunk_longer_than_rows": (1, 4, 128, 64, "bf16", [150], 90, 90, 0, 0, True, False),
    "prompt": (2, 8, 128, 64, "bf16", [513], 513, 513, 0, 0, True, False),
    "prompt_window": (1, 4, 128, 64, "fp16", [700], 700, 700, 129, 1, True, True),
    "long": (1, 4, 128, 64, "bf16", [1], 20011, 20011, 0, 0, True, False),
    # short tables: blocks of query rows, one launch
    "short_64_rows": (2, 8, 128, 64, "bf16", [16, 9, 0, 1], 16, 900, 0, 0, False, True),
    "short_128_rows": (1, 4, 64, 16, "fp16", [32, 31], 33, 2047, 0, 0, False, False),
    "short_g7": (2, 14, 128, 32, "bf16", [18, 2], 40, 3000, 0, 0, False, False),
    "short_window": (2, 8, 128, 64, "bf16", [20, 5], 300, 1500, 70, 5, False, True),
    "short_empty_rows": (1, 8, 128, 16, "bf16", [9, 5], 0, 4, 0, 0, False, False),
    "short_and_long_chunks": (2, 8, 64, 64, "bf16", [16, 200, 1], 201, 900, 0, 0, False, False),
    "short_512_rows": (1, 4, 128, 64, "bf16", [128], 700, 700, 0, 0, False, False),
    "short_too_many_items": (2, 8, 128, 64, "bf16", [30] * 30, 40, 300, 0, 0, False, False),
    "long_few_tokens": (2, 8, 128, 32, "bf16", [4, 1, 2], 300, 9001, 0, 0, True, False),
    "long_few_tokens_window": (2, 8, 64, 16, "fp16", [4, 1], 8000, 9001, 3001, 7, True, False),
    "many_requests": (2, 8, 128, 64, "bf16", [1] * 40, 1, 260, 0, 0, True, False),
    "long_chunk": (1, 8, 128, 64, "bf16", [96], 12345, 12345, 0, 0, True, False),
}


@pytest.mark.parametrize("name", CASES)
def test_against_the_formula(cuda_lib, name):
    from tests import paged
    H, Hq, d, page, dtype, counts, lo, hi, window, sinks, mass, strided = CASES[name]
    made = paged.Made(cuda_lib, _spread(len(counts), 2, H, lo, hi), Hq, d, page, dtype, mass=mass,
                      max_rows=hi + 3 * page, seed=len(name))
    q, out = _chunk_inputs(made, counts, Hq, strided, len(name))
    lse, status = _run(cuda_lib, made, counts, q, out, 1, window, sinks, mass)
    assert status == 0
    _check(made, counts, q, out, lse, 1, window, sinks, mass)


@pytest.mark.parametrize("counts,window,sinks", [([1, 1], 100, 4), ([1], 64, 0), ([70], 100, 4),
                                                 ([40, 20], 50, 0)])
@pytest.mark.parametrize("page", [16, 64])
def test_rows_no_query_sees_may_be_gone(cuda_lib, counts, window, sinks, page):
    """Rows between the sinks and the first query's window hold NaN and infinities, and the pages
    that they fill do not exist."""
    from tests import paged

    def unseen(r, l, h, n):
        return [(sinks, max(sinks, n - counts[r] - window + 1))]

    made = paged.Made(cuda_lib, _spread(len(counts), 1, 2, 700, 1100), 8, 128, page, seed=5,
                      unseen=unseen)
    q, out = _chunk_inputs(made, counts, 8, False, 5)
    lse, status = _run(cuda_lib, made, counts, q, out, 0, window, sinks)
    assert status == 0
    _check(made, counts, q, out, lse, 0, window, sinks)


@pytest.mark.parametrize("T", [1, 130])
def test_logits_far_from_zero(cuda_lib, T):
    """Large logits of both signs: the running maximum has to follow them."""
    from tests import paged
    made = paged.Made(cuda_lib, _spread(1, 1, 2, 600, 777), 8, 128, 64, seed=9, scale=4.0,
                      mass=True)
    q, out = _chunk_inputs(made, [T], 8, False, 9)
    lse, status = _run(cuda_lib, made, [T], q, out, 0, scale=0.25, mass=True)
    assert status == 0
    _check(made, [T], q, out, lse, 0, scale=0.25, mass=True)


@pytest.mark.parametrize("counts", [[1, 1], [64, 90]])
def test_rows_behind_the_last_token_stay(cuda_lib, counts):
    import torch
    from tests import paged
    kv = cuda_lib
    made = paged.Made(kv, _spread(2, 1, 2, 100, 200), 8, 128, 64, seed=3, mass=True)
    q, out = _chunk_inputs(made, counts + [7], 8, False, 3)
    tok = sum(counts)
    before = out.clone()
    lse, status = _run(kv, made, counts, q[:tok], out[:tok], mass=True)
    assert status == 0
    _check(made, counts, q[:tok], out[:tok], lse, mass=True)
    assert torch.equal(out[tok:], before[tok:])
    # pool rows of no unit keep their weights
    mine = torch.cat([made.rows(r, 0, h) for r in range(2) for h in range(2)])
    other = torch.ones(made.mass0.numel(), dtype=torch.bool, device="cuda")
    other[mine] = False
    assert torch.equal(made.cache.mass.view(-1)[other], made.mass0.view(-1)[other])


@pytest.mark.parametrize("counts,mass", [([1, 1, 1], True), ([3, 130], True), ([260], False)])
def test_the_same_call_gives_the_same_bits(cuda_lib, counts, mass):
    import torch
    from tests import paged
    kv = cuda_lib
    made = paged.Made(kv, _spread(len(counts), 1, 4, 300, 5000), 16, 128, 64, seed=4, mass=mass)
    q, out = _chunk_inputs(made, counts, 16, False, 4)
    got = []
    for _ in range(3):
        if mass:
            made.cache.mass.copy_(made.mass0)
        lse, status = _run(kv, made, counts, q, out, mass=mass)
        assert status == 0
        got.append([out.clone(), lse] + ([made.cache.mass.clone()] if mass else []))
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


def test_pool_offsets_past_32_bits(cuda_lib):
    """Pages at the far end of pools of more than 2^32 elements (past 2^31 in every unit of
    account but rows)."""
    import torch
    from tests import paged
    kv = cuda_lib
    d, page, H, Hq, n = 128, 64, 2, 8, 300
    pages = (1 << 32) // (page * d) + 40                       # 8.6 GB a pool
    small = paged.Made(kv, _spread(2, 1, H, 200, n), Hq, d, page, seed=6, mass=True)
    c = small.cache
    k = torch.empty((pages, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    mass = torch.zeros((pages, page), device="cuda")
    base = pages - c.num_pages
    k[base:], v[base:], mass[base:] = c.k_pages, c.v_pages, c.mass
    live = (c.page_table >= 0) & (c.page_table < c.num_pages)
    table = torch.where(live, c.page_table + base, -1).to(torch.int32)
    small.cache = kv.PagedCache(k, v, table, c.lens, Hq, mass=mass)
    for counts in ([1, 1], [100, 50]):
        mass[base:] = c.mass
        q, out = _chunk_inputs(small, counts, Hq, False, 6)
        lse, status = _run(kv, small, counts, q, out, mass=True)
        assert status == 0
        small.mass0 = torch.cat([torch.zeros((base, page), device="cuda"), c.mass])
        _check(small, counts, q, out, lse, mass=True)
        small.mass0 = None


@pytest.mark.parametrize("counts", [[1, 1], [90, 3]])
def test_bad_lengths_and_pages_are_reported(cuda_lib, counts):
    """A length no table can hold and a page that does not exist post KV_ERR_INVALID_ARG; units
    without either keep their results."""
    import torch
    from tests import paged
    kv = cuda_lib
    for what in ("length", "negative", "page"):
        made = paged.Made(kv, _spread(2, 1, 2, 200, 300), 8, 128, 64, seed=8)
        q, out = _chunk_inputs(made, counts, 8, False, 8)
        if what == "page":
            made.cache.page_table[0, 0, 1, 1] = made.cache.num_pages
        else:
            made.cache.lens[0, 0, 1] = -1 if what == "negative" else made.cache.max_pages * 64 + 1
        lse, status = _run(kv, made, counts, q, out)
        assert status == kv.KV_ERR_INVALID_ARG
        assert kv.kv_check_status(made.cache.status) == 0       # read and cleared
        # the other request is untouched by it
        t0 = counts[0]
        rest = paged.Made(kv, _spread(2, 1, 2, 200, 300), 8, 128, 64, seed=8)
        q2, out2 = _chunk_inputs(rest, counts, 8, False, 8)
        lse2, status2 = _run(kv, rest, counts, q2, out2)
        assert status2 == 0
        assert torch.equal(out[t0:], out2[t0:]) and torch.equal(lse[t0:], lse2[t0:])


@pytest.mark.parametrize("counts", [[1, 1], [40, 90]])
def test_graph_replays_follow_lengths_and_tables(cuda_lib, counts):
    """Captured once, replayed after lens, tables and queries changed in place."""
    import torch
    from tests import paged
    kv = cuda_lib
    a = paged.Made(kv, _spread(2, 1, 2, 100, 150), 8, 128, 64, seed=21, max_rows=2048, mass=True)
    b = paged.Made(kv, _spread(2, 1, 2, 900, 2000), 8, 128, 64, seed=22, max_rows=2048, mass=True)
    q, out = _chunk_inputs(a, counts, 8, False, 21)
    q2, _ = _chunk_inputs(a, counts, 8, False, 99)
    chunk = kv.Chunk(counts)
    c = a.cache
    ws = torch.empty(kv.kv_paged_attention_workspace_size(c, chunk, True), dtype=torch.uint8,
                     device="cuda")
    lse = torch.empty((sum(counts), 8), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def call():
        kv.kv_paged_attention(c, chunk, 0, q, out, ws, lse=lse, add_mass=True)

    with torch.cuda.stream(s):
        call()
    s.synchronize()
    c.mass.copy_(a.mass0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    g.replay()
    torch.cuda.synchronize()
    assert kv.kv_check_status(c.status) == 0
    _check(a, counts, q, out, lse, mass=True)
    c.k_pages.copy_(b.cache.k_pages)
    c.v_pages.copy_(b.cache.v_pages)
    c.page_table.copy_(b.cache.page_table)
    c.lens.copy_(b.cache.lens)
    c.mass.copy_(b.mass0)
    q.copy_(q2)
    a.K, a.V, a.lens_host, a.mass0 = b.K, b.V, b.lens_host, b.mass0
    g.replay()
    torch.cuda.synchronize()
    assert kv.kv_check_status(c.status) == 0
    _check(a, counts, q, out, lse, mass=True)


@pytest.mark.parametrize("counts,hi", [([1, 1], 900), ([1, 1], 9000), ([90, 40], 900)])
def test_an_expired_wait_is_reported(cuda_lib, counts, hi):
    """With a wait limit of 0 a wait that is not satisfied at once gives up: the call posts
    KV_ERR_TIMEOUT and returns (or none had to wait, and it is right); the next call with the
    usual limit is right."""
    from tests import paged
    kv = cuda_lib
    made = paged.Made(kv, _spread(2, 1, 2, 200, hi), 8, 128, 64, seed=8, mass=True)
    q, out = _chunk_inputs(made, counts, 8, False, 8)
    limit = kv.kv_get_wait_limit_ns()
    try:
        kv.kv_set_wait_limit_ns(0)
        for _ in range(5):
            made.cache.mass.copy_(made.mass0)
            lse, status = _run(kv, made, counts, q, out, mass=True)
            assert status in (kv.KV_OK, kv.KV_ERR_TIMEOUT)
            if status == kv.KV_OK:
                _check(made, counts, q, out, lse, mass=True)
    finally:
        kv.kv_set_wait_limit_ns(limit)
    made.cache.mass.copy_(made.mass0)
    lse, status = _run(kv, made, counts, q, out, mass=True)
    assert status == 0
    _check(made, counts, q, out, lse, mass=True)


def test_two_streams_at_once(cuda_lib):
    """Two calls with their own workspaces on two streams, while a third runs on the default."""
    import torch
    from tests import paged
    kv = cuda_lib
    sets = []
    for i, counts in enumerate([[1] * 6, [200, 3], [1, 40]]):
        made = paged.Made(kv, _spread(len(counts), 1, 4, 2000, 9000), 16, 128, 64, seed=30 + i,
                          mass=True)
        q, out = _chunk_inputs(made, counts, 16, False, 30 + i)
        chunk = kv.Chunk(counts)
        ws = torch.empty(kv.kv_paged_attention_workspace_size(made.cache, chunk, True),
                         dtype=torch.uint8, device="cuda")
        lse = torch.empty((sum(counts), 16), device="cuda")
        sets.append((made, counts, q, out, chunk, ws, lse, torch.cuda.Stream() if i else None))
    torch.cuda.synchronize()
    for made, counts, q, out, chunk, ws, lse, s in sets:
        kv.kv_paged_attention(made.cache, chunk, 0, q, out, ws, lse=lse, add_mass=True, stream=s)
    torch.cuda.synchronize()
    for made, counts, q, out, chunk, ws, lse, s in sets:
        assert kv.kv_check_status(made.cache.status, s) == 0
        _check(made, counts, q, out, lse, mass=True)


# Sinks that end in the very tile of 128 keys where an item's window begins: of the item's two
# blocks of 128 query rows, the second one's windows begin in a later tile, and it still sees them.
SINKS_AT_WINDOW = {
    "g4_lo97": (1, 4, 128, 64, "bf16", [300], 300, 300, 96, 4),
    "g4_lo98": (1, 4, 128, 64, "bf16", [300], 300, 300, 95, 4),
    "second_tile": (1, 1, 128, 64, "bf16", [600], 600, 600, 100, 150),
    "g7_ragged": (2, 14, 64, 16, "fp16", [400, 333], 400, 700, 260, 8),
    "window_4000": (1, 4, 128, 128, "bf16", [200], 4300, 4300, 4000, 4),
}


@pytest.mark.parametrize("name", SINKS_AT_WINDOW)
def test_sinks_in_the_tile_where_the_window_begins(cuda_lib, name):
    from tests import paged
    H, Hq, d, page, dtype, counts, lo, hi, window, sinks = SINKS_AT_WINDOW[name]
    made = paged.Made(cuda_lib, _spread(len(counts), 1, H, lo, hi), Hq, d, page, dtype, mass=True,
                      max_rows=hi + page, seed=41)
    q, out = _chunk_inputs(made, counts, Hq, False, 41)
    lse, status = _run(cuda_lib, made, counts, q, out, 0, window, sinks, True)
    assert status == 0
    _check(made, counts, q, out, lse, 0, window, sinks, True)
