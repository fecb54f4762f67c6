"""Attention over the pages with scores capped, lowered by distance and masked by position, against the
formula in 64 bits, at the sizes and masks where it can go wrong; unused memory is poison
(tests/paged.py)."""
import math

import pytest

pytestmark = pytest.mark.gpu


def _slopes(Hq, most=1.0):
    import torch
    return most * 2.0 ** (-8.0 * torch.arange(Hq, device="cuda") / Hq)


# rows of a page table that is too long for the kernel of short tables
LONG_TABLE = 8400

# (KV heads, query heads, d, page, dtype, counts, shortest, longest, cap, slopes, gaps, bounds, window, sinks, mass)
# gaps: positions beside the pages, the largest step (negative: steps of 0 too); 0: none are kept
CASES = {
    "one_row": (1, 1, 64, 16, "bf16", [1], 1, 1, 5.0, True, 0, None, 0, 0, True),
    "cap": (2, 8, 128, 16, "bf16", [1, 1, 1], 1, 70, 2.0, False, 0, None, 0, 0, False),
    "cap_g7": (2, 14, 128, 64, "bf16", [1, 1], 900, 1300, 30.0, False, 0, None, 0, 0, True),
    "slopes_rows": (2, 8, 128, 32, "bf16", [1, 1], 500, 1300, 0.0, True, 0, None, 0, 0, True),
    "slopes_gaps": (2, 8, 128, 32, "bf16", [1, 1, 1], 1, 1300, 0.0, True, 9, None, 0, 0, True),
    "slopes_g1": (3, 3, 64, 32, "fp16", [1] * 5, 63, 129, 20.0, True, 3, None, 0, 0, True),
    "slopes_g16": (1, 16, 128, 128, "bf16", [1, 1], 100, 500, 0.0, True, -2, None, 0, 0, True),
    "slopes_window": (2, 8, 128, 16, "bf16", [1, 1, 1], 400, 3000, 0.0, True, 3, None, 130, 4, False),
    "few_tokens": (2, 4, 128, 64, "bf16", [3, 0, 5, 1], 8, 400, 8.0, True, 4, None, 0, 0, True),
    "few_reach": (2, 4, 128, 64, "bf16", [3, 0, 5, 1], 8, 400, 0.0, True, 4, "reach", 0, 2, True),
    "few_docs": (2, 4, 64, 16, "fp16", [4, 8], 40, 900, 9.0, False, 4, "docs", 0, 0, False),
    "few_random": (2, 4, 128, 32, "bf16", [8, 3, 2], 40, 900, 9.0, True, -3, "random", 0, 0, True),
    "few_random_sinks": (2, 4, 128, 32, "bf16", [8, 3, 2], 40, 900, 0.0, False, -3, "random", 0, 70, False),
    "few_none": (2, 4, 128, 32, "bf16", [8, 3, 2], 40, 300, 9.0, True, 2, "none", 0, 0, True),
    "few_none_sinks": (2, 4, 128, 32, "bf16", [8, 3, 2], 40, 300, 9.0, True, 2, "none", 0, 5, True),
    "few_extremes": (2, 4, 128, 32, "bf16", [2, 3], 40, 300, 9.0, True, 2, "extremes", 0, 0, True),
    "few_halves": (1, 2, 64, 16, "bf16", [8], 700, 700, 0.0, False, 0, "halves", 0, 3, True),
    "empty_rows": (2, 4, 128, 16, "bf16", [4, 3], 0, 5, 3.0, True, 3, None, 0, 0, True),
    "all_empty": (1, 4, 64, 16, "bf16", [1, 2], 0, 0, 3.0, True, 3, "reach", 0, 0, True),
    "long": (1, 4, 128, 64, "bf16", [1], 20011, 20011, 30.0, True, 3, None, 0, 0, True),
    "long_few": (2, 8, 128, 32, "bf16", [4, 1, 2], 300, 9001, 0.0, True, 5, "docs", 0, 4, True),
    "long_reach": (2, 8, 64, 16, "fp16", [4, 1], 8000, 9001, 50.0, False, 2, "reach", 0, 7, False),
    "long_none": (2, 8, 64, 16, "fp16", [1, 1], 8000, 9001, 50.0, True, 2, "none", 0, 0, True),
    # short tables: blocks of query rows, one launch
    "short_64_rows": (2, 8, 128, 64, "bf16", [16, 9, 0, 1], 16, 900, 4.0, True, 3, None, 0, 0, False),
    "short_docs": (2, 14, 128, 32, "bf16", [18, 2], 40, 3000, 0.0, True, 0, "docs", 0, 0, False),
    "short_random": (1, 4, 64, 16, "fp16", [32, 31], 33, 2047, 7.0, True, 2, "random", 0, 3, False),
    "short_prefix": (1, 8, 128, 16, "bf16", [30, 17], 30, 400, 0.0, True, 1, "prefix", 0, 0, False),
    # prompt chunks
    "chunk_33": (2, 8, 128, 64, "bf16", [33] * 20, 33, 50, 3.0, True, 0, None, 0, 0, False),
    "chunk_cap": (2, 8, 128, 32, "bf16", [200, 1, 0, 37], 211, 700, 15.0, False, 0, None, 0, 0, False),
    "chunk_slopes": (2, 6, 64, 16, "fp16", [300, 131], 300, 500, 0.0, True, 0, None, 0, 0, False),
    "chunk_gaps": (2, 8, 128, 64, "bf16", [257, 150], 500, 1500, 0.0, True, 6, None, 0, 0, False),
    "chunk_both": (1, 7, 128, 64, "bf16", [150], 1000, 1000, 6.0, True, -4, None, 0, 0, False),
    "chunk_window": (2, 8, 128, 64, "bf16", [257, 140], 500, 1500, 9.0, True, 3, None, 100, 4, False),
    "chunk_docs": (2, 8, 128, 64, "bf16", [700, 160], 700, 1500, 9.0, True, 3, "docs", 0, 0, False),
    "chunk_docs_rows": (2, 8, 64, 32, "fp16", [400, 160], 900, 900, 0.0, True, 0, "docs", 0, 5, False),
    "chunk_reach": (1, 4, 128, 128, "bf16", [700], 1500, 1500, 9.0, False, 2, "reach", 0, 300, False),
    "chunk_prefix": (2, 8, 128, 64, "bf16", [513], 513, 513, 0.0, True, 0, "prefix", 0, 0, False),
    "chunk_random": (2, 2, 128, 64, "bf16", [600, 520], 600, 2500, 9.0, True, 2, "random", 0, 0, False),
    "chunk_random_sinks": (2, 2, 64, 16, "fp16", [600, 520], 600, 2500, 9.0, True, 2, "random", 0, 200, False),
    "chunk_halves": (1, 1, 128, 64, "bf16", [512], 2600, 2600, 0.0, True, 1, "halves", 0, 0, False),
    "chunk_halves_256": (1, 1, 128, 64, "bf16", [256 + 512], 2600, 2600, 5.0, False, 0, "halves", 0, 0, False),
    "chunk_halves_sinks": (1, 2, 64, 64, "bf16", [300, 520], 1400, 2600, 0.0, False, 1, "halves", 0, 9, False),
    "chunk_back": (2, 2, 128, 32, "bf16", [900, 640], 900, 2600, 0.0, True, 1, "back", 0, 0, False),
    "chunk_back_sinks": (2, 2, 128, 32, "bf16", [900, 640], 900, 2600, 6.0, True, 1, "back", 0, 400, False),
    "chunk_none": (2, 8, 128, 64, "bf16", [151, 140], 151, 500, 9.0, True, 3, "none", 0, 0, False),
    "chunk_none_sinks": (2, 8, 128, 64, "bf16", [151, 140], 151, 500, 9.0, True, 3, "none", 0, 130, False),
    "chunk_extremes": (2, 8, 128, 64, "bf16", [151, 140], 151, 500, 9.0, True, 3, "extremes", 0, 0, False),
    "chunk_longer_than_rows": (1, 4, 128, 64, "bf16", [650], 290, 290, 9.0, True, 2, "reach", 0, 0, False),
    # prompt chunks of more rows than short tables take in one launch
    "many_cap": (4, 32, 128, 32, "bf16", [200, 1, 0, 151], 211, 700, 15.0, False, 0, None, 0, 0, False),
    "many_cap_gaps": (8, 32, 128, 64, "bf16", [257, 190], 500, 1500, 9.0, False, 6, "reach", 0, 7, False),
    "many_slopes": (6, 18, 64, 16, "fp16", [500, 131], 500, 700, 0.0, True, 0, None, 0, 0, False),
    "many_gaps": (8, 32, 128, 64, "bf16", [257, 170], 500, 1500, 0.0, True, 6, None, 0, 0, False),
    "many_both": (8, 56, 128, 64, "bf16", [150, 8], 1000, 1000, 6.0, True, -4, None, 0, 0, False),
    "many_window": (8, 32, 128, 64, "bf16", [257, 140], 500, 1500, 9.0, True, 3, None, 100, 4, False),
    "many_docs": (8, 32, 128, 64, "bf16", [700, 160], 700, 1500, 9.0, True, 3, "docs", 0, 0, False),
    "many_docs_rows": (8, 32, 64, 32, "fp16", [400, 160], 900, 900, 0.0, False, 0, "docs", 0, 5, False),
    "many_docs_cap": (8, 32, 128, 128, "bf16", [611], 611, 611, 30.0, False, 0, "docs", 0, 0, False),
    "many_reach": (8, 32, 128, 128, "bf16", [700], 1500, 1500, 9.0, False, 2, "reach", 0, 300, False),
    "many_prefix": (8, 64, 128, 64, "bf16", [513], 513, 513, 0.0, True, 0, "prefix", 0, 0, False),
    "many_random": (8, 16, 128, 64, "bf16", [600, 520], 600, 2500, 9.0, True, 2, "random", 0, 0, False),
    "many_random_sinks": (8, 32, 64, 16, "fp16", [600, 520], 600, 2500, 9.0, True, 2, "random", 0, 200, False),
    "many_halves": (3, 3, 128, 64, "bf16", [4400], 4400, 4400, 0.0, True, 1, "halves", 0, 0, False),
    "many_halves_sinks": (4, 8, 64, 64, "bf16", [300, 1520], 1600, 2600, 5.0, False, 1, "halves", 0, 9, False),
    "many_back": (8, 32, 128, 32, "bf16", [900, 340], 900, 1300, 0.0, True, 1, "back", 0, 0, False),
    "many_none": (8, 64, 128, 64, "bf16", [151, 140], 151, 500, 9.0, True, 3, "none", 0, 130, False),
    "many_extremes": (8, 64, 128, 64, "bf16", [151, 140], 151, 500, 9.0, True, 3, "extremes", 0, 0, False),
    "many_longer_than_rows": (2, 8, 128, 64, "bf16", [1200], 290, 290, 9.0, True, 2, "reach", 0, 0, False),
    "long_chunk": (1, 8, 128, 64, "bf16", [96], 12345, 12345, 50.0, True, 4, "docs", 0, 4, False),
}


@pytest.mark.parametrize("name", CASES)
def test_against_the_formula(cuda_lib, name):
    import torch
    from tests import paged, scores
    from tests.test_gpu_paged_attention import _chunk_inputs, _spread
    H, Hq, d, page, dtype, counts, lo, hi, cap, slopes, gaps, kind, window, sinks, mass = CASES[name]
    lens = _spread(len(counts), 2, H, lo, hi)
    if kind and not gaps:
        lens = [[[x[0][0]] * H] * 2 for x in lens]         # rows' numbers are every head's positions
    made = paged.Made(cuda_lib, lens, Hq, d, page, dtype, mass=mass, max_rows=hi + 3 * page, seed=len(name))
    pos = scores.positions_of(made, gaps, len(name)) if gaps else None
    q, out = _chunk_inputs(made, counts, Hq, len(name) % 2 == 0, len(name))
    kw = dict(cap=cap, slopes=_slopes(Hq) if slopes else None, window=window, sinks=sinks)
    if kind:
        heads = [pos[r, 1, 0] if gaps else torch.arange(lens[r][1][0]) for r in range(len(counts))]
        kw["first"], kw["last"] = scores.bounds_of(kind, counts, [lens[r][1][0] for r in range(len(counts))], heads)
        if kind in ("docs", "reach"):
            kw["last"] = None
    lse, status = scores.run(cuda_lib, made, counts, q, out, 1, mass, **kw)
    assert status == 0
    scores.check(cuda_lib, made, pos, counts, q, out, lse, 1, mass=mass, **kw)


@pytest.mark.parametrize("counts", [[1, 1, 1], [3, 2], [200, 150]])
def test_plain_scores_are_those_of_plain_attention(cuda_lib, counts):
    """Without any change the call is kv_paged_attention; with bounds that hide nothing, almost."""
    import torch
    from tests import paged, scores
    from tests.test_gpu_paged_attention import _chunk_inputs, _run, _spread
    kv = cuda_lib
    made = paged.Made(kv, _spread(len(counts), 1, 2, 300, 9000), 8, 128, 64, seed=1)
    q, out = _chunk_inputs(made, counts, 8, False, 1)
    lse, _ = _run(kv, made, counts, q, out, 0, 200, 4)
    out2 = torch.empty_like(out)
    lse2, status = scores.run(kv, made, counts, q, out2, window=200, sinks=4)
    assert status == 0 and torch.equal(out, out2) and torch.equal(lse, lse2)
    zero = torch.zeros(sum(counts), dtype=torch.int32, device="cuda")
    lse3, status = scores.run(kv, made, counts, q, out2, window=200, sinks=4, first=zero, slopes=torch.zeros(8, device="cuda"))
    assert status == 0
    scores.check(kv, made, None, counts, q, out2, lse3, window=200, sinks=4)


@pytest.mark.parametrize("kind", ["few", "long", "short", "many"])
def test_caps_from_almost_flat_to_almost_none(cuda_lib, kind):
    """Logits far beyond the cap saturate; far below it they pass."""
    from tests import paged, scores
    from tests.test_gpu_paged_attention import _chunk_inputs, _spread
    counts, hi = {"few": ([1, 2], 777), "long": ([1, 1], 9000), "short": ([200, 150], 777),
                  "many": ([200, 150], 777)}[kind]
    made = paged.Made(cuda_lib, _spread(len(counts), 1, 2, 300, hi), 8, 128, 64, seed=9, scale=4.0,
                      max_rows=LONG_TABLE if kind == "many" else None)
    q, out = _chunk_inputs(made, counts, 8, False, 9)
    for cap in (1e-43, 1e-3, 0.5, 20.0, 300.0, 1e4, 1e30):
        lse, status = scores.run(cuda_lib, made, counts, q, out, cap=cap, scale=0.25)
        assert status == 0
        scores.check(cuda_lib, made, None, counts, q, out, lse, cap=cap, scale=0.25)


@pytest.mark.parametrize("counts,max_rows", [([1, 1], None), ([150, 90], None), ([150, 90], LONG_TABLE)])
def test_slopes_of_both_signs_and_far_positions(cuda_lib, counts, max_rows):
    """Positions past 2^24 from the start: only distances have to be below it."""
    import torch
    from tests import paged, scores
    from tests.test_gpu_paged_attention import _chunk_inputs, _spread
    made = paged.Made(cuda_lib, _spread(2, 1, 2, 150, 900), 8, 128, 32, seed=12, max_rows=max_rows)
    pos = scores.positions_of(made, 5, 12, start=2 ** 31 - 8000)
    q, out = _chunk_inputs(made, counts, 8, False, 12)
    slopes = torch.tensor([0.5, -0.01, 0.0, 3.0, -0.002, 1e-6, 0.1, 100.0], device="cuda")
    lse, status = scores.run(cuda_lib, made, counts, q, out, slopes=slopes)
    assert status == 0
    scores.check(cuda_lib, made, pos, counts, q, out, lse, slopes=slopes)


@pytest.mark.parametrize("counts,max_rows", [([1, 1], None), ([3, 4], None), ([120, 130], None),
                                             ([120, 130], LONG_TABLE)])
@pytest.mark.parametrize("page", [16, 128])
def test_rows_outside_the_bounds_may_be_gone(cuda_lib, counts, max_rows, page):
    """Rows before the first that any query of the chunk sees (behind the sinks), and rows behind the last,
    hold NaN and infinities, and the pages that they fill do not exist."""
    import torch
    from tests import paged, scores
    from tests.test_gpu_paged_attention import _chunk_inputs
    n, lo, hi, sinks = 1100, 333, 801, 5
    made = paged.Made(cuda_lib, [[[n] * 2]] * 2, 8, 128, page, seed=5, max_rows=max_rows,
                      unseen=lambda r, l, h, n: [(sinks, lo), (hi + 1, n)])
    q, out = _chunk_inputs(made, counts, 8, False, 5)
    first = torch.full((sum(counts),), lo, dtype=torch.int32, device="cuda")
    last = torch.full((sum(counts),), hi, dtype=torch.int32, device="cuda")
    first[-1] += 100
    kw = dict(first=first, last=last, sinks=sinks, cap=9.0)
    lse, status = scores.run(cuda_lib, made, counts, q, out, **kw)
    assert status == 0
    scores.check(cuda_lib, made, None, counts, q, out, lse, **kw)


@pytest.mark.parametrize("counts,mass", [([1, 1, 1], True), ([3, 130], False), ([260], False)])
def test_the_same_call_gives_the_same_bits_and_rows_behind_stay(cuda_lib, counts, mass):
    import torch
    from tests import paged, scores
    from tests.test_gpu_paged_attention import _chunk_inputs, _spread
    kv = cuda_lib
    made = paged.Made(kv, _spread(len(counts), 1, 4, 300, 5000), 16, 128, 64, seed=4, mass=mass)
    scores.positions_of(made, 4, 4)
    q, out = _chunk_inputs(made, counts + [5], 16, False, 4)
    tok = sum(counts)
    first = torch.full((tok,), 50, dtype=torch.int32, device="cuda")
    got = []
    for _ in range(3):
        if mass:
            made.cache.mass.copy_(made.mass0)
        lse, status = scores.run(kv, made, counts, q[:tok], out[:tok], mass=mass, cap=20.0, slopes=_slopes(16),
                                 first=first, sinks=2)
        assert status == 0
        got.append([out.clone(), lse] + ([made.cache.mass.clone()] if mass else []))
    assert (out[tok:] == -3.0).all()
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("counts,max_rows", [([1, 1], 2048), ([40, 90], 2048), ([40, 90], LONG_TABLE)])
def test_graph_replays_follow_lengths_positions_and_bounds(cuda_lib, counts, max_rows):
    import torch
    from tests import paged, scores
    from tests.test_gpu_paged_attention import _chunk_inputs, _spread
    kv = cuda_lib
    a = paged.Made(kv, _spread(2, 1, 2, 100, 150), 8, 128, 64, seed=21, max_rows=max_rows)
    b = paged.Made(kv, _spread(2, 1, 2, 900, 2000), 8, 128, 64, seed=22, max_rows=max_rows)
    pa, pb = scores.positions_of(a, 3, 21), scores.positions_of(b, 3, 22)
    q, out = _chunk_inputs(a, counts, 8, False, 21)
    chunk, c = kv.Chunk(counts), a.cache
    tok = sum(counts)
    slopes = _slopes(8)
    first = torch.full((tok,), 20, dtype=torch.int32, device="cuda")
    last = torch.full((tok,), 140, dtype=torch.int32, device="cuda")
    ws = torch.empty(kv.kv_paged_attention_scored_workspace_size(c, chunk), dtype=torch.uint8, device="cuda")
    lse = torch.empty((tok, 8), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def call():
        kv.kv_paged_attention_scored(c, chunk, 0, q, out, ws, softcap=10.0, slopes=slopes, first=first, last=last,
                                     lse=lse)

    with torch.cuda.stream(s):
        call()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for made, pos, f in ((a, pa, 30), (b, pb, 400)):
        for x, y in ((c.k_pages, made.cache.k_pages), (c.v_pages, made.cache.v_pages),
                     (c.page_table, made.cache.page_table), (c.lens, made.cache.lens),
                     (c.positions, made.cache.positions)):
            x.copy_(y)
        first.fill_(f)
        last.fill_(f + 700)
        g.replay()
        torch.cuda.synchronize()
        assert kv.kv_check_status(c.status) == 0
        a.K, a.V = made.K, made.V
        scores.check(kv, a, pos, counts, q, out, lse, cap=10.0, slopes=slopes, first=first, last=last)


@pytest.mark.parametrize("counts,hi,max_rows", [([1, 1], 900, None), ([1, 1], 9000, None), ([190, 140], 900, None),
                                                ([190, 140], 900, LONG_TABLE)])
def test_an_expired_wait_is_reported(cuda_lib, counts, hi, max_rows):
    """With a wait limit of 0 a call posts KV_ERR_TIMEOUT and returns, or none had to wait; the next call with
    the usual limit is right."""
    from tests import paged, scores
    from tests.test_gpu_paged_attention import _chunk_inputs, _spread
    kv = cuda_lib
    made = paged.Made(kv, _spread(2, 1, 2, 200, hi), 8, 128, 64, seed=8, max_rows=max_rows)
    pos = scores.positions_of(made, 3, 8)
    q, out = _chunk_inputs(made, counts, 8, False, 8)
    kw = dict(cap=10.0, slopes=_slopes(8))
    limit = kv.kv_get_wait_limit_ns()
    try:
        kv.kv_set_wait_limit_ns(0)
        for _ in range(5):
            lse, status = scores.run(kv, made, counts, q, out, **kw)
            assert status in (kv.KV_OK, kv.KV_ERR_TIMEOUT)
            if status == kv.KV_OK:
                scores.check(kv, made, pos, counts, q, out, lse, **kw)
    finally:
        kv.kv_set_wait_limit_ns(limit)
    lse, status = scores.run(kv, made, counts, q, out, **kw)
    assert status == 0
    scores.check(kv, made, pos, counts, q, out, lse, **kw)


@pytest.mark.parametrize("counts,hi", [([1] * 64, 8000), ([16] * 16, 1000), ([1] * 8, 30000), ([300, 200], 20000)])
def test_other_kernels_on_the_gpu_change_nothing(cuda_lib, counts, hi):
    """Calls beside copies on another stream, which share the SMs, give the bits of a quiet call."""
    import torch
    from tests import paged, scores
    from tests.test_gpu_paged_attention import _chunk_inputs, _spread
    kv = cuda_lib
    made = paged.Made(kv, _spread(len(counts), 1, 4, hi - 300, hi), 16, 128, 64, seed=55)
    scores.positions_of(made, 3, 55)
    q, out = _chunk_inputs(made, counts, 16, False, 55)
    chunk, c = kv.Chunk(counts), made.cache
    slopes = _slopes(16, 0.1)
    first = torch.zeros(sum(counts), dtype=torch.int32, device="cuda") + 700
    ws = torch.empty(kv.kv_paged_attention_scored_workspace_size(c, chunk), dtype=torch.uint8, device="cuda")
    lse = torch.empty((sum(counts), 16), device="cuda")
    busy = torch.empty((2, 1 << 30), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    want = None
    for i in range(20):
        out.fill_(-3.0)
        torch.cuda.synchronize()
        if want is not None:
            with torch.cuda.stream(side):
                for _ in range(3):
                    busy[0].copy_(busy[1])
        kv.kv_paged_attention_scored(c, chunk, 0, q, out, ws, softcap=30.0, slopes=slopes, first=first, lse=lse)
        assert kv.kv_check_status(c.status) == 0
        if want is None:
            want = [out.clone(), lse.clone()]
        for a, b in zip((out, lse), want):
            assert torch.equal(a, b), i
    torch.cuda.synchronize()                     # the copies end before their memory is free


@pytest.mark.parametrize("counts,max_rows", [([1, 1], None), ([190, 130], None), ([190, 130], LONG_TABLE)])
def test_bad_lengths_and_pages_are_reported(cuda_lib, counts, max_rows):
    from tests import paged, scores
    from tests.test_gpu_paged_attention import _chunk_inputs, _spread
    import torch
    kv = cuda_lib
    for what in ("length", "page"):
        got = []
        for bad in (True, False):
            made = paged.Made(kv, _spread(2, 1, 2, 200, 300), 8, 128, 64, seed=8, max_rows=max_rows)
            scores.positions_of(made, 3, 8)
            q, out = _chunk_inputs(made, counts, 8, False, 8)
            if bad and what == "page":
                made.cache.page_table[0, 0, 1, 1] = made.cache.num_pages
            elif bad:
                made.cache.lens[0, 0, 1] = made.cache.max_pages * 64 + 1
            first = torch.full((sum(counts),), 3, dtype=torch.int32, device="cuda")
            lse, status = scores.run(kv, made, counts, q, out, slopes=_slopes(8), first=first)
            assert status == (kv.KV_ERR_INVALID_ARG if bad else 0)
            got.append((out[counts[0]:], lse[counts[0]:]))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_two_steps_at_once(cuda_lib):
    """Two streams' calls on one cache, each with a workspace of its own, give the bits of one after the other."""
    import torch
    from tests import paged, scores
    from tests.test_gpu_paged_attention import _chunk_inputs, _spread
    kv = cuda_lib
    for counts, hi in (([1, 1], 900), ([1, 1], 9000), ([200, 300], 900), ([200, 300], 9000)):
        made = paged.Made(kv, _spread(2, 2, 4, 300, hi), 16, 128, 64, seed=3)
        scores.positions_of(made, 3, 3)
        c, chunk = made.cache, kv.Chunk(counts)
        q, out = _chunk_inputs(made, counts, 16, False, 3)
        slopes = 0.1 * torch.rand(16, device="cuda")
        first = torch.full((sum(counts),), 20, dtype=torch.int32, device="cuda")
        size = kv.kv_paged_attention_scored_workspace_size(c, chunk)

        def calls(streams):
            outs = [out.clone() for _ in streams]
            ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in streams]
            torch.cuda.synchronize()
            for _ in range(5):
                for layer, s in enumerate(streams):
                    kv.kv_paged_attention_scored(c, chunk, layer, q, outs[layer], ws[layer], softcap=20.0,
                                                 slopes=slopes, first=first, stream=s)
            torch.cuda.synchronize()
            assert kv.kv_check_status(c.status) == 0
            return outs

        one = torch.cuda.Stream()
        for a, b in zip(calls([one, one]), calls([torch.cuda.Stream(), torch.cuda.Stream()])):
            assert torch.equal(a, b)


def test_a_run_of_the_operators(cuda_lib):
    """A prompt read, two hypotheses that go on from it, tokens for each, one dropped, compaction, more
    tokens: every step's attention is that of rows turned and kept on the host."""
    import torch
    from tests import paged, scores
    kv = cuda_lib
    R, L, H, Hq, d, page, dt = 3, 2, 2, 8, 64, 16, torch.bfloat16
    c = kv.PagedCache.allocate(R, L, H, Hq, d, 200, page, dt, positions=True, refs=True)
    c.page_table.fill_(-1)
    rot = kv.Rotary.make(d, scaling="linear", scale=2.0)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    slopes, cap = _slopes(Hq, 0.2), 12.0
    rows = {(r, l): [] for r in range(R) for l in range(L)}     # (position, K [H][d], V [H][d]) on the host

    def step(counts, base):
        chunk = kv.Chunk(counts)
        tok = chunk.tokens
        kv.kv_paged_reserve(c, chunk, ws)
        where = torch.cat([base[r] + torch.arange(n) for r, n in enumerate(counts)]).int().cuda()
        for layer in range(L):
            q, k, v = (torch.randn((tok, n, d), generator=gen, device="cuda").to(dt) for n in (Hq, H, H))
            qt, kt = torch.empty_like(q), torch.empty_like(k)
            kv.kv_rotary(rot, where, q, qt)
            kv.kv_rotary(rot, where, k, kt)
            kv.kv_paged_append_rotary(c, chunk, layer, rot, where, q, q, k, v)
            assert torch.equal(q, qt)
            out, lse = torch.empty_like(q), torch.empty((tok, Hq), device="cuda")
            kv.kv_paged_attention_scored(c, chunk, layer, q, out, ws, softcap=cap, slopes=slopes, lse=lse)
            assert kv.kv_check_status(c.status) == 0
            t0 = 0
            for r, n in enumerate(counts):
                for i in range(n):
                    rows[r, layer].append((int(where[t0 + i]), kt[t0 + i].double(), v[t0 + i].double()))
                mine = rows[r, layer]
                assert int(c.lens[r, layer, 0]) == len(mine)
                for h in range(H if n else 0):
                    pos = torch.tensor([x[0] for x in mine], device="cuda")
                    K, V = (torch.stack([x[j][h] for x in mine]) for j in (1, 2))
                    g = slice(h * Hq // H, (h + 1) * Hq // H)
                    o, z, _, absv, pev, pe, _ = scores.scored_unit(q[t0:t0 + n, g].double(), K, V, pos, d ** -0.5, cap,
                                                                   slopes[g])
                    got = out[t0:t0 + n, g].double()
                    assert ((got - o).abs() <= scores.out_bound(o, absv, pev, pe, dt, len(mine))).all()
                    assert ((lse[t0:t0 + n, g].double() - z).abs() <= scores.lse_bound(z, pe, len(mine))).all()
                t0 += n

    step([37, 5, 0], [0, 0, 0])
    step([1, 1, 0], [37, 5, 0])
    kv.kv_paged_fork(c, torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda"))
    for l in range(L):
        for r in (1, 2):
            rows[r, l] = list(rows[0, l])
    used = int((c.refs > 0).sum())
    assert int(c.refs.max()) == 3 and used == L * H * 3
    step([1, 1, 1], [38] * 3)
    step([2, 20, 1], [39] * 3)
    kv.kv_paged_fork(c, torch.tensor([-1, 1, 2], dtype=torch.int32, device="cuda"))
    for l in range(L):
        rows[0, l] = []
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.kv_paged_compact(c, ws, live=live)
    assert int(live) == int((c.refs > 0).sum()) and not c.refs[int(live):].any()
    step([3, 1, 70], [1000, 59, 40])
    refs = c.refs.clone()
    kv.kv_paged_count_refs(c)
    assert torch.equal(refs, c.refs)
