"""Attention over the pages, form by form of its kernels: the weights' two 16-bit parts where few
query rows share a head's rows, long chunks whose units are taken in several groups, groups of more
than 16 query heads, and waits that run out."""
import math

import pytest

from tests.test_gpu_paged_attention import _chunk_inputs, _run, _spread

pytestmark = pytest.mark.gpu


# (query heads of a KV head, d, dtype, new tokens, earlier rows, rows that the tables can hold):
# tables to 8192 rows take the one-launch form, longer ones the cut one
TWO_PARTS = {
    "one_launch_g4": (4, 128, "bf16", 1, 20, 512),
    "one_launch_g7": (7, 64, "fp16", 1, 20, 512),
    "one_launch_g16": (16, 128, "fp16", 1, 20, 512),
    "one_launch_tiles": (4, 128, "bf16", 1, 200, 512),
    "row_blocks": (4, 64, "bf16", 16, 24, 512),
    "cut_g4": (4, 128, "bf16", 1, 200, 20000),
    "cut_g1": (1, 64, "fp16", 1, 20, 20000),
    "cut_16_rows": (4, 128, "fp16", 4, 20, 20000),
}


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("name", TWO_PARTS)
def test_few_rows_weights_keep_two_parts(cuda_lib, name, mass):
    """Values whose weighted average all but cancels: one 16-bit part of the weights would be past
    this bound several times over (tests/test_paged_bounds.py)."""
    import torch
    from tests import paged
    G, d, dtype, T, n, cap = TWO_PARTS[name]
    if mass and T * G > 16:
        pytest.skip("with weights added, more than 16 query rows take one part")
    H = 2
    made = paged.Made(cuda_lib, [[[n + T] * H]], H * G, d, 32, dtype, mass=mass, max_rows=cap,
                      seed=51)
    c = made.cache
    units = [paged.cancelling(n, T, d, made.dtype, 51 + h, "cuda") for h in range(H)]
    q = torch.empty((T, H * G, d), dtype=made.dtype, device="cuda")
    for h, (query, K, V, _) in enumerate(units):
        rows = made.rows(0, 0, h)
        c.k_pages.view(-1, d)[rows], c.v_pages.view(-1, d)[rows] = K, V
        q[:, h * G:(h + 1) * G] = query
    out = torch.full_like(q, -3.0)
    lse, status = _run(cuda_lib, made, [T], q, out, mass=mass)
    assert status == 0
    for h, (query, K, V, scale) in enumerate(units):
        o, z, _, absv, logit = paged.attend_unit(q[:, h * G:(h + 1) * G].double(), K.double(),
                                                 V.double(), 0, 0, scale)
        got = out[:, h * G:(h + 1) * G].double()
        ratio = (got - o).abs() / paged.out_bound(o, absv, made.dtype, d, n + T, logit, 2)
        assert float(ratio.max()) <= 1
        gz = lse[:, h * G:(h + 1) * G].double()
        assert ((gz - z).abs() <= paged.lse_bound(z, d, n + T, logit)).all()


def _groups(made, counts, window, sinks):
    """How many groups of units the many-rows kernel takes them in: as few as leave each 64 MB of
    K and V (4 at most), or 128 key tiles for each of 152 CTAs."""
    c = made.cache
    G = c.num_q_heads // c.num_kv_heads
    rows = c.num_requests * c.num_kv_heads * c.max_pages * c.page_size
    phases = min(4, -(-rows * c.head_dim * 4 // (64 << 20)))
    work = 0
    for r, count in enumerate(counts):
        items = -(-count * G // 256)
        for h in range(c.num_kv_heads):
            t0 = int(made.lens_host[r, 0, h]) - count
            r0 = items // 2 * 256
            t_hi = t0 + (min(count * G, r0 + 256) - 1) // G
            lo = max(0, t0 + r0 // G - window + 1) if window else 0
            first = lo >> 7
            work += items * (min(-(-min(sinks, lo) // 128), first) + (t_hi >> 7) + 1 - first)
    return min(phases, work // (152 * 128))


# (dtype, counts, shortest, longest, window, sinks, weights, groups)
LONG_CHUNKS = {
    "weights": ("bf16", [512, 420], 36000, 52000, 0, 0, True, 2),
    "window_weights": ("fp16", [600, 700], 36000, 52000, 30000, 300, True, 2),
    "four_groups": ("fp16", [1100, 1000], 36000, 52000, 0, 0, False, 4),
}


@pytest.mark.parametrize("name", LONG_CHUNKS)
def test_long_chunks_in_groups_of_units(cuda_lib, name):
    import torch
    from tests import paged
    dtype, counts, lo, hi, window, sinks, mass, groups = LONG_CHUNKS[name]
    H, G, d = 8, 4, 64
    made = paged.Made(cuda_lib, _spread(2, 1, H, lo, hi), H * G, d, 64, dtype, mass=mass, seed=52)
    assert _groups(made, counts, window, sinks) == groups
    q, out = _chunk_inputs(made, counts, H * G, False, 52)
    lse, status = _run(cuda_lib, made, counts, q, out, 0, window, sinks, mass)
    assert status == 0
    want_mass = made.mass0.double().view(-1).clone()
    tol = torch.zeros_like(want_mass)
    t0 = 0
    for r, count in enumerate(counts):
        for h in range(H):
            n = int(made.lens_host[r, 0, h])
            o, z, w, absv, logit = paged.attend_unit(
                q[t0:t0 + count, h * G:(h + 1) * G].double(), made.K[r, 0, h], made.V[r, 0, h],
                window, sinks, 1 / math.sqrt(d))
            # Additions that a value passes through.  A row's sum: 32 of a tile's 128 keys in each of
            # four accumulators and two joins, then a tile's sum after the other, then partials.  An
            # output: a product of 16 keys after the other, then partials.
            tiles = n // 128 + 1
            depth = 36 + tiles + 152
            steps = 16 + 8 * tiles + 152
            got = out[t0:t0 + count, h * G:(h + 1) * G].double()
            assert torch.isfinite(got).all()
            ratio = (got - o).abs() / paged.out_bound(o, absv, made.dtype, d, steps, logit, 1)
            assert float(ratio.max()) <= 1, (r, h, float(ratio.max()))
            gz = lse[t0:t0 + count, h * G:(h + 1) * G].double()
            ratio = (gz - z).abs() / paged.lse_bound(z, d, depth, logit)
            assert float(ratio.max()) <= 1, (r, h, float(ratio.max()))
            if mass:
                rows = made.rows(r, 0, h)
                tol[rows] = paged.mass_bound(w, want_mass[rows], d, depth, logit, count * G)
                want_mass[rows] += w
        t0 += count
    if mass:
        assert ((made.cache.mass.double().view(-1) - want_mass).abs() <= tol).all()


# (KV heads, query heads, d, page, dtype, counts, shortest, longest, window, sinks, weights)
WIDE_GROUPS = {
    "g17": (1, 17, 128, 64, "bf16", [1, 1], 100, 700, 0, 0, True),
    "g20_short": (2, 40, 64, 16, "fp16", [1, 1, 1], 1, 400, 0, 0, False),
    "g24_long": (1, 24, 128, 128, "bf16", [1], 9000, 9000, 0, 0, True),
    "g64_window": (1, 64, 128, 32, "bf16", [1, 1], 500, 9000, 300, 4, True),
    "g128": (1, 128, 64, 64, "fp16", [1, 2], 33, 900, 0, 0, False),
    "g300": (1, 300, 64, 64, "bf16", [1], 257, 257, 0, 0, True),
}


@pytest.mark.parametrize("name", WIDE_GROUPS)
def test_one_token_of_wide_groups(cuda_lib, name):
    from tests import paged
    from tests.test_gpu_paged_attention import _check
    H, Hq, d, page, dtype, counts, lo, hi, window, sinks, mass = WIDE_GROUPS[name]
    made = paged.Made(cuda_lib, _spread(len(counts), 1, H, lo, hi), Hq, d, page, dtype, mass=mass,
                      max_rows=hi + page, seed=53)
    q, out = _chunk_inputs(made, counts, Hq, False, 53)
    lse, status = _run(cuda_lib, made, counts, q, out, 0, window, sinks, mass)
    assert status == 0
    _check(made, counts, q, out, lse, 0, window, sinks, mass)


# (new tokens, longest unit, weights added): the one-launch form, the cut form, the many-rows kernel
EXPIRED = {
    "one_launch": ([1] * 64, 8000, False),
    "one_launch_weights": ([1] * 64, 8000, True),
    "cut": ([1] * 8, 30000, False),
    "cut_weights": ([1] * 8, 30000, True),
    "many": ([300, 200], 20000, False),
    "many_weights": ([300, 200], 20000, True),
}


@pytest.mark.parametrize("name", EXPIRED)
def test_a_wait_that_runs_out_is_reported(cuda_lib, name):
    """With a wait limit of 0, beside copies that keep the memory busy (a wait sleeps for some
    microseconds before it first looks at its limit): the timeout is posted, the call returns,
    and the next one with the usual limit is right."""
    import torch
    from tests import paged
    from tests.test_gpu_paged_attention import _check
    kv = cuda_lib
    counts, hi, mass = EXPIRED[name]
    made = paged.Made(kv, _spread(len(counts), 1, 4, hi - 300, hi), 16, 128, 64, seed=54, mass=mass)
    q, out = _chunk_inputs(made, counts, 16, False, 54)
    chunk, c = kv.Chunk(counts), made.cache
    ws = torch.empty(kv.kv_paged_attention_workspace_size(c, chunk, mass), dtype=torch.uint8,
                     device="cuda")
    busy = torch.empty((2, 1 << 30), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    limit = kv.kv_get_wait_limit_ns()
    status = kv.KV_OK
    try:
        kv.kv_set_wait_limit_ns(0)
        for _ in range(100):                     # more than half of the calls run into it
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                for _ in range(3):
                    busy[0].copy_(busy[1])
            kv.kv_paged_attention(c, chunk, 0, q, out, ws, add_mass=mass)
            status = kv.kv_check_status(c.status)
            if status != kv.KV_OK:
                break
    finally:
        kv.kv_set_wait_limit_ns(limit)
        torch.cuda.synchronize()                 # the copies end before their memory is free
    assert status == kv.KV_ERR_TIMEOUT
    if mass:
        c.mass.copy_(made.mass0)
    lse, status = _run(kv, made, counts, q, out, mass=mass)
    assert status == 0
    _check(made, counts, q, out, lse, mass=mass)


# (new tokens, longest unit, weights added)
BESIDE = {
    "one_launch": ([1] * 64, 8000, False),
    "one_launch_weights": ([1] * 64, 8000, True),
    "one_launch_clusters": ([1] * 8, 8000, False),
    "row_blocks": ([16] * 16, 1000, False),
    "cut": ([1] * 8, 30000, False),
    "cut_weights": ([1, 2] * 8, 30000, True),
    "many": ([300, 200], 20000, False),
    "many_weights": ([300, 200], 20000, True),
}


@pytest.mark.parametrize("name", BESIDE)
def test_other_kernels_on_the_gpu_change_nothing(cuda_lib, name):
    """Calls beside copies on another stream, which share the SMs, give the bits of a quiet call."""
    import torch
    from tests import paged
    kv = cuda_lib
    counts, hi, mass = BESIDE[name]
    made = paged.Made(kv, _spread(len(counts), 1, 4, hi - 300, hi), 16, 128, 64, seed=55, mass=mass)
    q, out = _chunk_inputs(made, counts, 16, False, 55)
    chunk, c = kv.Chunk(counts), made.cache
    ws = torch.empty(kv.kv_paged_attention_workspace_size(c, chunk, mass), dtype=torch.uint8,
                     device="cuda")
    lse = torch.empty((sum(counts), 16), device="cuda")
    busy = torch.empty((2, 1 << 30), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    want = None
    for i in range(30):
        out.fill_(-3.0)
        if mass:
            c.mass.copy_(made.mass0)
        torch.cuda.synchronize()
        if want is not None:
            with torch.cuda.stream(side):
                for _ in range(3):
                    busy[0].copy_(busy[1])
        kv.kv_paged_attention(c, chunk, 0, q, out, ws, lse=lse, add_mass=mass)
        assert kv.kv_check_status(c.status) == 0
        got = [out, lse] + ([c.mass] if mass else [])
        if want is None:
            want = [t.clone() for t in got]
        for a, b in zip(got, want):
            assert torch.equal(a, b), i
    torch.cuda.synchronize()                     # the copies end before their memory is free
