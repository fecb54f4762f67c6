"""Rows into pages, eviction by accumulated weight, and the whole life of a cache: prefill
eviction, load, append, attention, eviction again."""
import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu


def _bits(t):
    import torch
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16)


def _spread(R, L, H, lo, hi):
    return [[[lo + int((hi - lo + 1) * ((0.618 * ((r * L + l) * H + h) + 0.99) % 1))
              for h in range(H)] for l in range(L)] for r in range(R)]


@pytest.mark.parametrize("d,page,dtype,counts,lo,hi", [
    (128, 64, "bf16", [1, 1, 1], 1, 90), (64, 16, "fp16", [5, 0, 17, 1], 17, 60),
    (128, 32, "bf16", [40], 20, 30),        # longer than its units: the first tokens have no row
    (64, 128, "bf16", [1, 2], 0, 3), (128, 16, "fp16", [300], 300, 700)])
@pytest.mark.parametrize("strided", [False, True])
def test_append_writes_the_last_rows(cuda_lib, d, page, dtype, counts, lo, hi, strided):
    import torch
    from tests import paged
    kv = cuda_lib
    H, layer, tok = 3, 1, sum(counts)
    made = paged.Made(kv, _spread(len(counts), 2, H, lo, hi), 6, d, page, dtype, mass=True, seed=1)
    c = made.cache
    new = torch.randn((tok, 2 * H * d + (40 if strided else 0)), device="cuda").to(made.dtype)
    k_new = new[:, :H * d].view(tok, H, d)
    v_new = new[:, H * d:2 * H * d].view(tok, H, d)
    if not strided:
        k_new, v_new = k_new.contiguous(), v_new.contiguous()
    k, v, mass = c.k_pages.clone(), c.v_pages.clone(), c.mass.clone()
    t0 = 0
    for r, count in enumerate(counts):
        for h in range(H):
            n = int(made.lens_host[r, layer, h])
            rows = made.rows(r, layer, h)
            for i in range(count):
                if n - count + i >= 0:
                    x = int(rows[n - count + i])
                    k.view(-1, d)[x], v.view(-1, d)[x] = k_new[t0 + i, h], v_new[t0 + i, h]
                    mass.view(-1)[x] = 0
        t0 += count
    kv.kv_paged_append(c, kv.Chunk(counts), layer, k_new, v_new)
    torch.cuda.synchronize()
    for a, b in ((c.k_pages, k), (c.v_pages, v), (c.mass, mass)):
        assert torch.equal(_bits(a), _bits(b))
    assert kv.kv_check_status(c.status) == 0


def test_append_skips_pages_that_do_not_exist(cuda_lib):
    import torch
    from tests import paged
    kv = cuda_lib
    made = paged.Made(kv, _spread(2, 1, 2, 100, 100), 4, 64, 16, seed=2)
    c = made.cache
    c.page_table[0, 0, 0, 6] = c.num_pages
    c.page_table[1, 0, 1, 6] = -1
    c.lens[0, 0, 1] = c.max_pages * 16 + 1
    want = c.k_pages.clone()
    new = torch.ones((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    want.view(-1, 64)[int(made.rows(1, 0, 0)[-1])] = 1
    kv.kv_paged_append(c, kv.Chunk([1, 1]), 0, new, new)
    torch.cuda.synchronize()
    assert torch.equal(_bits(c.k_pages), _bits(want))
    assert kv.kv_check_status(c.status) == kv.KV_ERR_INVALID_ARG


@pytest.mark.parametrize("d,page,dtype,lo,hi", [(128, 64, "bf16", 0, 200), (64, 16, "fp16", 1, 33),
                                                (128, 128, "bf16", 600, 900), (64, 32, "bf16", 0, 0)])
@pytest.mark.parametrize("with_mass", [False, True])
def test_load_packed_rows(cuda_lib, d, page, dtype, lo, hi, with_mass):
    import torch
    from tests import paged
    kv = cuda_lib
    lens = _spread(2, 3, 2, lo, hi)
    made = paged.Made(kv, lens, 4, d, page, dtype, mass=True, seed=3)
    c = made.cache
    flat = np.asarray(lens).reshape(-1)
    offsets = np.concatenate([[0], np.cumsum(flat)]).astype(np.int64)
    total = int(offsets[-1])
    k = torch.randn((max(total, 1), d), device="cuda").to(made.dtype)
    v = torch.randn((max(total, 1), d), device="cuda").to(made.dtype)
    w = torch.rand(max(total, 1), device="cuda")
    ek, ev, em = c.k_pages.clone(), c.v_pages.clone(), c.mass.clone()
    for u, n in enumerate(flat):
        r, l, h = u // 6, u // 2 % 3, u % 2
        rows = made.rows(r, l, h)
        a = int(offsets[u])
        ek.view(-1, d)[rows], ev.view(-1, d)[rows] = k[a:a + n], v[a:a + n]
        em.view(-1)[rows] = w[a:a + n] if with_mass else 0.0
    c.lens.fill_(-9)
    kv.kv_paged_load(c, k, v, torch.from_numpy(offsets).cuda(), total,
                     mass_rows=w if with_mass else None)
    torch.cuda.synchronize()
    assert torch.equal(c.lens.cpu(), made.lens_host)
    for a, b in ((c.k_pages, ek), (c.v_pages, ev), (c.mass, em)):
        assert torch.equal(_bits(a), _bits(b))


def test_load_refuses_a_unit_that_does_not_fit(cuda_lib):
    import torch
    from tests import paged
    kv = cuda_lib
    made = paged.Made(kv, _spread(1, 1, 3, 40, 40), 3, 64, 16, seed=4)
    c = made.cache
    offsets = torch.tensor([0, 10, 10 + 49, 59 + 7], device="cuda")
    rows = torch.ones((66, 64), dtype=torch.bfloat16, device="cuda")
    kv.kv_paged_load(c, rows, rows, offsets, 66)
    torch.cuda.synchronize()
    assert c.lens.cpu().view(-1).tolist() == [10, -1, 7]
    # the unit without a length is reported by the calls after it
    q = torch.zeros((1, 3, 64), dtype=torch.bfloat16, device="cuda")
    chunk = kv.Chunk([1])
    ws = torch.empty(kv.kv_paged_attention_workspace_size(c, chunk), dtype=torch.uint8, device="cuda")
    kv.kv_paged_attention(c, chunk, 0, q, torch.empty_like(q), ws)
    assert kv.kv_check_status(c.status) == kv.KV_ERR_INVALID_ARG


def _evict(kv, made, into, budgets, sinks, recent, stride):
    import torch
    kept = torch.full((made.cache.num_units, stride), -1, dtype=torch.int32, device="cuda")
    ws = torch.full((kv.kv_paged_evict_workspace_size(made.cache),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    b = torch.as_tensor(budgets, dtype=torch.int32, device="cuda")
    kv.kv_paged_evict(made.cache, into, b, sinks, recent, kept, ws)
    return kept, kv.kv_check_status(ws)


@pytest.mark.parametrize("d,page,page2,dtype,lo,hi,blo,bhi,sinks,recent,levels", [
    (128, 64, 64, "bf16", 200, 400, 100, 150, 4, 16, 0),
    (64, 16, 64, "fp16", 30, 90, 40, 60, 0, 0, 5),          # many equal weights
    (128, 32, 16, "bf16", 1, 60, 30, 30, 2, 28, 1),         # all weights equal; pinned rows only
    (64, 128, 32, "bf16", 0, 300, 1, 299, 1, 0, 3),
    (128, 64, 64, "bf16", 9000, 20000, 1000, 9000, 4, 64, 4096),
    (64, 64, 64, "bf16", 33000, 70000, 3000, 65000, 4, 64, 0),
    (64, 32, 64, "bf16", 17000, 17500, 100, 1500, 3, 9, 2000),
    # more rows than a cluster's shared memory holds, and just as many
    (64, 64, 128, "fp16", 131072 + 68, 300000, 3000, 140000, 4, 64, 0),
    (64, 128, 64, "bf16", 131072 + 67, 200000, 5, 200, 2, 1, 600)])
def test_evict_keeps_the_largest_weights(cuda_lib, d, page, page2, dtype, lo, hi, blo, bhi, sinks,
                                         recent, levels):
    import torch
    from tests import paged
    kv = cuda_lib
    R, L, H = (2, 2, 2) if hi < 30000 else (1, 1, 3)
    if lo == 17000:                                          # more clusters than run at once
        R, L, H = 2, 3, 17
    lens = _spread(R, L, H, lo, hi)
    made = paged.Made(kv, lens, 2 * H, d, page, dtype, mass=True, seed=5)
    if levels:
        made.cache.mass.copy_(torch.floor(made.mass0 * levels) / 4)
    budgets = np.asarray(_spread(R, L, H, blo, bhi)).reshape(-1)[::-1].copy()
    most = int(min(budgets.max(), hi))
    into = kv.PagedCache.allocate(R, L, H, 2 * H, d, most, page2, made.dtype, mass=True)
    into.page_table.copy_(torch.flip(into.page_table, dims=[0, 1, 2, 3]))
    kept, status = _evict(kv, made, into, budgets, sinks, recent, most)
    assert status == 0
    src = made.cache
    mass = src.mass.view(-1)
    for u in range(R * L * H):
        r, l, h = u // (L * H), u // H % L, u % H
        n, b = lens[r][l][h], int(budgets[u])
        rows = made.rows(r, l, h)
        want = paged.evict_unit(mass[rows].cpu().tolist(), n, b, sinks, recent)
        m = len(want)
        assert int(into.lens[r, l, h]) == m
        assert kept[u, :m].cpu().tolist() == want
        assert (kept[u, m:] == -1).all()
        j = torch.arange(m, device="cuda")
        to = into.page_table[r, l, h].long()[j // page2] * page2 + j % page2
        frm = rows[torch.as_tensor(want, dtype=torch.long, device="cuda")]
        for a, z in ((src.k_pages, into.k_pages), (src.v_pages, into.v_pages)):
            assert torch.equal(_bits(z.view(-1, d)[to]), _bits(a.view(-1, d)[frm]))
        assert torch.equal(into.mass.view(-1)[to], mass[frm])


def test_evict_reports_bad_budgets_lengths_and_pages(cuda_lib):
    import torch
    from tests import paged
    kv = cuda_lib
    for what, code in (("budget", "KV_ERR_BUDGET"), ("stride", "KV_ERR_BUDGET"),
                       ("table", "KV_ERR_BUDGET"), ("length", "KV_ERR_INVALID_ARG"),
                       ("page", "KV_ERR_INVALID_ARG"), ("dst_page", "KV_ERR_INVALID_ARG")):
        made = paged.Made(kv, _spread(1, 1, 3, 200, 200), 3, 64, 16, mass=True, seed=6)
        into = kv.PagedCache.allocate(1, 1, 3, 3, 64, 50 if what == "table" else 100, 16, mass=True)
        budgets = [80, 80, 80]
        if what == "budget":
            budgets[1] = 19
        elif what == "length":
            made.cache.lens[0, 0, 1] = -4
        elif what == "page":
            made.cache.page_table[0, 0, 1, 0] = made.cache.num_pages + 3
        elif what == "dst_page":
            into.page_table[0, 0, 1, 2] = -1
        kept, status = _evict(kv, made, into, budgets, 4, 16, 70 if what == "stride" else 80)
        assert status == getattr(kv, code), what
        got = into.lens.cpu().view(-1).tolist()
        if what in ("stride", "table"):
            assert got == [-1, -1, -1]
        elif what in ("budget", "length"):
            assert got == [80, -1, 80]
        if what in ("budget", "length", "page", "dst_page"):    # the neighbours are not touched by it
            for h in (0, 2):
                rows = made.rows(0, 0, h)
                want = paged.evict_unit(made.cache.mass.view(-1)[rows].cpu().tolist(), 200, 80, 4, 16)
                assert kept[h, :80].cpu().tolist() == want


@pytest.mark.parametrize("page", [16, 64])
def test_from_prefill_eviction_to_decoding(cuda_lib, page):
    """The whole life of a cache: score, select and compact a prompt; load the kept rows; decode
    steps that append, attend and accumulate; eviction by the accumulated weight; another step."""
    import torch
    from synth.device import DeviceWorkload
    from tests import paged
    kv = cuda_lib
    wl = synth.small_variant(synth.RAGGED_MISTRAL, 0, requests=[700, 1100])
    dw = DeviceWorkload(wl)
    prob = kv.Problem.for_workload(wl, score_rule=kv.KV_SCORE_ATTN_SUM, head_budgets=True)
    R, L, H, Hq, d = wl.num_requests, wl.num_layers, wl.num_kv_heads, wl.num_q_heads, wl.head_dim
    bufs = kv.Buffers(prob, np.full((R, L, H), 150, dtype=np.int32))
    sel, k_out, v_out, offsets = kv.evict(prob, dw.q, dw.k, dw.v, bufs)
    cap = 2 * 150 + 40
    cache = kv.PagedCache.allocate(R, L, H, Hq, d, 2200, page, mass=True)
    # accumulated weight so far: the score (attention sum) of each kept row
    off = offsets.cpu().numpy()
    units = [(r, l, h) for r in range(R) for l in range(L) for h in range(H)]
    cu = dw.cu_host
    w0 = torch.cat([bufs.scores[l, h, int(cu[r]):int(cu[r + 1])][sel[off[u]:off[u + 1]].long()]
                    for u, (r, l, h) in enumerate(units)])
    kv.kv_paged_load(cache, k_out, v_out, offsets, bufs.total_rows, mass_rows=w0)
    ref = {x: [k_out[off[u]:off[u + 1]].double(), v_out[off[u]:off[u + 1]].double(),
               w0[off[u]:off[u + 1]].double()] for u, x in enumerate(units)}
    g = torch.Generator(device="cuda").manual_seed(1)
    G = Hq // H

    def step(cache, counts, window=0, sinks=0):
        chunk = kv.Chunk(counts)
        cache.advance(chunk)
        for layer in range(L):
            qkv = torch.randn((chunk.tokens, (Hq + 2 * H) * d), generator=g,
                              device="cuda").bfloat16()
            q = qkv[:, :Hq * d].view(-1, Hq, d)
            kn = qkv[:, Hq * d:(Hq + H) * d].view(-1, H, d)
            vn = qkv[:, (Hq + H) * d:].view(-1, H, d)
            kv.kv_paged_append(cache, chunk, layer, kn, vn)
            ws = torch.empty(kv.kv_paged_attention_workspace_size(cache, chunk, True),
                             dtype=torch.uint8, device="cuda")
            out = torch.empty((chunk.tokens, Hq, d), dtype=torch.bfloat16, device="cuda")
            kv.kv_paged_attention(cache, chunk, layer, q, out, ws, window=window, num_sinks=sinks,
                                  add_mass=True)
            assert kv.kv_check_status(cache.status) == 0
            t0 = 0
            for r, count in enumerate(counts):
                for h in range(H):
                    K, V, w = ref[r, layer, h]
                    K = torch.cat([K, kn[t0:t0 + count, h].double()])
                    V = torch.cat([V, vn[t0:t0 + count, h].double()])
                    w = torch.cat([w, torch.zeros(count, device="cuda", dtype=torch.float64)])
                    o, z, dw_, absv, logit = paged.attend_unit(
                        q[t0:t0 + count, h * G:(h + 1) * G].double(), K, V, window, sinks, d ** -0.5)
                    got = out[t0:t0 + count, h * G:(h + 1) * G].double()
                    assert ((got - o).abs() <= paged.out_bound(o, absv, torch.bfloat16, d,
                                                               K.shape[0], logit, 1)).all()
                    ref[r, layer, h] = [K, V, w + dw_]
                t0 += count

    for counts, window, sinks in (([20, 33], 0, 0), ([1, 1], 0, 0), ([1, 1], 64, 4), ([0, 1], 0, 0)):
        step(cache, counts, window, sinks)
    # eviction back to 100 rows a head, in other pages; the accumulated weights decide
    into = kv.PagedCache.allocate(R, L, H, Hq, d, 200, page, mass=True)
    kept = torch.empty((len(units), 100), dtype=torch.int32, device="cuda")
    ws = torch.empty(kv.kv_paged_evict_workspace_size(cache), dtype=torch.uint8, device="cuda")
    budgets = torch.full((len(units),), 100, dtype=torch.int32, device="cuda")
    kv.kv_paged_evict(cache, into, budgets, 4, 16, kept, ws)
    assert kv.kv_check_status(ws) == 0
    for u, x in enumerate(units):
        K, V, w = ref[x]
        n, m = K.shape[0], min(K.shape[0], 100)
        rows = cache.page_table[x].long().repeat_interleave(page) * page
        rows = (rows + torch.arange(page, device="cuda").repeat(cache.max_pages))[:n]
        have = cache.mass.view(-1)[rows].double()
        torch.testing.assert_close(have, w, rtol=1e-4, atol=1e-6)
        want = paged.evict_unit(have.cpu().tolist(), n, 100, 4, 16)
        assert int(into.lens[x]) == m and kept[u, :m].cpu().tolist() == want
        idx = torch.as_tensor(want, device="cuda")
        ref[x] = [K[idx], V[idx], have[idx]]
    step(into, [1, 5])


@pytest.mark.parametrize("d,H,counts", [(128, 8, [3001, 0, 5, 2000]), (64, 3, [4097])])
def test_append_of_a_prompts_rows(cuda_lib, d, H, counts):
    import torch
    from tests import paged
    kv = cuda_lib
    made = paged.Made(kv, _spread(len(counts), 2, H, 3100, 4500), H, d, 64, mass=True, seed=11)
    c, tok = made.cache, sum(counts)
    new = torch.randn((tok, 2 * H * d), device="cuda").to(made.dtype)
    k_new, v_new = new[:, :H * d].view(tok, H, d), new[:, H * d:].view(tok, H, d)
    want = [c.k_pages.clone(), c.v_pages.clone(), c.mass.clone()]
    t0 = 0
    for r, count in enumerate(counts):
        for h in range(H):
            n = int(made.lens_host[r, 1, h])
            skip = max(0, count - n)                    # tokens without a row
            rows = made.rows(r, 1, h)[n - (count - skip):]
            want[0].view(-1, d)[rows] = k_new[t0 + skip:t0 + count, h]
            want[1].view(-1, d)[rows] = v_new[t0 + skip:t0 + count, h]
            want[2].view(-1)[rows] = 0
        t0 += count
    kv.kv_paged_append(c, kv.Chunk(counts), 1, k_new, v_new)
    assert kv.kv_check_status(c.status) == 0
    for a, b in zip((c.k_pages, c.v_pages, c.mass), want):
        assert torch.equal(_bits(a), _bits(b))


@pytest.mark.parametrize("hi,levels", [(20000, 1), (20000, 2), (135000, 1)])
def test_evict_with_one_weight_for_all_rows(cuda_lib, hi, levels):
    """Rows loaded without weights all have 0: the first ones stay.  Units by clusters, and past
    what a cluster holds."""
    import torch
    from tests import paged
    kv = cuda_lib
    lens = _spread(1, 1, 3, hi - 3000, hi)
    made = paged.Made(kv, lens, 3, 64, 64, mass=True, seed=12)
    made.cache.mass.copy_(torch.floor(made.mass0 * levels))
    into = kv.PagedCache.allocate(1, 1, 3, 3, 64, 7000, 64, made.dtype, mass=True)
    kept, status = _evict(kv, made, into, [7000, 300, 80], 4, 64, 7000)
    assert status == 0
    for h, b in enumerate([7000, 300, 80]):
        rows = made.rows(0, 0, h)
        want = paged.evict_unit(made.cache.mass.view(-1)[rows].cpu().tolist(), lens[0][0][h], b, 4, 64)
        assert kept[h, :b].cpu().tolist() == want
        assert int(into.lens[0, 0, h]) == b


def test_load_reports_rows_that_it_could_not_write(cuda_lib):
    """A page that does not exist holds rows in use: they cannot be written, which is said."""
    import torch
    from tests import paged
    kv = cuda_lib
    for bad in (lambda c: c.num_pages, lambda c: -1):
        made = paged.Made(kv, _spread(1, 1, 3, 40, 40), 3, 64, 16, seed=13, mass=True)
        c = made.cache
        page = bad(c)
        want = [c.k_pages.clone(), c.v_pages.clone()]
        x = torch.randn((120, 64), device="cuda").to(made.dtype)
        for h in range(3):
            rows = made.rows(0, 0, h)
            j = torch.arange(40, device="cuda")
            if h == 1:
                rows, j = rows[j // 16 != 1], j[j // 16 != 1]
            want[0].view(-1, 64)[rows] = x[40 * h + j]
            want[1].view(-1, 64)[rows] = x[40 * h + j]
        c.page_table[0, 0, 1, 1] = page
        offsets = torch.tensor([0, 40, 80, 120], device="cuda")
        kv.kv_paged_load(c, x, x, offsets, 120)
        assert kv.kv_check_status(c.status) == kv.KV_ERR_INVALID_ARG
        assert c.lens.view(-1).tolist() == [40, 40, 40]
        for a, b in zip((c.k_pages, c.v_pages), want):
            assert torch.equal(_bits(a), _bits(b))
        assert kv.kv_check_status(c.status) == 0


def test_load_refuses_units_whose_rows_are_not_there(cuda_lib):
    """Offsets that run past the packed rows: such a unit gets length -1, and none of its rows."""
    import torch
    from tests import paged
    kv = cuda_lib
    made = paged.Made(kv, _spread(1, 1, 3, 40, 40), 3, 64, 16, seed=14)
    c = made.cache
    want = c.k_pages.clone()
    x = torch.randn((100, 64), device="cuda").to(made.dtype)
    want.view(-1, 64)[made.rows(0, 0, 0)] = x[:40]
    want.view(-1, 64)[made.rows(0, 0, 1)] = x[40:80]
    kv.kv_paged_load(c, x, x, torch.tensor([0, 40, 80, 120], device="cuda"), 100)
    torch.cuda.synchronize()
    assert c.lens.view(-1).tolist() == [40, 40, -1]
    assert torch.equal(_bits(c.k_pages), _bits(want))
