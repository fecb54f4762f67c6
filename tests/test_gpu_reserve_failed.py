"""Steps whose reservation failed: what is queued behind it leaves the cache as it was."""
import pytest

pytestmark = pytest.mark.gpu


def _model(kv, free=9, seed=3):
    """Three requests on the first one's 16 pages, of which the last four are part full, and `free` others."""
    from tests.test_gpu_pages import Model, _fork
    m = Model(kv, 3, 2, 2, 64, 16, 12, 4 * 4 + free, [50] * 4 + [0] * 8, seed=seed)
    m.fork([0, 0, 0])
    _fork(m, [0, 0, 0])
    m.check()
    return m


def _step(m, counts, ws, seed=0):
    """What a step queues: pages, rows in both ways, attention that adds weights."""
    import torch
    kv, c = m.kv, m.cache
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(counts)
    chunk = kv.Chunk(counts)
    rot = kv.Rotary.make(64)
    rows = [torch.randn((n, 2, 64), generator=g, device="cuda").bfloat16() for _ in range(3)]
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    kv.kv_paged_reserve(c, chunk, ws)
    kv.kv_paged_append(c, chunk, 0, rows[1], rows[2])
    kv.kv_paged_append_rotary(c, chunk, 1, rot, pos, rows[0], rows[0], rows[1], rows[2])
    for layer in range(2):
        out = torch.empty_like(rows[0])
        aw = torch.empty(kv.kv_paged_attention_workspace_size(c, chunk, True), dtype=torch.uint8, device="cuda")
        kv.kv_paged_attention(c, chunk, layer, rows[0], out, aw, add_mass=True)
        if max(counts) <= 16:
            kv.kv_paged_attention_scored(c, chunk, layer, rows[0], out, aw.new_empty(
                kv.kv_paged_attention_scored_workspace_size(c, chunk, True)), softcap=9.0, add_mass=True)
    return rows


@pytest.fixture
def ws(cuda_lib):
    import torch
    return torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda")


def _same(m, rows):
    """The appended rows are the last of every unit (k of layer 0 as it came, v of both)."""
    import torch
    c, t0 = m.cache, 0
    for r, count in enumerate(rows[0]):
        for l in range(2):
            for h in range(2):
                u = (r * 2 + l) * 2 + h
                for i in range(count):
                    j = m.lens[u] - count + i
                    at = m.table[u][j // 16], j % 16
                    assert torch.equal(c.v_pages[at], rows[1][2][t0 + i, h])
                    assert l or torch.equal(c.k_pages[at], rows[1][1][t0 + i, h])
                    assert not l or int(c.positions[at]) == t0 + i
        t0 += count


@pytest.mark.parametrize("counts", [[20, 20, 20], [4, 60, 0], [143, 0, 0]])
def test_a_step_without_pages_changes_nothing(cuda_lib, ws, counts):
    kv = cuda_lib
    m = _model(kv, 30 if counts[0] == 143 else 9)  # pages enough, a table too short
    assert not m.reserve(counts)
    _step(m, counts, ws)
    m.check(kv.KV_ERR_BUDGET)                     # rows, weights, positions, lengths, tables, counts
    # given pages, the step runs
    from tests.test_gpu_pages import _fork
    m.fork([0, -1, -1])
    _fork(m, [0, -1, -1])
    assert m.reserve([3, 0, 0])
    rows = _step(m, [3, 0, 0], ws)
    assert kv.kv_check_status(m.cache.status) == 0
    _same(m, ([3, 0, 0], rows))


def test_the_next_reservation_that_fits_ends_it(cuda_lib, ws):
    """Without the status being read: it keeps the first condition."""
    kv = cuda_lib
    m = _model(kv)
    _step(m, [20, 20, 20], ws)
    assert m.reserve([2, 1, 0])
    rows = _step(m, [2, 1, 0], ws)
    assert kv.kv_check_status(m.cache.status) == kv.KV_ERR_BUDGET
    _same(m, ([2, 1, 0], rows))
    assert kv.kv_check_status(m.cache.status) == 0


def test_a_length_that_cannot_be_stops_the_step(cuda_lib, ws):
    import torch
    kv = cuda_lib
    m = _model(kv)
    m.cache.lens.view(-1)[5] = -3
    tensors = [getattr(m.cache, x) for x in ("k_pages", "v_pages", "mass", "positions", "lens", "refs", "page_table")]
    before = [t.clone() for t in tensors]
    _step(m, [1, 2, 1], ws)
    assert kv.kv_check_status(m.cache.status) == kv.KV_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(tensors, before))


def test_an_earlier_condition_does_not_hide_it(cuda_lib, ws):
    """The status word keeps the first code; the step is stopped all the same."""
    import torch
    kv = cuda_lib
    m = _model(kv)
    kv.kv_paged_fork(m.cache, torch.tensor([0, 1, 7], dtype=torch.int32, device="cuda"))
    _step(m, [20, 20, 20], ws)
    m.check(kv.KV_ERR_INVALID_ARG)


def test_weights_of_a_long_chunk(cuda_lib, ws):
    """More query rows a head than the few-rows kernels take."""
    kv = cuda_lib
    m = _model(kv)
    assert not m.reserve([0, 80, 0])
    _step(m, [0, 80, 0], ws)
    m.check(kv.KV_ERR_BUDGET)


def test_a_captured_step(cuda_lib, ws):
    import torch
    kv = cuda_lib
    m = _model(kv, 30)
    c, counts = m.cache, [5, 5, 5]
    chunk = kv.Chunk(counts)
    rows = torch.randn((15, 2, 64), device="cuda").bfloat16()
    pos = torch.arange(15, dtype=torch.int32, device="cuda")
    rot = kv.Rotary.make(64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        kv.kv_paged_reserve(c, chunk, ws)
        for layer in range(2):
            kv.kv_paged_append_rotary(c, chunk, layer, rot, pos, None, None, rows, rows)
    steps = 0
    while m.reserve(counts):
        g.replay()
        steps += 1
    assert steps > 1
    torch.cuda.synchronize()
    before = [t.clone() for t in (c.k_pages, c.v_pages, c.mass, c.positions)]
    for _ in range(3):
        rows.normal_()
        g.replay()
    assert kv.kv_check_status(c.status) == kv.KV_ERR_BUDGET
    for t, old in zip((c.k_pages, c.v_pages, c.mass, c.positions), before):
        assert torch.equal(t, old)
    assert c.lens.view(-1).tolist() == m.lens
