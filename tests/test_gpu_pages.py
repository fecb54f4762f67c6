"""Pages given out, shared, copied before they are written and moved together, against the same rules
in plain Python; and a run of them with appends and attention."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


class Model:
    """A cache with counted pages, and the operators' rules on host lists."""

    def __init__(self, kv, R, L, H, d, page, cols, pages, lens, dtype="bf16", seed=0, shared=False):
        import torch
        from tests import paged
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = paged.DTYPES[dtype]
        self.R, self.U, self.per, self.ps, self.cols = R, R * L * H, L * H, page, cols
        rng = np.random.default_rng(seed)
        lens = np.asarray(lens, dtype=np.int64).reshape(self.U)
        table = rng.integers(-5, 2 ** 31 - 1, (self.U, cols))
        free = rng.permutation(pages).tolist()
        refs = [0] * pages
        for u, n in enumerate(lens.tolist()):
            for c in range(-(-n // page)):
                table[u, c] = free.pop()
                refs[table[u, c]] = 1
        self.table, self.lens, self.refs = table.tolist(), lens.tolist(), refs
        k, v = (torch.randn((pages, page, d), generator=g, device="cuda").to(dt) for _ in range(2))
        mass = torch.rand((pages, page), generator=g, device="cuda")
        pos = torch.randint(0, 1 << 20, (pages, page), generator=g, device="cuda").int()
        # what each page held at the start
        self.from_page = list(range(pages))
        self.start = [t.clone() for t in (k, v, mass, pos)]
        self.kv = kv
        self.cache = kv.PagedCache(k, v, torch.tensor(table, dtype=torch.int32, device="cuda").view(R, L, H, cols),
                                   torch.tensor(lens, dtype=torch.int32, device="cuda").view(R, L, H), H, mass=mass,
                                   positions=pos, refs=torch.tensor(refs, dtype=torch.int32, device="cuda"))

    def held(self, u):
        return -(-self.lens[u] // self.ps)

    def fork(self, parents):
        table, lens = [list(x) for x in self.table], list(self.lens)
        held = [self.held(u) for u in range(self.U)]
        for r, p in enumerate(parents):
            if p == r:
                continue
            for i in range(self.per):
                u, w = r * self.per + i, p * self.per + i
                for c in range(held[u]):
                    self.refs[table[u][c]] -= 1
                self.lens[u] = lens[w] if p >= 0 else 0
                for c in range(held[w] if p >= 0 else 0):
                    self.table[u][c] = table[w][c]
                    self.refs[table[w][c]] += 1

    def reserve(self, counts):
        """False, and no change, if it does not fit."""
        free = [p for p, n in enumerate(self.refs) if n == 0]
        need, copies = [], []
        for u in range(self.U):
            n, t = self.lens[u], counts[u // self.per]
            copy = t > 0 and n % self.ps > 0 and self.refs[self.table[u][self.held(u) - 1]] > 1
            copies.append(copy)
            need.append(-(-(n + t) // self.ps) - self.held(u) + copy)
            if n + t > self.cols * self.ps:
                return False
        if sum(need) > len(free):
            return False
        at = iter(free)
        for u in range(self.U):
            n, t, h = self.lens[u], counts[u // self.per], self.held(u)
            if copies[u]:
                old, new = self.table[u][h - 1], next(at)
                self.table[u][h - 1] = new
                self.refs[old] -= 1
                self.refs[new] = 1
                self.from_page[new] = self.from_page[old]
            for c in range(h, -(-(n + t) // self.ps)):
                self.table[u][c] = next(at)
                self.refs[self.table[u][c]] = 1
            self.lens[u] = n + t
        return True

    def compact(self):
        live = sum(n > 0 for n in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        far = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(far, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.from_page[b] = self.from_page[a]
        for u in range(self.U):
            for c in range(self.held(u)):
                self.table[u][c] = to.get(self.table[u][c], self.table[u][c])
        return live

    def check(self, status=0):
        import torch
        c = self.cache
        assert self.kv.kv_check_status(c.status) == status
        assert c.lens.view(-1).tolist() == self.lens
        assert c.refs.tolist() == self.refs
        assert c.page_table.view(self.U, -1).tolist() == self.table
        came = torch.tensor(self.from_page, device="cuda")
        for t, old in zip((c.k_pages, c.v_pages, c.mass, c.positions), self.start):
            assert torch.equal(t, old[came])
        # counted anew, the pages have as many references
        self.kv.kv_paged_count_refs(c)
        assert c.refs.tolist() == self.refs


# (requests, layers, heads, d, page, columns, free pages, shortest, longest, dtype)
SHAPES = {
    "one": (1, 1, 1, 64, 16, 4, 3, 5, 5, "bf16"),
    "empty": (2, 1, 2, 64, 16, 4, 20, 0, 0, "fp16"),
    "small": (3, 2, 2, 64, 16, 20, 300, 0, 150, "fp16"),
    "page_ends": (4, 1, 2, 128, 32, 9, 90, 64, 64, "bf16"),
    "wide": (5, 3, 4, 128, 64, 40, 700, 1, 1200, "bf16"),
    "page128": (2, 2, 3, 128, 128, 6, 60, 100, 400, "fp16"),
    "many_requests": (130, 1, 1, 64, 16, 6, 500, 0, 40, "bf16"),
    "many_units": (40, 32, 8, 64, 16, 3, 9000, 1, 20, "bf16"),
    "many_pages": (2, 1, 1, 64, 16, 40, 300011, 300, 400, "bf16"),
}


def _model(kv, name, seed=0):
    R, L, H, d, page, cols, free, lo, hi, dtype = SHAPES[name]
    rng = np.random.default_rng(seed + len(name))
    lens = rng.integers(lo, hi + 1, R * L * H)
    held = int(sum(-(-int(n) // page) for n in lens))
    return Model(kv, R, L, H, d, page, cols, held + free, lens, dtype, seed)


def _reserve(m, counts):
    import torch
    kv = m.kv
    ws = torch.full((kv.kv_paged_reserve_workspace_size(m.cache),), 0xFF, dtype=torch.uint8, device="cuda")
    kv.kv_paged_reserve(m.cache, kv.Chunk(counts), ws)


def _fork(m, parents):
    import torch
    m.kv.kv_paged_fork(m.cache, torch.tensor(parents, dtype=torch.int32, device="cuda"))


def _compact(m):
    import torch
    kv = m.kv
    ws = torch.full((kv.kv_paged_compact_workspace_size(m.cache),), 0xFF, dtype=torch.uint8, device="cuda")
    live = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    kv.kv_paged_compact(m.cache, ws, live=live)
    return live


@pytest.mark.parametrize("name", SHAPES)
def test_reserve_enters_the_lowest_free_pages(cuda_lib, name):
    m = _model(cuda_lib, name)
    room = m.cols * m.ps - max(m.lens)
    for t in (1, 0, 5, 17):
        counts = [min(t + r % 3 if t else r % 2, room // 4) for r in range(m.R)]
        fits = m.reserve(counts)
        _reserve(m, counts)
        m.check(0 if fits else cuda_lib.KV_ERR_BUDGET)


@pytest.mark.parametrize("name", SHAPES)
def test_forks_share_and_reserve_copies(cuda_lib, name):
    m = _model(cuda_lib, name, 1)
    rng = np.random.default_rng(7)
    for step in range(3):
        parents = rng.integers(-1, m.R, m.R).tolist() if step else [0] * m.R
        m.fork(parents)
        _fork(m, parents)
        m.check()
        room = m.cols * m.ps - max(m.lens)
        counts = [min(1 + step, room) if r % 4 != 3 else 0 for r in range(m.R)]
        fits = m.reserve(counts)
        _reserve(m, counts)
        m.check(0 if fits else cuda_lib.KV_ERR_BUDGET)


@pytest.mark.parametrize("parents", [[0, 1, 2, 3], [3, 2, 1, 0], [1, 2, 3, 0], [-1, -1, -1, -1], [2, 2, 2, 2],
                                     [1, -1, 1, 0]])
def test_fork_takes_the_tables_before_the_call(cuda_lib, parents):
    m = Model(cuda_lib, 4, 2, 2, 64, 16, 700, 9000, np.arange(16) * 500 + 3)
    m.fork(parents)
    _fork(m, parents)
    m.check()


@pytest.mark.parametrize("name", SHAPES)
def test_compaction_moves_the_last_pages_forward(cuda_lib, name):
    m = _model(cuda_lib, name, 2)
    # shared pages, and requests that are gone
    for parents in ([r // 2 for r in range(m.R)], [r if r % 3 else -1 for r in range(m.R)]):
        m.fork(parents)
        _fork(m, parents)
    live = m.compact()
    got = _compact(m)
    m.check()
    assert int(got) == live
    assert all(n > 0 for n in m.refs[:live]) and not any(m.refs[live:])
    # nothing to move
    assert int(_compact(m)) == live
    m.check()
    if live < len(m.refs) - 200:
        fits = m.reserve([1] * m.R)
        _reserve(m, [1] * m.R)
        m.check(0 if fits else cuda_lib.KV_ERR_BUDGET)


def test_a_full_pool_has_nothing_to_move(cuda_lib):
    m = Model(cuda_lib, 1, 1, 2, 64, 16, 9, 10, [80, 80])
    assert m.compact() == 10 and int(_compact(m)) == 10
    m.check()


def test_reserve_changes_nothing_unless_all_fit(cuda_lib):
    kv = cuda_lib
    # two pages short; then a unit that would outgrow its table; then just enough
    m = Model(kv, 3, 1, 2, 64, 16, 5, 6 * 2 + 4, [16, 17, 20, 32, 31, 17], seed=3)
    assert not m.reserve([1, 60, 0])
    _reserve(m, [1, 60, 0])
    m.check(kv.KV_ERR_BUDGET)
    assert not m.reserve([1, 0, 64])
    _reserve(m, [1, 0, 64])
    m.check(kv.KV_ERR_BUDGET)
    assert m.reserve([17, 1, 2])
    _reserve(m, [17, 1, 2])
    m.check()
    with pytest.raises(kv.KvError) as e:
        _reserve(m, [1 << 20, 0, 0])
    assert e.value.code == kv.KV_ERR_BUDGET
    m.check()


def test_lengths_and_pages_that_cannot_be_are_reported(cuda_lib):
    import torch
    kv = cuda_lib

    def fresh():
        return Model(kv, 2, 1, 2, 64, 16, 6, 40, [20, 33, 17, 50], seed=4)

    for break_it in (lambda c: c.lens.view(-1)[1].fill_(-1), lambda c: c.lens.view(-1)[1].fill_(97),
                     lambda c: c.page_table.view(4, -1)[1, 2].fill_(40)):
        m = fresh()
        break_it(m.cache)
        before = [t.clone() for t in (m.cache.lens, m.cache.page_table, m.cache.refs)]
        _reserve(m, [1, 1])
        assert kv.kv_check_status(m.cache.status) == kv.KV_ERR_INVALID_ARG
        for a, b in zip((m.cache.lens, m.cache.page_table, m.cache.refs), before):
            assert torch.equal(a, b)
        for call in (lambda: _fork(m, [0, 0]), lambda: kv.kv_paged_count_refs(m.cache)):
            call()
            assert kv.kv_check_status(m.cache.status) == kv.KV_ERR_INVALID_ARG
    # parents that are none: those requests stay
    for bad in (2, -2, 2 ** 31 - 1):
        m = fresh()
        _fork(m, [1, bad])
        m.fork([1, 1])
        m.check(kv.KV_ERR_INVALID_ARG)
    # a table that names a page without references
    m = fresh()
    far = max(p for p, n in enumerate(m.refs) if n)
    m.cache.refs[far] = 0
    _compact(m)
    used = sum(n > 0 for n in m.refs) - 1
    assert kv.kv_check_status(m.cache.status) == (kv.KV_ERR_INVALID_ARG if far >= used else 0)


def test_no_requests_and_no_tokens(cuda_lib):
    import torch
    kv = cuda_lib
    m = Model(kv, 2, 1, 2, 64, 16, 6, 40, [20, 33, 17, 50], seed=4)
    _reserve(m, [0, 0])
    m.check()
    c = kv.PagedCache.allocate(0, 1, 2, 2, 64, 10, refs=True)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    kv.kv_paged_fork(c, torch.empty(0, dtype=torch.int32, device="cuda"))
    kv.kv_paged_reserve(c, kv.Chunk([]), ws)
    kv.kv_paged_compact(c, ws)


def test_captured_steps_follow_the_cache(cuda_lib):
    """Fork, reserve and compact in one graph, replayed over a cache that each replay changes."""
    import torch
    kv = cuda_lib
    m = _model(kv, "wide", 5)
    chunk = kv.Chunk([1, 2, 0, 3, 1])
    parents = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device="cuda")
    sizes = [f(m.cache) for f in (kv.kv_paged_reserve_workspace_size, kv.kv_paged_compact_workspace_size)]
    ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        kv.kv_paged_fork(m.cache, parents)
        kv.kv_paged_reserve(m.cache, chunk, ws)
        kv.kv_paged_compact(m.cache, ws, live=live)
    for p in ([0, 1, 2, 3, 4], [0, 0, 2, 2, -1], [4, 3, 2, 1, 0], [1, 1, 1, 1, 1]):
        parents.copy_(torch.tensor(p, dtype=torch.int32))
        g.replay()
        m.fork(p)
        assert m.reserve([1, 2, 0, 3, 1])
        assert m.compact() == int(live)
        m.check()


def test_two_streams_at_once(cuda_lib):
    import torch
    kv = cuda_lib
    sets = [(_model(kv, "wide", 10 + i), torch.cuda.Stream()) for i in range(3)]
    chunk = kv.Chunk([2] * 5)
    parents = torch.tensor([0, 0, 0, 3, -1], dtype=torch.int32, device="cuda")
    spaces = [torch.empty(kv.kv_paged_reserve_workspace_size(m.cache), dtype=torch.uint8, device="cuda")
              for m, _ in sets]
    torch.cuda.synchronize()
    for (m, s), ws in zip(sets, spaces):
        kv.kv_paged_fork(m.cache, parents, stream=s)
        kv.kv_paged_reserve(m.cache, chunk, ws, stream=s)
    torch.cuda.synchronize()
    for m, _ in sets:
        m.fork([0, 0, 0, 3, -1])
        assert m.reserve([2] * 5)
        m.check()
