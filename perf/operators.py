"""Measured cases of the paged-cache operators: rows written into pages, attention of new tokens over
the pages (sliding window and sinks, accumulated attention weights), eviction by accumulated weight.

A cache holds, for every unit u = (request, layer, KV head), lens[u] rows of K and V in pages of
page_size rows; row j of u is row j % page_size of page page_table[u][j // page_size].  Eviction
leaves every unit with a length of its own, so pages belong to units, not to requests.

``run`` computes one pass in elementary torch operations (``own`` false) or through the package's
entry points (``own`` true); ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

# (KV heads, query heads, head dim) of the shapes the benchmark's configurations use
TINY, LLAMA, QWEN = (1, 4, 64), (8, 32, 128), (4, 28, 128)


def _case(name, op, shape, **kw):
    case = {"name": name, "op": op, "kv_heads": shape[0], "q_heads": shape[1], "head_dim": shape[2],
            "requests": 1, "layers": 1, "page": 64, "dtype": "bf16"}
    case.update(kw)
    return case


def _attend(name, shape, **kw):
    base = {"t_lo": 1, "t_hi": 1, "window": 0, "sinks": 0, "mass": False}
    base.update(kw)
    return _case(name, "attend", shape, **base)


def listed():
    return [
        # one decode step's new K/V rows of 8 requests, read from a fused QKV projection's output:
        # the smallest call of the serving loop
        _case("append_decode_8", "append", LLAMA, requests=8, n_lo=1200, n_hi=2400, t_lo=1, t_hi=1),
        # a prefill compacted to 5% (1638 rows a head, 32 layers) handed over to the pages
        _case("load_llama", "load", LLAMA, layers=32, n_lo=1638, n_hi=1638),
        # decode over that cache: one request, one layer's call; latency counts
        _attend("decode_1638", LLAMA, n_lo=1638, n_hi=1638),
        # decode of the ragged batch's kept caches (30% of 16384..131072), every head its own length
        _attend("decode_ragged_8", LLAMA, requests=8, layers=2, page=32, n_lo=4915, n_hi=39321),
        # decode over an uncompressed long context, weights accumulated for a later eviction
        _attend("decode_mass_131072", QWEN, n_lo=131072, n_hi=131072, mass=True),
        # decode in a sliding-window layer with 4 sinks, long caches, a batch of 16
        _attend("decode_window_16", LLAMA, requests=16, n_lo=8193, n_hi=32768, window=4096, sinks=4),
        # a short follow-up turn over the tiny configuration, small pages, fp16
        _attend("chunk_tiny_16", TINY, page=16, dtype="fp16", n_lo=2048, n_hi=2048, t_lo=16, t_hi=16),
        # a chunk of a prompt over a long cache
        _attend("chunk_2048_over_65536", LLAMA, page=128, n_lo=67584, n_hi=67584, t_lo=2048,
                t_hi=2048),
        # a prompt chunk with weights accumulated, ragged over 2 requests
        _attend("chunk_mass_511", LLAMA, requests=2, n_lo=13107, n_hi=32768, t_lo=301, t_hi=511,
                mass=True),
        # a whole prompt in a sliding-window layer
        _attend("prompt_window_8192", LLAMA, n_lo=8192, n_hi=8192, t_lo=8192, t_hi=8192, window=4096,
                sinks=4),
        # steady state of decoding under a budget: a page's worth of new rows evicted, all layers
        _case("evict_step", "evict", LLAMA, layers=32, n_lo=1702, n_hi=1702, budget=1638, sinks=4,
              recent=64),
        # one large eviction after a long prompt, all layers, 131072 rows down to 5%
        _case("evict_prompt", "evict", QWEN, layers=28, n_lo=131072, n_hi=131072, budget=6553,
              sinks=4, recent=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "load", "attend", "attend", "attend", "attend", "evict"])
    shape = rng.choice([TINY, LLAMA, QWEN, (2, 8, 128), (3, 3, 64)])
    case = _case("", op, shape, page=rng.choice([16, 32, 64, 128]),
                 dtype=rng.choice(["bf16", "bf16", "fp16"]))
    del case["name"]
    if op == "append":
        case.update(requests=_log_int(rng, 1, 64), t_lo=1, t_hi=_log_int(rng, 1, 100), n_lo=100,
                    n_hi=_log_int(rng, 200, 4000))
    elif op == "load":
        n = _log_int(rng, 17, 4000)
        case.update(requests=rng.randint(1, 3), layers=rng.randint(1, 16), n_lo=n,
                    n_hi=n + rng.randint(0, n))
    elif op == "evict":
        n = _log_int(rng, 200, 40000)
        sinks, recent = rng.randint(0, 8), rng.randint(1, 64)
        case.update(requests=rng.randint(1, 2), layers=rng.randint(1, 16), n_lo=n,
                    n_hi=n + rng.randint(0, n // 4), sinks=sinks, recent=recent,
                    budget=rng.randint(sinks + recent, n))
    else:
        t = rng.choice([1, 1, 1, _log_int(rng, 2, 1500)])
        n = _log_int(rng, 1, 40000) + t
        # no more than 1.2e8 (token, row) pairs a head, and 300000 rows
        r = rng.randint(1, max(1, min(12, 80000000 // (t * n), 200000 // n)))
        case.update(requests=r, n_lo=n, n_hi=n + rng.randint(0, n // 2), t_lo=max(1, t // 2), t_hi=t,
                    window=rng.choice([0, 0, 0, _log_int(rng, 1, 5000)]), sinks=rng.randint(0, 8),
                    mass=rng.random() < 0.3)
    return case


# --------------------------------------------------------------------------
# shapes that follow from a case alone
# --------------------------------------------------------------------------
def _spread(lo, hi, count, phase):
    """`count` whole numbers in [lo, hi], the same for every seed (multiples of the golden ratio)."""
    return [lo + int((hi - lo + 1) * ((0.6180339887498949 * i + phase) % 1.0)) for i in range(count)]


def _units(case):
    return case["requests"] * case["layers"] * case["kv_heads"]


def _lens(case):
    return _spread(case["n_lo"], case["n_hi"], _units(case), 0.99)


def _counts(case):
    return _spread(case["t_lo"], case["t_hi"], case["requests"], 0.99)


def _layer_lens(case):
    """Lengths [request][head] of the layer that the call works on: the last."""
    R, L, H = case["requests"], case["layers"], case["kv_heads"]
    n = _lens(case)
    return [[n[(r * L + L - 1) * H + h] for h in range(H)] for r in range(R)]


def work(case):
    d, H, Hq = case["head_dim"], case["kv_heads"], case["q_heads"]
    row = 2 * d * 2                                    # one K and one V row
    if case["op"] == "append":
        return {"bytes": 2 * row * H * sum(_counts(case)), "flops": 0}
    if case["op"] == "load":
        return {"bytes": 2 * row * sum(_lens(case)) + 8 * (_units(case) + 1), "flops": 0}
    if case["op"] == "evict":
        kept = [min(n, case["budget"]) for n in _lens(case)]
        return {"bytes": 4 * sum(_lens(case)) + (2 * row + 4 + 4) * sum(kept), "flops": 0}
    tokens = sum(_counts(case))
    rows = pairs = 0
    for n_r, t in zip(_layer_lens(case), _counts(case)):
        for n in n_r:
            w, s = case["window"], case["sinks"]
            first = max(0, n - t)                      # cache row of the first query
            lo = max(0, first - w + 1) if w else 0
            rows += n - lo + min(s if w else 0, lo)
            for p in range(first, n):
                lo = max(0, p - w + 1) if w else 0
                pairs += p + 1 - lo + min(s if w else 0, lo)
    out = 2 * tokens * Hq * d * 2 + tokens * Hq * 4    # q, out, lse
    return {"bytes": rows * (row + (8 if case["mass"] else 0)) + out,
            "flops": 4 * d * pairs * (Hq // H)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _dtype(case):
    return torch.float16 if case["dtype"] == "fp16" else torch.bfloat16


def _fill(shape, dtype, gen):
    """Normal values with a few outlier channels, as keys and values of language models have."""
    x = torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)
    x[..., 5::32] *= 4
    return x


def _cache(case, gen, capacity, extra_pages=3):
    """Pools and a page table in an allocator's order, for units of up to `capacity` rows."""
    R, L, H, d, ps = (case[k] for k in ("requests", "layers", "kv_heads", "head_dim", "page"))
    cols = -(-capacity // ps)
    pages = R * L * H * cols + extra_pages
    perm = torch.randperm(pages, generator=gen, device="cuda")[:R * L * H * cols].to(torch.int32)
    return {"k": _fill((pages, ps, d), _dtype(case), gen), "v": _fill((pages, ps, d), _dtype(case), gen),
            "table": perm.view(R, L, H, cols).contiguous(),
            "lens": torch.tensor(_lens(case), dtype=torch.int32, device="cuda").view(R, L, H)}


def _paged(c, q_heads, mass=None):
    import kv_cache_eviction_split_gb300 as kv
    return kv.PagedCache(c["k"], c["v"], c["table"], c["lens"], q_heads, mass=mass)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    H, Hq, d = case["kv_heads"], case["q_heads"], case["head_dim"]
    st = {"case": case}
    cap = case["n_hi"] + case["page"] // 2             # tables are as long as a step may need
    if case["op"] == "evict":
        # a source cache with its accumulated weights, and pages that the kept rows go to
        st["src"] = _cache(case, gen, cap)
        pages, ps = st["src"]["k"].shape[:2]
        mass = torch.empty((pages, ps), device="cuda").exponential_(generator=gen)
        st["mass"] = torch.round(mass * 4096) / 4096   # ties among them
        cols = -(-min(case["budget"], case["n_hi"]) // ps)
        st["budgets"] = torch.full((_units(case),), case["budget"], dtype=torch.int32, device="cuda")
        new = _units(case) * cols
        st["dst"] = {"k": torch.zeros((new, ps, d), dtype=_dtype(case), device="cuda"),
                     "v": torch.zeros((new, ps, d), dtype=_dtype(case), device="cuda"),
                     "table": torch.randperm(new, generator=gen, device="cuda").to(torch.int32)
                     .view(case["requests"], case["layers"], H, cols),
                     "lens": torch.zeros_like(st["src"]["lens"])}
        st["dst_mass"] = torch.zeros((new, ps), device="cuda")
        st["kept"] = torch.full((_units(case), min(case["budget"], case["n_hi"])), -1,
                                dtype=torch.int32, device="cuda")
        if own:
            import kv_cache_eviction_split_gb300 as kv
            st["from"] = _paged(st["src"], Hq, st["mass"])
            st["to"] = _paged(st["dst"], Hq, st["dst_mass"])
            st["ws"] = torch.empty(kv.kv_paged_evict_workspace_size(st["from"]), dtype=torch.uint8,
                                   device="cuda")
        return st
    if case["op"] == "load":
        n = _lens(case)
        off = [0]
        for x in n:
            off.append(off[-1] + x)
        st["offsets"] = torch.tensor(off, dtype=torch.int64, device="cuda")
        st["total"] = off[-1]
        st["k_rows"], st["v_rows"] = (_fill((off[-1], d), _dtype(case), gen) for _ in range(2))
        st["cache"] = _cache(case, gen, cap)
        if own:
            st["paged"] = _paged(st["cache"], Hq)
        return st
    st["cache"] = _cache(case, gen, cap)
    counts = _counts(case)
    off = [0]
    for x in counts:
        off.append(off[-1] + x)
    st["off"] = torch.tensor(off, dtype=torch.int64, device="cuda")
    tokens = off[-1]
    # the projection's output: queries, keys and values of a token side by side
    qkv = _fill((tokens, (Hq + 2 * H) * d), _dtype(case), gen)
    st["q"] = qkv[:, :Hq * d].view(tokens, Hq, d)
    st["k_new"] = qkv[:, Hq * d:(Hq + H) * d].view(tokens, H, d)
    st["v_new"] = qkv[:, (Hq + H) * d:].view(tokens, H, d)
    if own:
        import kv_cache_eviction_split_gb300 as kv
        st["chunk"] = kv.Chunk(counts, device="cuda")
    if case["op"] == "append":
        if own:
            st["paged"] = _paged(st["cache"], Hq)
        return st
    st["out"] = torch.empty((tokens, Hq, d), dtype=_dtype(case), device="cuda")
    st["lse"] = torch.empty((tokens, Hq), device="cuda")
    if case["mass"]:
        st["mass0"] = torch.empty(st["cache"]["k"].shape[:2], device="cuda").exponential_(generator=gen)
        st["mass"] = st["mass0"].clone()
    if own:
        st["paged"] = _paged(st["cache"], Hq, st.get("mass"))
        st["ws"] = torch.empty(
            kv.kv_paged_attention_workspace_size(st["paged"], st["chunk"], add_mass=case["mass"]),
            dtype=torch.uint8, device="cuda")
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    return {"append": _append, "load": _load, "attend": _attention, "evict": _evict}[st["case"]["op"]](st)


def _slots(table, ps, j):
    """Pool rows of cache rows j [..., n] of the units whose tables are table [..., cols]."""
    return torch.gather(table.long(), -1, j // ps) * ps + j % ps


def _append(st):
    case, c = st["case"], st["cache"]
    layer = case["layers"] - 1
    if own:
        import kv_cache_eviction_split_gb300 as kv
        kv.kv_paged_append(st["paged"], st["chunk"], layer, st["k_new"], st["v_new"])
        return [c["k"], c["v"]]
    ps, d, H = case["page"], case["head_dim"], case["kv_heads"]
    tok = torch.arange(st["q"].shape[0], device="cuda")
    req = torch.searchsorted(st["off"], tok, right=True) - 1
    # a request's new rows are the last of its units' rows
    j = c["lens"][:, layer].long()[req] - (st["off"][req + 1] - tok)[:, None]       # [tokens, H]
    rows = _slots(c["table"][:, layer][req], ps, j[..., None])[..., 0]
    c["k"].view(-1, d)[rows] = st["k_new"]
    c["v"].view(-1, d)[rows] = st["v_new"]
    return [c["k"], c["v"]]


def _load(st):
    case, c = st["case"], st["cache"]
    if own:
        import kv_cache_eviction_split_gb300 as kv
        kv.kv_paged_load(st["paged"], st["k_rows"], st["v_rows"], st["offsets"], st["total"])
        return [c["k"], c["v"], c["lens"]]
    ps, d = case["page"], case["head_dim"]
    row = torch.arange(st["total"], device="cuda")
    unit = torch.searchsorted(st["offsets"], row, right=True) - 1
    j = row - st["offsets"][unit]
    rows = c["table"].view(_units(case), -1)[unit, j // ps].long() * ps + j % ps
    c["k"].view(-1, d)[rows] = st["k_rows"]
    c["v"].view(-1, d)[rows] = st["v_rows"]
    c["lens"].copy_((st["offsets"][1:] - st["offsets"][:-1]).view_as(c["lens"]))
    return [c["k"], c["v"], c["lens"]]


def _attention(st):
    case, c = st["case"], st["cache"]
    layer = case["layers"] - 1
    if case["mass"]:
        st["mass"].copy_(st["mass0"])                  # the weights of the steps before this one
    if own:
        import kv_cache_eviction_split_gb300 as kv
        kv.kv_paged_attention(st["paged"], st["chunk"], layer, st["q"], st["out"], st["ws"],
                              window=case["window"], num_sinks=case["sinks"], lse=st["lse"],
                              add_mass=case["mass"])
        return [st["out"], st["lse"]] + ([st["mass"]] if case["mass"] else [])
    R, H, Hq, d, ps = (case[k] for k in ("requests", "kv_heads", "q_heads", "head_dim", "page"))
    G, T = Hq // H, case["t_hi"]
    n = c["lens"][:, layer].long()                                                    # [R, H]
    count = st["off"][1:] - st["off"][:-1]
    # queries padded to T a request: [R, H, T, G, d]
    i = torch.arange(T, device="cuda")
    tok = torch.minimum(st["off"][:-1, None] + i, st["off"][1:, None] - 1)
    q = st["q"][tok].float().view(R, T, H, G, d).permute(0, 2, 1, 3, 4)
    t = (n[:, :, None] - count[:, None, None] + i)[..., None]                         # [R, H, T, 1]
    j = torch.arange(case["n_hi"], device="cuda")
    held = j < n[..., None]
    rows = _slots(c["table"][:, layer], ps, j.expand(R, H, -1))
    K = c["k"].view(-1, d)[rows].float()
    V = torch.where(held[..., None], c["v"].view(-1, d)[rows].float(), 0.0)
    seen = (j <= t) & held[:, :, None]                                                # [R, H, T, n]
    if case["window"]:
        seen &= (j > t - case["window"]) | (j < case["sinks"])
    x = torch.matmul(q.reshape(R, H, T * G, d), K.transpose(-1, -2)).view(R, H, T, G, -1)
    x.mul_(1.0 / math.sqrt(d)).masked_fill_(~seen[:, :, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True).clamp_min(-1e30)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    x.div_(torch.where(total > 0, total, 1.0))
    o = torch.matmul(x.view(R, H, T * G, -1), V).view(R, H, T, G, d)
    lse = (top + torch.log(total))[..., 0]
    real = i < count[:, None]                                                         # [R, T]
    st["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(R, T, Hq, d)[real])
    st["lse"].copy_(lse.permute(0, 2, 1, 3).reshape(R, T, Hq)[real])
    if not case["mass"]:
        return [st["out"], st["lse"]]
    x.mul_(real[:, None, :, None, None])
    st["mass"].view(-1)[rows[held]] += x.sum((2, 3))[held]
    return [st["out"], st["lse"], st["mass"]]


def _evict(st):
    case, src, dst = st["case"], st["src"], st["dst"]
    out = [dst["k"], dst["v"], st["dst_mass"], dst["lens"], st["kept"]]
    if own:
        import kv_cache_eviction_split_gb300 as kv
        kv.kv_paged_evict(st["from"], st["to"], st["budgets"], case["sinks"], case["recent"], st["kept"],
                          st["ws"])
        return out
    ps, d, U, N = case["page"], case["head_dim"], _units(case), case["n_hi"]
    n = src["lens"].view(U, 1).long()
    b = torch.minimum(st["budgets"].view(U, 1).long(), n)
    j = torch.arange(N, device="cuda").expand(U, N)
    rows = _slots(src["table"].view(U, -1), ps, j)
    mass = st["mass"].view(-1)[rows]
    # first rows and recent rows before everything else, rows beyond the length after it
    pinned = (j < case["sinks"]) | (j >= n - case["recent"])
    rank = torch.where(pinned, float("inf"), mass).masked_fill_(j >= n, float("-inf"))
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices
    take = torch.arange(st["kept"].shape[1], device="cuda") < b                       # [U, kept]
    kept = torch.where(take, order[:, :take.shape[1]], N).sort(1).values
    st["kept"][take] = kept[take].int()
    at = kept.clamp(max=N - 1)
    i = torch.arange(take.shape[1], device="cuda").expand(U, -1)
    to = _slots(dst["table"].view(U, -1), ps, i)[take]
    frm = torch.gather(rows, 1, at)[take]
    dst["k"].view(-1, d)[to] = src["k"].view(-1, d)[frm]
    dst["v"].view(-1, d)[to] = src["v"].view(-1, d)[frm]
    st["dst_mass"].view(-1)[to] = st["mass"].view(-1)[frm]
    dst["lens"].copy_(b.view_as(dst["lens"]))
    return out


# --------------------------------------------------------------------------
# the same outputs from the definitions, in 64 bits, unit by unit
# --------------------------------------------------------------------------
def _rows_of(cache, ps, r, l, h, n):
    """Pool rows of the first n rows of unit (r, l, h)."""
    pages = cache["table"][r, l, h].long()
    return (pages[:, None] * ps + torch.arange(ps, device=pages.device)).reshape(-1)[:n]


def exact(case, seed):
    st = prepare(case, seed)
    R, L, H, Hq, d, ps = (case[k] for k in ("requests", "layers", "kv_heads", "q_heads", "head_dim",
                                            "page"))
    lens = _lens(case)
    units = [(r, l, h) for r in range(R) for l in range(L) for h in range(H)]
    if case["op"] in ("append", "load"):
        k, v = (st["cache"][x].double().view(-1, d) for x in "kv")
        a = 0
        for u, (r, l, h) in enumerate(units):
            rows = _rows_of(st["cache"], ps, r, l, h, lens[u])
            if case["op"] == "load":
                k[rows], v[rows] = (st[x][a:a + lens[u]].double() for x in ("k_rows", "v_rows"))
                a += lens[u]
            elif l == L - 1:
                t0, t1 = int(st["off"][r]), int(st["off"][r + 1])
                new = rows[lens[u] - (t1 - t0):]
                k[new], v[new] = (st[x][t0:t1, h].double() for x in ("k_new", "v_new"))
        pools = [k.view(-1, ps, d), v.view(-1, ps, d)]
        return pools + ([None] if case["op"] == "load" else [])
    if case["op"] == "evict":
        k, v = (st["dst"][x].double().view(-1, d) for x in "kv")
        mass = st["dst_mass"].double().view(-1)
        for u, (r, l, h) in enumerate(units):
            n, b = lens[u], min(lens[u], case["budget"])
            rows = _rows_of(st["src"], ps, r, l, h, n)
            w = st["mass"].view(-1)[rows].double()
            keep = torch.zeros(n, dtype=torch.bool, device=w.device)
            if n <= case["budget"]:
                keep[:] = True
            else:
                keep[:case["sinks"]] = True
                keep[n - case["recent"]:] = True
                mid = torch.arange(case["sinks"], n - case["recent"], device=w.device)
                more = b - case["sinks"] - case["recent"]
                # a weight's rank: how many are above it, and at lower indices equal to it
                least = torch.sort(w[mid]).values[mid.numel() - more] if more else math.inf
                above = w[mid] > least
                equal = w[mid] == least
                room = more - above.sum()
                keep[mid] = above | (equal & (torch.cumsum(equal, 0) <= room))
            frm, to = rows[keep], _rows_of(st["dst"], ps, r, l, h, b)
            k[to], v[to] = (st["src"][x].view(-1, d)[frm].double() for x in "kv")
            mass[to] = st["mass"].view(-1)[frm].double()
        return [k.view_as(st["dst"]["k"]), v.view_as(st["dst"]["v"]), mass.view_as(st["dst_mass"]), None,
                None]
    if work(case)["flops"] > 5e12:
        return None
    G = Hq // H
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    mass = st["mass0"].double().view(-1) if case["mass"] else None
    for u, (r, l, h) in enumerate(units):
        if l != L - 1:
            continue
        n, t0, t1 = lens[u], int(st["off"][r]), int(st["off"][r + 1])
        rows = _rows_of(st["cache"], ps, r, l, h, n)
        K, V = (st["cache"][x].view(-1, d)[rows].double() for x in "kv")
        pos = torch.arange(n - (t1 - t0), n, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")[None]
        hidden = key > pos
        if case["window"]:
            hidden |= (key <= pos - case["window"]) & (key >= case["sinks"])
        for g in range(G):
            s = st["q"][t0:t1, h * G + g].double() @ K.T / math.sqrt(d)
            s[hidden] = -math.inf
            z = torch.logsumexp(s, 1)
            p = torch.exp(s - z[:, None])
            out[t0:t1, h * G + g] = p @ V
            lse[t0:t1, h * G + g] = z
            if mass is not None:
                mass[rows] += p.sum(0)
    return [out, lse] + ([mass.view_as(st["mass0"])] if case["mass"] else [])
