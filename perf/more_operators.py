"""Measured cases of three more groups of paged-cache operators:

  rotary   rotary positions: new tokens' queries and keys turned, keys and values written into pages
           (kv_paged_append_rotary), and any rows turned forward or backward (kv_rotary)
  attend   attention over the pages with changed scores (kv_paged_attention_scored): capped by a tanh,
           lowered by distance, masked by positions (documents, prefixes, reach)
  beam     requests that go on from others' caches and get pages for their next tokens
           (kv_paged_fork, kv_paged_reserve): shared pages, copied before they are written
  compact  pages in use moved to the front of the pools (kv_paged_compact)

A cache holds, for every unit u = (request, layer, KV head), lens[u] rows of K and V in pages of
page_size rows; row j of u is row j % page_size of page table[u][j // page_size].  A row's position is
kept beside it (an eviction leaves gaps), or is its number j where a cache keeps none.  refs[p] counts
the table entries in use that name page p; 0 is a free page.

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
    base = {"t_lo": 1, "t_hi": 1, "cap": 0.0, "slopes": False, "gaps": 0, "docs": 0, "reach": 0, "prefix": 0,
            "sinks": 0}
    base.update(kw)
    return _case(name, "attend", shape, **base)


def listed():
    return [
        # one decode step's new rows of 8 requests whose caches were cut to 5%: rows far from their
        # positions; the smallest call of the serving loop
        _case("rotary_append_decode_8", "append", LLAMA, requests=8, n_lo=1200, n_hi=2400, t_lo=1, t_hi=1,
              gaps=20, dims=128, interleaved=False, scaling="none"),
        # a prompt's rows, frequencies scaled by parts for a long context
        _case("rotary_append_prompt_8192", "append", LLAMA, n_lo=8192, n_hi=8192, t_lo=8192, t_hi=8192, gaps=0,
              dims=128, interleaved=False, scaling="parts"),
        # the queries' gradient of a chunk, half of the head turned, neighbours paired, positions
        # deep in a long context
        _case("rotary_back_2047", "rotate", QWEN, dtype="fp16", tokens=2047, first=900000, dims=64,
              interleaved=True, scaling="linear"),
        # decode over a kept cache (5% of 32768), capped scores; latency counts
        _attend("decode_cap_1638", LLAMA, n_lo=1638, n_hi=1638, cap=30.0),
        # decode of a ragged batch's kept caches, scores lowered by the distance of positions, which
        # the eviction left with gaps
        _attend("decode_slopes_ragged_8", LLAMA, requests=8, layers=2, page=32, n_lo=4915, n_hi=39321,
                slopes=True, gaps=3),
        # a packed prompt of several documents, capped scores: a token sees its own document
        _attend("prompt_docs_8192", LLAMA, n_lo=8192, n_hi=8192, t_lo=8192, t_hi=8192, docs=5, cap=50.0),
        # a chunk of a prompt over a long cache, scores lowered by distance, a kept cache's positions
        _attend("chunk_slopes_2048_over_32768", LLAMA, page=128, n_lo=34816, n_hi=34816, t_lo=2048, t_hi=2048,
                slopes=True, gaps=2),
        # a short prompt whose first tokens see one another both ways, over the tiny configuration
        _attend("prefix_tiny_300", TINY, requests=2, page=16, dtype="fp16", n_lo=401, n_hi=401, t_lo=233,
                t_hi=300, prefix=180, cap=20.0, slopes=True),
        # 8 hypotheses of a beam go on from 3 of them; the next token's page is shared and copied
        _case("beam_step_8", "beam", LLAMA, requests=8, layers=32, n_lo=1638, n_hi=1700, t_lo=1, t_hi=1,
              parents=3, freed=0),
        # a short draft of tokens for hypotheses over the tiny configuration, some of them given up
        _case("beam_tiny_5", "beam", TINY, requests=5, layers=2, page=16, n_lo=200, n_hi=333, t_lo=3, t_hi=21,
              parents=2, freed=1),
        # a pool from which requests of a batch have gone, all layers
        _case("compact_batch", "compact", LLAMA, requests=10, layers=32, n_lo=1638, n_hi=3276, used=0.6),
        # a small pool with a few holes
        _case("compact_tiny", "compact", TINY, requests=3, layers=2, page=16, dtype="fp16", n_lo=100, n_hi=900,
              used=0.8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "rotate", "attend", "attend", "attend", "attend", "beam", "compact"])
    shape = rng.choice([TINY, LLAMA, QWEN, (2, 8, 128), (3, 3, 64)])
    case = _case("", op, shape, page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "bf16", "fp16"]))
    del case["name"]
    if op in ("append", "rotate"):
        case.update(dims=16 * rng.randint(1, shape[2] // 16), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "base", "parts"]))
    if op == "append":
        t = _log_int(rng, 1, 2000)
        n = t + _log_int(rng, 1, 4000)
        case.update(requests=rng.randint(1, max(1, min(32, 6000 // t))), t_lo=max(1, t // 2), t_hi=t, n_lo=n,
                    n_hi=n + rng.randint(0, n // 2), gaps=rng.choice([0, 3, 20]))
        if not case["gaps"]:
            case["n_hi"] = n
    elif op == "rotate":
        case.update(tokens=_log_int(rng, 1, 8000), first=_log_int(rng, 1, 2000000))
    elif op == "attend":
        t = rng.choice([1, 1, 1, _log_int(rng, 2, 1500)])
        n = _log_int(rng, 1, 40000) + t
        r = rng.randint(1, max(1, min(12, 80000000 // (t * n), 200000 // n)))
        gaps = rng.choice([0, 1, 4])
        case.update(requests=r, n_lo=n, n_hi=n + (rng.randint(0, n // 2) if gaps else 0), t_lo=max(1, t // 2),
                    t_hi=t, gaps=gaps, cap=rng.choice([0.0, rng.uniform(5, 60)]), slopes=rng.random() < 0.5,
                    docs=rng.choice([0, rng.randint(1, 6)]) if t > 1 else 0,
                    reach=rng.choice([0, 0, _log_int(rng, 1, 9000)]),
                    prefix=rng.choice([0, 0, rng.randint(1, t)]), sinks=rng.choice([0, rng.randint(1, 8)]))
    elif op == "beam":
        r = rng.randint(1, 16)
        n = _log_int(rng, 17, 2000)
        t = _log_int(rng, 1, 100)
        case.update(requests=r, layers=rng.randint(1, 12), n_lo=n, n_hi=n + rng.randint(0, n), t_lo=max(1, t // 2),
                    t_hi=t, parents=rng.randint(1, r), freed=rng.randint(0, r // 3))
    else:
        n = _log_int(rng, 17, 3000)
        case.update(requests=rng.randint(1, 8), layers=rng.randint(1, 16), n_lo=n, n_hi=n + rng.randint(0, n),
                    used=rng.uniform(0.3, 0.98))
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


def _parents(case):
    """Whose cache each request goes on from: the first `parents` requests; the last `freed` are given
    up (-1)."""
    R, p, f = case["requests"], case["parents"], case["freed"]
    return [-1 if r >= R - f else (r if r < p else r % p) for r in range(R)]


def _layer_lens(case):
    """Lengths [request][head] of the layer that the call works on: the last."""
    R, L, H = case["requests"], case["layers"], case["kv_heads"]
    n = _lens(case)
    return [[n[(r * L + L - 1) * H + h] for h in range(H)] for r in range(R)]


def _token_plan(case, counts):
    """Of every token of a request's chunk: where its document begins and the last token of the chunk
    that it sees, counted in tokens of the chunk (a negative begin: the rows before the chunk)."""
    plan = []
    for t in counts:
        d = case["docs"]
        # the first document may have begun before the chunk
        starts = sorted(_spread(0, t - 1, d, 0.37)) if d else []
        plan.append(([max([s for s in starts if s <= i], default=-1) for i in range(t)],
                     [max(i, min(case["prefix"], t) - 1) for i in range(t)]))
    return plan


def work(case):
    d, H, Hq, ps = case["head_dim"], case["kv_heads"], case["q_heads"], case["page"]
    row = 2 * d * 2                                    # one K and one V row
    if case["op"] == "append":
        tokens = sum(_counts(case))
        return {"bytes": 2 * tokens * (H * row + Hq * d * 2) + 4 * tokens * (H + 1), "flops": 0}
    if case["op"] == "rotate":
        return {"bytes": case["tokens"] * (2 * Hq * d * 2 + 4), "flops": 0}
    if case["op"] == "compact":
        held = sum(-(-n // ps) for n in _lens(case))
        moved = held * (1 - case["used"])
        pages = held / case["used"]
        return {"bytes": moved * ps * (2 * row + 8) + 4 * (pages + held) + 8 * moved, "flops": 0}
    if case["op"] == "beam":
        counts, parents, lens = _counts(case), _parents(case), _lens(case)
        per = case["layers"] * H
        copied = new = entries = 0
        for r, p in enumerate(parents):
            kin = sum(q == p for q in parents)
            for u in range(per):
                n = lens[(p if p >= 0 else r) * per + u]
                held = -(-n // ps)
                entries += held if p != r else 0
                if p >= 0:
                    copied += kin > 1 and n % ps != 0
                    new += -(-(n + counts[r]) // ps) - held
        return {"bytes": copied * ps * (2 * row + 8) + 8 * entries + 4 * (copied + new) + 12 * per * len(parents),
                "flops": 0}
    tokens = sum(_counts(case))
    counts = _counts(case)
    rows = pairs = 0
    for n_r, t, (begin, end) in zip(_layer_lens(case), counts, _token_plan(case, counts)):
        for n in n_r:
            old = n - t                                # rows before the chunk
            step = case["gaps"] + 1                    # positions from one of them to the next, on average
            low, high = n, -1
            for i in range(t):
                lo = 0 if begin[i] < 0 else old + begin[i]
                if case["reach"]:
                    back = case["reach"] - 1
                    lo = max(lo, old + i - back if back <= i else old - (back - i) // step)
                    lo = max(lo, 0)
                hi = old + end[i]
                low, high = min(low, lo), max(high, hi)
                pairs += hi + 1 - lo + min(case["sinks"], lo)
            rows += high + 1 - low + min(case["sinks"], low)
    out = 2 * tokens * Hq * d * 2 + tokens * Hq * 4    # q, out, lse
    return {"bytes": rows * (row + (4 if case["gaps"] else 0)) + out, "flops": 4 * d * pairs * (Hq // H)}


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


def _frequencies(case):
    """Angles per position of the dims / 2 pairs, float32, and the factor of the turned values, for a
    context 8 times as long as 4096 positions (linear: positions divided; base: a larger base; parts:
    short waves kept, long ones divided, those between mixed)."""
    m, s, base = case["dims"], 8.0, 10000.0
    if case["scaling"] == "base":
        base *= s ** (m / max(m - 2, 1))
    w = base ** (-torch.arange(0, m, 2, dtype=torch.float64) / m)
    factor = 1.0
    if case["scaling"] == "linear":
        w = w / s
    elif case["scaling"] == "parts":
        turns = 4096 * w / (2 * math.pi)
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        w = w * keep + w / s * (1 - keep)
        factor = 0.1 * math.log(s) + 1
    return w.float().cuda(), factor


def _rotary(st):
    import kv_cache_eviction_split_gb300 as kv
    return kv.Rotary(st["freq"], factor=st["factor"], interleaved=st["case"]["interleaved"])


def _pack(*parts):
    """Whole-number tensors side by side in one, each at a multiple of 64 entries; and views of them."""
    size = [-(-p.numel() // 64) * 64 for p in parts]
    one, views, at = torch.zeros(sum(size), dtype=torch.int32, device="cuda"), [], 0
    for p, s in zip(parts, size):
        views.append(one[at:at + p.numel()].view(p.shape))
        views[-1].copy_(p)
        at += s
    return one, views


def _cache(case, gen, capacity, extra_pages=3):
    """Pools and a page table in an allocator's order, for units of up to `capacity` rows."""
    R, L, H, d, ps = (case[k] for k in ("requests", "layers", "kv_heads", "head_dim", "page"))
    cols = -(-capacity // ps)
    pages = R * L * H * cols + extra_pages
    perm = torch.randperm(pages, generator=gen, device="cuda")[:R * L * H * cols].to(torch.int32)
    return {"k": _fill((pages, ps, d), _dtype(case), gen), "v": _fill((pages, ps, d), _dtype(case), gen),
            "table": perm.view(R, L, H, cols).contiguous(),
            "lens": torch.tensor(_lens(case), dtype=torch.int32, device="cuda").view(R, L, H)}


def _slots(table, ps, j):
    """Pool rows of cache rows j [..., n] of the units whose tables are table [..., cols]."""
    return torch.gather(table.long(), -1, j // ps) * ps + j % ps


def _place_positions(case, c, counts, gen):
    """Positions of the cached rows, and of the new tokens [tokens]: rows of an evicted cache lie 1 to
    2 gaps + 1 apart, the new tokens follow one another behind the furthest of them."""
    R, L, H, ps, gaps = (case[k] for k in ("requests", "layers", "kv_heads", "page", "gaps"))
    n = c["lens"].long()
    t = torch.tensor(counts, device="cuda")
    if not gaps:
        # a row's position is its number: every head has the same length
        start = n[:, 0, 0] - t
    else:
        N = case["n_hi"]
        step = torch.randint(1, 2 * gaps + 2, (R, L, H, N), generator=gen, device="cuda")
        pos = torch.cumsum(step, -1) - 1
        j = torch.arange(N, device="cuda")
        old = (n - t[:, None, None])[..., None]                                       # rows before the chunk
        last = torch.where(j < old, pos, -1).amax(-1)
        start = last.amax((1, 2)) + 1
        pos = torch.where(j < old, pos, start[:, None, None, None] + j - old).int()
        c["pos"] = torch.full(c["k"].shape[:2], -1, dtype=torch.int32, device="cuda")
        held = j < n[..., None]
        c["pos"].view(-1)[_slots(c["table"], ps, j.expand(R, L, H, N))[held]] = pos[held]
    return torch.cat([start[r] + torch.arange(k, device="cuda") for r, k in enumerate(counts)]).int(), start


def _paged(c, q_heads):
    import kv_cache_eviction_split_gb300 as kv
    return kv.PagedCache(c["k"], c["v"], c["table"], c["lens"], q_heads, positions=c.get("pos"),
                         refs=c.get("refs"))


def _share(case, gen):
    """A cache whose pages are counted; of a compaction's, some are free and lie among the others."""
    R, L, H, d, ps = (case[k] for k in ("requests", "layers", "kv_heads", "head_dim", "page"))
    lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda").view(R, L, H)
    held = [-(-n // ps) for n in _lens(case)]
    if case["op"] == "beam":
        cols = -(-(case["n_hi"] + case["t_hi"]) // ps)
        # the tables' pages, and for every unit a copied tail and the new tokens' pages
        pages = sum(held) + len(held) * (2 + case["t_hi"] // ps) + 5
    else:
        cols = max(held)
        pages = max(sum(held), int(round(sum(held) / case["used"])))
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(cols, device="cuda")
    mine = col < torch.tensor(held, device="cuda")[:, None]
    table = torch.full((len(held), cols), -1, dtype=torch.int32, device="cuda")
    table[mine] = perm[:sum(held)]
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[perm[:sum(held)].long()] = 1
    state, (table, lens, refs) = _pack(table.view(R, L, H, cols), lens, refs)
    c = {"k": _fill((pages, ps, d), _dtype(case), gen), "v": _fill((pages, ps, d), _dtype(case), gen),
         "table": table, "lens": lens, "refs": refs,
         "pos": torch.randint(0, 1 << 20, (pages, ps), generator=gen, device="cuda").int()}
    return c, state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    H, Hq, d = case["kv_heads"], case["q_heads"], case["head_dim"]
    st = {"case": case}
    if case["op"] == "rotate":
        st["freq"], st["factor"] = _frequencies(case)
        st["x"] = _fill((case["tokens"], Hq, d), _dtype(case), gen)
        st["out"] = torch.empty_like(st["x"])
        st["positions"] = case["first"] + torch.arange(case["tokens"], dtype=torch.int32, device="cuda") + seed % 7
        if own:
            st["rotary"] = _rotary(st)
        return st
    if case["op"] in ("beam", "compact"):
        st["cache"], st["state"] = _share(case, gen)
        st["saved"] = st["state"].clone()
        st["live"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["op"] == "beam":
            # the order of the hypotheses is the seed's
            order = torch.randperm(case["requests"], generator=gen, device="cuda").cpu().tolist()
            parents, counts = [0] * case["requests"], [0] * case["requests"]
            for r, (p, t) in enumerate(zip(_parents(case), _counts(case))):
                parents[order[r]] = order[p] if p >= 0 else -1
                counts[order[r]] = t if p >= 0 else 0
            st["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda")
            st["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
        if own:
            import kv_cache_eviction_split_gb300 as kv
            st["paged"] = _paged(st["cache"], Hq)
            if case["op"] == "beam":
                st["chunk"] = kv.Chunk(counts, device="cuda")
                size = kv.kv_paged_reserve_workspace_size(st["paged"])
            else:
                size = kv.kv_paged_compact_workspace_size(st["paged"])
            st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        return st
    counts = _counts(case)
    # tables are as long as a step may need
    st["cache"] = c = _cache(case, gen, case["n_hi"] + case["page"] // 2)
    st["positions"], start = _place_positions(case, c, counts, gen)
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
    st["out"] = torch.empty((tokens, Hq, d), dtype=_dtype(case), device="cuda")
    if own:
        import kv_cache_eviction_split_gb300 as kv
        st["paged"] = _paged(c, Hq)
        st["chunk"] = kv.Chunk(counts, device="cuda")
    if case["op"] == "append":
        st["freq"], st["factor"] = _frequencies(case)
        if own:
            st["rotary"] = _rotary(st)
        return st
    st["lse"] = torch.empty((tokens, Hq), device="cuda")
    st["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq) if case["slopes"] else None
    plan = _token_plan(case, counts)
    begin, end = (torch.tensor(sum((p[i] for p in plan), []), device="cuda") for i in (0, 1))
    base = start[torch.searchsorted(st["off"], torch.arange(tokens, device="cuda"), right=True) - 1]
    first = torch.where(begin < 0, 0, base + begin)
    if case["reach"]:
        first = torch.maximum(first, st["positions"] - (case["reach"] - 1))
    st["first"] = first.int() if case["reach"] or case["docs"] else None
    st["last"] = (base + end).int() if case["prefix"] else None
    if own:
        st["ws"] = torch.empty(kv.kv_paged_attention_scored_workspace_size(st["paged"], st["chunk"]),
                               dtype=torch.uint8, device="cuda")
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    return {"append": _append, "rotate": _rotate, "attend": _attention, "beam": _beam,
            "compact": _compact}[st["case"]["op"]](st)


def _turned(st, x, positions, back=False):
    """x [tokens, heads, d] turned by its positions' angles, in 32 bits from angles in 64."""
    case = st["case"]
    m = case["dims"]
    a = positions.double()[:, None] * st["freq"].double()
    cos, sin = ((f(a) * st["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
    if back:
        sin = -sin
    y = x.float()
    one, two = (y[..., 0:m:2], y[..., 1:m:2]) if case["interleaved"] else (y[..., :m // 2], y[..., m // 2:m])
    pair = [one * cos - two * sin, one * sin + two * cos]
    t = torch.stack(pair, -1).flatten(-2) if case["interleaved"] else torch.cat(pair, -1)
    return torch.cat([t, y[..., m:]], -1).to(x.dtype)


def _rotate(st):
    if own:
        import kv_cache_eviction_split_gb300 as kv
        kv.kv_rotary(st["rotary"], st["positions"], st["x"], st["out"], backward=True)
        return st["out"]
    st["out"].copy_(_turned(st, st["x"], st["positions"], back=True))
    return st["out"]


def _append(st):
    case, c = st["case"], st["cache"]
    layer = case["layers"] - 1
    out = [st["out"], c["k"], c["v"]] + ([c["pos"]] if case["gaps"] else [])
    if own:
        import kv_cache_eviction_split_gb300 as kv
        kv.kv_paged_append_rotary(st["paged"], st["chunk"], layer, st["rotary"], st["positions"], st["q"],
                                  st["out"], st["k_new"], st["v_new"])
        return out
    ps, d = case["page"], case["head_dim"]
    st["out"].copy_(_turned(st, st["q"], st["positions"]))
    tok = torch.arange(st["q"].shape[0], device="cuda")
    req = torch.searchsorted(st["off"], tok, right=True) - 1
    # a request's new rows are the last of its units' rows
    j = c["lens"][:, layer].long()[req] - (st["off"][req + 1] - tok)[:, None]       # [tokens, H]
    rows = _slots(c["table"][:, layer][req], ps, j[..., None])[..., 0]
    c["k"].view(-1, d)[rows] = _turned(st, st["k_new"], st["positions"])
    c["v"].view(-1, d)[rows] = st["v_new"]
    if case["gaps"]:
        c["pos"].view(-1)[rows] = st["positions"][:, None].expand_as(rows)
    return out


def _attention(st):
    case, c = st["case"], st["cache"]
    layer = case["layers"] - 1
    if own:
        import kv_cache_eviction_split_gb300 as kv
        kv.kv_paged_attention_scored(st["paged"], st["chunk"], layer, st["q"], st["out"], st["ws"],
                                     softcap=case["cap"], slopes=st["slopes"], first=st["first"],
                                     last=st["last"], num_sinks=case["sinks"], lse=st["lse"])
        return [st["out"], st["lse"]]
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
    at = c["pos"].view(-1)[rows].long() if case["gaps"] else j.expand(R, H, -1)       # [R, H, n]
    p = st["positions"][tok].long()[:, None, :, None]                                 # [R, 1, T, 1]
    seen = held[:, :, None] & ((at[:, :, None] <= st["last"][tok][:, None, :, None]) if st["last"] is not None
                               else (j <= t))
    if st["first"] is not None:
        seen &= (at[:, :, None] >= st["first"][tok][:, None, :, None]) | (j < case["sinks"])
    x = torch.matmul(q.reshape(R, H, T * G, d), K.transpose(-1, -2)).view(R, H, T, G, -1)
    x.mul_(1.0 / math.sqrt(d))
    if case["cap"]:
        x.div_(case["cap"]).tanh_().mul_(case["cap"])
    if case["slopes"]:
        far = (at[:, :, None] - p).abs().float()                                      # [R, H, T, n]
        x.sub_(st["slopes"].view(H, 1, G, 1) * far[:, :, :, None])
    x.masked_fill_(~seen[:, :, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True).clamp_min(-1e30)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    x.div_(torch.where(total > 0, total, 1.0))
    o = torch.matmul(x.view(R, H, T * G, -1), V).view(R, H, T, G, d)
    lse = (top + torch.log(total))[..., 0]
    real = i < count[:, None]                                                         # [R, T]
    st["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(R, T, Hq, d)[real])
    st["lse"].copy_(lse.permute(0, 2, 1, 3).reshape(R, T, Hq)[real])
    return [st["out"], st["lse"]]


def _beam(st):
    case, c = st["case"], st["cache"]
    out = [c[x] for x in ("k", "v", "pos", "table", "lens", "refs")]
    st["state"].copy_(st["saved"])                     # the step before this one
    if own:
        import kv_cache_eviction_split_gb300 as kv
        kv.kv_paged_fork(st["paged"], st["parents"])
        kv.kv_paged_reserve(st["paged"], st["chunk"], st["ws"])
        return out
    ps, R = case["page"], case["requests"]
    table, lens, refs = c["table"], c["lens"], c["refs"]
    cols = table.shape[-1]
    col = torch.arange(cols, device="cuda")
    # every request takes its parent's entries and lengths
    parents = st["parents"].long()
    moves = (parents != torch.arange(R, device="cuda"))[:, None, None, None]
    before = table.clone()
    had = (col < (lens[..., None] + ps - 1) // ps) & moves
    new_lens = torch.where((parents >= 0)[:, None, None], lens[parents.clamp_min(0)], 0)
    has = (col < (new_lens[..., None] + ps - 1) // ps) & moves
    table.copy_(torch.where(has, before[parents.clamp_min(0)], before))
    gone, come = before[had].long(), table[has].long()
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    refs.index_add_(0, come, torch.ones_like(come, dtype=torch.int32))
    lens.copy_(new_lens)
    # pages for the next tokens: the lowest free ones, unit after unit, a shared tail's copy first
    free = torch.nonzero(refs == 0)[:, 0]
    flat, n = table.view(-1, cols), lens.view(-1).long()
    t = st["counts"].long()[:, None].expand(R, flat.shape[0] // R).reshape(-1)
    old, new = (n + ps - 1) // ps, (n + t + ps - 1) // ps
    tail = torch.gather(flat, 1, (old - 1).clamp_min(0)[:, None])[:, 0].long()
    copy = (t > 0) & (n % ps != 0) & (refs[tail.clamp_min(0)] > 1)
    first, need = old - copy.long(), new - old + copy.long()
    k = torch.cumsum(need, 0) - need
    take = (col >= first[:, None]) & (col < new[:, None])
    pages = free[(k[:, None] + col - first[:, None])[take]]
    flat[take] = pages.int()
    refs[pages] = 1
    src, dst = tail[copy], torch.gather(flat, 1, (old - 1).clamp_min(0)[:, None])[:, 0].long()[copy]
    refs.index_add_(0, src, torch.full_like(src, -1, dtype=torch.int32))
    for x in ("k", "v", "pos"):
        c[x][dst] = c[x][src]
    lens.add_(st["counts"][:, None, None])
    return out


def _compact(st):
    case, c = st["case"], st["cache"]
    out = [c[x] for x in ("k", "v", "pos", "table", "lens", "refs")] + [st["live"]]
    st["state"].copy_(st["saved"])
    if own:
        import kv_cache_eviction_split_gb300 as kv
        kv.kv_paged_compact(st["paged"], st["ws"], live=st["live"])
        return out
    ps, table, lens, refs = case["page"], c["table"], c["lens"], c["refs"]
    page = torch.arange(refs.numel(), device="cuda")
    st["live"].copy_((refs > 0).sum())
    hole = torch.nonzero((refs == 0) & (page < st["live"]))[:, 0]
    far = torch.nonzero((refs > 0) & (page >= st["live"]))[:, 0]
    for x in ("k", "v", "pos"):
        c[x][hole] = c[x][far]
    refs[hole] = refs[far]
    refs[far] = 0
    page[far] = hole
    used = torch.arange(table.shape[-1], device="cuda") < (lens[..., None] + ps - 1) // ps
    table[used] = page[table[used].long()].int()
    return out


# --------------------------------------------------------------------------
# the same outputs from the definitions, in 64 bits, unit by unit
# --------------------------------------------------------------------------
def _rows_of(cache, ps, r, l, h, n):
    """Pool rows of the first n rows of unit (r, l, h)."""
    pages = cache["table"][r, l, h].long()
    return (pages[:, None] * ps + torch.arange(ps, device=pages.device)).reshape(-1)[:n]


def _turned64(case, freq, factor, x, positions, sign):
    """Pair by pair: a product of complex numbers."""
    y = x.double().clone()
    m = case["dims"]
    for i in range(m // 2):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + m // 2)
        angle = sign * positions.double() * freq[i].double()
        z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.full_like(angle, factor), angle)[:, None]
        y[..., a], y[..., b] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotate":
        return _turned64(case, st["freq"], st["factor"], st["x"], st["positions"], -1.0)
    c = st["cache"]
    R, L, H, Hq, d, ps = (case[k] for k in ("requests", "layers", "kv_heads", "q_heads", "head_dim", "page"))
    lens = _lens(case)
    if case["op"] == "compact":
        refs, table = c["refs"].tolist(), c["table"].view(-1, c["table"].shape[-1]).tolist()
        live = sum(x > 0 for x in refs)
        holes = [p for p in range(live) if not refs[p]]
        far = [p for p in range(live, len(refs)) if refs[p]]
        k, v = (c[x].double() for x in "kv")
        for a, b in zip(holes, far):
            k[a], v[a] = c["k"][b].double(), c["v"][b].double()
        return [k, v, None, None, None, None, None]
    if case["op"] == "beam":
        cols, per = c["table"].shape[-1], L * H
        table, refs = c["table"].view(-1, cols).tolist(), c["refs"].tolist()
        parents, counts = st["parents"].tolist(), st["counts"].tolist()
        k, v = (c[x].double() for x in "kv")
        held = [table[u][:-(-lens[u] // ps)] for u in range(R * per)]
        mine = [[held[p * per + i] if p >= 0 else [] for i in range(per)] for p in parents]
        refs = [0] * len(refs)
        for unit in (x for r in mine for x in r):
            for p in unit:
                refs[p] += 1
        free = iter([p for p, x in enumerate(refs) if not x])
        for r in range(R):
            for i in range(per):
                n = lens[parents[r] * per + i] if parents[r] >= 0 else 0
                if counts[r] and n % ps and refs[mine[r][i][-1]] > 1:
                    a, b = mine[r][i][-1], next(free)
                    k[b], v[b] = c["k"][a].double(), c["v"][a].double()
                for _ in range(-(-(n + counts[r]) // ps) - -(-n // ps)):
                    next(free)
        return [k, v, None, None, None, None]
    if case["op"] == "append":
        k, v = (c[x].double().view(-1, d) for x in "kv")
        turned = _turned64(case, st["freq"], st["factor"], st["k_new"], st["positions"], 1.0)
        off = st["off"].tolist()
        for r in range(R):
            for h in range(H):
                n, t0, t1 = lens[(r * L + L - 1) * H + h], off[r], off[r + 1]
                new = _rows_of(c, ps, r, L - 1, h, n)[n - (t1 - t0):]
                k[new], v[new] = turned[t0:t1, h], st["v_new"][t0:t1, h].double()
        return [_turned64(case, st["freq"], st["factor"], st["q"], st["positions"], 1.0),
                k.view(c["k"].shape), v.view(c["v"].shape)] + ([None] if case["gaps"] else [])
    if work(case)["flops"] > 5e12:
        return None
    G = Hq // H
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    for r in range(R):
        for h in range(H):
            n, t0, t1 = lens[(r * L + L - 1) * H + h], int(st["off"][r]), int(st["off"][r + 1])
            rows = _rows_of(c, ps, r, L - 1, h, n)
            K, V = (c[x].view(-1, d)[rows].double() for x in "kv")
            key = torch.arange(n, device="cuda")
            at = c["pos"].view(-1)[rows].double() if case["gaps"] else key.double()
            own_row = torch.arange(n - (t1 - t0), n, device="cuda")
            here = at[own_row][:, None]
            hidden = at[None] > (st["last"][t0:t1, None].double() if case["prefix"] else here)
            if st["first"] is not None:
                hidden |= (at[None] < st["first"][t0:t1, None].double()) & (key >= case["sinks"])
            for g in range(G):
                s = st["q"][t0:t1, h * G + g].double() @ K.T / math.sqrt(d)
                if case["cap"]:
                    s = case["cap"] * torch.tanh(s / case["cap"])
                if case["slopes"]:
                    s = s - st["slopes"][h * G + g].double() * (here - at[None]).abs()
                s[hidden] = -math.inf
                z = torch.logsumexp(s, 1)
                out[t0:t1, h * G + g] = torch.nan_to_num(torch.exp(s - z[:, None])) @ V
                lse[t0:t1, h * G + g] = z
    return [out, lse]
