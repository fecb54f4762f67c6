"""Attention with changed scores in 64 bits, unit by unit, and how far the kernels may be from it."""
import math

import torch

from tests import paged


def positions_of(made, gaps, seed, start=0):
    """Rising positions for every unit's rows (gaps: largest step), the last rows of all of a
    request's heads at the same ones; poison elsewhere.  {(r, l, h): int64 [n]}."""
    g = torch.Generator().manual_seed(seed + 77)
    c = made.cache
    pool = torch.full(c.k_pages.shape[:2], -(1 << 30), dtype=torch.int32, device="cuda")
    found = {}
    for key, K in made.K.items():
        n = K.shape[0]
        step = torch.randint(0 if gaps < 0 else 1, abs(gaps) + 1, (n,), generator=g)
        pos = start + torch.cumsum(step, 0) - (step[:1] if n else 0)
        found[key] = pos.cuda()
        pool.view(-1)[made.rows(*key)] = found[key].int()
    c.positions = pool
    return found


def scored_unit(q, K, V, pos, scale, cap=0.0, slopes=None, first=None, last=None, window=0, sinks=0):
    """q [count][G][d], K/V [n][d] double, pos [n], slopes [G], first/last [count]: out, lse, weights summed
    per row, sum p |v|, and per output the first order of what errors of the logits do to it and to lse.

    A logit is off by its d products (2^-23 of the sum of magnitudes each), its 2^x (2^-22 and 2^-22 of
    itself); capped, by 2^-20 of cap (2^x to 2^-22, which counts a quarter, a reciprocal to
    2^-23 of two factors with three roundings, one fused product: 6.5 2^-23), and with
    caps beyond 4096 softmax scales by 2^-17 of itself at most (a polynomial whose first coefficient is 2.8e-6 off,
    or the series; above a quarter of the cap the same);
    lowered, by 2^-22 of what is taken off (slope log2(e), the product, the difference)."""
    count, G, d = q.shape
    n = K.shape[0]
    t = torch.arange(n - count, n, device=q.device)
    j = torch.arange(n, device=q.device)
    here = pos[t.clamp_min(0)] if n else torch.zeros(count, device=q.device)
    ok = (t >= 0)[:, None] & ((pos[None] <= last[:, None]) if last is not None else (j[None] <= t[:, None]))
    low = torch.ones_like(ok)
    if first is not None:
        low &= pos[None] >= first[:, None]
    if window:
        low &= j[None] > t[:, None] - window
    if first is not None or window:
        low |= j[None] < sinks
    ok &= low
    s = scale * torch.einsum("igd,jd->gij", q, K)
    err = d * 2.0 ** -23 * scale * torch.einsum("igd,jd->gij", q.abs(), K.abs())
    if cap:
        s = cap * torch.tanh(s / cap)
        own = 2.0 ** -17 * s.abs() if cap > 4096 * scale else torch.full_like(s, math.inf)
        err = err + own.clamp_max(2.0 ** -20 * cap)
    if slopes is not None:
        off = slopes.double()[:, None, None] * (here[:, None] - pos[None]).abs().double()
        s = s - off
        err = err + 2.0 ** -22 * off.abs()
    err = err + 2.0 ** -22 * (s.abs() + 1)
    s = s.masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(s, -1) if n else torch.full((G, count), -math.inf, device=q.device,
                                                      dtype=torch.float64)
    p = torch.where(ok, torch.exp(s - lse.clamp_min(-1e300)[..., None]), 0.0)
    pe = p * err
    return (torch.einsum("gij,jd->igd", p, V), lse.T, p.sum((0, 1)), torch.einsum("gij,jd->igd", p, V.abs()),
            torch.einsum("gij,jd->igd", pe, V.abs()), pe.sum(-1).T, pe.sum((0, 1)))


def out_bound(o, absv, pev, pe, dtype, n):
    """As tests/paged.py's, with the logits' errors weighted: each weight's own and the normaliser's."""
    half = torch.finfo(dtype).eps / 2
    return half * o.abs() + 1.01 * ((half + 2 * n * 2.0 ** -23) * absv + pev + pe[..., None] * absv) + 1e-7


def lse_bound(z, pe, n):
    return pe + n * 2.0 ** -23 + 2.0 ** -22 * z.abs() + 2.0 ** -22


def check(kv, made, pos, counts, q, out, lse, layer=0, cap=0.0, slopes=None, first=None, last=None, window=0,
          sinks=0, scale=None, mass=False):
    c = made.cache
    G, d = c.num_q_heads // c.num_kv_heads, made.d
    scale = scale or 1 / math.sqrt(d)
    want = made.mass0.double().clone().view(-1)
    tol = torch.zeros_like(want)
    t0 = 0
    for r, count in enumerate(counts):
        t1 = t0 + count
        for h in range(c.num_kv_heads):
            K, V = made.K[r, layer, h], made.V[r, layer, h]
            n = K.shape[0]
            at = pos[r, layer, h] if pos is not None else torch.arange(n, device="cuda")
            g = slice(h * G, (h + 1) * G)
            o, z, w, absv, pev, pe, wpe = scored_unit(
                q[t0:t1, g].double(), K, V, at, scale, cap, None if slopes is None else slopes[g],
                None if first is None else first[t0:t1].long(), None if last is None else last[t0:t1].long(),
                window, sinks)
            got = out[t0:t1, g].double()
            assert torch.isfinite(got).all()
            ratio = (got - o).abs() / out_bound(o, absv, pev, pe, made.dtype, n)
            assert count == 0 or float(ratio.max()) <= 1, (r, h, float(ratio.max()))
            gz = lse[t0:t1, g].double()
            empty = torch.isinf(z)
            assert torch.equal(torch.isinf(gz) & (gz < 0), empty)
            ratio = ((gz - z).abs() / lse_bound(z, pe, n))[~empty]
            assert ratio.numel() == 0 or float(ratio.max()) <= 1, (r, h, float(ratio.max()))
            if mass and n and count:
                rows = made.rows(r, layer, h)
                # a weight's own error and its normaliser's
                tol[rows] = wpe + w * (float(pe.max()) + n * 2.0 ** -23 + count * G * 2.0 ** -24) \
                    + 2.0 ** -23 * (want[rows].abs() + w) + 1e-30
                want[rows] += w
        t0 = t1
    if mass:
        assert ((c.mass.double().view(-1) - want).abs() <= tol).all()


def run(kv, made, counts, q, out, layer=0, mass=False, stream=None, **kw):
    chunk = kv.Chunk(counts)
    c = made.cache
    lse = torch.full((q.shape[0], c.num_q_heads), 7.0, device="cuda")
    ws = torch.full((kv.kv_paged_attention_scored_workspace_size(c, chunk, mass),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    kw = dict(kw)
    kv.kv_paged_attention_scored(c, chunk, layer, q, out, ws, softcap=kw.pop("cap", 0.0), num_sinks=kw.pop("sinks", 0),
                                 softmax_scale=kw.pop("scale", None), lse=lse, add_mass=mass, stream=stream, **kw)
    return lse, kv.kv_check_status(c.status, stream)


def bounds_of(kind, counts, lens, pos, seed=0):
    """first and last [tokens] int32 (or None) of a kind; lens[r] the rows of a head, pos[r] the positions
    of one head's rows."""
    g = torch.Generator().manual_seed(seed)
    first, last = [], []
    for count, n, p in zip(counts, lens, pos):
        p = p.cpu().long()
        top = int(p[-1]) if n else 0
        own = torch.tensor([int(p[max(n - count + i, 0)]) if n else 0 for i in range(count)])
        if kind == "docs":
            cuts = torch.sort(torch.randint(0, top + 1, (4,), generator=g)).values
            first.append(torch.stack([torch.where(own >= c, c, 0) for c in cuts]).amax(0) if count else own)
            last.append(own)
        elif kind == "reach":
            first.append(own - 100)
            last.append(own)
        elif kind == "prefix":
            first.append(torch.zeros_like(own))
            last.append(torch.maximum(own, own[count // 2] if count else own))
        elif kind == "random":
            a = torch.randint(-5, top + 5, (count,), generator=g)
            first.append(a)
            last.append(a + torch.randint(-3, top // 2 + 4, (count,), generator=g))
        elif kind == "halves":
            # the first queries see the first rows, the others the last ones, and none those between
            early = torch.arange(count) < count // 2
            first.append(torch.where(early, 0, max(0, top - 60)))
            last.append(torch.where(early, min(top, 60), top))
        elif kind == "back":
            # later queries see earlier rows
            first.append((top * (count - torch.arange(count))) // (count + 1))
            last.append(first[-1] + 40)
        elif kind == "none":
            first.append(torch.full((count,), top + 1))
            last.append(torch.full((count,), top + 9) if count % 2 else torch.full((count,), -1))
        elif kind == "extremes":
            first.append(torch.full((count,), -2 ** 31))
            last.append(torch.full((count,), 2 ** 31 - 1))
    one = [torch.cat(x).to(torch.int32).cuda() if x else torch.zeros(0, dtype=torch.int32, device="cuda")
           for x in (first, last)]
    return one
