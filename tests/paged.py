"""Caches in pages for the tests, and the operators on them in 64 bits, unit by unit."""
import math

import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Made:
    """A cache whose unused memory is poison: rows past a unit's length hold NaN, table
    entries past its last page do not exist, and neither do pages that `unseen` rows fill."""

    def __init__(self, kv, lens, num_q_heads, d, page, dtype="bf16", max_rows=None, mass=False,
                 seed=0, spare=2, device="cuda", scale=1.0, unseen=None):
        g = torch.Generator(device=device).manual_seed(seed)
        self.lens_host = torch.as_tensor(lens, dtype=torch.int32)       # [R][L][H]
        R, L, H = self.lens_host.shape
        cols = -(-max(int(max_rows or self.lens_host.max()), 1) // page)
        units, dt = R * L * H, DTYPES[dtype]
        pages = units * cols + spare
        kp = torch.randn((pages, page, d), generator=g, device=device) * scale
        vp = torch.randn((pages, page, d), generator=g, device=device) * scale
        kp[..., 3::16] *= 3
        perm = torch.randperm(pages, generator=g, device=device)[:units * cols].to(torch.int32)
        table = perm.view(R, L, H, cols).clone()
        ps = torch.arange(page, device=device)
        self.mass0 = torch.rand((pages, page), generator=g, device=device)
        kp, vp = kp.to(dt), vp.to(dt)
        self.K, self.V = {}, {}
        for r in range(R):
            for l in range(L):
                for h in range(H):
                    n = max(int(self.lens_host[r, l, h]), 0)
                    rows = (table[r, l, h].long()[:, None] * page + ps).reshape(-1)
                    self.K[r, l, h] = kp.view(-1, d)[rows[:n]].double()
                    self.V[r, l, h] = vp.view(-1, d)[rows[:n]].double()
                    kp.view(-1, d)[rows[n:]] = float("nan")
                    vp.view(-1, d)[rows[n:]] = float("nan")
                    self.mass0.view(-1)[rows[n:]] = -7.0
                    used = -(-n // page)
                    table[r, l, h, used:] = -1 if (r + h) % 2 else 2 ** 31 - 1
                    if unseen is not None:
                        for a, b in unseen(r, l, h, n):           # whole pages inside are gone
                            kp.view(-1, d)[rows[a:b]] = float("nan")
                            vp.view(-1, d)[rows[a:b]] = float("inf")
                            p0, p1 = -(-a // page), b // page
                            if p1 > p0:
                                table[r, l, h, p0:p1] = -5
        self.page, self.d, self.dtype = page, d, dt
        self.cache = kv.PagedCache(kp, vp, table, self.lens_host.to(device), num_q_heads,
                                   mass=self.mass0.clone() if mass else None)

    def rows(self, r, l, h, n=None):
        """Pool rows of the first n rows of a unit."""
        t = self.cache.page_table[r, l, h].long()
        n = int(self.lens_host[r, l, h]) if n is None else n
        j = torch.arange(n, device=t.device)
        return t[j // self.page] * self.page + j % self.page


def seen_mask(n, count, window, sinks, device):
    """[count][n]: which rows query i of the last `count` sees."""
    t = torch.arange(n - count, n, device=device)[:, None]
    j = torch.arange(n, device=device)[None]
    ok = j <= t
    if window > 0:
        ok &= (j > t - window) | (j < sinks)
    return ok


def attend_unit(q, K, V, window, sinks, scale):
    """q [count][G][d], K/V [n][d], all double -> out, lse, weights summed per row, and what the
    tolerances need: sum p |v| [count][G][d] and the largest sum |q||k| of a logit."""
    count, G, d = q.shape
    n = K.shape[0]
    ok = seen_mask(n, count, window, sinks, q.device)
    s = scale * torch.einsum("igd,jd->gij", q, K)
    big = scale * torch.einsum("igd,jd->gij", q.abs(), K.abs())
    s = s.masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(s, -1) if n else torch.full((G, count), -math.inf, device=q.device,
                                                      dtype=torch.float64)
    p = torch.exp(s - lse.clamp_min(-1e300)[..., None])
    p = torch.where(ok, p, 0.0)
    out = torch.einsum("gij,jd->igd", p, V)
    absv = torch.einsum("gij,jd->igd", p, V.abs())
    logit = float(big.masked_fill(~ok, 0).max()) if n and count else 0.0
    return out, lse.T, p.sum((0, 1)), absv, logit


# Error bounds.  A logit sums d exact products in fp32, each addition off by at most 2^-23 of the
# sum of magnitudes so far (the tensor core may truncate): d 2^-23 sum|q||k|.  Its 2^x adds 2^-22
# relative (the fp32 power of two and the fused multiply-add before it).
def logit_error(d, logit):
    return d * 2.0 ** -23 * logit + 2.0 ** -22 * (logit + 1)


def out_bound(out, absv, dtype, d, n, logit, parts):
    """parts = 1: weights rounded to the dtype before they multiply V; 2: to two such parts.
    A weight is off by its rounding and by twice the logit's error (its own and the normaliser's);
    n additions in fp32 (twice: weights' sum and products' sum); the output is rounded once."""
    half = torch.finfo(dtype).eps / 2
    p_err = half ** parts + 2 * logit_error(d, logit) + 2 * n * 2.0 ** -23
    return half * out.abs() + 1.01 * p_err * absv + 1e-7


def lse_bound(lse, d, n, logit):
    return logit_error(d, logit) + n * 2.0 ** -23 + 2.0 ** -22 * lse.abs()


def mass_bound(added, before, d, n, logit, terms):
    rel = 2 * logit_error(d, logit) + n * 2.0 ** -23 + terms * 2.0 ** -24
    return rel * added + 2.0 ** -23 * (before.abs() + added) + 1e-30


def evict_unit(mass, n, b, sinks, recent):
    """Kept rows of a unit, by a sort on (weight descending, row ascending)."""
    if n <= b:
        return list(range(n))
    mid = sorted(range(sinks, n - recent), key=lambda j: (-float(mass[j]), j))
    mid = sorted(mid[:b - sinks - recent])
    return list(range(sinks)) + mid + list(range(n - recent, n))


def cancelling(n, new, d, dtype, seed, device="cpu"):
    """A query, n + new keys and values (in `dtype`) whose softmax average is all but zero while
    sum p |v| is not: the output's own rounding then hides nothing of an error in the weights.
    The last `new` rows have values 0, so queries that see different numbers of them agree up to
    a factor.  Returns (q [d], K [n + new][d], V [n + new][d], softmax scale)."""
    g = torch.Generator(device=device).manual_seed(seed)
    q, K, V = (torch.zeros(s, dtype=torch.float64, device=device)
               for s in ((d,), (n + new, d), (n + new, d)))
    scale = 1 / math.sqrt(d)
    q[0] = 0.5 / scale
    q = q.to(dtype)
    # logits in -0.5 .. 0.5: one product each
    K[:n, 0] = torch.rand(n, generator=g, device=device, dtype=torch.float64) * 2 - 1
    K = K.to(dtype)
    p = torch.exp(scale * (K[:n].double() @ q.double()))
    v = torch.randn((n, d), generator=g, device=device, dtype=torch.float64)
    V[:n] = v - torch.outer(p, (p @ v) / (p @ p))
    return q, K, V.to(dtype), scale
