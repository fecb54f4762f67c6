"""Attention over the pages where a query or a key that is seen holds NaN: the rows that see it are NaN, output
and lse, in every form of the kernels and with every change of the scores; the others follow the
formula in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu

# (KV heads, query heads, d, page, dtype, counts, shortest, longest, rows of a table)
FORMS = {
    "clusters": (2, 8, 128, 16, "bf16", [1, 2], 500, 900, 1000),
    "one_block": (2, 4, 64, 16, "fp16", [1] * 80, 20, 60, 60),
    "row_blocks": (1, 8, 128, 32, "bf16", [30, 9], 40, 400, 400),
    "long": (2, 8, 128, 64, "bf16", [1, 3], 8500, 9001, 9001),
    "many": (4, 32, 128, 32, "bf16", [200, 1, 0, 151], 211, 700, 700),
    "many_fp16": (8, 32, 64, 64, "fp16", [140, 257], 300, 1300, 1300),
}
# cap 200: below half of it; cap 2: far above it (softmax scales 1 / sqrt(d) and 1)
CHANGES = {
    "plain": {},
    "slopes": dict(slopes=True),
    "docs": dict(docs=True),
    "docs_slopes": dict(docs=True, slopes=True),
    "cap": dict(cap=200.0),
    "cap_exact": dict(cap=2.0, scale=1.0),
    "both": dict(cap=200.0, slopes=True),
    "both_exact": dict(cap=2.0, scale=1.0, slopes=True),
    "docs_cap": dict(docs=True, cap=200.0),
    "docs_cap_exact": dict(docs=True, cap=2.0, scale=1.0),
}


@pytest.mark.parametrize("where", ["query", "key"])
@pytest.mark.parametrize("change", CHANGES)
@pytest.mark.parametrize("form", FORMS)
def test_nan_reaches_the_rows_that_see_it(cuda_lib, form, change, where):
    import torch
    from tests import paged, scores
    from tests.test_gpu_paged_attention import _chunk_inputs, _spread
    from tests.test_gpu_paged_scores import _slopes
    kv = cuda_lib
    H, Hq, d, page, dtype, counts, lo, hi, table = FORMS[form]
    G = Hq // H
    lens = [[[n] * H] for (n, *_), in _spread(len(counts), 1, H, lo, hi)]
    made = paged.Made(kv, lens, Hq, d, page, dtype, max_rows=table, seed=len(form))
    q, out = _chunk_inputs(made, counts, Hq, False, len(change))
    kw = dict(CHANGES[change])
    if kw.pop("slopes", False):
        kw["slopes"] = _slopes(Hq)
    if kw.pop("docs", False):
        kw["first"], kw["last"] = scores.bounds_of("docs", counts, [x[0][0] for x in lens],
                                                   [torch.arange(x[0][0]) for x in lens])
        kw["last"] = None
    bad = torch.zeros((q.shape[0], Hq), dtype=torch.bool, device="cuda")
    nan_key = {}
    if where == "query":
        # a token of every request, one head of each; and all heads of the last token
        t0 = 0
        for r, count in enumerate(counts):
            if count:
                bad[t0 + count // 2, (3 * r) % Hq] = True
            t0 += count
        bad[-1] = True
        q[bad, 5] = math.nan
    else:
        # the row of a query in the middle of its request's chunk, which earlier ones do not see, in one head
        for r, count in enumerate(counts):
            if count:
                h, j = r % H, lens[r][0][0] - (count + 1) // 2
                nan_key[r, h] = j
                made.cache.k_pages.view(-1, d)[made.rows(r, 0, h)[j], 7] = math.nan
    lse, status = scores.run(kv, made, counts, q, out, **kw)
    assert status == 0
    scale = kw.pop("scale", 1 / math.sqrt(d))
    slopes = kw.pop("slopes", None)
    t0 = 0
    for r, count in enumerate(counts):
        t1 = t0 + count
        for h in range(H if count else 0):
            K, V = made.K[r, 0, h], made.V[r, 0, h]
            g = slice(h * G, (h + 1) * G)
            n = K.shape[0]
            first = None if kw.get("first") is None else kw["first"][t0:t1].long()
            # Made's copies of K are from before: the rows that do not see the NaN are those of the clean cache
            o, z, _, absv, pev, pe, _ = scores.scored_unit(
                q[t0:t1, g].double().nan_to_num(0.0), K, V, torch.arange(n, device="cuda"), scale,
                kw.get("cap", 0.0), None if slopes is None else slopes[g], first)
            nan = bad[t0:t1, g].clone()
            if (r, h) in nan_key:
                j = nan_key[r, h]
                t = torch.arange(n - count, n, device="cuda")
                sees = t >= j
                if first is not None:
                    sees &= first <= j
                nan |= sees[:, None]
            got, gz = out[t0:t1, g].double(), lse[t0:t1, g].double()
            assert torch.isnan(got).all(-1).equal(nan) and torch.isnan(got).any(-1).equal(nan), (r, h)
            assert torch.isnan(gz).equal(nan), (r, h)
            fine = ~nan
            ratio = ((got - o).abs() / scores.out_bound(o, absv, pev, pe, made.dtype, n))[fine]
            assert ratio.numel() == 0 or float(ratio.max()) <= 1, (r, h, float(ratio.max()))
            ratio = ((gz - z).abs() / scores.lse_bound(z, pe, n))[fine]
            assert ratio.numel() == 0 or float(ratio.max()) <= 1, (r, h, float(ratio.max()))
        t0 = t1
