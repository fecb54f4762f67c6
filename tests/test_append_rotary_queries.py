"""kv_paged_append_rotary takes queries and a place for them, or neither (no GPU needed)."""
import pytest


@pytest.mark.parametrize("given", ["q", "q_out"])
def test_queries_without_a_place_or_the_reverse(given):
    import torch
    import kv_cache_eviction_split_gb300 as kv
    kv.build()
    kv.load()
    c = kv.PagedCache.allocate(2, 1, 2, 8, 128, 100, 64, torch.bfloat16, device="cpu")
    t = kv.Chunk([1, 5], device="cpu")
    q, k = (torch.zeros((6, h, 128), dtype=torch.bfloat16) for h in (8, 2))
    both = {"q": None, "q_out": None, given: q}
    with pytest.raises(ValueError, match="q and q_out"):
        kv.kv_paged_append_rotary(c, t, 0, kv.Rotary.make(64, device="cpu"), torch.zeros(6, dtype=torch.int32),
                                  both["q"], both["q_out"], k, k)
