"""What the page-keeping calls leave where there is nothing to keep."""
import pytest

pytestmark = pytest.mark.gpu


def test_a_cache_without_requests_has_no_live_pages(cuda_lib):
    import torch
    kv = cuda_lib
    c = kv.PagedCache.allocate(0, 1, 2, 2, 64, 10, refs=True)
    ws = torch.empty(kv.kv_paged_compact_workspace_size(c), dtype=torch.uint8, device="cuda")
    live = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    kv.kv_paged_compact(c, ws, live=live)
    assert int(live) == 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        kv.kv_paged_compact(c, ws, live=live)
    live.fill_(7)
    g.replay()
    assert int(live) == 0
