"""Scoring beside other kernels: copies on another stream share the SMs and the memory, and the
scores keep the bits of a quiet call."""
import pytest

import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rule", [0, 2], ids=["dropkv", "attn_sum"])
@pytest.mark.parametrize("wl", [
    synth.small_variant(synth.LONG_128K, 20003),     # two row chunks per unit
    synth.small_variant(synth.LLAMA8B_32K, 20003),   # one row chunk, alternate tiles
], ids=lambda w: w.name)
def test_scores_beside_copies(cuda_lib, wl, rule):
    import torch
    from synth.device import DeviceWorkload
    kv = cuda_lib
    dw = DeviceWorkload(wl)
    prob = kv.Problem.for_workload(wl, score_rule=rule)
    ws = torch.zeros(kv.kv_score_workspace_size(prob), dtype=torch.uint8, device="cuda")
    scores = torch.zeros((wl.num_layers, wl.num_kv_heads, dw.N_tot), dtype=torch.float32,
                         device="cuda")
    busy = torch.empty((2, 1 << 30), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    want = None
    for i in range(20):
        scores.fill_(-1.0)
        torch.cuda.synchronize()
        if want is not None:
            with torch.cuda.stream(side):
                for _ in range(3):
                    busy[0].copy_(busy[1])
        kv.kv_score(prob, dw.q, dw.k, dw.v, scores, ws)
        assert kv.kv_check_status(ws) == kv.KV_OK
        if want is None:
            want = scores.clone()
        assert torch.equal(scores, want), i
    torch.cuda.synchronize()                         # the copies end before their memory is free
