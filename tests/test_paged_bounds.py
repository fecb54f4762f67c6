"""The bound that the few-rows kernels' outputs are held to tells weights in two 16-bit parts from
weights in one: shown on the formula itself (no GPU needed)."""
import pytest


@pytest.mark.parametrize("dtype,d,n", [("bf16", 128, 20), ("bf16", 64, 20), ("bf16", 128, 200),
                                       ("fp16", 128, 20), ("fp16", 64, 20)])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_one_part_weights_exceed_the_two_part_bound(dtype, d, n, seed):
    import torch
    from tests import paged
    dt = paged.DTYPES[dtype]
    q, K, V, scale = paged.cancelling(n, 0, d, dt, seed)
    o, _, _, absv, logit = paged.attend_unit(q.double().view(1, 1, d), K.double(), V.double(), 0, 0,
                                             scale)
    s = scale * (K.double() @ q.double())
    p = torch.exp(s - s.max())
    high = p.to(dt).double()
    low = (p - high).to(dt).double()
    bound = paged.out_bound(o, absv, dt, d, n, logit, 2)[0, 0]
    for parts, weights in ((1, high), (2, high + low)):
        got = ((weights @ V.double()) / p.sum()).to(dt).double()
        worst = float(((got - o[0, 0]).abs() / bound).max())
        assert (worst > 1.5) if parts == 1 else (worst <= 1), (parts, worst)
