"""Rows turned by frequencies that a caller brings: above 1, negative, tiny; near and far positions."""
import pytest

pytestmark = pytest.mark.gpu

FREQUENCIES = [1000.0, -1000.0, 3.5, -0.75, 1.0, 1e-9, 0.0, 123456.789]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("first", [0, 5000, 1 << 24, (1 << 31) - 64, -(1 << 31)])
def test_any_frequency(cuda_lib, first, interleaved):
    """An angle is off by 2^-52 p w and 2^-23 (tests/test_gpu_rotary.py's bound), and so by that of its own
    frequency; the reference's product of 64 bits by 2^-53 p w."""
    import torch
    from tests.test_gpu_rotary import _bound, _turn64
    kv = cuda_lib
    freq = torch.tensor(FREQUENCIES, device="cuda")
    m = len(FREQUENCIES)
    rot = kv.Rotary(freq, 1.0, interleaved)
    pos = (first + torch.arange(64, device="cuda")).to(torch.int32)
    x = torch.randn((64, 3, 64), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    out = torch.empty_like(x)
    kv.kv_rotary(rot, pos, x, out)
    want, mag = _turn64(x.double(), pos, freq, 1.0, interleaved)
    assert torch.equal(out[..., 2 * m:], x[..., 2 * m:])
    for i in range(m):
        pair = [2 * i, 2 * i + 1] if interleaved else [i, i + m]
        own = _bound(want[..., pair], mag[..., pair], pos, freq[i:i + 1], x.dtype)
        far = 2.0 ** -53 * float(pos.double().abs().max()) * abs(FREQUENCIES[i])
        assert ((out[..., pair].double() - want[..., pair]).abs() <= own + 1.01 * far * mag[..., pair]).all(), i
