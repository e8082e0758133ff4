"""The arithmetic that the 8-bit cache's attention relies on for its weights."""
import pytest

torch = pytest.importorskip("torch")


def test_three_e5m2_parts_hold_every_weight():
    """fp16 from 0 to 2^15: the nearest code, 16 times the rest, 16 times the rest of that, nothing left."""
    h = torch.arange(0x7801, dtype=torch.int32).to(torch.int16).view(torch.float16)
    assert h[-1] == 2.0 ** 15
    left, held = h, torch.zeros(h.shape, dtype=torch.float64)
    for k in range(3):
        code = left.to(torch.float8_e5m2)
        half = (code.view(torch.uint8).to(torch.int16) << 8).view(torch.float16)      # a code is its half float's upper byte
        assert torch.equal(half, code.to(torch.float16))
        held += half.double() / 16.0 ** k
        left = (left - half) * 16
        assert left.abs().max() <= 2.0 ** 15
    assert torch.equal(held, h.double())
