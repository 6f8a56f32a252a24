"""Rotary positions' angles at the ends of the positions' range, for frequencies of either sign and
any size, against angles reduced in whole numbers."""
from fractions import Fraction

import pytest
import torch

import embedding_columns_amd as E
import encoder_reference as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# 2 pi to 60 digits
TURN = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)
FREQUENCIES = [0.0, 0.7, 1e-3, 1e-5, 1e-12, 1e-16, 3e-16, 1e-20, 3.3e-16, 123.456, 6.283185307179586, 1e6, 1e9, 999999999.9]
ENDS = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 20, -2 ** 20, 2 ** 30 + 12345]


def angles(pos, freq):
    """Angles within one turn, exact before they become doubles."""
    t = [[float((Fraction(f) * p) % TURN) for f in freq] for p in pos]
    return torch.tensor(t, dtype=torch.float64)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_far_positions(sign, layout, dtype):
    """The angle's own rounding to fp32 (up to pi / 4: 5e-8) and the sine's and cosine's are 1e-7,
    two products and a sum follow."""
    gen = torch.Generator().manual_seed(41)
    freq = [sign * f for f in FREQUENCIES]
    pos = ENDS + torch.randint(-2 ** 31, 2 ** 31, (40,), generator=gen).tolist()
    pairs = len(freq)
    x = torch.randn(len(pos), 2, 2 * pairs, generator=gen).to(dtype)
    f = torch.tensor(freq, dtype=torch.float64, device="cuda")
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    q = x.cuda().requires_grad_()
    y, _ = E.rotary(q, None, p, None, f, layout)
    back, = torch.autograd.grad(y, q, q.detach())
    t = angles(pos, freq)[:, None]
    i = torch.arange(pairs)
    at, bt = (i, i + pairs) if layout == "half" else (2 * i, 2 * i + 1)
    a, b = x[..., at].double(), x[..., bt].double()
    for got, s in ((y.detach(), 1.0), (back, -1.0)):
        want = torch.empty_like(x, dtype=torch.float64)
        want[..., at] = a * t.cos() - s * b * t.sin()
        want[..., bt] = b * t.cos() + s * a * t.sin()
        bound = torch.empty_like(want)
        bound[..., at] = bound[..., bt] = (1e-7 + 4 * R.E32) * (a.abs() + b.abs())
        off = (got.cpu().double() - want).abs()
        bound += R.unit(dtype) * want.abs()
        assert (off <= bound).all(), float((off / bound).max())


def test_a_negative_frequency_turns_back():
    """To the bit what the negative position turns."""
    gen = torch.Generator().manual_seed(42)
    q = torch.randn(50, 1, 2 * len(FREQUENCIES), generator=gen).cuda()
    p = torch.randint(-2 ** 31 + 1, 2 ** 31, (50,), generator=gen).int().cuda()
    f = torch.tensor(FREQUENCIES, dtype=torch.float64, device="cuda")
    assert torch.equal(E.rotary(q, None, p, None, -f)[0], E.rotary(q, None, -p, None, f)[0])
