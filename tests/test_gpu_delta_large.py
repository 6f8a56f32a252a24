"""The gated delta rule over more than 2^25 rows times heads, read in place and packed: the samples at
the far end to the bit what they are by themselves."""
import pytest
import torch

import embedding_columns_amd as E

pytestmark = pytest.mark.gpu


def inputs(lens, heads, dk, dv):
    gen = torch.Generator(device="cuda").manual_seed(51)
    n = sum(lens)

    def randn(*s):
        return torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)
    k = randn(n, heads, dk)
    k.mul_(0.9 * dk ** -0.5)
    t = [randn(n, heads, dk), k, randn(n, heads, dv), randn(n, heads).add_(2), randn(n, heads)]
    return t, torch.tensor([0] + lens).cumsum(0).int().cuda()


def run(t, off, dv, train):
    if not train:
        return E.gated_delta(*t, off)
    leaves = [x.detach().requires_grad_() for x in t]
    o, last = E.gated_delta(*leaves, off)
    return (o.detach(), last.detach()) + torch.autograd.grad([o, last], leaves, [t[2], torch.ones_like(last)])


@pytest.mark.parametrize("rows,dk,dv,train", [(9_000_000, 32, 32, True), (34_000_000, 8, 8, False)])
def test_far_rows(rows, dk, dv, train):
    lens = [rows // 90] * 90 + [77, 1, 130]
    t, off = inputs(lens, 4, dk, dv)
    got = run(t, off, dv, train)
    cut = int(off[90])
    want = run([x[cut:] for x in t], off[90:] - cut, dv, train)
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a[90:] if i == 1 else a[cut:], b), i
