"""The gated delta rule's backward on saved tensors that lie otherwise than the forward's did."""
import pytest
import torch

from test_gpu_delta import BF16, F32, call, make

pytestmark = pytest.mark.gpu


class Shifted:
    """Saved tensors come back at addresses that no 16 bytes divide, and forth."""

    def __init__(self, by):
        self.by = by

    def pack(self, t):
        return t.clone()

    def unpack(self, t):
        if t.dtype not in (F32, BF16) or t.dim() < 2:
            return t
        room = t.new_empty(t.numel() + self.by)
        room[self.by:] = t.reshape(-1)
        return room[self.by:].view(t.shape)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("by", [0, 1])
@pytest.mark.parametrize("unaligned", [False, True])
def test_other_places(unaligned, by, dtype):
    t = make([100, 33], 2, 4, 64, 32, dtype, masked=0.1, seed=61)
    want = call(t)
    if unaligned:
        for x in ("q", "k", "v", "do"):
            wide = torch.zeros(t[x].shape[:2] + (t[x].shape[2] + 1,), dtype=dtype, device="cuda")
            wide[..., 1:] = t[x]
            t[x] = wide[..., 1:]
    hooks = Shifted(by)
    with torch.autograd.graph.saved_tensors_hooks(hooks.pack, hooks.unpack):
        got = call(t)
    for name in want:
        assert torch.equal(got[name], want[name]), name
