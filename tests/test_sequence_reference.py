"""The 64-bit forms that the GPU tests compare with, against torch's own differentiation of
the definitions (CPU, float64)."""
import torch

import sequence_reference as ref


def offsets(lengths):
    return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32)


def test_attention_gradients_are_those_of_its_definition():
    gen = torch.Generator().manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64)

    q_len, k_len = [3, 0, 4], [5, 2, 6]
    q, k, v, dout = normal(7, 4, 8), normal(13, 2, 8), normal(13, 2, 8), normal(7, 4, 8)
    bias, boundaries = normal(4, 4), torch.tensor([-3, 0, 5], dtype=torch.int32)
    q_pos, k_pos = torch.arange(7, dtype=torch.int32), torch.arange(13, dtype=torch.int32) - 4
    mask = torch.ones(13, dtype=torch.uint8)
    mask[[1, 8]] = 0
    args = dict(mask=mask, bias=bias, boundaries=boundaries, q_pos=q_pos, k_pos=k_pos)
    got = ref.attention(q, k, v, offsets(q_len), offsets(k_len), dout=dout, **args)
    for t in (q, k, v, bias):
        t.requires_grad_()
    qo, ko, outs = offsets(q_len).tolist(), offsets(k_len).tolist(), []
    for b in range(3):
        for i in range(qo[b], qo[b + 1]):
            for h in range(4):
                score, value = [], []
                for j in range(ko[b], ko[b + 1]):
                    if mask[j]:
                        m = int((boundaries <= q_pos[i] - k_pos[j]).sum())
                        score.append(q[i, h] @ k[j, h // 2] * 8 ** -0.5 + bias[m, h])
                        value.append(v[j, h // 2])
                outs.append(torch.softmax(torch.stack(score), 0) @ torch.stack(value))
    out = torch.stack(outs).view(7, 4, 8)
    grads = torch.autograd.grad(out, (q, k, v, bias), dout)
    for name, want in zip(("out", "dq", "dk", "dv", "dbias"), (out,) + grads):
        assert torch.allclose(got[name][0], want, rtol=1e-12, atol=1e-13), name


def test_recurrence_gradients_are_those_of_its_definition():
    gen = torch.Generator().manual_seed(2)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64)

    lengths = [4, 0, 5]
    x, gate, state, dy, dlast = normal(9, 3), normal(9, 3), normal(3, 3), normal(9, 3), normal(3, 3)
    mask = torch.ones(9, dtype=torch.uint8)
    mask[[2, 8]] = 0
    got = ref.recurrence(x, gate, offsets(lengths), state=state, mask=mask, dy=dy, dlast=dlast)
    for t in (x, gate, state):
        t.requires_grad_()
    off, ys, last = offsets(lengths).tolist(), [], []
    for b in range(3):
        h = state[b]
        for t in range(off[b], off[b + 1]):
            a = torch.sigmoid(gate[t])
            h = a * h + (1 - a) * x[t] if mask[t] else h
            ys.append(h)
        last.append(h)
    y, last = torch.stack(ys), torch.stack(last)
    grads = torch.autograd.grad([y, last], (x, gate, state), [dy, dlast])
    for name, want in zip(("y", "last", "dx", "dgate", "dstate"), (y, last) + grads):
        assert torch.allclose(got[name][0], want, rtol=1e-12, atol=1e-13), name
