"""What the sequence operators' autograd nodes hand to the library, on the CPU: the library's
calls are recorded instead of made."""
import pytest
import torch
import torch.utils.checkpoint

import embedding_columns_amd as E


class Calls:
    """Stands in for the library: keeps every call's arguments, a copy of its descriptor first."""

    def __init__(self):
        self.made = []

    def __getattr__(self, name):
        def call(desc, *args):
            if hasattr(desc, "_obj"):
                desc = type(desc._obj).from_buffer_copy(desc._obj)
            self.made.append((name, desc, args))
            if name == "emb_recurrence_query":
                args[0]._obj.value = 4
            return 0
        return call

    def last(self, name):
        return [(desc, args) for n, desc, args in self.made if n == name][-1]


@pytest.fixture
def calls(monkeypatch):
    made = Calls()
    monkeypatch.setattr(E, "lib", lambda: made)
    monkeypatch.setattr(E, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(E, "_rows_ptr", lambda t, ndim: t.data_ptr())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)     # a CPU tensor's device index
    return made


def attention():
    i32 = torch.int32
    d = dict(q=torch.randn(3, 2, 8), k=torch.randn(5, 1, 8), v=torch.randn(5, 1, 8),
             q_offsets=torch.tensor([0, 3], dtype=i32), k_offsets=torch.tensor([0, 5], dtype=i32),
             mask=torch.ones(5, dtype=torch.bool), bias=torch.randn(3, 2),
             boundaries=torch.tensor([-1, 1], dtype=i32), q_pos=torch.zeros(3, dtype=i32),
             k_pos=torch.zeros(5, dtype=i32))
    for name in ("q", "k", "v", "bias"):
        d[name].requires_grad_()
    return d


def recurrence():
    d = dict(x=torch.randn(5, 4), gate=torch.randn(5, 4), state=torch.randn(1, 4),
             offsets=torch.tensor([0, 5], dtype=torch.int32), mask=torch.ones(5, dtype=torch.uint8))
    for name in ("x", "gate", "state"):
        d[name].requires_grad_()
    return d


class Moved:
    """Saved-tensor hooks that keep a copy and give another one back, as offloading does."""

    def __init__(self):
        self.given = []

    def __enter__(self):
        self.hooks = torch.autograd.graph.saved_tensors_hooks(lambda t: t.detach().clone(), self.unpack)
        self.hooks.__enter__()
        return self

    def __exit__(self, *args):
        self.hooks.__exit__(*args)

    def unpack(self, t):
        self.given.append(t.clone())
        return self.given[-1]


def test_attention_backward_reads_the_tensors_that_autograd_gives_back(calls):
    d = attention()
    with Moved() as moved:
        out = E.cross_attention(**d)
        out.sum().backward()
    desc, args = calls.last("emb_attention_backward")
    q, k, v, bias, qo, ko, mask, boundaries, q_pos, k_pos, out, lse = [t.data_ptr() for t in moved.given]
    assert (desc.q, desc.k, desc.v, desc.bias, desc.q_offsets, desc.k_offsets, desc.mask) == (
        q, k, v, bias, qo, ko, mask)
    assert (desc.boundaries, desc.q_pos, desc.k_pos) == (boundaries, q_pos, k_pos)
    assert args[0] == out and args[2] == lse


def test_recurrence_backward_reads_the_tensors_that_autograd_gives_back(calls):
    d = recurrence()
    with Moved() as moved:
        y, last = E.gated_recurrence(**d)
        (y.sum() + last.sum()).backward()
    desc, args = calls.last("emb_recurrence_backward")
    x, gate, state, offsets, mask, saved = [t.data_ptr() for t in moved.given]
    assert (desc.x, desc.gate, desc.state, desc.offsets, desc.mask) == (x, gate, state, offsets, mask)
    assert args[0] == saved


def test_strides_are_those_of_the_tensors_given_back(calls):
    """A hook may lay a tensor out anew: rows out of a wider one come back contiguous."""
    d = attention()
    wide = torch.randn(5, 1, 24, requires_grad=True)
    with Moved():
        E.cross_attention(**{**d, "k": wide[:, :, 8:16]}).sum().backward()
    assert calls.last("emb_attention_forward")[0].k_stride == 24
    assert calls.last("emb_attention_backward")[0].k_stride == 8
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: t.t().contiguous().t()
                                                  if t.shape == (5, 4) else t):
        y, _ = E.gated_recurrence(**recurrence())
        y.sum().backward()
    desc = calls.last("emb_recurrence_backward")[0]
    assert (desc.x_stride, desc.gate_stride) == (4, 4)


def test_checkpointed_blocks_read_what_was_recomputed(calls):
    d = attention()
    seen = []

    def block(q):
        q2 = q * 2
        seen.append(q2.data_ptr())
        keep.append(q2.detach())       # no address is used twice
        return E.cross_attention(**{**d, "q": q2})
    keep = []
    torch.utils.checkpoint.checkpoint(block, d["q"], use_reentrant=False).sum().backward()
    assert len(seen) == 2
    assert calls.last("emb_attention_backward")[0].q == seen[1]


def direction(t):
    return torch.ones_like(t)


def test_forward_mode_is_refused(calls):
    """No tangent is computed, so none may be lost without a word."""
    fw = torch.autograd.forward_ad
    for make, call, names in ((attention, E.cross_attention, ("q", "k", "v", "bias")),
                              (recurrence, E.gated_recurrence, ("x", "gate", "state"))):
        for name in names:
            for grad in (False, True):
                d = {n: t.detach().requires_grad_(grad and t.is_floating_point()) for n, t in make().items()}
                with fw.dual_level():
                    d[name] = fw.make_dual(d[name], direction(d[name]))
                    with pytest.raises(RuntimeError, match="forward"):
                        call(**d)
                    with torch.no_grad(), pytest.raises(RuntimeError, match="forward"):
                        call(**d)
                    d[name] = fw.unpack_dual(d[name]).primal
                    call(**d)                    # without a tangent it goes through
    x = torch.randn(3, 4)
    with fw.dual_level():
        for i in range(3):
            step = [x, x, x.clone()]
            step[i] = fw.make_dual(step[i], x)
            with pytest.raises(RuntimeError, match="forward"):
                E.gated_recurrence_step(*step)
        E.gated_recurrence_step(x, x, x.clone())


def test_forward_mode_through_a_backward_pass_is_refused(calls):
    fw = torch.autograd.forward_ad
    d, r = attention(), recurrence()
    out, (y, last) = E.cross_attention(**d), E.gated_recurrence(**r)
    with fw.dual_level():
        for outs, given, at in (([out], [torch.ones_like(out)], 0), ([y, last], [torch.ones_like(y), direction(last)], 0),
                                ([y, last], [torch.ones_like(y), direction(last)], 1)):
            given[at] = fw.make_dual(given[at], direction(given[at]))
            with pytest.raises(RuntimeError, match="forward"):
                torch.autograd.grad(outs, d["q"] if outs[0] is out else r["x"], given, retain_graph=True)


def test_function_transforms_do_not_go_through(calls):
    d = {n: t.detach() for n, t in attention().items()}

    def of_q(q):
        return E.cross_attention(**{**d, "q": q})
    for call in (lambda: torch.func.jvp(of_q, (d["q"],), (direction(d["q"]),)),
                 lambda: torch.func.grad(lambda q: of_q(q).sum())(d["q"]),
                 lambda: torch.func.vmap(of_q)(d["q"][None])):
        with pytest.raises(Exception):
            call()
    assert not any(name == "emb_attention_forward" for name, _, _ in calls.made)


def test_second_derivatives_are_refused(calls):
    out = E.cross_attention(**(d := attention()))
    with pytest.raises(RuntimeError, match="first derivatives"):
        torch.autograd.grad(out.sum(), d["q"], create_graph=True)
    y, _ = E.gated_recurrence(**(r := recurrence()))
    with pytest.raises(RuntimeError, match="first derivatives"):
        torch.autograd.grad(y.sum(), r["x"], create_graph=True)


def test_a_step_tells_autograd_that_it_writes(calls):
    """What a step overwrites, a graph that saved it may not use any more."""
    x, state, out, w = torch.randn(3, 4), torch.randn(3, 4), torch.zeros(3, 4), torch.ones(3, 4)
    w.requires_grad_()
    for saved in (state, out):
        graph = (w * saved).sum()
        E.gated_recurrence_step(x, x, state, out=out)
        with pytest.raises(RuntimeError, match="inplace"):
            graph.backward()
    versions = state._version, out._version
    E.gated_recurrence_step(x, x, state, out=out)
    assert (state._version, out._version) == (versions[0] + 1, versions[1] + 1)
    assert x._version == 0


def test_a_step_in_inference_mode(calls):
    """There tensors have no versions, and ordinary ones may be mixed in."""
    plain = torch.randn(3, 4)
    with torch.inference_mode():
        x, state = torch.randn(3, 4), torch.randn(3, 4)
        assert E.gated_recurrence_step(x, x, state).shape == (3, 4)
        E.gated_recurrence_step(x, x, plain, out=state)
    E.gated_recurrence_step(x, x, state, out=plain)
