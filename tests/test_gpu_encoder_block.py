"""Layer norm, rotary positions and the gated delta rule one after another, as a block of a
sequence encoder uses them: every stage of the run against the 64-bit form of that stage, from
what the stage was given and what came back to it, and what autograd, streams and graphs do to them."""
import importlib.util
import os

import pytest
import torch
import torch.utils.checkpoint

import embedding_columns_amd as E
import encoder_reference as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KH, H, DK, DV, C = 2, 4, 32, 24, 72


def make(dtype, lens=(40, 0, 1, 95), seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = 2 + sum(lens) + 1                                # rows of no sample before and behind

    def randn(*s):
        return torch.randn(*s, generator=gen).cuda()
    leaves = {"x": randn(n, C).to(dtype), "w": 1 + 0.1 * randn(C), "b": 0.1 * randn(C),
              "weight": randn(C, 2 * KH * DK + H * DV + 2 * H) / C ** 0.5, "state": 0.3 * randn(len(lens), H, DK, DV),
              "w2": 1 + 0.1 * randn(DV), "b2": 0.1 * randn(DV)}
    rest = {"offsets": torch.tensor([2] + list(lens)).cumsum(0).int().cuda(),
            "mask": (torch.rand(n, generator=gen) < 0.9).cuda(),
            "pos": torch.randint(0, 1 << 30, (n,), generator=gen).int().cuda(),
            "f": E.rotary_frequencies(DK - 8), "dz": randn(n, H, DV).to(dtype), "dlast": randn(len(lens), H, DK, DV)}
    return leaves, rest


def block(leaves, rest):
    """Every tensor that one of the operators made or was given."""
    t = dict(leaves)
    dtype = t["x"].dtype
    t["y"] = E.layer_norm(t["x"], t["w"], t["b"])
    made = (t["y"].float() @ t["weight"]).to(dtype)
    q, k, v, gate, beta = made.split([KH * DK, KH * DK, H * DV, H, H], dim=1)
    t["q"], t["v"] = q.unflatten(1, (KH, DK)), v.unflatten(1, (H, DV))
    t["k"] = torch.nn.functional.normalize(k.unflatten(1, (KH, DK)).float(), dim=-1).to(dtype)
    t["gate"], t["beta"] = gate + 2, beta
    t["tq"], t["tk"] = E.rotary(t["q"], t["k"], rest["pos"], rest["pos"], rest["f"])
    t["o"], t["last"] = E.gated_delta(t["tq"], t["tk"], t["v"], t["gate"], t["beta"], rest["offsets"], t["state"],
                                      rest["mask"])
    t["z"] = E.layer_norm(t["o"], t["w2"], t["b2"])
    return t


def run(leaves, rest, keep=False):
    leaves = {x: t.detach().requires_grad_() for x, t in leaves.items()}
    t = block(leaves, rest)
    if keep:
        for x in t.values():
            if not x.is_leaf:
                x.retain_grad()
    torch.autograd.backward([t["z"], t["last"]], [rest["dz"], rest["dlast"]])
    return t


def grads(t):
    return {x: t[x].grad for x in ("x", "w", "b", "weight", "state", "w2", "b2")}


def near(got, ref, name):
    val, bound = ref
    off = (got.detach().cpu().double() - val).abs()
    assert got.shape == val.shape and (off <= bound).all(), (name, float((off / bound).max()))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_every_stage(dtype):
    leaves, rest = make(dtype)
    t = run(leaves, rest, keep=True)
    for x, w, b, y in (("x", "w", "b", "y"), ("o", "w2", "b2", "z")):
        ref = R.layer_norm(t[x], t[w], t[b], 1e-5, t[y].grad)
        near(t[y], ref["y"], y)
        near(t[x].grad, ref["dx"], "d" + x)
        near(t[w].grad, ref["dweight"], "d" + w)
        near(t[b].grad, ref["dbias"], "d" + b)
    for x, y in (("q", "tq"), ("k", "tk")):
        near(t[y], R.rotary(t[x], rest["pos"], rest["f"]), y)
        near(t[x].grad, R.rotary(t[y].grad, rest["pos"], rest["f"], back=True), "d" + x)
    ref = R.delta(*(t[x] for x in ("tq", "tk", "v", "gate", "beta")), rest["offsets"], t["state"], rest["mask"], None,
                  t["o"].grad, rest["dlast"])
    near(t["o"], ref["o"], "o")
    near(t["last"], ref["last"], "last")
    for x, d in (("tq", "dq"), ("tk", "dk"), ("v", "dv"), ("gate", "dgate"), ("beta", "dbeta"), ("state", "dstate")):
        near(t[x].grad, ref[d], d)


def test_each_gradient_alone():
    """What else is wanted changes no gradient."""
    leaves, rest = make(BF16, seed=1)
    want = grads(run(leaves, rest))
    for x in leaves:
        one = {y: t.detach().requires_grad_(y == x) for y, t in leaves.items()}
        t = block(one, rest)
        outs = [(t["z"], rest["dz"]), (t["last"], rest["dlast"])]
        outs = [(o, d) for o, d in outs if o.requires_grad]
        got, = torch.autograd.grad([o for o, _ in outs], [one[x]], [d for _, d in outs])
        assert torch.equal(got, want[x]), x


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_recomputed_and_offloaded(dtype):
    """Activation checkpointing and saved tensors kept on the host give the same bits."""
    leaves, rest = make(dtype, seed=2)
    want = grads(run(leaves, rest))
    with torch.autograd.graph.save_on_cpu():
        got = grads(run(leaves, rest))
    for x in want:
        assert torch.equal(got[x], want[x]), x
    names = list(leaves)
    ins = [leaves[x].detach().requires_grad_() for x in names]

    def out(*ins):
        t = block(dict(zip(names, ins)), rest)
        return t["z"], t["last"]
    z, last = torch.utils.checkpoint.checkpoint(out, *ins, use_reentrant=False)
    for x, g in zip(names, torch.autograd.grad([z, last], ins, [rest["dz"], rest["dlast"]])):
        assert torch.equal(g, want[x]), x


def test_other_streams():
    """Calls on two streams at once, each with scratch memory of its own."""
    leaves, rest = make(BF16, lens=(700, 300), seed=3)
    other, rest2 = make(BF16, lens=(5, 900, 64), seed=4)
    want, want2 = grads(run(leaves, rest)), grads(run(other, rest2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            got2 = grads(run(other, rest2))
        got = grads(run(leaves, rest))
        torch.cuda.synchronize()
        for x in want:
            assert torch.equal(got[x], want[x]) and torch.equal(got2[x], want2[x]), x


def test_two_captured_blocks():
    """Two captured steps of training, replayed in turn and with eager work between."""
    cases = [make(BF16, lens=(64, 33), seed=5), make(BF16, lens=(3, 128), seed=6)]
    side = torch.cuda.Stream()
    graphs = []
    for leaves, rest in cases:
        ins = {x: t.clone() for x, t in leaves.items()}
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            run(ins, rest)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run(ins, rest)
        graphs.append((graph, ins, {**grads(got), "z": got["z"], "last": got["last"]}))
    for i in range(3):
        others = [make(BF16, lens=lens, seed=10 * i + 7)[0] for lens in ((64, 33), (3, 128))]
        for (graph, ins, _), new in zip(graphs, others):
            for x in ins:
                ins[x].copy_(new[x])
            graph.replay()
        for (_, _, got), new, (_, rest) in zip(graphs, others, cases):
            eager = run(new, rest)
            torch.cuda.synchronize()
            for x, t in {**grads(eager), "z": eager["z"], "last": eager["last"]}.items():
                assert torch.equal(got[x], t), x


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,c", [(8300, 1030), (1400, 1100), (800, 3000), (300, 16384), (35000, 9), (9000, 1000)])
def test_more_rows_than_a_round_of_workgroups(rows, c, dtype):
    """Layer norm's workgroups take several rows one after another."""
    gen = torch.Generator().manual_seed(rows)
    x, dy = ((torch.randn(rows, c, generator=gen) + 0.5).to(dtype).cuda() for _ in range(2))
    w, b = torch.randn(c, generator=gen).cuda(), torch.randn(c, generator=gen).cuda()
    leaves = [t.detach().requires_grad_() for t in (x, w, b)]
    y = E.layer_norm(*leaves)
    ref = R.layer_norm(x, w, b, 1e-5, dy)
    near(y, ref["y"], "y")
    for name, g in zip(("dx", "dweight", "dbias"), torch.autograd.grad(y, leaves, dy)):
        near(g, ref[name], name)


def example():
    spec = importlib.util.spec_from_file_location("sequence_ranking",
                                                  os.path.join(ROOT, "examples", "sequence_ranking.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_ranking_example_runs_with_a_matrix_state():
    loss, right, repeat = example().main(steps=3, quiet=True, encoder="delta")
    assert all(x == x and abs(x) < 1e3 for x in (loss, right, repeat))


def test_the_ranking_examples_gradients():
    """Along the gradient and a random direction together, against differences of the loss.  A loss
    is off by 2^-24 of the logits' size (about 1) for each of some 300 steps of arithmetic that
    lead to it, and a difference by that over its step; what a difference leaves out falls with
    the step's square, so that the two steps' differ by three times what the smaller leaves out."""
    module = example()
    dev = torch.device("cuda")
    torch.manual_seed(3)
    gen = torch.Generator().manual_seed(4)
    model = module.DeltaRanker(dev, most=16 * 70)
    b = module.batch(16, gen, dev)
    n = b.items.numel()
    with torch.no_grad():
        rows = model.rows(torch.cat([b.items, b.cands])).clone()
    params = list(model.parameters())

    def loss():
        kv, _ = model.encode(rows[:n], b.ko, b.k_pos)
        scores = model.rank(rows[n:], b.qo, b.q_pos, kv, b.ko, b.k_pos)
        return torch.nn.functional.binary_cross_entropy_with_logits(scores.double(), b.label.double())
    grad = torch.autograd.grad(loss(), params)
    step = 0.05
    rounding = 300 * 2.0 ** -24 / step
    for p, g in zip(params, grad):
        assert torch.isfinite(g).all()
        way = torch.randn(p.shape, generator=gen).to(dev)
        way = way / way.norm() + g / g.norm().clamp(min=1e-30)
        slopes = []
        start = p.detach().clone()
        with torch.no_grad():
            for s in (2 * step, step):
                p.copy_(start + s * way)
                up = loss()
                p.copy_(start - s * way)
                slopes.append(((up - loss()) / (2 * s)).item())
            p.copy_(start)
        slope = (4 * slopes[1] - slopes[0]) / 3
        off = abs((g * way).double().sum().item() - slope)
        assert off <= abs(slopes[0] - slopes[1]) + 2 * rounding, (p.shape, off, slopes)
