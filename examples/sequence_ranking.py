"""Ranking candidates against a user's behaviour sequence, end to end: the embedding
stage looks up the rows of behaviours and candidates, the gated recurrence makes states
of the behaviours, candidates attend to them with a bias by elapsed time, and a logistic
loss trains everything, the tables by the stage's own sparse Adagrad.  Afterwards the
same model serves one new event and one candidate at a time.

    python examples/sequence_ranking.py [--steps N]

Synthetic data: a candidate is clicked iff it equals an item of the last hour.
Needs the GPU and the built library; prints the loss and how many are told right."""
import argparse
import os
import sys
from types import SimpleNamespace

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import embedding_columns_amd as E  # noqa: E402

ITEMS, DIM, HEADS, BUCKETS = 64, 64, 2, 16


def batch(samples, gen, dev):
    """Jagged behaviours (item, time) and candidates (item, time, label) of `samples` users."""
    k_len = torch.randint(0, 60, (samples,), generator=gen)
    q_len = torch.randint(1, 8, (samples,), generator=gen)
    ko = torch.cat([torch.zeros(1, dtype=torch.long), k_len.cumsum(0)])
    qo = torch.cat([torch.zeros(1, dtype=torch.long), q_len.cumsum(0)])
    items = torch.randint(0, ITEMS, (int(ko[-1]),), generator=gen)
    cands = torch.randint(0, ITEMS, (int(qo[-1]),), generator=gen)
    k_pos, label = torch.zeros(len(items), dtype=torch.int32), torch.zeros(len(cands))
    q_pos = torch.full((len(cands),), 100_000, dtype=torch.int32)
    for b in range(samples):
        n = int(k_len[b])
        rows = slice(int(ko[b]), int(ko[b + 1]))
        k_pos[rows] = torch.sort(100_000 - torch.randint(1, 40_000, (n,), generator=gen)).values.int()
        recent = items[rows][k_pos[rows] > 100_000 - 3600]
        for i in range(int(qo[b]), int(qo[b + 1])):
            if len(recent) and torch.rand((), generator=gen) < 0.5:
                cands[i] = recent[int(torch.randint(0, len(recent), (), generator=gen))]
            label[i] = float((recent == cands[i]).any())
    return SimpleNamespace(items=items.to(dev), cands=cands.to(dev), k_pos=k_pos.to(dev),
                           q_pos=q_pos.to(dev), label=label.to(dev), ko=ko.int().to(dev),
                           qo=qo.int().to(dev))


class Ranker(torch.nn.Module):
    def __init__(self, dev, most):
        super().__init__()
        column = SimpleNamespace(kind=E.IDENTITY, pool=E.SUM, dtype=E.F32, dim=DIM, rows=ITEMS,
                                 id_lo=0, id_hi=ITEMS)
        self.table = 0.5 * torch.randn(ITEMS, DIM, device=dev)
        self.stage = E.EmbeddingColumns([column], [self.table], [torch.zeros_like(self.table)],
                                        batch=most, max_ids=most, opt=E.OPT_ADAGRAD, lr=0.02,
                                        eps=1e-8, device=dev)
        self.most = most
        make = {"device": dev}
        self.gates = torch.nn.Linear(DIM, 2 * DIM, **make)      # the recurrence's x and gate
        self.keys = torch.nn.Linear(2 * DIM, 2 * DIM, **make)   # attention's k and v
        self.query = torch.nn.Linear(DIM, DIM, **make)
        self.score = torch.nn.Linear(2 * DIM, 1, **make)
        self.bias = torch.nn.Parameter(torch.zeros(BUCKETS, HEADS, **make))
        self.boundaries = (60 * 1.6 ** torch.arange(BUCKETS - 1, device=dev)).int()

    def rows(self, ids):
        """One row an id: bags of one, and empty ones up to the stage's batch."""
        n = ids.numel()
        offsets = torch.arange(self.most + 1, dtype=torch.int32, device=ids.device).clamp(max=n)
        return self.stage(offsets, ids=ids)[:n]

    def encode(self, rows, offsets):
        x, gate = self.gates(rows).split(DIM, dim=1)
        states, last = E.gated_recurrence(x, gate, offsets)
        return self.key_values(rows, states), last

    def key_values(self, rows, states):
        k, v = self.keys(torch.cat([rows, states], 1)).split(DIM, dim=1)
        return k.view(-1, HEADS, DIM // HEADS), v.view(-1, HEADS, DIM // HEADS)

    def rank(self, cand_rows, qo, q_pos, kv, ko, k_pos):
        q = self.query(cand_rows).view(-1, HEADS, DIM // HEADS)
        read = E.cross_attention(q, kv[0], kv[1], qo, ko, bias=self.bias, boundaries=self.boundaries,
                                 q_pos=q_pos, k_pos=k_pos).reshape(-1, DIM)
        return self.score(torch.cat([read * cand_rows, read], 1))[:, 0]

    def forward(self, b):
        n = b.items.numel()
        rows = self.rows(torch.cat([b.items, b.cands]))     # one lookup, one update of the table
        kv, _ = self.encode(rows[:n], b.ko)
        return self.rank(rows[n:], b.qo, b.q_pos, kv, b.ko, b.k_pos)


def main(steps=300, samples=128, quiet=False):
    dev = torch.device("cuda")
    torch.manual_seed(1)
    gen = torch.Generator().manual_seed(2)
    model = Ranker(dev, most=samples * 70)
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    for step in range(steps):
        b = batch(samples, gen, dev)
        loss = torch.nn.functional.binary_cross_entropy_with_logits(model(b), b.label)
        opt.zero_grad()
        loss.backward()
        opt.step()
        if not quiet and (step % 50 == 0 or step == steps - 1):
            print(f"step {step}: loss {loss.item():.3f}", flush=True)
    b = batch(samples, gen, dev)
    with torch.no_grad():
        right = float(((model(b) > 0) == (b.label > 0.5)).float().mean())
        # serving: a stored state takes one event, one candidate reads the longer sequence
        rows = model.rows(b.items)
        kv, last = model.encode(rows, b.ko)
        event = torch.randint(0, ITEMS, (samples,), generator=gen).to(dev)
        event_rows = model.rows(event)
        x, gate = model.gates(event_rows).split(DIM, dim=1)
        state = last.clone()
        states = E.gated_recurrence_step(x, gate, state)
        new_kv = model.key_values(event_rows, states)
        ends = b.ko[1:].long()
        at = torch.arange(samples, device=dev)
        spots = torch.ones(len(b.items) + samples, dtype=torch.bool, device=dev)
        spots[ends + at] = False

        def grown(old, new):
            t = new.new_empty((len(spots),) + new.shape[1:])
            t[spots], t[~spots] = old, new
            return t
        ko = (b.ko + torch.arange(samples + 1, device=dev)).int()
        one = torch.arange(samples + 1, dtype=torch.int32, device=dev)
        now = torch.full((samples,), 100_000, dtype=torch.int32, device=dev)
        scores = model.rank(event_rows, one, now, [grown(o, n) for o, n in zip(kv, new_kv)], ko,
                            grown(b.k_pos, now - 30))
    repeat = float((scores > 0).float().mean())
    if not quiet:
        print(f"told right: {right:.3f}; repeats of a served event called clicks: {repeat:.3f}")
    return loss.item(), right, repeat


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=300)
    main(ap.parse_args().steps)
