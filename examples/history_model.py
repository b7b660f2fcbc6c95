"""A small model on users' event histories: table lookups, a gated recurrence over each history, a
linear layer for each domain, dropout.

    python examples/history_model.py [--steps 50] [--users 2048]

Each event is looked up as one row of 2 * dim values, the recurrence's input and gate.  A user's
last state goes through the linear layer of the user's domain (users are sorted by domain), whose
output is dropped out and added to the state.  Training runs the gradients back into the tables,
whose touched rows get one SGD update each; serving takes one new event of each user.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import table_embedding_bag_amd as tbe  # noqa: E402


def batch(users, rows, domains, dim, seed, device="cuda"):
    """Histories of 0 to 40 events, users sorted by domain, and what the model should answer."""
    g = np.random.default_rng(seed)
    lengths = g.integers(0, 41, users)
    sizes = g.multinomial(users, np.full(domains, 1.0 / domains))
    offsets = lambda n: torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).to(device)  # noqa: E731
    return {"ids": torch.from_numpy(g.integers(0, rows, int(lengths.sum()))).to(device),
            "histories": offsets(lengths), "domains": offsets(sizes),
            "target": torch.from_numpy(g.standard_normal((users, dim))).float().to(device)}


class HistoryModel:
    def __init__(self, rows, dim, domains, p=0.1, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        randn = lambda *n: torch.randn(*n, generator=g, device=device)  # noqa: E731
        self.dim, self.p, self.seed, self.offset = dim, p, seed, 0
        self.table = randn(rows * 2 * dim)
        self.tables = tbe.TBE([rows], [2 * dim], self.table)
        self.weight = randn(domains, dim, dim) * dim ** -0.5
        self.bias = torch.zeros(domains, dim, device=device)

    def _events(self, ids):
        """The rows of the events, and their halves: input and gate."""
        n = ids.numel()
        one_each = torch.arange(n + 1, device=ids.device)
        rows = self.tables.forward(n, ids, one_each)
        return one_each, rows[:, :self.dim], rows[:, self.dim:]

    def loss_and_update(self, b, lr):
        """The mean squared error of a batch; the parameters take one SGD step down its gradient."""
        one_each, x, gate = self._events(b["ids"])
        _, last, carry = tbe.scan_forward(x, gate, b["histories"])
        y = tbe.grouped_linear(last, self.weight, b["domains"], bias=self.bias)
        out = tbe.dropout(y, self.p, self.seed, self.offset, residual=last)
        error = out - b["target"]

        dout = error * (2 / error.numel())
        dy = tbe.dropout_backward(dout, self.p, self.seed, self.offset)
        dlast, dweight, dbias = tbe.grouped_linear_backward(last, self.weight, b["domains"], dy, bias=True)
        drows = torch.empty(x.shape[0], 2 * self.dim, device=x.device)
        tbe.scan_backward(x, gate, b["histories"], carry, grad_final=dlast.add_(dout),
                          out=(drows[:, :self.dim], drows[:, self.dim:]))
        self.tables.backward_update(x.shape[0], b["ids"], one_each, None, drows, lr)
        self.weight.sub_(dweight, alpha=lr)
        self.bias.sub_(dbias, alpha=lr)
        self.offset += (out.numel() + 3) // 4
        return error.square().mean()

    def states(self, ids, histories):
        """Every user's state after a whole history."""
        _, x, gate = self._events(ids)
        return tbe.scan_forward(x, gate, histories, need_carry=False)[1]

    def serve(self, ids, state, domains):
        """One new event of each user: the answers; state is brought up to date in place."""
        _, x, gate = self._events(ids)
        last, _ = tbe.scan_step(x, gate, state, out_state=state)
        return tbe.grouped_linear(last, self.weight, domains, bias=self.bias).add_(last)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--users", type=int, default=2048)
    a = ap.parse_args()
    rows, dim, domains = 10000, 128, 8
    model = HistoryModel(rows, dim, domains)
    b = batch(a.users, rows, domains, dim, seed=1)
    for step in range(a.steps):
        loss = model.loss_and_update(b, lr=0.2 * b["target"].numel() / a.users)
        if step % 10 == 0 or step == a.steps - 1:
            print(f"step {step}: loss {loss.item():.4f}", flush=True)
    state = model.states(b["ids"], b["histories"])
    events = torch.randint(rows, (a.users,), device="cuda")
    print("served", tuple(model.serve(events, state, b["domains"]).shape))


if __name__ == "__main__":
    main()
