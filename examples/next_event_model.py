"""What comes next in users' event histories: table lookups, a gated recurrence over each history, layer
norm, experts chosen for each user, and the softmax loss over the rows of a table of events.

    python examples/next_event_model.py [--steps 50] [--users 2048]

A user's last state is normalised and sent to the two experts (linear layers) that a router chooses for
it; their outputs, weighted, are added to the state.  The result, normalised, is compared with every row
of the events' output table; the user's next event is the target (users without one are left out).
Training takes SGD steps; the expert choice is kept even by a bias that counts in the choice alone.
Serving gives every user's best next events.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import table_embedding_bag_amd as tbe  # noqa: E402


def batch(users, events, seed, device="cuda"):
    """Histories of 0 to 40 events and the event that follows each: the history's last one plus 1,
    mostly; -1 for users whose next event is not known."""
    g = np.random.default_rng(seed)
    lengths = g.integers(0, 41, users)
    ids = g.integers(0, events, int(lengths.sum()))
    offsets = np.concatenate([[0], np.cumsum(lengths)])
    target = g.integers(0, events, users)
    full = lengths > 0
    target[full] = (ids[offsets[1:][full] - 1] + 1) % events
    target[g.random(users) < 0.05] = -1
    to = lambda a: torch.from_numpy(a).to(device)  # noqa: E731
    return {"ids": to(ids), "histories": to(offsets), "target": to(target)}


class NextEventModel:
    def __init__(self, events, dim, experts, k=2, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        randn = lambda *n: torch.randn(*n, generator=g, device=device)  # noqa: E731
        self.dim, self.experts, self.k = dim, experts, k
        self.table = randn(events * 2 * dim)
        self.tables = tbe.TBE([events], [2 * dim], self.table)
        self.p = {"norm1": torch.ones(dim, device=device), "bias1": torch.zeros(dim, device=device),
                  "router": randn(1, experts, dim) * dim ** -0.5, "expert": randn(experts, dim, dim) * dim ** -0.5,
                  "norm2": torch.ones(dim, device=device), "bias2": torch.zeros(dim, device=device),
                  "events": randn(events, dim) * dim ** -0.5}
        self.balance = torch.zeros(experts, device=device)

    def _events(self, ids):
        """The rows of the events, and their halves: input and gate."""
        n = ids.numel()
        one_each = torch.arange(n + 1, device=ids.device)
        rows = self.tables.forward(n, ids, one_each)
        return one_each, rows[:, :self.dim], rows[:, self.dim:]

    def _answer(self, last):
        """What is compared with the events' rows, from the users' last states, and what the way back
        needs of the way there."""
        p = self.p
        x, stats1 = tbe.layer_norm(last, p["norm1"], p["bias1"])
        all_users = torch.tensor([0, last.shape[0]], device=last.device)
        logits = tbe.grouped_linear(x, p["router"], all_users)
        ids, weights = tbe.route(logits, self.k, scores="sigmoid", bias=self.balance)
        plan = tbe.dispatch_plan(ids, self.experts)
        rows = tbe.dispatch(x, plan)
        y = tbe.grouped_linear(rows, p["expert"], plan.offsets)
        z = tbe.combine(y, plan, weights, residual=last)
        out, stats2 = tbe.layer_norm(z, p["norm2"], p["bias2"])
        return out, (x, stats1, all_users, logits, ids, weights, plan, rows, y, z, stats2)

    def gradients(self, b):
        """The users' losses, the gradients of their mean by parameter and of the looked-up rows, and
        how many users each expert got."""
        p = self.p
        one_each, x0, gate = self._events(b["ids"])
        _, last, carry = tbe.scan_forward(x0, gate, b["histories"])
        out, (x, stats1, all_users, logits, ids, weights, plan, rows, y, z, stats2) = self._answer(last)
        loss, lse = tbe.softmax_loss(out, p["events"], b["target"])

        d = {}
        real = b["target"] >= 0
        each = real.float() / real.sum().clamp(min=1)
        dout, d["events"] = tbe.softmax_loss_backward(out, p["events"], b["target"], lse, each)
        dz, d["norm2"], d["bias2"] = tbe.layer_norm_backward(z, stats2, dout, weight=p["norm2"], bias=True)
        dy, dweights = tbe.combine_backward(y, plan, weights, dz)
        drows, d["expert"], _ = tbe.grouped_linear_backward(rows, p["expert"], plan.offsets, dy)
        dlogits = tbe.route_backward(logits, ids, dweights, scores="sigmoid")
        dx, d["router"], _ = tbe.grouped_linear_backward(x, p["router"], all_users, dlogits)
        dx.add_(tbe.dispatch_backward(drows, plan))
        dlast, d["norm1"], d["bias1"] = tbe.layer_norm_backward(last, stats1, dx, weight=p["norm1"], bias=True)
        d["rows"] = torch.empty(x0.shape[0], 2 * self.dim, device=x0.device)
        tbe.scan_backward(x0, gate, b["histories"], carry, grad_final=dlast.add_(dz),
                          out=(d["rows"][:, :self.dim], d["rows"][:, self.dim:]))
        return loss, d, plan.offsets.diff(), one_each

    def loss_and_update(self, b, lr):
        """The mean loss of a batch; the parameters take one SGD step down its gradient, and the
        balance one towards even experts."""
        loss, d, users_of, one_each = self.gradients(b)
        rows = d.pop("rows")
        self.tables.backward_update(rows.shape[0], b["ids"], one_each, None, rows, lr)
        for name, g in d.items():
            self.p[name].sub_(g, alpha=lr)
        self.balance.add_(torch.sign(users_of.float().mean() - users_of), alpha=1e-3)
        return loss.sum() / (b["target"] >= 0).sum().clamp(min=1)

    def serve(self, ids, histories, best=5):
        """The best next events of every user."""
        _, x, gate = self._events(ids)
        last = tbe.scan_forward(x, gate, histories, need_carry=False)[1]
        return (self._answer(last)[0] @ self.p["events"].t()).topk(best).indices


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--users", type=int, default=2048)
    ap.add_argument("--lr", type=float, default=1.0)
    a = ap.parse_args()
    events, dim, experts, lr = 10000, 128, 16, a.lr
    model = NextEventModel(events, dim, experts)
    b = batch(a.users, events, seed=1)
    for step in range(a.steps):
        loss = model.loss_and_update(b, lr=lr)
        if step % 10 == 0 or step == a.steps - 1:
            print(f"step {step}: loss {loss.item():.4f}", flush=True)
    print("served", tuple(model.serve(b["ids"], b["histories"]).shape))


if __name__ == "__main__":
    main()
