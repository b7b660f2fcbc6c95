"""The layers together, as examples/history_model.py uses them."""
import os
import subprocess
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def _loss(lr):
    """The losses before and after one step at this rate, the gradient's squared norm from the
    change of the parameters, and the users' count."""
    from history_model import HistoryModel, batch
    model = HistoryModel(500, 32, 3, seed=3)
    b = batch(200, 500, 3, 32, seed=4)
    before = [t.double().clone() for t in (model.table, model.weight, model.bias)]
    first = model.loss_and_update(b, lr).double().item()
    square = sum(((new.double() - old) / lr).square().sum().item()
                 for new, old in zip((model.table, model.weight, model.bias), before))
    model.offset = 0   # the same mask
    return first, model.loss_and_update(b, 0.0).double().item(), square


def test_gradients_by_differences():
    """A step of rate r takes r |gradient|^2 off the loss, but for a term of r^2: of the two rates'
    ratios to that, extrapolated to r = 0, what is left is of r^2 (1% here: the ratios themselves
    are some 5% off), and the losses' rounding (2^-24 of sums of 6400 terms, 1e-4 of their change)."""
    ratios = []
    for lr in (8.0, 4.0):
        first, second, square = _loss(lr)
        ratios.append((first - second) / (lr * square))
    print(f"[history] ratios {ratios}", flush=True)
    assert abs(2 * ratios[1] - ratios[0] - 1) < 0.01 + 1e-4


def test_serving_goes_on_from_training():
    """One new event for each user gives the state of the history with that event at its end."""
    from history_model import HistoryModel, batch
    users, rows, dim = 100, 300, 20
    model = HistoryModel(rows, dim, 4, seed=5)
    b = batch(users, rows, 4, dim, seed=6)
    ids, off = b["ids"].cpu(), b["histories"].cpu()
    new = torch.randint(rows, (users,), generator=torch.Generator().manual_seed(7))
    longer = torch.cat([torch.cat([ids[off[u]:off[u + 1]], new[u:u + 1]]) for u in range(users)])
    state = model.states(b["ids"], b["histories"])
    answer = model.serve(new.cuda(), state, b["domains"])
    want = model.states(longer.cuda(), b["histories"] + torch.arange(users + 1, device="cuda"))
    # both are off by at most 8 half steps for each of up to 41 events, of states within the
    # largest input (a convex combination of inputs)
    bound = 2 * 41 * 8 * 2.0 ** -24 * model.table.abs().max().item()
    assert (state - want).abs().max().item() <= bound
    assert answer.shape == (users, dim) and answer.isfinite().all()


def test_command():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "history_model.py"), "--steps", "21",
                        "--users", "300"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr
    losses = [float(line.split()[-1]) for line in r.stdout.splitlines() if line.startswith("step")]
    assert len(losses) == 3 and losses[2] < losses[1] < losses[0], r.stdout
