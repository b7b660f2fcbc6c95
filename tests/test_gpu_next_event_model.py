"""Layer norm, routing, dispatch and combine, and the softmax loss together with the tables, the recurrence
and the grouped linear layer, as examples/next_event_model.py uses them."""
import os
import subprocess
import sys

import pytest
import torch

import heads_reference as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def _definition(model, b):
    """The mean loss by 64-bit autograd, and its gradients."""
    p = {n: t.double().cpu().requires_grad_() for n, t in model.p.items()}
    rows = model.table.double().cpu().view(-1, 2 * model.dim)[b["ids"].cpu()].requires_grad_()
    off = b["histories"].tolist()
    last = []
    for s in range(len(off) - 1):
        h = torch.zeros(model.dim, dtype=torch.float64)
        for t in range(off[s], off[s + 1]):
            a = torch.sigmoid(rows[t, model.dim:])
            h = a * h + (1 - a) * rows[t, :model.dim]
        last.append(h)
    last = torch.stack(last)
    norm = torch.nn.functional.layer_norm
    x = norm(last, (model.dim,), p["norm1"], p["bias1"], eps=1e-5)
    logits = x @ p["router"][0].t()
    ids = ref.route(logits.detach(), model.k, scores="sigmoid", bias=model.balance.cpu())["ids"].long()
    w = torch.sigmoid(logits).gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    y = torch.einsum("nkod,nd->nko", p["expert"][ids], x)
    z = last + (w[:, :, None] * y).sum(1)
    out = norm(z, (model.dim,), p["norm2"], p["bias2"], eps=1e-5)
    target = b["target"].cpu()
    loss = torch.nn.functional.cross_entropy(out @ p["events"].t(), target, ignore_index=-1)
    loss.backward()
    return loss.item(), {**{n: t.grad for n, t in p.items()}, "rows": rows.grad}


def test_gradients_of_the_whole_model():
    """Every gradient against 64-bit autograd.  A value passes through some ten layers of sums of up to 300
    terms in fp32, each off by some ten half steps of its terms' size: 2^-24 * 10 * 10 of the largest
    gradient, and as much again for terms that cancel."""
    from next_event_model import NextEventModel, batch
    model = NextEventModel(300, 24, 5, seed=3)
    model.balance.copy_(torch.tensor([0.02, -0.01, 0.0, 0.01, -0.03]))
    b = batch(60, 300, seed=4)
    loss, d, users_of, _ = model.gradients(b)
    want_loss, want = _definition(model, b)
    real = (b["target"] >= 0).sum().item()
    assert abs(loss.double().sum().item() / real - want_loss) < 200 * 2.0 ** -24 * want_loss
    assert int(users_of.sum()) == 60 * model.k
    for name, g in want.items():
        off = (d[name].double().cpu() - g).abs().max().item()
        print(f"[next event] {name}: off {off:.2e} of {g.abs().max().item():.2e}", flush=True)
        assert off <= 200 * 2.0 ** -24 * g.abs().max().item(), name


def test_training_changes_every_parameter_and_serving_runs():
    from next_event_model import NextEventModel, batch
    model = NextEventModel(300, 24, 5, seed=5)
    b = batch(80, 300, seed=6)
    before = {**{n: t.clone() for n, t in model.p.items()}, "table": model.table.clone()}
    assert torch.isfinite(model.loss_and_update(b, 0.1))
    for name, t in before.items():
        assert not torch.equal(t, model.table if name == "table" else model.p[name]), name
    best = model.serve(b["ids"], b["histories"])
    assert best.shape == (80, 5) and int(best.min()) >= 0 and int(best.max()) < 300


def test_example_runs():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, os.path.join(root, "examples", "next_event_model.py"), "--steps", "3", "--users",
                          "256"], capture_output=True, text=True, timeout=100)
    assert out.returncode == 0, out.stderr
    assert "served (256, 5)" in out.stdout
