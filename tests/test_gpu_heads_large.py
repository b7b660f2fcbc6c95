"""Heads of models on tensors of more than 2^32 bytes: what lies at their ends."""
import math

import pytest
import torch

import table_embedding_bag_amd as tbe

pytestmark = pytest.mark.gpu


def test_layer_norm():
    """The last rows, bit for bit those of a call with them alone."""
    x = torch.randn(70000, 32768, dtype=torch.float16, device="cuda")
    y, stats = tbe.layer_norm(x)
    dx, _, _ = tbe.layer_norm_backward(x, stats, x)
    end = x[-4:].clone()
    want, few = tbe.layer_norm(end)
    assert torch.equal(y[-4:], want) and torch.equal(stats[-4:], few)
    assert torch.equal(dx[-4:], tbe.layer_norm_backward(end, few, end)[0])


def test_route():
    logits = torch.randn(2200000, 1024, dtype=torch.float16, device="cuda")
    ids, weights = tbe.route(logits, 2)
    grad = torch.ones_like(weights)
    grad[:, 1] = -1
    dlogits = tbe.route_backward(logits, ids, grad)
    end = logits[-7:].clone()
    want, few = tbe.route(end, 2)
    assert torch.equal(ids[-7:], want) and torch.equal(weights[-7:], few)
    assert torch.equal(dlogits[-7:], tbe.route_backward(end, want, grad[-7:].clone()))


def test_dispatch_and_combine():
    """Whole numbers: every result exact."""
    N, k, D = 70000, 2, 16384
    x = (torch.arange(N, device="cuda") % 251).to(torch.bfloat16)[:, None].repeat(1, D)
    ids = torch.arange(N * k, device="cuda").flip(0).view(N, k) * 8 // (N * k)
    plan = tbe.dispatch_plan(ids.contiguous(), 8)
    rows = tbe.dispatch(x, plan)
    for n in (0, 1, N // 2, N - 2, N - 1):
        for p in plan.places[n].tolist():
            assert torch.equal(rows[p], x[n])
    half = torch.full((N, k), 0.5, device="cuda")
    assert torch.equal(tbe.combine(rows, plan, half), x)
    drows, _ = tbe.combine_backward(rows, plan, 2 * half, x)
    assert torch.equal(drows, rows)


@pytest.mark.parametrize("V,D,dtype", [(17000000, 128, torch.bfloat16), (16500000, 136, torch.float16),
                                       (17000000, 64, torch.float32)])
def test_softmax_loss(V, D, dtype):
    """A table of zeros but for its last three rows, whose logits are about 16, 16 and -16."""
    N = 8
    x = torch.full((N, D), 16 / D * 2, dtype=torch.float32, device="cuda").to(dtype)
    table = torch.zeros(V, D, dtype=dtype, device="cuda")
    table[-3:] = torch.tensor([[-0.5], [0.5], [0.5]], device="cuda").to(dtype)
    z = 0.5 * float(x[0].double().sum())
    targets = torch.full((N,), V - 1, device="cuda")
    grad = torch.full((N,), 4096.0, device="cuda")
    loss, lse = tbe.softmax_loss(x, table, targets)
    dx, dtable = tbe.softmax_loss_backward(x, table, targets, lse, grad)
    total = V - 3 + 2 * math.exp(z) + math.exp(-z)
    want = math.log(total)
    # half steps of fp32: two of the result's, four of the logit's (sum of the products, scale,
    # power, its reference), each also a relative error of the powers
    error = 2.0 ** -24 * (2 * want + 4 * z) + D * 2.0 ** -24
    assert float((lse.double() - want).abs().max()) <= error
    assert float((loss.double() - (want - z)).abs().max()) <= error + 2.0 ** -24 * z
    step = torch.finfo(dtype).eps / 2
    p, first, last = 1 / total, math.exp(-z) / total, math.exp(z) / total
    # the logits' gradients, and the output, each off by half a step; the powers by lse's error
    xs = N * 4096 * float(x[0, 0])
    rel = 2 * step + 2 * error + 2.0 ** -20
    for v, d in ((0, p), (V // 2, p), (V - 4, p), (V - 3, first), (V - 2, last), (V - 1, last - 1)):
        # fp16: the smallest subnormal's half
        bound = rel * max(abs(d), last if v == V - 1 else 0) * xs + 2.0 ** -25
        assert float((dtable[v].double() - d * xs).abs().max()) <= bound, v
    dx_want = 4096 * 0.5 * (last + (last - 1) - first)
    bound = 4096 * 0.5 * rel * (2 * last + 1) + step * abs(dx_want)
    assert float((dx.double() - dx_want).abs().max()) <= bound
