"""Layer norm, the choice of experts, dispatch and combine, and the softmax loss without a GPU: every
refusal, in Python and at the C interface, and the 64-bit definitions' gradients by autograd."""
import ctypes

import pytest
import torch

import heads_reference as ref
import table_embedding_bag_amd as tbe

X = torch.zeros(6, 4)
STATS = torch.zeros(6, 2)
IDS = torch.zeros(6, 2, dtype=torch.int32)
G2 = torch.zeros(6, 2)
PLAN = tbe.DispatchPlan(torch.zeros(4, dtype=torch.int64), IDS)
Y = torch.zeros(12, 4)
T = torch.zeros(9, 4)
TARGETS = torch.zeros(6, dtype=torch.int64)
N6 = torch.zeros(6)


def refuses(f, a, change, what):
    a.update(change)
    with pytest.raises(ValueError, match=what):
        f(**a)


# --- the definitions ---------------------------------------------------------------------------

def _leaf(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64).requires_grad_()


def test_norm_gradients_of_the_definition():
    x, w, b, g = _leaf(5, 7), _leaf(7, seed=1), _leaf(7, seed=2), _leaf(5, 7, seed=3).detach()
    torch.nn.functional.layer_norm(x, (7,), w, b, eps=1e-5).backward(g)
    out = ref.norm(x.detach(), w.detach(), b.detach(), 1e-5, g)
    for name, t in (("dx", x), ("dweight", w), ("dbias", b)):
        assert (out[name][0] - t.grad).abs().max() < 1e-13, name


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradients_of_the_definition(scores, renormalize):
    x, g = _leaf(5, 12), _leaf(5, 3, seed=1).detach()
    out = ref.route(x.detach(), 3, scores=scores, renormalize=renormalize, scale=1.5, g=g)
    p = torch.softmax(x, 1) if scores == "softmax" else torch.sigmoid(x)
    w = p.gather(1, out["ids"].long())
    w = 1.5 * (w / w.sum(1, keepdim=True) if renormalize else w)
    assert (w - out["weights"][0]).abs().max() < 1e-14
    w.backward(g)
    assert (out["dlogits"][0] - x.grad).abs().max() < 1e-14


def test_combine_gradients_of_the_definition():
    places = torch.tensor([[2, -1], [0, 1], [-1, 3]], dtype=torch.int32)
    y, w, g = _leaf(6, 5), _leaf(3, 2, seed=1), _leaf(3, 5, seed=2).detach()
    out = ref.combine(y.detach(), places, w.detach(), g=g)
    rows = y[places.clamp(min=0).long()] * (w * (places >= 0))[:, :, None]
    assert (rows.sum(1) - out["out"][0]).abs().max() < 1e-14
    rows.sum(1).backward(g)
    assert (out["dy"][0] - y.grad).abs().max() < 1e-14 and (out["dweights"][0] - w.grad).abs().max() < 1e-14


def test_loss_gradients_of_the_definition():
    x, t, g = _leaf(5, 4), _leaf(9, 4, seed=1), _leaf(5, seed=2).detach()
    targets = torch.tensor([3, -1, 8, 0, 9])
    on = (targets >= 0) & (targets < 9)
    out = ref.loss(x.detach(), t.detach(), targets, 0.7, g)
    loss = torch.nn.functional.cross_entropy(0.7 * x @ t.t(), torch.where(on, targets, -100), reduction="none")
    assert (loss - out["loss"][0]).abs().max() < 1e-13
    loss.backward(g)
    assert (out["dx"][0] - x.grad).abs().max() < 1e-13 and (out["dtable"][0] - t.grad).abs().max() < 1e-13


def test_plan_of_the_definition():
    offsets, places = ref.plan(torch.tensor([[2, 0], [0, 5], [-1, 2]]), 3)
    assert offsets.tolist() == [0, 2, 2, 4] and places.tolist() == [[2, 0], [1, -1], [-1, 3]]


# --- refusals in Python ------------------------------------------------------------------------

@pytest.mark.parametrize("change,what", [
    ({"x": torch.zeros(6)}, "2 dimensions"), ({"x": X.int()}, "float32"), ({"x": torch.zeros(6, 0)}, "at least one"),
    ({"x": X.t().contiguous().t()}, "adjacent"), ({"weight": torch.zeros(5)}, "weight"), ({"weight": torch.zeros(4).half()}, "weight"),
    ({"bias": torch.zeros(8)[::2]}, "contiguous"), ({"eps": -1.0}, "eps"), ({"eps": float("nan")}, "eps"),
    ({"out": torch.zeros(6, 5)}, "out"), ({"out": torch.zeros(1, 4).expand(6, 4)}, "overlap"), ({}, "GPU"),
])
def test_layer_norm_refuses(change, what):
    refuses(tbe.layer_norm, dict(x=X), change, what)


@pytest.mark.parametrize("change,what", [
    ({"stats": None}, "stats"), ({"stats": torch.zeros(6, 3)}, "stats"), ({"stats": STATS.half()}, "stats"),
    ({"grad": torch.zeros(5, 4)}, "grad"), ({"grad": X.half()}, "grad"), ({"weight": torch.zeros(3)}, "weight"),
    ({"out": X.half()}, "out"), ({}, "GPU"),
])
def test_layer_norm_backward_refuses(change, what):
    refuses(tbe.layer_norm_backward, dict(x=X, stats=STATS, grad=X), change, what)


@pytest.mark.parametrize("change,what", [
    ({"k": 0}, "k must"), ({"k": 5}, "k must"), ({"scores": "relu"}, "scores"), ({"group_score": "sum"}, "group_score"),
    ({"groups": 3}, "groups must"), ({"groups": 0}, "groups must"), ({"groups": 2, "top_groups": 3}, "top_groups"),
    ({"groups": 2, "top_groups": 0}, "top_groups"), ({"groups": 2, "k": 3}, "k must"), ({"bias": torch.zeros(5)}, "bias"),
    ({"bias": torch.zeros(4).half()}, "bias"), ({"scale": float("inf")}, "scale"), ({"scale": float("nan")}, "scale"),
    ({"logits": X.double()}, "float32"), ({"logits": torch.zeros(6, 0)}, "groups must"), ({}, "GPU"),
])
def test_route_refuses(change, what):
    refuses(tbe.route, dict(logits=X, k=2), change, what)


@pytest.mark.parametrize("change,what", [
    ({"ids": IDS.long()}, "ids"), ({"ids": IDS[:5]}, "ids"), ({"ids": torch.zeros(6, dtype=torch.int32)}, "ids"),
    ({"ids": torch.zeros(6, 5, dtype=torch.int32)}, "ids"), ({"grad": G2.half()}, "grad"), ({"grad": torch.zeros(6, 3)}, "grad"),
    ({"scores": 1}, "scores"), ({"out": X.half()}, "out"), ({}, "GPU"),
])
def test_route_backward_refuses(change, what):
    refuses(tbe.route_backward, dict(logits=X, ids=IDS, grad=G2), change, what)


@pytest.mark.parametrize("change,what", [
    ({"ids": G2}, "ids"), ({"ids": torch.zeros(6, dtype=torch.int32)}, "ids"), ({"ids": torch.zeros(6, 0, dtype=torch.int32)}, "ids"),
    ({"ids": torch.zeros(2, 6, dtype=torch.int32).t()}, "contiguous"), ({"experts": 0}, "experts"), ({}, "GPU"),
])
def test_dispatch_plan_refuses(change, what):
    refuses(tbe.dispatch_plan, dict(ids=IDS, experts=3), change, what)


@pytest.mark.parametrize("plan,what", [
    (tbe.DispatchPlan(PLAN.offsets, IDS.long()), "places"), (tbe.DispatchPlan(PLAN.offsets, IDS[:, 0]), "places"),
    (tbe.DispatchPlan(PLAN.offsets.int(), IDS), "offsets"), (tbe.DispatchPlan(PLAN.offsets[:1], IDS), "offsets"),
    (tbe.DispatchPlan(PLAN.offsets, torch.zeros(2, 6, dtype=torch.int32).t()), "contiguous"), (PLAN, "GPU"),
])
def test_moves_refuse_plans(plan, what):
    for f, a in ((tbe.dispatch, (X, plan)), (tbe.combine, (Y, plan)), (tbe.dispatch_backward, (Y, plan)),
                 (tbe.combine_backward, (Y, plan, G2, X))):
        with pytest.raises(ValueError, match=what):
            f(*a)


def test_moves_refuse():
    for f, a, kw, what in (
            (tbe.dispatch, (torch.zeros(5, 4), PLAN), {}, "rows"), (tbe.dispatch, (X, PLAN), {"out": X}, "out"),
            (tbe.dispatch, (torch.zeros(6, 0), PLAN), {}, "rows"), (tbe.combine, (X, PLAN), {}, "rows"),
            (tbe.combine, (Y, PLAN, G2.half()), {}, "weights"), (tbe.combine, (Y, PLAN, G2[:, :1]), {}, "weights"),
            (tbe.combine, (Y, PLAN), {"residual": X.half()}, "residual"), (tbe.combine, (Y, PLAN), {"out": Y}, "out"),
            (tbe.combine_backward, (Y, PLAN, G2, X.half()), {}, "grad"), (tbe.combine_backward, (X, PLAN, G2, X), {}, "rows"),
            (tbe.combine_backward, (Y, PLAN, torch.zeros(6, 3), X), {}, "weights")):
        with pytest.raises(ValueError, match=what):
            f(*a, **kw)


@pytest.mark.parametrize("change,what", [
    ({"x": X.double()}, "float32"), ({"table": T.half()}, "table"), ({"table": torch.zeros(9, 5)}, "table"),
    ({"table": T[:0]}, "table"), ({"x": torch.zeros(6, 0), "table": torch.zeros(9, 0)}, "table"),
    ({"targets": N6}, "targets"), ({"targets": TARGETS[:5]}, "targets"), ({"targets": torch.zeros(12, dtype=torch.int64)[::2]}, "contiguous"),
    ({"scale": 0.0}, "scale"), ({"scale": -1.0}, "scale"), ({"scale": float("nan")}, "scale"), ({}, "GPU"),
])
def test_softmax_loss_refuses(change, what):
    refuses(tbe.softmax_loss, dict(x=X, table=T, targets=TARGETS), change, what)
    refuses(tbe.softmax_loss_backward, dict(x=X, table=T, targets=TARGETS, lse=N6, grad=N6), change, what)


@pytest.mark.parametrize("change,what", [({"lse": N6.half()}, "lse"), ({"lse": N6[:5]}, "lse"), ({"grad": N6.double()}, "grad"),
                                         ({"grad": torch.zeros(6, 1)}, "grad")])
def test_softmax_loss_backward_refuses(change, what):
    refuses(tbe.softmax_loss_backward, dict(x=X, table=T, targets=TARGETS, lse=N6, grad=N6), change, what)


# --- refusals at the C interface: nothing is enqueued, no GPU is touched -------------------------

INVALID, UNSUPPORTED, SMALL = 1, 2, 4
A = 4096  # an aligned address that is never read


def call(name, defaults, kw):
    a = dict(defaults)
    a.update(kw)
    return getattr(tbe.load(), name)(*a.values())


NORM = dict(x=A, xs=4, w=A, b=A, y=A, ys=4, stats=A, rows=6, cols=4, dtype=0, eps=1e-5, stream=None)
NORM_BACK = dict(x=A, xs=4, stats=A, g=A, gs=4, w=A, dx=A, ds=4, dw=A, db=A, rows=6, cols=4, dtype=0, ws=A, nws=1 << 40,
                 stream=None)


@pytest.mark.parametrize("kw,status", [
    ({"x": None}, INVALID), ({"y": None}, INVALID), ({"rows": -1}, INVALID), ({"cols": 0}, INVALID), ({"dtype": 3}, INVALID),
    ({"x": A + 2}, INVALID), ({"w": A + 1}, INVALID), ({"b": A + 2}, INVALID), ({"y": A + 1}, INVALID), ({"stats": A + 4}, INVALID),
    ({"xs": -1}, INVALID), ({"ys": 3}, INVALID), ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID),
    ({"rows": 1 << 31}, UNSUPPORTED), ({"cols": 1 << 21}, UNSUPPORTED), ({"rows": 0, "x": None}, 0),
])
def test_c_layer_norm_refuses(kw, status):
    assert call("tbe_layer_norm", NORM, kw) == status


@pytest.mark.parametrize("kw,status", [
    ({"x": None}, INVALID), ({"stats": None}, INVALID), ({"g": None}, INVALID), ({"gs": -1}, INVALID), ({"ds": 3}, INVALID),
    ({"dx": A + 2}, INVALID), ({"dw": A + 2}, INVALID), ({"db": A + 1}, INVALID), ({"stats": A + 4}, INVALID), ({"ws": None}, INVALID),
    ({"ws": A + 64}, INVALID), ({"nws": 0}, SMALL), ({"rows": 1 << 31}, UNSUPPORTED),
    ({"rows": 0, "dw": None, "db": None, "ws": None}, 0), ({"dx": None, "dw": None, "db": None}, 0),
])
def test_c_layer_norm_backward_refuses(kw, status):
    assert call("tbe_layer_norm_backward", NORM_BACK, kw) == status


ROUTE = dict(l=A, ls=64, bias=None, ids=A, w=A, rows=6, E=64, k=4, groups=8, top=4, dtype=0, scores=0, gscore=0, renorm=1,
             scale=1.0, stream=None)
ROUTE_BACK = dict(l=A, ls=64, ids=A, g=A, d=A, ds=64, rows=6, E=64, k=4, dtype=0, scores=0, renorm=1, scale=1.0, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({"l": None}, INVALID), ({"l": A + 2}, INVALID), ({"ls": -1}, INVALID), ({"rows": -1}, INVALID), ({"E": 0}, INVALID), ({"k": 0}, INVALID),
    ({"k": 65}, INVALID), ({"dtype": 9}, INVALID), ({"scores": 2}, INVALID), ({"scale": float("inf")}, INVALID), ({"scale": 1e300}, INVALID),
    ({"ids": None}, INVALID), ({"ids": A + 2}, INVALID), ({"E": 1040}, UNSUPPORTED), ({"k": 17}, UNSUPPORTED), ({"rows": 1 << 30}, UNSUPPORTED),
])
def test_c_route_refuses(kw, status):
    assert call("tbe_route", ROUTE, kw) == status
    assert call("tbe_route_backward", ROUTE_BACK, kw) == status


def test_c_route_refuses_more():
    for kw in ({"w": None}, {"w": A + 2}, {"bias": A + 2}, {"groups": 0}, {"groups": 5}, {"top": 0}, {"top": 9}, {"top": 1, "k": 9},
               {"gscore": 2}, {"groups": 128, "E": 64}):
        assert call("tbe_route", ROUTE, kw) == INVALID, kw
    assert call("tbe_route", ROUTE, {"groups": 32}) == UNSUPPORTED
    for kw in ({"g": None}, {"d": None}, {"ds": 63}, {"d": A + 1}, {"g": A + 2}):
        assert call("tbe_route_backward", ROUTE_BACK, kw) == INVALID, kw
    assert call("tbe_route", ROUTE, {"rows": 0, "l": None}) == 0 and call("tbe_route_backward", ROUTE_BACK, {"rows": 0}) == 0


PLAN_C = dict(ids=A, index=0, rows=6, k=2, E=3, offsets=A, places=A, ws=None, nws=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({"ids": None}, INVALID), ({"offsets": None}, INVALID), ({"places": None}, INVALID), ({"index": 2}, INVALID), ({"rows": -1}, INVALID),
    ({"k": 0}, INVALID), ({"E": 0}, INVALID), ({"offsets": A + 4}, INVALID), ({"places": A + 2}, INVALID), ({"ids": A + 4, "index": 1}, INVALID),
    ({"k": 65}, UNSUPPORTED), ({"E": 2049}, UNSUPPORTED), ({"rows": 1 << 30}, UNSUPPORTED),
    ({"rows": 100000}, INVALID), ({"rows": 100000, "ws": A}, SMALL), ({"rows": 100000, "ws": A + 64, "nws": 1 << 30}, INVALID),
])
def test_c_dispatch_plan_refuses(kw, status):
    assert call("tbe_dispatch_plan", PLAN_C, kw) == status
    n = ctypes.c_size_t(1)
    assert tbe.load().tbe_dispatch_plan_size(6, 2, 3, None) == INVALID
    assert tbe.load().tbe_dispatch_plan_size(6, 2, 3, ctypes.byref(n)) == 0 and n.value == 0


DISPATCH = dict(x=A, xs=4, places=A, total=A, out=A, os=4, rows=6, k=2, cols=4, dtype=0, stream=None)
COMBINE = dict(y=A, ys=4, places=A, w=A, r=A, rs=4, out=A, os=4, rows=6, k=2, cols=4, dtype=0, stream=None)
COMBINE_BACK = dict(y=A, ys=4, places=A, total=A, w=A, g=A, gs=4, dy=A, dys=4, dw=A, rows=6, k=2, cols=4, dtype=0, stream=None)


def test_c_moves_refuse():
    for name, base, bad in (
            ("tbe_dispatch", DISPATCH, ({"x": None}, {"total": None}, {"out": None}, {"os": 3}, {"xs": -1}, {"total": A + 4}, {"x": A + 2})),
            ("tbe_combine", COMBINE, ({"y": None}, {"out": None}, {"os": 3}, {"ys": -1}, {"rs": -1}, {"w": A + 2}, {"r": A + 1})),
            ("tbe_combine_backward", COMBINE_BACK, ({"y": None}, {"total": None}, {"w": None}, {"g": None}, {"dy": None}, {"dys": 3},
                                                    {"gs": -1}, {"ys": -1}, {"dw": A + 2}, {"dy": A + 1}))):
        for kw in bad + ({"places": None}, {"places": A + 2}, {"rows": -1}, {"k": 0}, {"cols": 0}, {"dtype": 3}):
            assert call(name, base, kw) == INVALID, (name, kw)
        for kw in ({"k": 65}, {"rows": 1 << 30}, {"cols": 1 << 21}):
            assert call(name, base, kw) == UNSUPPORTED, (name, kw)
        assert call(name, base, {"rows": 0}) == 0


LOSS = dict(x=A, xs=4, t=A, ts=4, targets=A, index=1, scale=1.0, loss=A, lse=A, rows=6, V=9, D=4, dtype=0, ws=A, nws=1 << 40, stream=None)
LOSS_BACK = dict(x=A, xs=4, t=A, ts=4, targets=A, index=1, scale=1.0, lse=A, g=A, dx=A, dt=A, rows=6, V=9, D=4, dtype=0, ws=A, nws=1 << 40,
                 stream=None)


@pytest.mark.parametrize("kw,status", [
    ({"x": None}, INVALID), ({"t": None}, INVALID), ({"targets": None}, INVALID), ({"index": 2}, INVALID), ({"scale": 0.0}, INVALID),
    ({"scale": float("nan")}, INVALID), ({"scale": float("inf")}, INVALID), ({"rows": -1}, INVALID), ({"V": 0}, INVALID), ({"D": 0}, INVALID),
    ({"dtype": 3}, INVALID), ({"x": A + 2}, INVALID), ({"t": A + 1}, INVALID), ({"targets": A + 4}, INVALID), ({"xs": -1}, INVALID),
    ({"ts": -1}, INVALID), ({"lse": A + 2}, INVALID), ({"lse": None}, INVALID), ({"ws": None}, INVALID), ({"ws": A + 64}, INVALID), ({"nws": 0}, SMALL),
    ({"rows": 1 << 25}, UNSUPPORTED), ({"V": 1 << 31}, UNSUPPORTED), ({"D": 1 << 21}, UNSUPPORTED), ({"xs": 1 << 21}, UNSUPPORTED),
    ({"ts": 1 << 21}, UNSUPPORTED),
])
def test_c_softmax_loss_refuses(kw, status):
    assert call("tbe_softmax_loss", LOSS, kw) == status
    assert call("tbe_softmax_loss_backward", LOSS_BACK, kw) == status


def test_c_softmax_loss_refuses_more():
    f, b = ctypes.c_size_t(1), ctypes.c_size_t(1)
    sizes = tbe.load().tbe_softmax_loss_sizes
    assert sizes(6, 9, 4, 0, None, ctypes.byref(b)) == INVALID and sizes(6, 0, 4, 0, ctypes.byref(f), ctypes.byref(b)) == INVALID
    assert sizes(6, 1 << 31, 4, 0, ctypes.byref(f), ctypes.byref(b)) == UNSUPPORTED
    for rows, V, D, dtype in ((6, 9, 4, 0), (3000, 70001, 136, 2), (1, 1, 1, 1)):
        assert sizes(rows, V, D, dtype, ctypes.byref(f), ctypes.byref(b)) == 0
        kw = dict(rows=rows, V=V, D=D, dtype=dtype, xs=D, ts=D)
        assert call("tbe_softmax_loss", LOSS, {**kw, "nws": f.value - 1}) == SMALL
        assert call("tbe_softmax_loss_backward", LOSS_BACK, {**kw, "nws": b.value - 1}) == SMALL
    assert call("tbe_softmax_loss", LOSS, {"loss": None}) == INVALID and call("tbe_softmax_loss", LOSS, {"rows": 0, "x": None}) == 0
    for kw in ({"g": None}, {"dx": A + 2}, {"dt": A + 1}, {"g": A + 1}):
        assert call("tbe_softmax_loss_backward", LOSS_BACK, kw) == INVALID, kw
    assert call("tbe_softmax_loss_backward", LOSS_BACK, {"dx": None, "dt": None}) == 0
