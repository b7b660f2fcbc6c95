"""Rows to their experts and back: the plan, dispatch, combine and their gradients."""
import pytest
import torch

import heads_reference as ref
import table_embedding_bag_amd as tbe

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def ids_of(N, k, E, seed=0, left_out=0.1, index=torch.int32):
    g = torch.Generator().manual_seed(seed)
    ids = (E * torch.rand(N, k, generator=g) ** 2).to(index)
    return torch.where(torch.rand(N, k, generator=g) < left_out, torch.tensor(-1, dtype=index), ids).cuda()


def check_plan(ids, E, plan=None):
    plan = plan or tbe.dispatch_plan(ids, E)
    offsets, places = ref.plan(ids, E)
    assert torch.equal(plan.offsets.cpu(), offsets), "offsets"
    assert torch.equal(plan.places.cpu(), places), "places"
    return plan


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("N,k,E", [(1, 1, 1), (1, 2, 64), (64, 2, 64), (63, 3, 5), (257, 8, 256), (1000, 4, 130),
                                   (1024, 4, 16), (1025, 4, 16), (4099, 3, 13), (9001, 8, 512), (300, 64, 2048)])
def test_plan(N, k, E, index):
    check_plan(ids_of(N, k, E, seed=N + k, index=index), E)


def test_plan_of_many_tiles():
    check_plan(ids_of(150001, 8, 300, seed=1), 300)
    check_plan(ids_of(1100003, 1, 7, seed=2), 7)


def test_plan_of_one_expert_none_and_wrong_ids():
    check_plan(torch.zeros(5000, 2, dtype=torch.int64, device="cuda"), 3)
    check_plan(torch.full((5000, 2), -1, dtype=torch.int32, device="cuda"), 3)
    wrong = torch.tensor([[0, 3], [2, 1 << 40], [-(1 << 40), 4], [2, 2]], device="cuda")
    check_plan(wrong, 3)
    plan = tbe.dispatch_plan(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 3)
    assert not plan.offsets.any() and plan.places.shape == (0, 2)


class Rows:
    def __init__(self, N, k, D, E, dtype, seed=0, wide=0, left_out=0.1):
        g = torch.Generator().manual_seed(seed)
        make = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
        self.ids = ids_of(N, k, E, seed, left_out)
        self.E, self.N, self.k, self.D, self.dtype = E, N, k, D, dtype
        self.x, self.residual, self.grad = (make(N, D + wide)[:, :D] for _ in range(3))
        self.y, self.grad_rows = (make(N * k, D + wide)[:, :D] for _ in range(2))
        self.weights = torch.rand(N, k, generator=g).cuda()

    def run(self):
        plan = tbe.dispatch_plan(self.ids, self.E)
        dy, dw = tbe.combine_backward(self.y, plan, self.weights, self.grad)
        return {"offsets": plan.offsets, "places": plan.places, "rows": tbe.dispatch(self.x, plan),
                "out": tbe.combine(self.y, plan, self.weights, residual=self.residual), "dy": dy, "dweights": dw,
                "dx": tbe.dispatch_backward(self.grad_rows, plan), "plain": tbe.combine(self.y, plan)}

    def check(self, got=None):
        got = got or self.run()
        check_plan(self.ids, self.E, tbe.DispatchPlan(got["offsets"], got["places"]))
        places = got["places"]
        rows = torch.zeros(self.N * self.k, self.D, dtype=self.dtype, device="cuda")
        n, j = (places >= 0).nonzero(as_tuple=True)
        rows[places[n, j].long()] = self.x[n]
        assert torch.equal(got["rows"], rows), "rows"
        d = lambda t: t.double()  # noqa: E731
        want = ref.combine(d(self.y), places, d(self.weights), d(self.residual), d(self.grad))
        for name in ("out", "dy", "dweights"):
            ref.assert_close(got[name], *want[name], name)
        ref.assert_close(got["dx"], *ref.combine(d(self.grad_rows), places)["out"], "dx")
        ref.assert_close(got["plain"], *ref.combine(d(self.y), places)["out"], "plain")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("N,k,D,E", [(1, 1, 1, 1), (1, 8, 512, 64), (7, 2, 3, 4), (64, 2, 130, 16), (33, 3, 1000, 9),
                                     (500, 5, 257, 31), (100, 16, 2056, 40), (3, 64, 4100, 100)])
def test_rows(N, k, D, E, dtype):
    Rows(N, k, D, E, DTYPES[dtype], seed=N + D).check()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_of_wider_buffers(dtype):
    Rows(90, 3, 70, 8, DTYPES[dtype], seed=3, wide=5).check()


@pytest.mark.parametrize("left_out", [0.0, 1.0])
def test_all_and_none(left_out):
    Rows(70, 4, 136, 8, torch.bfloat16, seed=4, left_out=left_out).check()


def test_many_rows():
    Rows(20001, 4, 96, 50, torch.float32, seed=5).check()


def test_what_nobody_has_reaches_nothing():
    """NaN in rows that have no place, and in weights of assignments that have none."""
    p = Rows(60, 3, 40, 6, torch.float32, seed=6, left_out=0.4)
    plan = tbe.dispatch_plan(p.ids, p.E)
    total = int(plan.offsets[-1])
    p.y[total:] = float("nan")
    p.weights[plan.places < 0] = float("nan")
    out = tbe.combine(p.y, plan, p.weights)
    dy, dw = tbe.combine_backward(p.y, plan, p.weights, p.grad)
    assert not torch.isnan(out).any() and not torch.isnan(dy).any() and not torch.isnan(dw).any()
    assert not dy[total:].any() and not dw[plan.places < 0].any()


def test_outputs_given():
    p = Rows(50, 2, 64, 5, torch.bfloat16, seed=7)
    plan = tbe.dispatch_plan(p.ids, p.E)
    wide = torch.full((100, 80), 3.0, dtype=torch.bfloat16, device="cuda")
    tbe.dispatch(p.x, plan, out=wide[:, 8:72])
    assert torch.equal(wide[:, 8:72], tbe.dispatch(p.x, plan)) and (wide[:, :8] == 3).all() and (wide[:, 72:] == 3).all()
    want = tbe.combine(p.y, plan, p.weights, residual=p.residual)
    tbe.combine(p.y, plan, p.weights, residual=p.residual, out=p.residual)
    assert torch.equal(p.residual, want)


def test_wrong_places_reach_nothing():
    p = Rows(8, 2, 16, 4, torch.float32, seed=8)
    places = torch.full((8, 2), 1 << 20, dtype=torch.int32, device="cuda")
    places[3] = torch.tensor([-7, 16])
    plan = tbe.DispatchPlan(torch.tensor([0, 0, 0, 0, 16], device="cuda"), places)
    assert torch.equal(tbe.combine(p.y, plan, p.weights, residual=p.residual), p.residual)
    _, dw = tbe.combine_backward(p.y, plan, p.weights, p.grad)
    assert not dw.any()


def test_same_bits_every_time_and_graphs():
    p = Rows(3000, 4, 200, 32, torch.bfloat16, seed=9)
    p.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = p.run()
    for i in range(4):
        q = Rows(3000, 4, 200, 32, torch.bfloat16, seed=40 + i)
        for name in ("ids", "x", "y", "residual", "grad", "grad_rows", "weights"):
            getattr(p, name).copy_(getattr(q, name))
        want = p.run()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[n]) for n in want), i


def test_with_the_grouped_linear_layer():
    """Every expert's product, added up by hand."""
    p = Rows(200, 2, 64, 6, torch.float32, seed=10)
    w = torch.randn(6, 48, 64, generator=torch.Generator().manual_seed(11)).cuda()
    plan = tbe.dispatch_plan(p.ids, 6)
    out = tbe.combine(tbe.grouped_linear(tbe.dispatch(p.x, plan), w, plan.offsets), plan, p.weights)
    want = torch.zeros(200, 48, dtype=torch.float64, device="cuda")
    size = want.clone()
    for j in range(2):
        for e in range(6):
            n = (p.ids[:, j] == e).nonzero()[:, 0]
            want[n] += p.weights[n, j:j + 1].double() * (p.x[n].double() @ w[e].double().t())
            size[n] += p.weights[n, j:j + 1].double() * (p.x[n].double().abs() @ w[e].double().abs().t())
    assert ((out.double() - want).abs() <= 72 * ref.U32 * size + 1e-30).all()
