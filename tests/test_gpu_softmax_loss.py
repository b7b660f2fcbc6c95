"""The softmax loss over a table's rows and its gradients."""
import pytest
import torch

import heads_reference as ref
import table_embedding_bag_amd as tbe

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


# Sizes whose tests compare every output with 64 bits; tests/test_loss_plan.py asserts that they reach
# every kernel.
SMALL = [(n, v, d) for d in (1, 33, 64, 100, 130, 256)
         for n, v in ((1, 1), (1, 300), (5, 64), (33, 129), (64, 1000), (130, 257), (300, 2500))]
NARROW = [(n, v, d) for d in (8, 16, 40, 64, 72, 104, 120, 128)
          for n, v in ((1, 127), (63, 128), (64, 129), (65, 63), (256, 64), (257, 65), (600, 1999))] + [
              (8, 70000, 16), (66000, 300, 16)]
LARGER = [(600, 5000, 128), (40, 30000, 72), (2049, 1030, 520), (5000, 65, 40), (700, 9000, 264), (3000, 4001, 131),
          (3000, 4001, 130), (3000, 4001, 132), (20, 9000, 301), (20, 9000, 302), (20, 9000, 304),
          (3000, 6000, 301), (3000, 6000, 302), (3000, 6000, 304)]
LARGE = [(11000, 12000, 520), (11000, 12000, 521), (11000, 12000, 522)]
SIZES = [(*s, t) for s in SMALL + LARGER for t in DTYPES] + [(*s, t) for s in NARROW + LARGE for t in ("fp16", "bf16")] + [
    (70000, 5000, 16, "bf16"), (70000, 5000, 17, "bf16")]


class Problem:
    def __init__(self, N, V, D, dtype, seed=0, wide=0, scale=1.0, index=torch.int64, left_out=0.1, spread=2.0):
        g = torch.Generator().manual_seed(seed)
        self.N, self.V, self.D, self.dtype, self.scale = N, V, D, dtype, scale
        table = spread * D ** -0.5 * torch.randn(V, D + wide, generator=g)
        targets = torch.randint(0, V, (N,), generator=g)
        x = torch.randn(N, D + wide, generator=g) + table[targets]
        self.x, self.table = x.to(dtype).cuda()[:, :D], table.to(dtype).cuda()[:, :D]
        self.targets = torch.where(torch.rand(N, generator=g) < left_out, -1, targets).to(index).cuda()
        self.grad = (0.5 + torch.rand(N, generator=g)).cuda() / N
        if dtype == torch.float16:
            self.grad *= 4096

    def run(self):
        loss, lse = tbe.softmax_loss(self.x, self.table, self.targets, scale=self.scale)
        dx, dtable = tbe.softmax_loss_backward(self.x, self.table, self.targets, lse, self.grad, scale=self.scale)
        return {"loss": loss, "lse": lse, "dx": dx, "dtable": dtable}

    def check(self, got=None):
        got = got or self.run()
        want = ref.loss(self.x.double(), self.table.double(), self.targets, self.scale, self.grad.double(), self.dtype)
        for name in ("lse", "loss", "dx", "dtable"):
            ref.assert_close(got[name], *want[name], name)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("N,V,D", SMALL)
def test_forward_and_backward(N, V, D, dtype):
    Problem(N, V, D, DTYPES[dtype], seed=N + V + D).check()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("N,V,D", LARGER)
def test_larger(N, V, D, dtype):
    Problem(N, V, D, DTYPES[dtype], seed=1).check()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("N,V,D", LARGE)
def test_large(N, V, D, dtype):
    Problem(N, V, D, DTYPES[dtype], seed=1).check()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [64, 128, 200])
def test_logits_far_below_and_above_zero(D, dtype):
    """Tables that end inside a tile: a row past the end would have the logit 0, which is e^200 times
    the largest here (or nothing beside the others)."""
    for sign in (-1, 1):
        p = Problem(100, 321, D, DTYPES[dtype], seed=6)
        p.x[:] = 0.05 * p.x + 1
        p.table[:] = 0.1 * p.table + sign * 200.0 / D
        p.check()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("N,V,D", NARROW)
def test_narrow_rows(N, V, D, dtype):
    """Rows of whole 16-byte chunks, which stay in registers."""
    Problem(N, V, D, DTYPES[dtype], seed=N + V + D).check()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [64, 128, 200])
def test_negative_and_zero_gradients(D, dtype):
    for negative in (0.3, 1.0):
        p = Problem(300, 500, D, DTYPES[dtype], seed=D)
        way = torch.rand(300, generator=torch.Generator().manual_seed(1)).cuda()
        p.grad[way < negative] *= -1
        p.grad[way > 0.8] = 0
        p.check()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_logits_that_grow_along_the_table(dtype):
    """Each tile of the table brings larger logits than all before it, or smaller ones."""
    for way in (1, -1):
        p = Problem(70, 2000, 64, DTYPES[dtype], seed=5, left_out=0.0)
        p.x[:] = 0.5
        ramp = torch.linspace(-way * 100, way * 100, 2000, device="cuda") / 32
        p.table[:] = ramp[:, None].to(p.dtype) + 0.01 * p.table
        p.check()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("wide", [3, 4, 8])
def test_rows_of_wider_buffers(wide, dtype):
    Problem(150, 700, 96, DTYPES[dtype], seed=2, wide=wide).check()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("N,V,D", [(300, 500, 64), (300, 500, 120), (70, 500, 130)])
def test_rows_that_start_inside_others(N, V, D, dtype):
    """x and the table one value into their buffers, each alone and both."""
    for x_from, table_from in ((1, 0), (0, 1), (1, 1)):
        p = Problem(N, V, D + 1, DTYPES[dtype], seed=17)
        p.x = p.x[:, x_from:x_from + D] if x_from else p.x[:, :D].contiguous()
        p.table = p.table[:, table_from:table_from + D] if table_from else p.table[:, :D].contiguous()
        p.check()


@pytest.mark.parametrize("scale", [0.05, 3.0])
def test_scale_and_index_types(scale):
    Problem(70, 500, 64, torch.float32, seed=3, scale=scale, index=torch.int32).check()
    Problem(70, 500, 64, torch.bfloat16, seed=3, scale=scale).check()


def test_confident_rows():
    """Targets whose probability is nearly one, and logits of some hundreds."""
    Problem(100, 400, 64, torch.float32, seed=4, spread=12.0).check()
    Problem(100, 400, 64, torch.bfloat16, seed=4, spread=12.0).check()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_without_a_target_reach_nothing(dtype):
    """Padding that holds NaN or infinities: losses of 0, gradients of 0, the table's untouched."""
    p = Problem(200, 600, 64, DTYPES[dtype], seed=5)
    p.targets[:50] = torch.tensor([-1, -100, 600, 1 << 40, -(1 << 40)], device="cuda").repeat(10)
    p.check()
    clean = p.run()
    out = p.targets < 0
    out |= p.targets >= 600
    p.x[out] = float("nan")
    p.x[3] = torch.inf
    p.grad[out] = float("nan")
    got = p.run()
    assert not got["loss"][out].any() and not got["dx"][out].any()
    for name in ("loss", "dx", "dtable"):
        assert torch.equal(got[name], clean[name]), name


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("N,V,D", [(300, 1300, 40), (300, 1300, 130), (11000, 12000, 520)])
def test_rows_of_nan_in_the_table_reach_every_row(N, V, D, dtype):
    """Whole blocks of the table that hold nothing else, before and behind others."""
    for first in (0, V // 2):
        p = Problem(N, V, D, DTYPES[dtype])
        p.table[first:first + 512] = float("nan")
        _, lse = tbe.softmax_loss(p.x, p.table, p.targets)
        assert bool(lse.isnan().all())


def test_no_targets_at_all():
    p = Problem(30, 200, 64, torch.float16, seed=6, left_out=2.0)
    got = p.run()
    assert not got["loss"].any() and not got["dx"].any() and not got["dtable"].any()
    p.check(got)


def test_no_rows():
    x, t = torch.zeros(0, 16, device="cuda"), torch.ones(1031, 16, device="cuda")
    loss, lse = tbe.softmax_loss(x, t, torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert loss.shape == (0,) and lse.shape == (0,)
    dx, dt = tbe.softmax_loss_backward(x, t, torch.zeros(0, dtype=torch.int64, device="cuda"), lse, loss)
    assert dx.shape == (0, 16) and dt.shape == (1031, 16) and not dt.any()


def test_one_gradient_alone():
    for dtype in DTYPES.values():
        p = Problem(150, 1000, 96, dtype, seed=7)
        both = p.run()
        for need in ("dx", "dtable"):
            dx, dt = tbe.softmax_loss_backward(p.x, p.table, p.targets, both["lse"], p.grad, need_dx=need == "dx",
                                               need_dtable=need == "dtable")
            assert (dx is None) == (need != "dx") and (dt is None) == (need != "dtable")
            assert torch.equal(both[need], dx if need == "dx" else dt), need


def test_gradients_of_very_different_rows():
    """fp16: rows whose gradients are 2^-12 of the largest keep theirs."""
    p = Problem(100, 800, 64, torch.float16, seed=8)
    p.grad[::2] *= 2.0 ** -12
    p.grad *= 64
    p.check()
    p.grad *= 2.0 ** -30
    p.check()
    p.grad.zero_()
    p.check()


@pytest.mark.parametrize("D", [16, 17])
def test_many_rows(D):
    """More rows than one piece of the logits' gradients has room for, the last piece short (17)."""
    N, V = 70000, 5000
    p = Problem(N, V, D, torch.bfloat16, seed=9)
    got = p.run()
    z = p.x.float() @ p.table.float().t()
    # 32-bit reference, some roundings of its own: sums of 5000 terms, as the kernels'
    logp = torch.log_softmax(z, 1)
    real = p.targets >= 0
    d = logp.exp()
    d[torch.arange(N, device="cuda"), p.targets.clamp(min=0)] -= 1
    d = torch.where(real[:, None], d * p.grad[:, None], 0)
    dx = (d.double() @ p.table.double())
    dt = (d.double().t() @ p.x.double())
    size_x, size_t = d.double().abs() @ p.table.double().abs(), d.double().abs().t() @ p.x.double().abs()
    half = ref.half_step(torch.bfloat16)
    assert ((got["dx"].double() - dx).abs() <= 2 * half * size_x + half * dx.abs()).all()
    assert ((got["dtable"].double() - dt).abs() <= 2 * half * size_t + half * dt.abs()).all()


def test_same_bits_every_time():
    p = Problem(700, 3000, 136, torch.bfloat16, seed=10)
    first = p.run()
    for _ in range(3):
        again = p.run()
        assert all(torch.equal(first[n], again[n]) for n in first)


def test_another_stream():
    p = Problem(300, 2000, 128, torch.bfloat16, seed=11)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = p.run()
    side.synchronize()
    p.check(got)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_graph_replays_match_eager_calls(dtype):
    p = Problem(200, 1500, 100, DTYPES[dtype], seed=12)
    p.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = p.run()
    for i in range(4):
        q = Problem(200, 1500, 100, DTYPES[dtype], seed=50 + i)
        for name in ("x", "table", "targets", "grad"):
            getattr(p, name).copy_(getattr(q, name))
        want = p.run()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[n]) for n in want), i


def test_gradients_by_differences():
    """Along a random direction, in fp32: the difference's third-order rest is below 1e-6 of it and
    the losses' rounding 2^-22 of sums of 60 values of about 6, over a step of 2^-6."""
    p = Problem(60, 300, 32, torch.float32, seed=13)
    got = p.run()
    g = torch.Generator().manual_seed(14)
    for name, grad in (("x", got["dx"]), ("table", got["dtable"])):
        t = getattr(p, name)
        keep, way = t.clone(), torch.randn(t.shape, generator=g).cuda()
        way /= way.norm()
        values = []
        for sign in (1, -1):
            t.copy_(keep + sign * 2.0 ** -6 * way)
            values.append((tbe.softmax_loss(p.x, p.table, p.targets)[0].double() * p.grad.double()).sum().item())
        t.copy_(keep)
        slope = (values[0] - values[1]) * 2.0 ** 5
        want = (grad.double() * way.double()).sum().item()
        assert abs(slope - want) < 1e-4, (name, slope, want)
