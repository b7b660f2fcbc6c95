"""Layer norm and its gradients."""
import pytest
import torch

import heads_reference as ref
import table_embedding_bag_amd as tbe

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def inputs(N, D, dtype, seed=0, wide=0, shift=1.0):
    g = torch.Generator().manual_seed(seed)
    make = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (make(N, D + wide) * (0.5 + torch.rand(N, 1, generator=g)) + shift).to(dtype).cuda()[:, :D]
    grad = make(N, D + wide).to(dtype).cuda()[:, :D]
    return x, make(D).to(dtype).cuda(), make(D).to(dtype).cuda(), grad


def check(x, w, b, grad, eps=1e-5, got=None):
    if got is None:
        y, stats = tbe.layer_norm(x, w, b, eps=eps)
        got = (y, stats, *tbe.layer_norm_backward(x, stats, grad, weight=w, bias=True))
    y, stats, dx, dw, db = got
    d = lambda t: None if t is None else t.double()  # noqa: E731
    want = ref.norm(d(x), d(w), d(b), eps, d(grad))
    ref.assert_close(stats[:, 0], *want["mean"], "mean")
    ref.assert_close(stats[:, 1], *want["r"], "r")
    for name, t in (("y", y), ("dx", dx), ("dweight", dw), ("dbias", db)):
        if t is not None:
            ref.assert_close(t, *want[name], name)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("N", [1, 7, 300])
@pytest.mark.parametrize("D", [1, 3, 64, 130, 256, 513, 1000, 1024, 2047, 4096, 8192, 16384])
def test_forward_and_backward(N, D, dtype):
    check(*inputs(N, D, DTYPES[dtype], seed=D + N))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("N,D", [(3, 20001), (40, 17000)])
def test_rows_too_long_for_registers(N, D, dtype):
    check(*inputs(N, D, DTYPES[dtype], seed=1))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [130, 1000, 9000])
def test_rows_of_wider_buffers(D, dtype):
    check(*inputs(50, D, DTYPES[dtype], seed=2, wide=7))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_many_rows(dtype):
    check(*inputs(20011, 96, DTYPES[dtype], seed=3))
    check(*inputs(5003, 1536, DTYPES[dtype], seed=4))


def test_without_weight_and_bias():
    x, w, b, grad = inputs(33, 200, torch.float32, seed=5)
    y, stats = tbe.layer_norm(x)
    dx, dw, db = tbe.layer_norm_backward(x, stats, grad)
    assert dw is None and db is None
    check(x, None, None, grad, got=(y, stats, dx, None, None))
    y, stats = tbe.layer_norm(x, bias=b)
    dx, dw, db = tbe.layer_norm_backward(x, stats, grad, bias=True)
    assert dw is None
    check(x, None, b, grad, got=(y, stats, dx, None, db))
    y, none = tbe.layer_norm(x, w, need_stats=False)
    assert none is None and torch.equal(y, tbe.layer_norm(x, w)[0])


def test_weights_gradients_alone():
    x, w, b, grad = inputs(700, 200, torch.bfloat16, seed=6)
    _, stats = tbe.layer_norm(x, w, b)
    full = tbe.layer_norm_backward(x, stats, grad, weight=w, bias=True)
    dx, dw, db = tbe.layer_norm_backward(x, stats, grad, weight=w, bias=True, need_dx=False)
    assert dx is None and torch.equal(dw, full[1]) and torch.equal(db, full[2])


def test_rows_with_large_means():
    """The squares are of differences from the mean: means 1000 times the spread cost no more than
    the mean's own rounding."""
    check(*inputs(20, 512, torch.float32, seed=7, shift=1000.0))


def test_equal_values_and_eps():
    x = torch.full((4, 100), 3.0, device="cuda")
    w, b = torch.ones(100, device="cuda"), torch.full((100,), 0.5, device="cuda")
    y, stats = tbe.layer_norm(x, w, b)
    assert (y == 0.5).all()
    assert (stats[:, 0] == 3).all()
    x, w, b, grad = inputs(9, 100, torch.float32, seed=8)
    check(x, w, b, grad, eps=0.0)
    check(x, w, b, grad, eps=10.0)


def test_no_rows():
    x, w = torch.zeros(0, 10, device="cuda"), torch.ones(10, device="cuda")
    y, stats = tbe.layer_norm(x, w, w)
    assert y.shape == (0, 10) and stats.shape == (0, 2)
    dx, dw, db = tbe.layer_norm_backward(x, stats, x, weight=w, bias=True)
    assert dx.shape == (0, 10) and not dw.any() and not db.any()


def test_nan_stays_in_its_row():
    x, w, b, grad = inputs(10, 300, torch.float32, seed=9)
    clean, _ = tbe.layer_norm(x, w, b)
    x[4, 17] = float("nan")
    y, stats = tbe.layer_norm(x, w, b)
    assert torch.isnan(y[4]).all()
    keep = torch.arange(10) != 4
    assert torch.equal(y[keep], clean[keep])
    dx, _, _ = tbe.layer_norm_backward(x, stats, grad, weight=w)
    assert torch.isnan(dx[4]).all() and not torch.isnan(dx[keep]).any()


def test_in_place():
    x, w, b, grad = inputs(77, 1000, torch.bfloat16, seed=10)
    y, stats = tbe.layer_norm(x, w, b)
    dx, _, _ = tbe.layer_norm_backward(x, stats, grad, weight=w)
    into = grad.clone()
    tbe.layer_norm_backward(x, stats, into, weight=w, out=into)
    assert torch.equal(into, dx)
    z = x.clone()
    tbe.layer_norm(z, w, b, out=z)
    assert torch.equal(z, y)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("N,D", [(300, 130), (77, 1000), (60, 4096), (30, 8192), (20, 16384), (9, 20001)])
def test_every_gradient_in_place(N, D, dtype):
    """dx into grad itself: the weight's and the bias's gradients are of what grad held before."""
    x, w, b, grad = inputs(N, D, DTYPES[dtype], seed=14)
    y, stats = tbe.layer_norm(x, w, b)
    want = tbe.layer_norm_backward(x, stats, grad, weight=w, bias=True)
    check(x, w, b, grad, got=(y, stats, *want))
    got = tbe.layer_norm_backward(x, stats, grad, weight=w, bias=True, out=grad)
    assert got[0] is grad
    for name, p, q in zip(("dx", "dweight", "dbias"), got, want):
        assert torch.equal(p, q), name


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("N,D", [(1 << 24, 8), (4000001, 520), (300007, 1100), (200001, 16400)])
def test_sums_whose_rounding_does_not_grow_with_the_rows(N, D, dtype):
    """Equal rows (one, N times over), whose terms' roundings all go the same way: whatever N is, a sum
    is off by at most 512 + 8 half steps of fp32, those of 512 terms and of what joins them."""
    t = DTYPES[dtype]
    g = torch.Generator().manual_seed(15)
    x = torch.randn(1, D, generator=g).to(t).cuda()
    grad = (torch.rand(1, D, generator=g) + 1 / 3).to(t).cuda()
    grad *= 2.0 ** -10      # fp16's sums stay below its largest value
    w = torch.ones(D, dtype=t, device="cuda")
    _, stats = tbe.layer_norm(x, w, w)
    _, dw, db = tbe.layer_norm_backward(x.expand(N, D), stats.expand(N, 2).contiguous(), grad.expand(N, D), weight=w,
                                        bias=True, need_dx=False)
    # one row's terms, exact for the bias; the weight's as the kernel has them, in fp32: a difference and
    # two products
    n = (x.double() - stats[:, :1].double()) * stats[:, 1:].double()
    for got, one, own in ((dw, grad.double() * n, 3), (db, grad.double(), 0)):
        want = N * one[0]
        ref.assert_close(got, want, (520 + own) * ref.U32 * want.abs(), "sum")


def test_same_bits_every_time():
    a = inputs(9000, 520, torch.float16, seed=11)
    one = [tbe.layer_norm(*a[:3])]
    one += [tbe.layer_norm_backward(a[0], one[0][1], a[3], weight=a[1], bias=True)]
    for _ in range(3):
        y, stats = tbe.layer_norm(*a[:3])
        back = tbe.layer_norm_backward(a[0], stats, a[3], weight=a[1], bias=True)
        assert torch.equal(y, one[0][0]) and all(torch.equal(p, q) for p, q in zip(back, one[1]))


def test_graph_replays_match_eager_calls():
    x, w, b, grad = inputs(900, 264, torch.bfloat16, seed=12)

    def both():
        y, stats = tbe.layer_norm(x, w, b)
        return (y, stats, *tbe.layer_norm_backward(x, stats, grad, weight=w, bias=True))

    both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    for i in range(4):
        new = inputs(900, 264, torch.bfloat16, seed=20 + i)
        for t, n in zip((x, w, b, grad), new):
            t.copy_(n)
        want = both()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), i


def test_another_stream():
    a = inputs(400, 520, torch.float32, seed=13)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y, stats = tbe.layer_norm(*a[:3])
        back = tbe.layer_norm_backward(a[0], stats, a[3], weight=a[1], bias=True)
    side.synchronize()
    check(*a, got=(y, stats, *back))
