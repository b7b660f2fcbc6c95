"""The linear layer of each ragged row group and its gradients."""
import numpy as np
import pytest
import torch

import layers_reference as ref
import table_embedding_bag_amd as tbe
from gpu_check import guarded_empty, guards_intact

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def _np(t):
    return None if t is None else t.double().cpu().numpy()


class Problem:
    def __init__(self, sizes, K, M, dtype, seed=0, bias=True, wide=0, index=torch.int64):
        g = torch.Generator().manual_seed(seed)
        self.dtype = dtype
        self.off = np.concatenate([[0], np.cumsum(np.asarray(sizes, dtype=np.int64))])
        N, G = int(self.off[-1]), len(sizes)
        self.N, self.G, self.K, self.M = N, G, K, M
        make = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
        self.x = make(N, K + wide)[:, :K]
        self.w = make(G, M, K)
        self.bias = make(G, M) if bias else None
        self.grad = make(N, M + wide)[:, :M]
        self.offsets = torch.from_numpy(self.off).to(index).cuda()

    def run(self):
        y = tbe.grouped_linear(self.x, self.w, self.offsets, bias=self.bias)
        dx, dw, db = tbe.grouped_linear_backward(self.x, self.w, self.offsets, self.grad,
                                                 bias=self.bias is not None)
        return {"y": y, "dx": dx, "dw": dw, "db": db}

    def check(self, got=None):
        got = got or self.run()
        torch.cuda.synchronize()
        want = ref.grouped(_np(self.x), _np(self.w), self.off, _np(self.bias), _np(self.grad))
        for name, t in got.items():
            if t is not None:
                v, bound = want[name]
                ref.assert_close(t, v, ref.rounded(bound, v, self.dtype), name)


SIZES = {
    "one-row": [1],
    "ones": [1] * 9,
    "empty": [0, 0, 5, 0],
    "tile-ends": [64, 16, 17, 15, 128, 129, 1],
    "skewed": [300, 2, 0, 40, 7],
}


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("K,M", [(1, 1), (8, 16), (64, 64), (250, 130), (33, 65), (136, 200)])
def test_forward_and_backward(sizes, K, M, dtype):
    print(f"[grouped] {sizes} K={K} M={M} {dtype}", flush=True)
    Problem(SIZES[sizes], K, M, DTYPES[dtype], seed=K + M, bias=K != 64, wide=3 if K == 33 else 0,
            index=torch.int32 if M == 65 else torch.int64).check()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("sizes,K,M,wide", [([700, 0, 513, 1], 320, 272, 8), ([511, 1025], 1032, 264, 0),
                                            ([257, 300], 264, 1100, 4)])
def test_larger(sizes, K, M, wide, dtype):
    print(f"[grouped] {sizes} K={K} M={M} {dtype}", flush=True)
    Problem(sizes, K, M, DTYPES[dtype], seed=1, wide=wide).check()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_many_groups_of_few_rows(dtype):
    g = np.random.default_rng(2)
    print(f"[grouped] many {dtype}", flush=True)
    Problem(g.integers(0, 4, 130), 72, 144, DTYPES[dtype], seed=3).check()
    Problem(g.integers(0, 3, 64), 512, 96, DTYPES[dtype], seed=4).check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name,G,N,K,M,wide", [("forward", 12, 12801, 264, 4104, 0), ("dx", 12, 12801, 4104, 264, 8),
                                               ("dw", 64, 2600, 1040, 1040, 0), ("unaligned", 12, 12801, 263, 4099, 0),
                                               ("128", 3, 16000, 1096, 1032, 0)])
def test_many_tiles(name, G, N, K, M, wide, dtype):
    """Sizes whose products take the largest tiles (and, last, those of 128 on all sides), held to
    64-bit products on the GPU."""
    print(f"[grouped] many tiles {name} {dtype}", flush=True)
    g = np.random.default_rng(20)
    p = Problem(g.multinomial(N, g.dirichlet(np.ones(G))), K, M, DTYPES[dtype], seed=21, wide=wide)
    got = p.run()
    for i in list(range(G))[:: max(1, G // 6)]:
        r = slice(int(p.off[i]), int(p.off[i + 1]))
        x, w, dy = p.x[r].double(), p.w[i].double(), p.grad[r].double().contiguous()
        b = p.bias[i].double()
        n = r.stop - r.start
        for what, mine, want, size, terms in (
                ("y", got["y"][r], x @ w.t().contiguous() + b, x.abs() @ w.abs().t().contiguous() + b.abs(), K),
                ("dx", got["dx"][r], dy @ w, dy.abs() @ w.abs(), M),
                ("dw", got["dw"][i], dy.t().contiguous() @ x, dy.abs().t().contiguous() @ x.abs(), n),
                ("db", got["db"][i], dy.sum(0), dy.abs().sum(0), n)):
            off = (mine.double() - want).abs()
            bound = (terms + 2) * ref.U32 * size
            bound = bound + ref.half_step(p.dtype) * (want.abs() + bound) + ref.TINY[p.dtype]
            assert (off <= bound).all(), (what, i, float((off / bound).max()))


def test_no_rows_and_no_groups():
    for G in (0, 3):
        off = torch.zeros(G + 1, dtype=torch.int64, device="cuda")
        x, w = torch.empty(0, 8, device="cuda"), torch.randn(G, 4, 8, device="cuda")
        assert tbe.grouped_linear(x, w, off).shape == (0, 4)
        dx, dw, db = tbe.grouped_linear_backward(x, w, off, torch.empty(0, 4, device="cuda"), bias=True)
        assert dx.shape == (0, 8) and (dw == 0).all() and (db == 0).all()
        assert dw.shape == (G, 4, 8) and db.shape == (G, 4)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("K,M", [(136, 72), (129, 70)])
def test_groups_and_rows_do_not_mix(K, M, dtype):
    """NaN and infinities in one group's rows and weights stay out of the others' results, one
    row's out of the other rows', and those behind the rows' ends out of all."""
    sizes = [40, 3, 130, 0, 70]
    p = Problem(sizes, K, M, DTYPES[dtype], seed=5, wide=8)
    clean = p.run()
    q = Problem(sizes, K, M, DTYPES[dtype], seed=5, wide=8)
    lo, hi = int(p.off[2]), int(p.off[3])
    for t in (q.x, q.grad):
        t._base[:, -8:] = float("nan")       # behind the rows' ends
        t[lo:hi] = float("nan")
    q.w[2] = float("inf")
    q.w[3] = float("nan")                    # the weights of an empty group
    q.bias[2] = float("nan")
    dirty = q.run()
    rest = torch.ones(p.N, dtype=torch.bool)
    rest[lo:hi] = False
    for name in ("y", "dx"):
        assert torch.equal(clean[name].cpu()[rest], dirty[name].cpu()[rest]), name
    for name in ("dw", "db"):
        for g in (0, 1, 3, 4):
            assert torch.equal(clean[name][g], dirty[name][g]), (name, g)
    r = Problem(sizes, K, M, DTYPES[dtype], seed=5, wide=8)
    r.x[lo + 3] = float("inf")
    y = r.run()["y"]
    rest = torch.arange(p.N) != lo + 3
    assert torch.equal(clean["y"].cpu()[rest], y.cpu()[rest])


def test_parts_of_the_gradient_and_outputs_in_their_buffers():
    p = Problem([40, 0, 33], 72, 56, torch.bfloat16, seed=6)
    full = p.run()
    b = lambda **kw: tbe.grouped_linear_backward(p.x, p.w, p.offsets, p.grad, **kw)  # noqa: E731
    dx, dw, db = b()
    assert db is None and torch.equal(dx, full["dx"]) and torch.equal(dw, full["dw"])
    dx, dw, db = b(need_dx=False, bias=True)
    assert dx is None and torch.equal(dw, full["dw"]) and torch.equal(db, full["db"])
    dx, dw, db = b(need_dweight=False)
    assert dw is None and torch.equal(dx, full["dx"])
    buf, out = guarded_empty((p.N, p.M), p.dtype)
    assert tbe.grouped_linear(p.x, p.w, p.offsets, bias=p.bias, out=out) is out
    assert torch.equal(out, full["y"]) and guards_intact(buf)
    wide = torch.full((p.N, p.M + 5), 7.0, dtype=p.dtype, device="cuda")
    tbe.grouped_linear(p.x, p.w, p.offsets, bias=p.bias, out=wide[:, :p.M])
    assert torch.equal(wide[:, :p.M], full["y"]) and (wide[:, p.M:] == 7).all()


@pytest.mark.parametrize("dtype,K,M", [("bf16", 264, 520), ("bf16", 77, 131), ("fp32", 70, 66)])
def test_every_output_within_its_buffer(dtype, K, M):
    """The C calls into guarded buffers, workspaces among them."""
    p = Problem([300, 1, 0, 213], K, M, DTYPES[dtype], seed=7)
    _, N, G, K, M, fw, bw = tbe.layers._grouped(p.x, p.w, p.offsets)
    made = {}

    def buf(name, shape, dt):
        made[name], v = guarded_empty(shape, dt)
        return v

    y, dx = buf("y", (N, M), p.dtype), buf("dx", (N, K), p.dtype)
    dw, db = buf("dw", (G, M, K), p.dtype), buf("db", (G, M), p.dtype)
    wf, wb = buf("wf", (fw,), torch.uint8), buf("wb", (bw,), torch.uint8)
    st = torch.cuda.current_stream().cuda_stream
    code = {"fp32": 0, "fp16": 1, "bf16": 2}[dtype]
    assert tbe.load().tbe_grouped_linear(p.x.data_ptr(), K, p.w.data_ptr(), p.bias.data_ptr(),
                                         p.offsets.data_ptr(), 1, y.data_ptr(), M, N, G, K, M, code,
                                         wf.data_ptr(), fw, st) == 0
    assert tbe.load().tbe_grouped_linear_backward(
        p.x.data_ptr(), K, p.w.data_ptr(), p.offsets.data_ptr(), 1, p.grad.data_ptr(), M,
        dx.data_ptr(), K, dw.data_ptr(), db.data_ptr(), N, G, K, M, code, wb.data_ptr(), bw, st) == 0
    p.check({"y": y, "dx": dx, "dw": dw, "db": db})
    for name, b in made.items():
        assert guards_intact(b), name


def test_differences():
    """y is linear in x, weight and bias: a finite step gives the projected gradients."""
    p = Problem([30, 0, 65, 2], 48, 40, torch.float32, seed=9)
    got = {k: v.double() for k, v in p.run().items()}

    def loss():
        y = tbe.grouped_linear(p.x, p.w, p.offsets, bias=p.bias)
        return (y.double() * p.grad.double()).sum()

    g = torch.Generator(device="cuda").manual_seed(10)
    for name, t in (("dx", p.x), ("dw", p.w), ("db", p.bias)):
        d = torch.randn(t.shape, generator=g, device="cuda")
        keep = t.clone()
        t.copy_(keep + d)
        hi, up = loss(), (t - keep).double()
        t.copy_(keep - d)
        lo, down = loss(), (keep - t).double()
        t.copy_(keep)
        want = (got[name] * (up + down)).sum()
        # N M outputs of magnitude sqrt(2 K) at most some times over, off by K U32 of the terms
        rest = 4 * p.N * p.M * p.K * ref.U32 * (2 * p.K) ** 0.5
        assert abs((hi - lo) - want) <= rest, (name, float(hi - lo), float(want), rest)


def test_same_bits_every_time():
    p = Problem([900, 3, 0, 400], 200, 264, torch.bfloat16, seed=11)
    first = p.run()
    for _ in range(4):
        again = p.run()
        for name in first:
            assert torch.equal(first[name], again[name]), name


def test_another_stream_than_the_tensors_own():
    p = Problem([100, 0, 31], 80, 48, torch.float16, seed=12)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = p.run()
    side.synchronize()
    p.check(got)


def test_graph_replays_match_eager_calls():
    p = Problem([500, 0, 31, 90], 136, 128, torch.bfloat16, seed=13)
    p.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            out = p.run()
    torch.cuda.current_stream().wait_stream(side)
    for i in range(5):
        q = Problem([90, 31, 400, 100], 136, 128, torch.bfloat16, seed=30 + i)
        for name in ("x", "w", "bias", "grad", "offsets"):
            getattr(p, name).copy_(getattr(q, name))
        want = p.run()
        g.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(out[name], want[name]), (i, name)


@pytest.mark.parametrize("name,G,N,K,M,dtype", [("128", 75, 23200, 128, 896, "bf16"), ("128", 75, 23200, 128, 896, "fp32"),
                                                ("256", 41, 42000, 1280, 1280, "bf16")])
def test_both_gradients_in_workgroups_rounded_up(name, G, N, K, M, dtype):
    """The gradients' products in one launch, where the first's workgroups (75 x 7, 41 x 25) are no
    multiple of 8 and the ones that fill it up have nothing to do."""
    print(f"[grouped] rounded up {name} {dtype}", flush=True)
    g = np.random.default_rng(22)
    p = Problem(g.multinomial(N, np.full(G, 1 / G)), K, M, DTYPES[dtype], seed=23)
    dx, dw, db = tbe.grouped_linear_backward(p.x, p.w, p.offsets, p.grad, bias=True)
    for i in (0, G // 2, G - 1):
        r = slice(int(p.off[i]), int(p.off[i + 1]))
        x, w, dy = p.x[r].double(), p.w[i].double(), p.grad[r].double().contiguous()
        n = r.stop - r.start
        for what, mine, want, size, terms in (
                ("dx", dx[r], dy @ w, dy.abs() @ w.abs(), M),
                ("dw", dw[i], dy.t().contiguous() @ x, dy.abs().t().contiguous() @ x.abs(), n),
                ("db", db[i], dy.sum(0), dy.abs().sum(0), n)):
            off = (mine.double() - want).abs()
            bound = (terms + 2) * ref.U32 * size
            bound = bound + ref.half_step(p.dtype) * (want.abs() + bound) + ref.TINY[p.dtype]
            assert (off <= bound).all(), (what, i, float((off / bound).max()))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("K,M,wide", [(130, 134, 0), (2, 6, 2), (66, 258, 6), (262, 70, 4)])
def test_rows_of_words(sizes, K, M, wide, dtype):
    """Rows of 2-byte values that start at multiples of 4 bytes, but not of 16."""
    print(f"[grouped] words {sizes} {K} {M} {wide} {dtype}", flush=True)
    Problem(SIZES[sizes], K, M, DTYPES[dtype], seed=24, wide=wide).check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_odd_columns_in_rows_of_words(dtype):
    """An odd number of columns, whose last shares its word with what follows the row: that is NaN
    here, and reaches no output."""
    print(f"[grouped] odd columns {dtype}", flush=True)
    p = Problem([70, 0, 3, 200], 34, 37, DTYPES[dtype], seed=25)
    for name, cols in (("x", 34), ("grad", 37)):
        buf = torch.full((p.N, 40 if name == "grad" else 34 + 4), float("nan"), dtype=p.dtype, device="cuda")
        buf[:, :cols] = getattr(p, name)
        setattr(p, name, buf[:, :cols])
    p.check()


@pytest.mark.parametrize("name,G,N,K,M", [("forward", 12, 12801, 262, 4098), ("dx", 12, 12801, 4098, 262),
                                          ("dw", 64, 2600, 1042, 1038), ("128", 3, 16000, 1098, 1030)])
def test_many_tiles_of_rows_of_words(name, G, N, K, M):
    test_many_tiles(name, G, N, K, M, 0, "bf16")
