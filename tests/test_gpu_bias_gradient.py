"""The bias's gradient of the grouped linear layer: sums over many rows of one sign, beside the
weights' gradient (whole groups and chunks of rows) and alone."""
import pytest
import torch

import layers_reference as ref
import table_embedding_bag_amd as tbe

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def _check(db, grad, offsets, dtype):
    """A sum is off by the tree of a fragment (3 additions), the long sum's last one, the two halves'
    or the 16 waves' (and the chunks') joins, 3 each, and what the long sum's second float loses of
    itself: n / 8 additions of at most n / 8 half steps of the sum, (n / 8)^2 U32 half steps (a few
    here).  12 and those, relative to the sum of the magnitudes."""
    for g, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        v = grad[lo:hi].double()
        want, size = v.sum(0), v.abs().sum(0)
        bound = (12 + ((hi - lo) / 8) ** 2 * ref.U32) * ref.U32 * size
        bound = bound + ref.half_step(dtype) * (want.abs() + bound) + ref.TINY[dtype]
        off = (db[g].double() - want).abs()
        assert (off <= bound).all(), (g, float((off / bound).max()), float((off / size.clamp(min=1e-30)).max()))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("data", ["equal", "positive"])
@pytest.mark.parametrize("name,sizes,K,M", [("chunks", [40001], 96, 80), ("128", [33000, 3, 0, 40001], 2100, 1000),
                                            ("256", [40001], 4096, 4096), ("64-chunks", [30000, 0, 17], 40, 24)])
def test_sums_over_many_rows(name, sizes, K, M, data, dtype):
    print(f"[bias gradient] {name} {data} {dtype}", flush=True)
    dt = DTYPES[dtype]
    off = [0]
    for n in sizes:
        off.append(off[-1] + n)
    N, G = off[-1], len(sizes)
    gen = torch.Generator(device="cuda").manual_seed(40)
    grad = torch.rand(N, M, generator=gen, device="cuda") if data == "positive" else torch.full((N, M), 0.1, device="cuda")
    grad = grad.to(dt)
    x = torch.zeros(N, K, dtype=dt, device="cuda")
    w = torch.zeros(G, M, K, dtype=dt, device="cuda")
    offsets = torch.tensor(off, device="cuda")
    _, dw, db = tbe.grouped_linear_backward(x, w, offsets, grad, bias=True, need_dx=False)
    _check(db, grad, off, dt)
    _, _, alone = tbe.grouped_linear_backward(x, w, offsets, grad, bias=True, need_dx=False, need_dweight=False)
    _check(alone, grad, off, dt)


def test_infinite_sums():
    """An infinity is the sum's, two of different signs make NaN, and neighbours keep their values."""
    grad = torch.ones(5000, 70, device="cuda")
    grad[1234, 3] = float("inf")
    grad[77, 5], grad[4000, 5] = float("inf"), -float("inf")
    grad[4999, 7] = float("nan")
    x, w = torch.zeros(5000, 64, device="cuda"), torch.zeros(1, 70, 64, device="cuda")
    off = torch.tensor([0, 5000], device="cuda")
    for need in (True, False):
        db = tbe.grouped_linear_backward(x, w, off, grad, bias=True, need_dx=False, need_dweight=need)[2][0].cpu()
        assert db[3] == float("inf") and torch.isnan(db[5]) and torch.isnan(db[7])
        keep = torch.ones(70, dtype=torch.bool)
        keep[[3, 5, 7]] = False
        assert (db[keep] == 5000).all()


def test_no_workspace_without_the_weights_gradient():
    """Sizes whose weights' gradient is summed in chunks of rows, with a workspace of megabytes."""
    N, G, K, M = 20000, 2, 320, 256
    assert tbe.layers._grouped_sizes(N, G, K, M, torch.float32)[1] > 1 << 20
    x, w, grad = torch.ones(N, K, device="cuda"), torch.ones(G, M, K, device="cuda"), torch.ones(N, M, device="cuda")
    off = torch.tensor([0, 7000, N], device="cuda")
    tbe.grouped_linear_backward(x, w, off, grad, bias=True, need_dx=False, need_dweight=False)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    db = tbe.grouped_linear_backward(x, w, off, grad, bias=True, need_dx=False, need_dweight=False)[2]
    assert torch.cuda.max_memory_allocated() - before <= 1 << 16
    assert (db[0] == 7000).all() and (db[1] == 13000).all()
