"""Every kernel of the grouped linear layer (each product, tile, row layout and type), held to
products in 64 bits on the GPU, its outputs in guarded buffers."""
import numpy as np
import pytest
import torch

import grouped_cases
import layers_reference as ref
import table_embedding_bag_amd as tbe
from gpu_check import guarded_empty, guards_intact

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def _close(what, g, mine, want, size, terms, dtype):
    """Sums of n products in fp32, in any order: off by n + 2 half steps of the sum of magnitudes."""
    bound = (terms + 2) * ref.U32 * size
    bound = bound + ref.half_step(dtype) * (want.abs() + bound) + ref.TINY[dtype]
    off = (mine.double() - want).abs()
    assert (off <= bound).all(), (what, g, float((off / bound).max()))


@pytest.mark.parametrize("case", list(grouped_cases.cases()), ids=grouped_cases.name)
def test_kernel(case):
    product, tile, chunked, layout, N, G, K, M, dtype = case
    print(f"[grouped kernel] {grouped_cases.name(case)} {N} rows {G} groups {K} -> {M}", flush=True)
    dt = DTYPES[dtype]
    r = np.random.default_rng(tile + layout)
    p = r.dirichlet(np.full(G, 1.5))
    p[r.integers(G)] = 0.0                       # an empty group
    off = np.concatenate([[0], np.cumsum(r.multinomial(N, p / p.sum()))])
    gen = torch.Generator(device="cuda").manual_seed(60)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dt)  # noqa: E731
    x, w, bias, grad = randn(N, K), randn(G, M, K), randn(G, M), randn(N, M)
    offsets = torch.from_numpy(off).cuda()
    made, stream = [], torch.cuda.current_stream().cuda_stream

    def buf(*shape):
        b, v = guarded_empty(shape, dt)
        made.append(b)
        return v

    y = dx = dw = db = None
    if product == "forward":
        y = buf(N, M)
        tbe.grouped_linear(x, w, offsets, bias=bias, out=y)
    else:
        dx = buf(N, K) if product != "dw" else None
        dw, db = (buf(G, M, K), buf(G, M)) if product != "dx" else (None, None)
        need = tbe.layers._grouped_sizes(N, G, K, M, dt)[1] if dw is not None else 0
        wb, ws = guarded_empty((need,), torch.uint8)
        made.append(wb)
        at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        assert tbe.load().tbe_grouped_linear_backward(
            x.data_ptr(), K, w.data_ptr(), offsets.data_ptr(), 1, grad.data_ptr(), M, at(dx), K, at(dw), at(db), N, G, K,
            M, tbe.layers._DTYPE[dt], ws.data_ptr(), need, stream) == 0
    torch.cuda.synchronize()
    assert all(guards_intact(b) for b in made)
    for g in range(G):
        rows = slice(int(off[g]), int(off[g + 1]))
        n = rows.stop - rows.start
        xg, wg, gg, b = x[rows].double(), w[g].double(), grad[rows].double(), bias[g].double()
        if y is not None:
            wt = wg.t().contiguous()
            _close("y", g, y[rows], xg @ wt + b, xg.abs() @ wt.abs() + b.abs(), K, dt)
        if dx is not None:
            _close("dx", g, dx[rows], gg @ wg, gg.abs() @ wg.abs(), M, dt)
        if dw is not None:
            gt = gg.t().contiguous()
            _close("dw", g, dw[g], gt @ xg, gt.abs() @ xg.abs(), n, dt)
            _close("db", g, db[g], gg.sum(0), gg.abs().sum(0), n, dt)
