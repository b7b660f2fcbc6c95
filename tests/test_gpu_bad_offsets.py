"""Offsets that decrease, overlap or lie outside the rows: values may be wrong, but nothing outside
the buffers is written, and calls end."""
import ctypes

import numpy as np
import pytest
import torch

import table_embedding_bag_amd as tbe
from gpu_check import guarded_empty, guards_intact

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _bad(name, ranges, rows, index):
    r = np.random.default_rng(5)
    far = 2 ** 62 if index == torch.int64 else 2 ** 30
    off = {"decreasing": np.linspace(rows, 0, ranges + 1).astype(np.int64),
           "overlapping": np.arange(ranges + 1) % 2 * rows,
           "outside": r.integers(-far, far, ranges + 1),
           "shuffled": r.permutation(np.linspace(0, rows, ranges + 1).astype(np.int64)),
           "short": np.linspace(rows // 4, rows // 2, ranges + 1).astype(np.int64),
           "all-before": np.full(ranges + 1, -5), "all-behind": np.full(ranges + 1, rows + 9)}[name]
    return torch.from_numpy(off).to(index).cuda()


NAMES = ["decreasing", "overlapping", "outside", "shuffled", "short", "all-before", "all-behind"]


@pytest.mark.parametrize("index", [torch.int64, torch.int32], ids=["i64", "i32"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("G,N,K,M", [(3, 500, 72, 56), (130, 900, 33, 65), (70, 5000, 264, 136)])
def test_grouped_linear(G, N, K, M, name, dtype, index):
    """The products and both ways to the bias's gradient, every output and workspace guarded."""
    print(f"[bad offsets] grouped {G} {N} {K} {M} {name} {dtype} {index}", flush=True)
    dt = DTYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(6)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dt)  # noqa: E731
    made = []

    def buf(shape, t):
        b, v = guarded_empty(shape, t)
        made.append(b)
        return v

    off = _bad(name, G, N, index)
    x, w, grad, bias = randn(N, K), randn(G, M, K), randn(N, M), randn(G, M)
    y, dx, dw, db = buf((N, M), dt), buf((N, K), dt), buf((G, M, K), dt), buf((G, M), dt)
    code, icode = {torch.float32: 0, torch.bfloat16: 2}[dt], int(index == torch.int64)
    fw, bw = tbe.layers._grouped_sizes(N, G, K, M, dt)
    wb = buf((max(bw, 256),), torch.uint8)
    st = torch.cuda.current_stream().cuda_stream
    lib = tbe.load()
    assert lib.tbe_grouped_linear(x.data_ptr(), K, w.data_ptr(), bias.data_ptr(), off.data_ptr(), icode, y.data_ptr(),
                                  M, N, G, K, M, code, wb.data_ptr(), fw, st) == 0
    for dw_ in (dw.data_ptr(), None):
        assert lib.tbe_grouped_linear_backward(x.data_ptr(), K, w.data_ptr(), off.data_ptr(), icode, grad.data_ptr(),
                                               M, dx.data_ptr(), K, dw_, db.data_ptr(), N, G, K, M, code,
                                               wb.data_ptr(), bw, st) == 0
    torch.cuda.synchronize()
    assert all(guards_intact(b) for b in made)


@pytest.mark.parametrize("index", [torch.int64, torch.int32], ids=["i64", "i32"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("S,N,D", [(3, 900, 40), (200, 700, 67), (5, 3000, 130)])
def test_scan(S, N, D, name, dtype, index):
    print(f"[bad offsets] scan {S} {N} {D} {name} {dtype} {index}", flush=True)
    dt = DTYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(7)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    made = []

    def buf(shape, t):
        b, v = guarded_empty(shape, t)
        made.append(b)
        return v

    off = _bad(name, S, N, index)
    x, gate, grad_h = (randn(N, D).to(dt) for _ in range(3))
    initial, grad_final = randn(S, D), randn(S, D)
    nc, nw = tbe.layers._scan_sizes(N, S, D, dt)
    h, final, carry = buf((N, D), dt), buf((S, D), torch.float32), buf((nc // 4,), torch.float32)
    dx, dgate, dinitial = buf((N, D), dt), buf((N, D), dt), buf((S, D), torch.float32)
    ws = buf((nw,), torch.uint8)
    st = torch.cuda.current_stream().cuda_stream
    _, inp = tbe.layers._scan_input(x, gate, off, initial, "sigmoid")
    lib = tbe.load()
    assert lib.tbe_scan_forward(ctypes.byref(inp), h.data_ptr(), final.data_ptr(), carry.data_ptr(), ws.data_ptr(),
                                nw, st) == 0
    assert lib.tbe_scan_backward(ctypes.byref(inp), carry.data_ptr(), grad_h.data_ptr(), D, grad_final.data_ptr(), D,
                                 dx.data_ptr(), D, dgate.data_ptr(), D, dinitial.data_ptr(), ws.data_ptr(), nw,
                                 st) == 0
    torch.cuda.synchronize()
    assert all(guards_intact(b) for b in made)
