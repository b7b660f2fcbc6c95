"""The bias's gradient of the grouped linear layer without the weights', with and without dx."""
import numpy as np
import pytest
import torch

import layers_reference as ref
import table_embedding_bag_amd as tbe
from gpu_check import guarded_empty, guards_intact

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"one-row": [1], "empty": [0, 5, 0, 0], "ragged": [0, 1, 130, 0, 63, 64, 65, 2, 16, 17, 900],
         "many": [3, 0, 1] * 40}


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("K,M,wide", [(8, 1, 0), (9, 63, 0), (16, 64, 8), (7, 65, 3), (72, 200, 1)])
@pytest.mark.parametrize("need_dx", [False, True], ids=["alone", "dx"])
def test_matches_definition(need_dx, K, M, wide, sizes, dtype):
    print(f"[bias alone] {sizes} {K} {M} {wide} {dtype} dx={need_dx}", flush=True)
    dt = DTYPES[dtype]
    g = torch.Generator().manual_seed(50)
    off = np.concatenate([[0], np.cumsum(SIZES[sizes])])
    N, G = int(off[-1]), len(SIZES[sizes])
    x, w = torch.randn(N, K, generator=g).to(dt).cuda(), torch.randn(G, M, K, generator=g).to(dt).cuda()
    buf = torch.full((N, M + wide), float("nan"), dtype=dt)      # behind the rows' ends
    buf[:, :M] = torch.randn(N, M, generator=g).to(dt)
    grad = buf.cuda()[:, :M]
    offsets = torch.from_numpy(off).cuda()
    code, stream = tbe.layers._DTYPE[dt], torch.cuda.current_stream().cuda_stream
    bb, db = guarded_empty((G, M), dt)
    xb, dx = guarded_empty((N, K), dt)
    assert tbe.load().tbe_grouped_linear_backward(
        x.data_ptr(), K, w.data_ptr(), offsets.data_ptr(), 1, grad.data_ptr(), M + wide,
        dx.data_ptr() if need_dx else None, K, None, db.data_ptr(), N, G, K, M, code, None, 0, stream) == 0
    torch.cuda.synchronize()
    want = ref.grouped(x.double().cpu().numpy(), w.double().cpu().numpy(), off, None, grad.double().cpu().numpy())
    for name, got in (("db", db),) + ((("dx", dx),) if need_dx else ()):
        v, bound = want[name]
        ref.assert_close(got, v, ref.rounded(bound, v, dt), name)
    assert guards_intact(bb) and guards_intact(xb)
    again = tbe.grouped_linear_backward(x, w, offsets, grad, bias=True, need_dx=need_dx, need_dweight=False)
    assert again[1] is None and torch.equal(again[2], db)
    assert torch.equal(again[0], dx) if need_dx else again[0] is None


def test_no_rows():
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    dx, dw, db = tbe.grouped_linear_backward(torch.empty(0, 8, device="cuda"), torch.ones(3, 70, 8, device="cuda"), off,
                                             torch.empty(0, 70, device="cuda"), bias=True, need_dweight=False)
    assert dx.shape == (0, 8) and dw is None and db.shape == (3, 70) and (db == 0).all()
