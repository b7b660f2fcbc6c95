"""Dropout with the mask recomputed from (p, seed, offset), against its definition."""
import numpy as np
import pytest
import torch

import layers_reference as ref
import table_embedding_bag_amd as tbe
from gpu_check import guarded_empty, guards_intact

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
IDS = ["fp32", "fp16", "bf16"]


def _randn(shape, dtype, seed, wide=0):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn((*shape[:-1], shape[-1] + wide), generator=g).to(dtype).cuda()
    return t[..., :shape[-1]] if wide else t


def _expected(x, residual, p, seed, offset):
    v = x.double().cpu().numpy()
    mask = ref.kept(v.size, p, seed, offset).reshape(v.shape)
    y = np.where(mask, v / (1 - p) if p < 1 else 0.0, 0.0)
    bound = 2 * ref.U32 * np.abs(y)          # the scale's rounding and the product's
    if residual is not None:
        y = y + residual.double().cpu().numpy()
        bound = bound + ref.U32 * (np.abs(y) + bound)
    return y, ref.rounded(bound, y, x.dtype), mask


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("shape,wide", [((1, 1), 0), ((1, 3), 0), ((5, 1), 7), ((7, 33), 0), ((7, 33), 3),
                                        ((64, 128), 0), ((33, 100), 4), ((9, 1000), 24), ((13, 5), 1),
                                        ((3, 2049), 0)])
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
def test_matches_definition(shape, wide, residual, dtype):
    print(f"[dropout] {shape} wide={wide} residual={residual} {dtype}", flush=True)
    x = _randn(shape, dtype, 1, wide)
    r = _randn(shape, dtype, 2) if residual else None
    buf, out = guarded_empty(shape, dtype)
    y = tbe.dropout(x, 0.3, 12345678901234567890, 77, residual=r, out=out)
    assert y is out
    want, bound, mask = _expected(x, r, 0.3, 12345678901234567890, 77)
    ref.assert_close(y, want, bound, "y")
    assert guards_intact(buf)
    assert torch.equal(tbe.dropout(x, 0.3, 12345678901234567890, 77, residual=r), y)
    if not residual:
        assert (y.cpu()[torch.from_numpy(~mask)] == 0).all()
        dx = tbe.dropout_backward(x, 0.3, 12345678901234567890, 77)
        assert torch.equal(dx, y)


@pytest.mark.parametrize("p", [0.0, 1e-12, 0.5, 1 - 2.0 ** -32, 1.0])
def test_probabilities_and_values_that_are_not_finite(p):
    x = _randn((16, 64), torch.float32, 3)
    x[0, :] = float("inf")
    x[1, :] = float("nan")
    x[2, :] = -float("inf")
    y = tbe.dropout(x, p, 9, 0).cpu()
    mask = torch.from_numpy(ref.kept(16 * 64, p, 9, 0).reshape(16, 64))
    assert (y[~mask] == 0).all()              # a dropped element is 0 whatever it was
    rest = mask.clone()
    rest[:3] = False
    if p < 1:
        want = x.cpu().double()[rest] / (1 - p)
        assert ((y.double()[rest] - want).abs() <= 4 * ref.U32 * want.abs()).all()
        assert torch.isnan(y[1][mask[1]]).all() and (y[0][mask[0]] == float("inf")).all()
    if p == 0.0:
        assert mask.all()
    if p == 1.0:
        assert not mask.any() and (y == 0).all()


@pytest.mark.parametrize("offset", [2 ** 32 - 3, 2 ** 63, 2 ** 64 - 2], ids=["word", "sign", "wrap"])
def test_counters_over_their_words_ends(offset):
    x = torch.ones(1, 64, device="cuda")
    y = tbe.dropout(x, 0.5, 2 ** 64 - 1, offset).cpu().numpy()
    assert np.array_equal(y != 0, ref.kept(64, 0.5, 2 ** 64 - 1, offset).reshape(1, 64))


def test_mask_is_split_by_offsets():
    """Two halves of a tensor, the second with the counters that follow, drop as the whole."""
    x = _randn((8, 64), torch.bfloat16, 5)
    whole = tbe.dropout(x, 0.25, 3, 10)
    halves = torch.cat([tbe.dropout(x[:4], 0.25, 3, 10), tbe.dropout(x[4:], 0.25, 3, 10 + 4 * 64 // 4)])
    assert torch.equal(whole, halves)


def test_in_place_other_ranks_and_empty():
    x = _randn((5, 6, 7), torch.float16, 6)
    want = tbe.dropout(x, 0.4, 1, 2)
    assert want.shape == x.shape
    assert torch.equal(want.view(1, -1), tbe.dropout(x.view(1, -1), 0.4, 1, 2))
    assert tbe.dropout(x, 0.4, 1, 2, out=x) is x and torch.equal(x, want)
    for shape in ((0, 8), (8, 0), (0,)):
        assert tbe.dropout(torch.empty(shape, device="cuda"), 0.4, 1, 2).shape == shape


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("wide", [0, 5])
def test_many_elements(dtype, wide):
    """Sizes past the switch to several groups a thread, against the same map taken in slices."""
    rows, cols = 8193, 2050
    x = _randn((rows, cols), dtype, 7, wide)
    y = tbe.dropout(x, 0.1, 5, 0)
    step = 512                                # rows of a whole number of counters
    for lo in range(0, rows, step):
        part = tbe.dropout(x[lo:lo + step], 0.1, 5, lo * cols // 4)
        assert torch.equal(part, y[lo:lo + step])
    share = (y != 0).float().mean().item()
    assert abs(share - 0.9) < 6 * (0.09 / y.numel()) ** 0.5 + 1e-6


def test_graph_replays_match_eager_calls():
    x = _randn((300, 130), torch.bfloat16, 8)
    r = _randn((300, 130), torch.bfloat16, 9)
    out = torch.empty_like(x)
    tbe.dropout(x, 0.2, 4, 4, residual=r, out=out)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            tbe.dropout(x, 0.2, 4, 4, residual=r, out=out)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        x.copy_(_randn((300, 130), torch.bfloat16, 20 + i))
        want = tbe.dropout(x, 0.2, 4, 4, residual=r)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
