"""The choice of experts and its gradient."""
import pytest
import torch

import heads_reference as ref
import table_embedding_bag_amd as tbe

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def check(logits, k, bias=None, grad_seed=0, got=None, **kw):
    N, E = logits.shape
    g = torch.Generator().manual_seed(grad_seed)
    grad = torch.randn(N, k, generator=g).cuda()
    want = ref.route(logits.double(), k, bias=bias, g=grad.double(), **kw)
    back = {n: v for n, v in kw.items() if n in ("scores", "renormalize", "scale")}
    if got is None:
        ids, weights = tbe.route(logits, k, bias=bias, **kw)
        got = ids, weights, tbe.route_backward(logits, ids, grad, **back)
    ids, weights, dlogits = got
    assert torch.equal(ids, want["ids"]), (ids != want["ids"]).nonzero()[:3]
    ref.assert_close(weights, *want["weights"], "weights")
    ref.assert_close(dlogits, *want["dlogits"], "dlogits")
    return got


def logits_of(N, E, dtype, seed=0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(N, E, generator=g)).to(dtype).cuda()


def bias_of(E, seed=0):
    return (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(seed + 100))).cuda()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (5, 3), (16, 16), (17, 4), (33, 5), (64, 2), (100, 8), (128, 6),
                                 (250, 8), (256, 8), (257, 1), (300, 16), (1024, 8)])
def test_one_group(E, k, renormalize, scores, dtype):
    for N in (1, 37):
        check(logits_of(N, E, DTYPES[dtype], seed=E + k), k, scores=scores, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(2, 1), (13, 3), (64, 6), (160, 6), (256, 8), (512, 10)])
def test_bias(E, k, scores, dtype):
    check(logits_of(200, E, DTYPES[dtype], seed=E), k, bias=bias_of(E), scores=scores)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("E,k,groups,top", [(4, 1, 4, 1), (12, 3, 3, 2), (64, 8, 8, 4), (256, 8, 8, 4), (250, 5, 5, 1),
                                            (256, 16, 16, 16), (1024, 16, 16, 3), (16, 8, 16, 8), (30, 2, 15, 3)])
def test_groups(E, k, groups, top, with_bias, group_score, scores, dtype):
    check(logits_of(150, E, DTYPES[dtype], seed=E + top), k, bias=bias_of(E) if with_bias else None, scores=scores,
          groups=groups, top_groups=top, group_score=group_score)


@pytest.mark.parametrize("E,k,groups,top", [(8, 3, 1, 1), (64, 8, 8, 3), (400, 9, 4, 2)])
def test_ties_go_to_the_lowest_index(E, k, groups, top):
    x = torch.randint(0, 3, (300, E), generator=torch.Generator().manual_seed(1)).float().cuda()
    for dtype in DTYPES.values():
        for bias in (None, torch.zeros(E, device="cuda"), torch.randint(0, 2, (E,)).float().cuda()):
            for scores in ("softmax", "sigmoid"):
                check(x.to(dtype), k, bias=bias, scores=scores, groups=groups, top_groups=top, group_score="top2")


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_scores_closer_than_fp32_tells(scores):
    """Logits that differ in their last bits, at sizes where their fp32 scores agree: the choice is
    still that of the exact scores."""
    g = torch.Generator().manual_seed(2)
    steps = torch.randint(-3, 4, (500, 96), generator=g)
    base = torch.rand(500, 1, generator=g) * 2 + 0.5
    x = (base * (1 + steps * 2.0 ** -23)).float().cuda()
    check(x, 8, bias=torch.zeros(96, device="cuda"), scores=scores)
    check(x, 8, scores=scores)
    check(x, 8, scores=scores, groups=8, top_groups=3, group_score="top2")
    far = (17 + 3 * torch.rand(500, 96, generator=g)).cuda()   # sigmoids of 1 - 2^-25 and above
    check(far, 8, bias=torch.zeros(96, device="cuda"), scores=scores)
    check(far, 8, bias=bias_of(96), scores=scores)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_masked_experts(dtype, renormalize, scores):
    """Rows whose logits are partly or wholly -inf, the type's lowest value, NaN or +inf."""
    t = DTYPES[dtype]
    x = logits_of(12, 40, t, seed=3)
    low = torch.finfo(t).min
    x[0, 5:] = -torch.inf
    x[1, 2:] = -torch.inf
    x[2] = -torch.inf
    x[3, 3:] = low
    x[4] = low
    x[5, ::2] = float("nan")
    x[6] = float("nan")
    x[7, 9] = torch.inf
    x[8, 10:] = torch.finfo(t).max
    for bias in (None, bias_of(40)):
        for groups, top in ((1, 1), (4, 2)):
            ids, w, d = check(x, 5, bias=bias, scores=scores, renormalize=renormalize, groups=groups, top_groups=top)
            assert not w[2].any() and not w[6].any() and not d[2].any() and not torch.isnan(w).any()


@pytest.mark.parametrize("E,groups,top", [(48, 1, 1), (256, 8, 3), (320, 16, 9)])
def test_biases_that_close_experts(E, groups, top):
    """-inf and NaN biases: the expert is chosen for want of others only, the lowest index first."""
    x = logits_of(50, E, torch.float32, seed=11)
    for first in (E // 2, 3, 0):
        bias = bias_of(E)
        bias[first:] = -torch.inf
        for scores in ("softmax", "sigmoid"):
            want = check(x, 6, bias=bias, scores=scores, groups=groups, top_groups=top, group_score="max")
            other = bias.clone()
            other[first + 1::2] = float("nan")
            got = tbe.route(x, 6, bias=other, scores=scores, groups=groups, top_groups=top, group_score="max")
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k", [(12, 3, 1, 3), (16, 8, 4, 8), (24, 3, 2, 12), (32, 4, 2, 9), (48, 3, 2, 4), (48, 3, 2, 16),
                                            (64, 8, 4, 6), (64, 8, 4, 16), (250, 5, 2, 7), (256, 8, 4, 16), (512, 4, 2, 16),
                                            (1024, 16, 3, 16)])
def test_groups_without_an_open_expert(E, groups, top, k, scores, dtype):
    """Rows with fewer open groups than are taken: the rest are the lowest ones, whatever a lane's
    experts are of a group."""
    t, per = DTYPES[dtype], E // groups
    shut = -torch.inf
    x = torch.full((6 + 3 * groups, E), shut, dtype=t, device="cuda")
    some = logits_of(x.shape[0], E, t, seed=12)
    x[1] = float("nan")
    x[2, ::2] = float("nan")
    x[3, 0], x[4, E - 1], x[5, E // 2] = some[3, 0], torch.inf, torch.finfo(t).min
    for g in range(groups):
        at = slice(g * per, (g + 1) * per)
        row = 6 + 3 * g
        x[row, at] = some[row, at]                       # one open group
        x[row + 1, g * per + per // 2] = some[row + 1, 0]  # one open expert
        x[row + 2] = some[row + 2]                       # all but one group open
        x[row + 2, at] = shut
    for renormalize in (True, False):
        ids, w, d = check(x, k, scores=scores, groups=groups, top_groups=top, renormalize=renormalize)
        assert bool(((ids >= 0) & (ids < E)).all()) and not w[:3].any() and not d[:3].any()
    check(x, k, bias=bias_of(E), scores=scores, groups=groups, top_groups=top, group_score="top2")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top", [(16, 8, 3), (32, 4, 2), (64, 8, 4), (256, 8, 3), (256, 16, 5), (1024, 16, 3), (250, 5, 2)])
def test_biases_that_close_parts_of_groups(E, groups, top, scores, dtype):
    """A group's score is the sum of its best two open experts, wherever its closed ones lie."""
    per = E // groups
    x = logits_of(60, E, DTYPES[dtype], seed=13)
    lane = max(1, min(16, E // 16))     # experts side by side in a lane
    random = torch.rand(E, generator=torch.Generator().manual_seed(14)) < 0.8
    for name in ("first", "last", "all but one", "all but two", "random"):
        bias = bias_of(E)
        for g in range(0, groups, 2):
            at = torch.arange(g * per, (g + 1) * per)
            shut = {"first": at[:lane], "last": at[-lane:], "all but one": at[at != g * per + g % per],
                    "all but two": at[1:-1], "random": at[random[at]]}[name]
            bias[shut] = -torch.inf
        want = check(x, min(6, per * top), bias=bias, scores=scores, groups=groups, top_groups=top, group_score="top2")
        bias[bias == -torch.inf] = float("nan")
        got = tbe.route(x, min(6, per * top), bias=bias, scores=scores, groups=groups, top_groups=top, group_score="top2")
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), name


def test_strided_rows_and_outputs():
    wide = logits_of(60, 90, torch.bfloat16, seed=4)
    view = wide[:, 3:80]
    out = torch.full((60, 100), 7.0, dtype=torch.bfloat16, device="cuda")
    ids, w, d = check(view, 6, scores="sigmoid", bias=bias_of(77))
    grad = torch.randn(60, 6, generator=torch.Generator().manual_seed(0)).cuda()
    tbe.route_backward(view, ids, grad, scores="sigmoid", out=out[:, :77])
    assert torch.equal(out[:, :77], d) and (out[:, 77:] == 7).all()


def test_an_expert_given_twice_and_wrong_ids():
    """route never gives an expert twice; a caller's ids may: each has its part."""
    x = logits_of(6, 20, torch.float32, seed=5)
    ids = torch.tensor([[3, 3, 5], [1, 2, 2], [0, 19, 20], [-1, 4, 1 << 30], [7, 7, 7], [-5, -1, 99]],
                       dtype=torch.int32, device="cuda")
    grad = torch.randn(6, 3, generator=torch.Generator().manual_seed(6)).cuda()
    for scores in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            got = tbe.route_backward(x, ids, grad, scores=scores, renormalize=renormalize)
            leaf = x.double().cpu().requires_grad_()
            p = torch.softmax(leaf, 1) if scores == "softmax" else torch.sigmoid(leaf)
            i = ids.cpu().long()
            on = (i >= 0) & (i < 20)
            w = torch.where(on, p.gather(1, torch.where(on, i, 0)), 0)
            if renormalize:
                total = w.sum(1, keepdim=True)
                w = torch.where(total > 0, w / torch.where(total > 0, total, 1), 0)
            (torch.where(on, w * grad.double().cpu(), 0)).sum().backward()
            # values of size 1, some tens of roundings
            assert (got.double().cpu() - leaf.grad).abs().max() < 100 * ref.U32 * grad.abs().max().item()


def test_no_rows():
    ids, w = tbe.route(torch.zeros(0, 8, device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    assert tbe.route_backward(torch.zeros(0, 8, device="cuda"), ids, w).shape == (0, 8)


def test_many_rows():
    check(logits_of(20003, 64, torch.bfloat16, seed=7), 6, scores="sigmoid", bias=bias_of(64), groups=8, top_groups=4,
          group_score="top2")
    check(logits_of(40001, 24, torch.float32, seed=8), 3)


def test_graph_replays_match_eager_calls():
    x = logits_of(300, 128, torch.float32, seed=9)
    b = bias_of(128)
    grad = torch.randn(300, 8, device="cuda")

    def both():
        ids, w = tbe.route(x, 8, scores="sigmoid", bias=b, groups=8, top_groups=4, group_score="top2")
        return ids, w, tbe.route_backward(x, ids, grad, scores="sigmoid")

    both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    for i in range(4):
        x.copy_(logits_of(300, 128, torch.float32, seed=30 + i))
        want = both()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), i
