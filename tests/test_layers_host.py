"""The layers on looked-up rows without a GPU: their 64-bit definitions (published vectors,
differences) and every refusal, in Python and at the C interface."""
import ctypes

import numpy as np
import pytest
import torch

import layers_reference as ref
import table_embedding_bag_amd as tbe


# --- the definitions ---------------------------------------------------------------------------

def test_philox_known_answers():
    """Random123's known answers of philox4x32 with 7 rounds for all-zero and all-one inputs need a
    full 128-bit counter; the zero one is reachable here."""
    assert ref.philox(0, 0) == [0x5f6fb709, 0x0d893f64, 0x4f121f81, 0x4f730a48]


def _loss(x, g, off, init, kind, gh, gf):
    out = ref.scan(x, g, off, init, kind)
    return (out["h"][0] * gh).sum() + (out["final"][0] * gf).sum()


@pytest.mark.parametrize("kind", ["sigmoid", "decay"])
def test_scan_gradients_by_differences(kind):
    r = np.random.default_rng(0)
    off = np.array([0, 4, 4, 5, 12])
    x, g, init = r.normal(size=(12, 3)), r.normal(size=(12, 3)), r.normal(size=(4, 3))
    gh, gf = r.normal(size=(12, 3)), r.normal(size=(4, 3))
    out = ref.scan(x, g, off, init, kind, gh, gf)
    for name, t in (("dx", x), ("dgate", g), ("dinitial", init)):
        for i in np.ndindex(t.shape):
            keep = t[i]
            t[i] = keep + 1e-5
            hi = _loss(x, g, off, init, kind, gh, gf)
            t[i] = keep - 1e-5
            lo = _loss(x, g, off, init, kind, gh, gf)
            t[i] = keep
            # third-order rest 1e-10 of terms of some magnitude, and 1e-16 / 1e-5 of rounding
            assert abs((hi - lo) / 2e-5 - out[name][0][i]) < 1e-7, (name, i)


def test_grouped_gradients_by_differences():
    r = np.random.default_rng(1)
    off = np.array([0, 3, 3, 5])
    x, w, b, gy = r.normal(size=(5, 4)), r.normal(size=(3, 2, 4)), r.normal(size=(3, 2)), r.normal(size=(5, 2))
    out = ref.grouped(x, w, off, b, gy)
    for name, t in (("dx", x), ("dw", w), ("db", b)):
        for i in np.ndindex(t.shape):
            keep = t[i]
            t[i] = keep + 1.0          # linear: any step
            hi = (ref.grouped(x, w, off, b)["y"][0] * gy).sum()
            t[i] = keep
            lo = (ref.grouped(x, w, off, b)["y"][0] * gy).sum()
            assert abs(hi - lo - out[name][0][i]) < 1e-12


# --- refusals in Python ------------------------------------------------------------------------

X = torch.zeros(6, 4)
OFF = torch.tensor([0, 2, 6])
W = torch.zeros(2, 3, 4)


@pytest.mark.parametrize("args,kw,what", [
    ((X, 1.5, 0, 0), {}, "p must"), ((X, -0.1, 0, 0), {}, "p must"), ((X, float("nan"), 0, 0), {}, "p must"),
    ((X, 0.5, -1, 0), {}, "seed"), ((X, 0.5, 0, 1 << 64), {}, "offset"),
    ((X, 0.5, 0, 0), {"residual": torch.zeros(6, 5)}, "residual"),
    ((X, 0.5, 0, 0), {"residual": torch.zeros(6, 4).half()}, "residual"),
    ((X, 0.5, 0, 0), {"out": torch.zeros(4, 6)}, "out"),
    ((X, 0.5, 0, 0), {"out": torch.zeros(1, 4).expand(6, 4)}, "overlap"),
    ((X.t(), 0.5, 0, 0), {}, "adjacent"), ((X.double(), 0.5, 0, 0), {}, "float32"),
    ((torch.zeros(2, 3, 4).transpose(0, 1), 0.5, 0, 0), {}, "contiguous"),
    ((X, 0.5, 0, 0), {}, "GPU"),
])
def test_dropout_refuses(args, kw, what):
    with pytest.raises(ValueError, match=what):
        tbe.dropout(*args, **kw)


@pytest.mark.parametrize("change,what", [
    ({"gate": torch.zeros(6, 5)}, "gate"), ({"gate": X.half()}, "gate"), ({"gate_kind": "relu"}, "gate_kind"),
    ({"offsets": OFF.float()}, "offsets"), ({"offsets": OFF[:, None]}, "offsets"),
    ({"offsets": torch.zeros(0, dtype=torch.int64)}, "offsets"), ({"offsets": OFF[:1]}, "no sequence"),
    ({"offsets": torch.zeros(6, dtype=torch.int64)[::2]}, "contiguous"),
    ({"initial": torch.zeros(3, 4)}, "initial"), ({"initial": torch.zeros(2, 4).half()}, "initial"),
    ({"x": torch.zeros(6, 4, 1)}, "2 dimensions"), ({"x": X.int()}, "x must"),
    ({"x": torch.zeros(6, 0), "gate": torch.zeros(6, 0)}, "at least one"), ({}, "GPU"),
])
def test_scan_forward_refuses(change, what):
    a = dict(x=X, gate=X, offsets=OFF)
    a.update(change)
    with pytest.raises(ValueError, match=what):
        tbe.scan_forward(**a)


@pytest.mark.parametrize("change,what", [
    ({"carry": None}, "carry"), ({"carry": torch.zeros(1 << 20)}, "carry"),
    ({"grad_h": X.half()}, "grad_h"), ({"grad_h": torch.zeros(6, 5)}, "grad_h"),
    ({"grad_final": torch.zeros(6, 4)}, "grad_final"), ({"out": (X, X.half())}, "dgate"),
    ({"out": (torch.zeros(1, 4).expand(6, 4), X)}, "overlap"), ({}, "GPU"),
])
def test_scan_backward_refuses(change, what):
    carry = torch.zeros(tbe.layers._scan_sizes(6, 2, 4, torch.float32)[0] // 4)
    a = dict(x=X, gate=X, offsets=OFF, carry=carry)
    a.update(change)
    with pytest.raises(ValueError, match=what):
        tbe.scan_backward(**a)


@pytest.mark.parametrize("change,what", [
    ({"gate": torch.zeros(6, 5)}, "gate"), ({"state": X.half()}, "state"), ({"state": torch.zeros(5, 4)}, "state"),
    ({"gate_kind": None}, "gate_kind"), ({"out_state": torch.zeros(6, 8)[:, :4]}, "contiguous"), ({}, "GPU"),
])
def test_scan_step_refuses(change, what):
    a = dict(x=X, gate=X, state=X)
    a.update(change)
    with pytest.raises(ValueError, match=what):
        tbe.scan_step(**a)


@pytest.mark.parametrize("change,what", [
    ({"weight": torch.zeros(3, 3, 4)}, "weight"), ({"weight": torch.zeros(2, 3, 5)}, "weight"),
    ({"weight": W.half()}, "weight"), ({"weight": torch.zeros(2, 4, 3).transpose(1, 2)}, "contiguous"),
    ({"offsets": OFF.double()}, "offsets"), ({"offsets": OFF[:1], "weight": W[:0]}, "no group"),
    ({"bias": torch.zeros(2, 4)}, "bias"), ({"bias": torch.zeros(2, 3).half()}, "bias"),
    ({"out": torch.zeros(6, 4)}, "out"), ({"x": X.t().contiguous().t()}, "adjacent"), ({}, "GPU"),
])
def test_grouped_linear_refuses(change, what):
    a = dict(x=X, weight=W, offsets=OFF)
    a.update(change)
    with pytest.raises(ValueError, match=what):
        tbe.grouped_linear(**a)


@pytest.mark.parametrize("grad,what", [(torch.zeros(6, 4), "grad"), (torch.zeros(6, 3).half(), "grad"),
                                       (torch.zeros(6, 3), "GPU")])
def test_grouped_linear_backward_refuses(grad, what):
    with pytest.raises(ValueError, match=what):
        tbe.grouped_linear_backward(X, W, OFF, grad)


# --- refusals at the C interface: nothing is enqueued, no GPU is touched -------------------------

INVALID, UNSUPPORTED, SMALL = 1, 2, 4
A = 4096  # an aligned address that is never read


def _dropout(**kw):
    a = dict(x=A, xs=8, r=None, rs=0, y=A, ys=8, rows=4, cols=8, dtype=0, p=0.5, seed=0, offset=0, stream=None)
    a.update(kw)
    return tbe.load().tbe_dropout(*a.values())


@pytest.mark.parametrize("kw,status", [
    ({"x": None}, INVALID), ({"y": None}, INVALID), ({"rows": -1}, INVALID), ({"cols": -1}, INVALID),
    ({"dtype": 3}, INVALID), ({"dtype": -1}, INVALID), ({"p": -1.0}, INVALID), ({"p": 1.1}, INVALID),
    ({"p": float("nan")}, INVALID), ({"ys": 7}, INVALID), ({"xs": -8}, INVALID), ({"x": A + 2}, INVALID),
    ({"y": A + 1, "dtype": 1}, INVALID), ({"r": A + 1, "dtype": 2}, INVALID), ({"r": A, "rs": -1}, INVALID),
    ({"rows": 1 << 33, "cols": 8, "ys": 8}, UNSUPPORTED), ({"rows": 0, "x": None}, 0),
])
def test_c_dropout_refuses(kw, status):
    assert _dropout(**kw) == status


def _scan_input(**kw):
    a = dict(tokens=6, seqs=2, dim=4, dtype=0, gate_kind=0, index_dtype=1, max_polls=0, x=A, x_stride=4, gate=A,
             gate_stride=4, offsets=A, initial=None, initial_stride=0)
    a.update(kw)
    return tbe._ScanInput(*a.values())


def _forward(inp, **kw):
    a = dict(h=A, final=A, carry=A, ws=A, nws=1 << 30, stream=None)
    a.update(kw)
    return tbe.load().tbe_scan_forward(None if inp is None else ctypes.byref(inp), *a.values())


def _backward(inp, **kw):
    a = dict(carry=A, gh=None, ghs=0, gf=None, gfs=0, dx=A, dxs=4, dg=A, dgs=4, di=None, ws=A, nws=1 << 30,
             stream=None)
    a.update(kw)
    return tbe.load().tbe_scan_backward(None if inp is None else ctypes.byref(inp), *a.values())


@pytest.mark.parametrize("kw,status", [
    ({"tokens": -1}, INVALID), ({"seqs": -1}, INVALID), ({"seqs": 0}, INVALID), ({"dim": 0}, INVALID),
    ({"dtype": 5}, INVALID), ({"gate_kind": 2}, INVALID), ({"index_dtype": 2}, INVALID), ({"x": None}, INVALID),
    ({"gate": None}, INVALID), ({"offsets": None}, INVALID), ({"offsets": A + 4}, INVALID), ({"x": A + 2}, INVALID),
    ({"x_stride": -4}, INVALID), ({"gate_stride": -1}, INVALID), ({"initial": A + 2}, INVALID),
    ({"tokens": 1 << 31}, UNSUPPORTED), ({"seqs": 1 << 31}, UNSUPPORTED), ({"dim": 1 << 31}, UNSUPPORTED),
    ({"tokens": 1 << 30, "dim": 1 << 20}, UNSUPPORTED),
])
def test_c_scan_refuses_inputs(kw, status):
    assert _forward(_scan_input(**kw)) == status
    assert _backward(_scan_input(**kw)) == status


def test_c_scan_refuses_outputs():
    assert _forward(None) == INVALID and _backward(None) == INVALID
    for kw in ({"h": None}, {"final": None}, {"h": A + 2}, {"final": A + 1}, {"carry": A + 8}):
        assert _forward(_scan_input(), **kw) == INVALID
    for kw in ({"carry": None}, {"dx": None}, {"dg": None}, {"dxs": 3}, {"dgs": 0}, {"gh": A, "ghs": -1},
               {"gf": A, "gfs": -1}, {"gh": A + 2}, {"gf": A + 2}, {"di": A + 2}, {"dx": A + 1}):
        assert _backward(_scan_input(), **kw) == INVALID
    assert _forward(_scan_input(tokens=0, seqs=0)) == 0


def test_c_scan_sizes_and_workspace():
    c, w = ctypes.c_size_t(1), ctypes.c_size_t(1)
    sizes = tbe.load().tbe_scan_sizes
    assert sizes(6, 2, 4, 0, ctypes.byref(c), ctypes.byref(w)) == 0
    assert sizes(6, 2, 4, 0, None, ctypes.byref(w)) == INVALID
    assert sizes(6, 0, 4, 0, ctypes.byref(c), ctypes.byref(w)) == INVALID
    assert sizes(1 << 31, 2, 4, 0, ctypes.byref(c), ctypes.byref(w)) == UNSUPPORTED
    if w.value:
        for call in (_forward, _backward):
            assert call(_scan_input(), nws=w.value - 1) == SMALL
            assert call(_scan_input(), ws=None, nws=w.value) == INVALID
            assert call(_scan_input(), ws=A + 64) == INVALID


def _step(**kw):
    a = dict(x=A, xs=4, gate=A, gs=4, state=A, ss=4, h=A, nxt=A, seqs=2, dim=4, dtype=0, kind=0, stream=None)
    a.update(kw)
    return tbe.load().tbe_scan_step(*a.values())


@pytest.mark.parametrize("kw,status", [
    ({"x": None}, INVALID), ({"gate": None}, INVALID), ({"h": None}, INVALID), ({"nxt": None}, INVALID),
    ({"dtype": 3}, INVALID), ({"kind": 2}, INVALID), ({"dim": 0}, INVALID), ({"seqs": -1}, INVALID),
    ({"xs": -1}, INVALID), ({"ss": -1}, INVALID), ({"state": A + 1}, INVALID),
    ({"seqs": 1 << 30, "dim": 64}, UNSUPPORTED), ({"seqs": 0, "x": None}, 0),
])
def test_c_scan_step_refuses(kw, status):
    assert _step(**kw) == status


def _linear(**kw):
    a = dict(x=A, xs=4, w=A, b=None, off=A, index=1, y=A, ys=3, rows=6, groups=2, K=4, M=3, dtype=0, ws=A,
             nws=1 << 40, stream=None)
    a.update(kw)
    return tbe.load().tbe_grouped_linear(*a.values())


def _linear_back(**kw):
    a = dict(x=A, xs=4, w=A, off=A, index=1, grad=A, gs=3, dx=A, dxs=4, dw=A, db=A, rows=6, groups=2, K=4, M=3,
             dtype=0, ws=A, nws=1 << 40, stream=None)
    a.update(kw)
    return tbe.load().tbe_grouped_linear_backward(*a.values())


@pytest.mark.parametrize("kw,status", [
    ({"rows": -1}, INVALID), ({"groups": -1}, INVALID), ({"groups": 0}, INVALID), ({"K": 0}, INVALID),
    ({"M": 0}, INVALID), ({"dtype": 3}, INVALID), ({"index": 2}, INVALID), ({"x": None}, INVALID),
    ({"w": None}, INVALID), ({"off": None}, INVALID), ({"off": A + 4}, INVALID), ({"x": A + 2}, INVALID),
    ({"w": A + 2}, INVALID), ({"xs": -4}, INVALID), ({"rows": 1 << 31}, UNSUPPORTED),
    ({"xs": 1 << 21}, UNSUPPORTED), ({"K": 1 << 21}, UNSUPPORTED), ({"M": 1 << 21}, UNSUPPORTED), ({"groups": 1 << 17}, UNSUPPORTED),
])
def test_c_grouped_linear_refuses(kw, status):
    assert _linear(**kw) == status
    assert _linear_back(**kw) == status


def test_c_grouped_linear_refuses_outputs():
    for kw in ({"y": None}, {"ys": 2}, {"y": A + 2}, {"b": A + 2}):
        assert _linear(**kw) == INVALID
    for kw in ({"grad": None}, {"gs": -1}, {"dxs": 3}, {"dx": A + 2}, {"dw": A + 2}, {"db": A + 1},
               {"grad": A + 2}):
        assert _linear_back(**kw) == INVALID
    assert _linear(rows=0) == 0 and _linear_back(rows=0, groups=0) == 0


def test_c_grouped_linear_workspace():
    f, b = ctypes.c_size_t(1), ctypes.c_size_t(1)
    sizes = tbe.load().tbe_grouped_linear_sizes
    assert sizes(6, 2, 4, 3, 0, None, ctypes.byref(b)) == INVALID
    assert sizes(6, 0, 4, 3, 0, ctypes.byref(f), ctypes.byref(b)) == INVALID
    assert sizes(6, 2, 1 << 21, 3, 0, ctypes.byref(f), ctypes.byref(b)) == UNSUPPORTED
    for rows, groups, K, M, dtype in ((6, 2, 4, 3, 0), (4096, 8, 512, 512, 2)):
        assert sizes(rows, groups, K, M, dtype, ctypes.byref(f), ctypes.byref(b)) == 0
        a = dict(rows=rows, groups=groups, K=K, M=M, dtype=dtype, xs=K)
        for call, n, kw in ((_linear, f.value, {"ys": M}), (_linear_back, b.value, {"gs": M, "dxs": K})):
            if n:
                assert call(**a, **kw, nws=n - 1) == SMALL
                assert call(**a, **kw, ws=None, nws=n) == INVALID
                assert call(**a, **kw, ws=A + 64) == INVALID
