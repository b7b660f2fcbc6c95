"""Decay gates above 1: states and gradients of 0 stay 0 however long such gates go on, though the
gates' products over a part of a sequence are infinite."""
import pytest
import torch

import layers_reference as ref
import table_embedding_bag_amd as tbe
from test_gpu_scan import DTYPES, Problem

pytestmark = pytest.mark.gpu
CASES = [(dtype, big) for dtype in DTYPES for big in (2.0, 6e4, 1e30) if dtype != "fp16" or big < 65504]
# few long sequences, and one among many short ones (tiles of either size)
LENGTHS = {"long": [3, 2500, 2], "among-short": [2] * 60 + [900, 0, 1]}


def _long(p):
    s = int(p.lengths.argmax())
    return s, int(p.off[s]), int(p.off[s + 1])


def _check(p, got, names):
    torch.cuda.synchronize()
    want = p.reference()
    for name in names:
        dt = torch.float32 if name in ("final", "dinitial") else p.dtype
        v, bound = want[name]
        ref.assert_close(got[name], v, ref.rounded(bound, v, dt), name)


@pytest.mark.parametrize("polls", [0, -1], ids=["waits", "walks"])
@pytest.mark.parametrize("dim", [40, 130])
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dtype,big", CASES)
def test_states_of_zero(dtype, big, lengths, dim, polls, monkeypatch):
    """No input and no initial state under gates above 1, then gates below 1 and inputs."""
    print(f"[scan] range forward {dtype} {big} {lengths} {dim} {polls}", flush=True)
    monkeypatch.setattr(tbe.layers, "_MAX_POLLS", polls)
    p = Problem(LENGTHS[lengths], dim, DTYPES[dtype], "decay", seed=30, grads=False)
    s, lo, hi = _long(p)
    end = lo + (hi - lo) * 4 // 5 + 3
    p.initial[s] = 0.0
    p.x[lo:end] = 0.0
    p.gate[lo:end] = big
    h, final, _ = tbe.scan_forward(p.x, p.gate, p.offsets, initial=p.initial, gate_kind="decay")
    assert (h[lo:end] == 0).all()
    _check(p, {"h": h, "final": final}, ("h", "final"))


@pytest.mark.parametrize("polls", [0, -1], ids=["waits", "walks"])
@pytest.mark.parametrize("dim", [40, 130])
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dtype,big", CASES)
def test_gradients_of_zero(dtype, big, lengths, dim, polls, monkeypatch):
    """A gate of 0, then no input and no gradient under gates above 1 to the sequence's end."""
    print(f"[scan] range backward {dtype} {big} {lengths} {dim} {polls}", flush=True)
    monkeypatch.setattr(tbe.layers, "_MAX_POLLS", polls)
    p = Problem(LENGTHS[lengths], dim, DTYPES[dtype], "decay", seed=31)
    s, lo, hi = _long(p)
    begin = lo + (hi - lo) // 5 + 3
    p.x[begin:hi] = 0.0
    p.gate[begin:hi] = big
    p.gate[begin] = 0.0
    p.grad_h[begin:hi] = 0.0
    p.grad_final[s] = 0.0
    got = p.run()
    assert (got["dx"][begin:hi] == 0).all()
    _check(p, got, ("h", "final", "dx", "dgate", "dinitial"))


def test_short_sequences_end_inside_a_span_of_infinite_products():
    """Gates of 1e30 in sequences of one or two tokens, many of them in a wave's tokens."""
    p = Problem([1, 2, 0, 2, 1] * 40, 36, torch.float32, "decay", seed=32)
    p.gate[:] = 1e30
    p.x[:] = 0.0
    p.initial[:] = 0.0
    p.grad_h[:] = 0.0
    p.grad_final[:, ::2] = 0.0
    p.grad_final *= 1e-25     # times two gates: 1e35
    _check(p, p.run(), ("h", "final", "dx", "dgate", "dinitial"))
