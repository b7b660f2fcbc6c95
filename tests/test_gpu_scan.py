"""The gated linear recurrence over jagged sequences, its gradient and its step."""
import numpy as np
import pytest
import torch

import layers_reference as ref
import table_embedding_bag_amd as tbe
from gpu_check import guarded_copy, guarded_empty, guards_intact

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def _np(t):
    return t.double().cpu().numpy()


class Problem:
    def __init__(self, lengths, D, dtype, kind, seed=0, halves=False, index=torch.int64,
                 initial=True, grads=True):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.dtype = kind, dtype
        self.lengths = np.asarray(lengths, dtype=np.int64)
        self.off = np.concatenate([[0], np.cumsum(self.lengths)])
        N, S = int(self.off[-1]), len(lengths)
        self.N, self.S, self.D = N, S, D
        both = torch.randn(N, 2 * D + 3, generator=g)
        gate = both[:, D:2 * D] + 2
        if kind == "decay":
            gate = torch.sigmoid(gate)
        both[:, D:2 * D] = gate
        both = both.to(dtype).cuda()
        self.x, self.gate = both[:, :D], both[:, D:2 * D]
        if not halves:
            self.x, self.gate = self.x.contiguous(), self.gate.contiguous()
        self.offsets = torch.from_numpy(self.off).to(index).cuda()
        self.initial = torch.randn(S, D, generator=g).cuda() if initial else None
        self.grad_h = torch.randn(N, D, generator=g).to(dtype).cuda() if grads else None
        self.grad_final = torch.randn(S, D, generator=g).cuda() if grads else None

    def reference(self):
        opt = lambda t: None if t is None else _np(t)  # noqa: E731
        return ref.scan(_np(self.x), _np(self.gate), self.off, opt(self.initial), self.kind,
                        opt(self.grad_h), opt(self.grad_final))

    def run(self):
        h, final, carry = tbe.scan_forward(self.x, self.gate, self.offsets, initial=self.initial,
                                           gate_kind=self.kind)
        dx, dgate, dinitial = tbe.scan_backward(self.x, self.gate, self.offsets, carry, self.grad_h,
                                                grad_final=self.grad_final, initial=self.initial,
                                                gate_kind=self.kind)
        return {"h": h, "final": final, "dx": dx, "dgate": dgate, "dinitial": dinitial}

    def check(self, got=None):
        got = got or self.run()
        torch.cuda.synchronize()
        for name, (want, bound) in self.reference().items():
            dt = torch.float32 if name in ("final", "dinitial") else self.dtype
            ref.assert_close(got[name], want, ref.rounded(bound, want, dt), name)


LENGTHS = {
    "one-token": [1],
    "ones": [1] * 70,
    "empty-ones": [0, 0, 3, 0, 1, 0, 0, 17, 0],
    "all-empty": [0, 0, 0],
    "tile-ends": [16, 16, 15, 17, 32, 1, 31, 64, 128, 127, 129],
    "ragged": [5, 40, 0, 1, 2, 33, 100, 7, 0, 250, 3],
    "one-long": [1500],
    "long-among-short": [2, 1, 700, 0, 1, 1, 333],
    "many-empty": [0] * 300 + [5] + [0] * 200 + [1, 1] + [0] * 70,
}


@pytest.mark.parametrize("kind", ["sigmoid", "decay"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dim", [1, 33, 100, 130])
def test_forward_and_backward(lengths, dim, dtype, kind):
    print(f"[scan] {lengths} D={dim} {dtype} {kind}", flush=True)
    Problem(LENGTHS[lengths], dim, DTYPES[dtype], kind, seed=dim, halves=dim % 2 == 1,
            index=torch.int32 if dim == 33 else torch.int64).check()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_wide_rows_and_many_sequences(dtype):
    g = np.random.default_rng(3)
    print(f"[scan] wide {dtype}", flush=True)
    Problem(g.integers(0, 60, 40), 520, DTYPES[dtype], "sigmoid", seed=4, halves=True).check()
    Problem(g.integers(0, 9, 700), 64, DTYPES[dtype], "decay", seed=5).check()


def test_long_sequences():
    """Some thousands of tokens over few channels: states pass many tiles."""
    print("[scan] long", flush=True)
    p = Problem([6000, 1, 0, 5001], 8, torch.float32, "sigmoid", seed=6)
    p.gate.add_(4)                      # long memories
    p.check()
    # one among many short ones (tiles of the size for those), and few of some tiles each
    Problem([2] * 60 + [4000, 0, 1], 33, torch.bfloat16, "decay", seed=7, halves=True).check()
    Problem([300] * 9, 130, torch.float16, "sigmoid", seed=8).check()


@pytest.mark.parametrize("kind", ["sigmoid", "decay"])
def test_optional_inputs(kind):
    Problem([4, 0, 90], 36, torch.float32, kind, initial=False).check()
    Problem([4, 0, 90], 36, torch.float32, kind, grads=False).check()
    p = Problem([4, 0, 90], 36, torch.float32, kind)
    p.initial = p.initial[:1].expand(3, 36)       # one row for all sequences
    p.grad_final = p.grad_final[1:2].expand(3, 36)
    p.check()


def test_no_tokens_and_no_sequences():
    for S in (0, 3):
        off = torch.zeros(S + 1, dtype=torch.int64, device="cuda")
        x = torch.empty(0, 5, device="cuda")
        init = torch.randn(S, 5, device="cuda")
        h, final, carry = tbe.scan_forward(x, x, off, initial=init)
        assert h.shape == (0, 5) and torch.equal(final, init)
        dx, dg, di = tbe.scan_backward(x, x, off, carry, grad_final=init)
        assert dx.shape == (0, 5) and torch.equal(di, init)


def test_a_sequence_does_not_reach_its_neighbours():
    """Infinities and NaN stay in their sequence and channel, forwards and backwards."""
    for dtype in DTYPES.values():
        lengths = [20, 3, 0, 40, 150, 1, 10]
        p = Problem(lengths, 40, dtype, "sigmoid", seed=8)
        clean = p.run()
        q = Problem(lengths, 40, dtype, "sigmoid", seed=8)
        lo, hi = int(p.off[3]), int(p.off[4])
        q.x[lo + 5, 7] = float("inf")
        q.x[lo + 6, 8] = float("nan")
        q.initial[3, 9] = float("inf")
        q.grad_h[lo + 30, 10] = float("nan")
        q.grad_final[3, 11] = -float("inf")
        dirty = q.run()
        cols = torch.ones(40, dtype=torch.bool)
        cols[7:12] = False
        for name in clean:
            a, b = clean[name].cpu(), dirty[name].cpu()
            inside = slice(3, 4) if name in ("final", "dinitial") else slice(lo, hi)
            rest = torch.ones(a.shape[0], dtype=torch.bool)
            rest[inside] = False
            assert torch.equal(a[rest], b[rest]), name
            assert torch.equal(a[:, cols], b[:, cols]), name
        assert torch.isinf(dirty["h"][lo + 5, 7]) and torch.isnan(dirty["h"][lo + 6:hi, 8]).all()
        assert torch.isnan(dirty["dx"][lo:lo + 31, 10]).all()


@pytest.mark.parametrize("polls", [-1, 1])
@pytest.mark.parametrize("dtype,kind", [("fp32", "decay"), ("bf16", "sigmoid")])
def test_waits_that_give_up(polls, dtype, kind, monkeypatch):
    """A part of a sequence that does not wait for the one before works its state out itself."""
    monkeypatch.setattr(tbe.layers, "_MAX_POLLS", polls)
    for D in (40, 130, 131):
        Problem([5, 700, 0, 3, 300, 64, 128, 1], D, DTYPES[dtype], kind, seed=20).check()


def test_extreme_gates():
    """Gates of the types' ends: a is 0 or 1, and nothing but the state is lost or kept."""
    p = Problem([50, 200], 16, torch.float32, "sigmoid", seed=9)
    p.gate[:, :4] = 1e4
    p.gate[:, 4:8] = -1e4
    p.gate[:, 8:10] = float("inf")
    p.gate[:, 10:12] = -float("inf")
    p.check()
    q = Problem([50, 200], 16, torch.float32, "decay", seed=9)
    q.gate[:, :4] = 0.0
    q.gate[:, 4:8] = 1.0
    q.gate[:, 8:12] = -0.5
    q.check()


def test_same_bits_every_time():
    p = Problem([3000, 5, 0, 900] + [7] * 50, 200, torch.bfloat16, "sigmoid", seed=10)
    first = p.run()
    for _ in range(5):
        again = p.run()
        for name in first:
            assert torch.equal(first[name], again[name]), name


def test_another_stream_than_the_tensors_own():
    p = Problem([300, 5, 0, 900], 64, torch.float32, "decay", seed=11)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = p.run()
    side.synchronize()
    p.check(got)


def test_outputs_stay_within_their_buffers():
    """dx and dgate as the halves of one guarded buffer; h, the states and the carry through the
    C interface into guarded buffers."""
    import ctypes
    p = Problem([16, 33, 0, 130, 1], 37, torch.bfloat16, "sigmoid", seed=12)
    N, S, D = p.N, p.S, p.D
    nc, nw = tbe.layers._scan_sizes(N, S, D, p.dtype)
    hb, h = guarded_empty((N, D), p.dtype)
    fb, final = guarded_empty((S, D), torch.float32)
    cb, carry = guarded_empty((nc // 4,), torch.float32)
    wb, ws = guarded_empty((nw,), torch.uint8)
    _, inp = tbe.layers._scan_input(p.x, p.gate, p.offsets, p.initial, "sigmoid")
    st = torch.cuda.current_stream().cuda_stream
    assert tbe.load().tbe_scan_forward(ctypes.byref(inp), h.data_ptr(), final.data_ptr(),
                                       carry.data_ptr(), ws.data_ptr(), nw, st) == 0
    ob, both = guarded_empty((N, 2 * D), p.dtype)
    dx, dgate, dinitial = tbe.scan_backward(p.x, p.gate, p.offsets, carry, p.grad_h,
                                            grad_final=p.grad_final, initial=p.initial,
                                            out=(both[:, :D], both[:, D:]))
    p.check({"h": h, "final": final, "dx": dx, "dgate": dgate, "dinitial": dinitial})
    for b in (hb, fb, cb, wb, ob):
        assert guards_intact(b)


@pytest.mark.parametrize("kind", ["sigmoid", "decay"])
def test_differences(kind):
    """The states are linear in x and initial, so a finite step gives their gradients' projection;
    gates by a small central step."""
    p = Problem([9, 0, 40, 130], 24, torch.float32, kind, seed=14)
    got = {k: v.double() for k, v in p.run().items()}

    def loss():
        h, final, _ = tbe.scan_forward(p.x, p.gate, p.offsets, initial=p.initial, gate_kind=kind)
        return (h.double() * p.grad_h.double()).sum() + (final.double() * p.grad_final.double()).sum()

    g = torch.Generator(device="cuda").manual_seed(15)
    n = p.N * p.D
    for name, t, step in (("dx", p.x, 1.0), ("dinitial", p.initial, 1.0), ("dgate", p.gate, 2.0 ** -8)):
        d = torch.randn(t.shape, generator=g, device="cuda")
        keep = t.clone()
        t.copy_(keep + step * d)
        hi, up = loss(), (t - keep).double()
        t.copy_(keep - step * d)
        lo, down = loss(), (keep - t).double()
        t.copy_(keep)
        want = (got[name] * (up + down)).sum()
        # a loss sums 2 n terms of order 1 that are off by some U32 each; a gate's step of 2^-8
        # leaves a third-order rest of 2^-16 of the sum's spread
        rest = 64 * ref.U32 * n + (2.0 ** -16 * 2 * step * n if name == "dgate" else 0.0)
        assert abs((hi - lo) - want) <= rest, (name, float(hi - lo), float(want), rest)


@pytest.mark.parametrize("kind", ["sigmoid", "decay"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("S,D", [(1, 1), (7, 3), (65, 128), (33, 101), (3, 1024)])
def test_step(S, D, dtype, kind):
    p = Problem([1] * S, D, DTYPES[dtype], kind, seed=S, halves=True)
    want = p.reference()
    before = p.initial.clone()
    h, state = tbe.scan_step(p.x, p.gate, p.initial, gate_kind=kind)
    ref.assert_close(h, want["h"][0], ref.rounded(want["h"][1], want["h"][0], p.dtype), "h")
    ref.assert_close(state, want["final"][0], ref.rounded(want["final"][1], want["final"][0], torch.float32),
                     "state")
    assert torch.equal(p.initial, before)
    h2, again = tbe.scan_step(p.x, p.gate, p.initial, gate_kind=kind, out_state=p.initial)
    assert again is p.initial and torch.equal(again, state) and torch.equal(h, h2)
    zero, _ = tbe.scan_step(p.x, p.gate, gate_kind=kind)
    assert torch.equal(zero, tbe.scan_step(p.x, p.gate, torch.zeros_like(state), gate_kind=kind)[0])


def test_steps_follow_a_sequence():
    """A prompt through scan_forward and the rest by steps gives the states of the whole."""
    p = Problem([40] * 3, 48, torch.float32, "sigmoid", seed=16)
    want = p.reference()
    x, gate = p.x.view(3, 40, 48), p.gate.view(3, 40, 48)
    off = torch.arange(0, 31, 10, device="cuda")
    _, state, none = tbe.scan_forward(x[:, :10].reshape(30, 48), gate[:, :10].reshape(30, 48), off,
                                      initial=p.initial, need_carry=False)
    assert none is None
    for t in range(10, 40):
        _, state = tbe.scan_step(x[:, t], gate[:, t], state, out_state=state)
    ref.assert_close(state, want["final"][0], ref.rounded(want["final"][1], want["final"][0], torch.float32),
                     "state")


def test_graph_replays_match_eager_calls():
    p = Problem([300, 5, 0, 900, 20], 96, torch.bfloat16, "sigmoid", seed=17)
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
        q = Problem([300, 5, 0, 900, 20][::-1], 96, torch.bfloat16, "sigmoid", seed=30 + i)
        for name in ("x", "gate", "offsets", "initial", "grad_h", "grad_final"):
            getattr(p, name).copy_(getattr(q, name))
        want = p.run()
        g.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(out[name], want[name]), (i, name)


@pytest.mark.parametrize("kind", ["sigmoid", "decay"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [64, 67, 200])
def test_short_sequences_within_spans_of_long_ones(dim, dtype, kind):
    """Several sequences start and end inside one wave's tokens, among ones that span many tiles."""
    lengths = [2100, 3, 0, 1, 4, 2, 2, 1, 0, 1900, 15, 16, 1, 2500, 0]
    Problem(lengths, dim, DTYPES[dtype], kind, seed=21, halves=True, index=torch.int32).check()
    Problem(lengths, dim, DTYPES[dtype], kind, seed=22, initial=False, grads=False).check()
