"""The recurrence forwards without a carry, as a prompt is read for serving."""
import pytest
import torch

import layers_reference as ref
import table_embedding_bag_amd as tbe
from test_gpu_scan import DTYPES, LENGTHS, Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["sigmoid", "decay"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lengths", ["ones", "empty-ones", "ragged", "one-long", "long-among-short"])
@pytest.mark.parametrize("dim", [33, 130])
def test_no_carry(dim, lengths, dtype, kind):
    """The same bits as with one, which is the part that a backward pass needs."""
    print(f"[scan serving] {lengths} {dim} {dtype} {kind}", flush=True)
    p = Problem(LENGTHS[lengths], dim, DTYPES[dtype], kind, seed=70, halves=dim == 33, grads=False)
    h, final, carry = tbe.scan_forward(p.x, p.gate, p.offsets, initial=p.initial, gate_kind=kind, need_carry=False)
    assert carry is None
    with_carry = tbe.scan_forward(p.x, p.gate, p.offsets, initial=p.initial, gate_kind=kind)
    assert torch.equal(h, with_carry[0]) and torch.equal(final, with_carry[1])
    want = {"h": h, "final": final}
    for name, (v, bound) in p.reference().items():
        if name in want:
            dt = torch.float32 if name == "final" else p.dtype
            ref.assert_close(want[name], v, ref.rounded(bound, v, dt), name)
