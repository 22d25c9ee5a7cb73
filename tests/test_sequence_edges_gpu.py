"""Edges of the sequence operators on the GPU: empty plans, rows and widths at the limits, infinities, arguments far from
zero, and calls that have to be refused."""
import numpy as np
import pytest
import torch

from sparse_spd_selected_b200 import selinv
from tests.test_sequence_gpu import TYPES, arith, dev, host, scan_inputs, unit

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_state", [False, True])
@pytest.mark.parametrize("tail", [0, 3])
def test_backward_of_sequences_without_rows(cuda_ok, with_state, tail):
    """A plan of sequences without rows: the final states' cotangents are the initial ones', all else is zero."""
    v, yb, stateb = scan_inputs(31, torch.float32, (tail,), 12, 5, 2, states=(2,))
    state = v["state"] if with_state else None
    plan = selinv.SequencePlan([0, 0])
    args = (v["x"], v["dt"], v["A"], v["B"], v["C"])
    more = dict(D=v["D"], z=v["z"], dt_bias=v["dt_bias"], softplus=True, state=state, plan=plan)
    r = selinv.selective_scan(*args, keep=True, **more)
    b = selinv.selective_scan_backward(r["kept"], *args, yb, stateb=stateb, **more)
    for k in ("xb", "dtb", "Bb", "Cb", "zb", "Ab", "Db", "dt_biasb"):
        assert not b[k].any(), k
    assert torch.equal(b["stateb"], stateb) if with_state else b["stateb"] is None
    w = torch.ones(12, 4, device="cuda")
    cs, csb = (dev(np.random.default_rng(i).standard_normal((2, 3, 12)), torch.float32) for i in (1, 2))
    c = selinv.causal_conv_backward(v["x"], w, yb, bias=v["D"], stateb=csb, state=cs if with_state else None, plan=plan)
    assert not c["xb"].any() and not c["weightb"].any() and not c["biasb"].any()
    assert torch.equal(c["stateb"], csb) if with_state else c["stateb"] is None


def test_gradients_of_sequences_without_rows(cuda_ok):
    v, _, stateb = scan_inputs(32, torch.float32, (0,), 12, 5, 2, states=(2,))
    leaves = {k: a.requires_grad_(True) for k, a in v.items()}
    y, state = selinv.selective_scan_ad(**leaves, softplus=True, plan=selinv.SequencePlan([0, 0]))
    ((state * stateb).sum() + y.sum()).backward()
    assert torch.equal(v["state"].grad, stateb)
    for k in ("A", "D", "dt_bias"):
        assert not v[k].grad.any(), k
