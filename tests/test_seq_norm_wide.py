"""Gradients of the norms over rows so wide that not all column sums fit the shared memory at once: what the forward
pass takes, the backward pass takes."""
import pytest
import torch

import _seq_ref as R
import linear_spatial_propagation_gspn_b200 as g
from test_seq_norm import NAMES, PARTS, make, reach

pytestmark = pytest.mark.gpu


def check(t, kw, center, got, rows):
    """The bounds of test_seq_norm.test_backward."""
    ref = R.norm(t["y"], None, *(kw.get(k) for k in ("gate", "w_post", "b_post", "scale", "w_pre", "b_pre")), 1e-5, center,
                 t["r"], t["dr"], t["do"])
    for name, a in zip(NAMES, got):
        r = ref[name]
        mag = r.abs() + r.abs().max(-1, keepdim=True).values if r.dim() == 2 else ref[name + "_m"] + ref[name + "_m"].max()
        R.check(a, r, mag, 8 * 96.0 * reach(t, kw, center) + (0 if r.dim() == 2 else rows), name)


@pytest.mark.parametrize("C", [10240, 10241, 12808, 16384])
@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_all_five_sums(C, types):
    t = make(3, C, *types, seed=1)
    kw = {k: t[k] for k in PARTS["all"]}
    got = g.norm_backward(t["y"], t["r"], t["dr"], t["do"], center=True, **kw)
    again = g.norm_backward(t["y"], t["r"], t["dr"], t["do"], center=True, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    check(t, kw, True, got, 3)


def test_autograd_of_the_widest_rows():
    t = make(2, 16384, "f32", "f32", seed=2)
    kw = {k: t[k].clone().requires_grad_(True) for k in PARTS["all"]}
    y, r = (t[k].clone().requires_grad_(True) for k in ("y", "r"))
    r_out, o = g.block_norm(y, r, center=True, **kw)
    torch.autograd.backward([r_out, o], [t["dr"], t["do"]])
    want = g.norm_backward(y.detach(), r_out.detach(), t["dr"], t["do"], center=True, **{k: v.detach() for k, v in kw.items()})
    got = [y.grad, r.grad, *(kw[k].grad for k in ("gate", "w_post", "b_post", "scale", "w_pre", "b_pre"))]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
