"""The token-sequence kernels in the forms and loops that small calls do not reach: single tokens whose states fill
their lanes, rows enough for several to a block, pieces of sequences with wide states, many packed sequences.
Bounds are those of each operator's own tests."""
import pytest
import torch

import _seq_ref as R
import linear_spatial_propagation_gspn_b200 as g
import test_seq_conv as conv
import test_seq_norm as norm
import test_seq_scan as scan

pytestmark = pytest.mark.gpu


# (rows, C, G, N): whole blocks of states as they lie, for each lane count; then the general form with four channels
# a lane, which takes some 600 blocks
PLAIN = [(1, 128, 1, 16), (12, 256, 1, 16), (256, 128, 1, 16), (1, 64, 1, 32), (256, 192, 1, 32), (12, 32, 1, 64), (256, 96, 1, 64)]
GENERAL = [(25, 1600, 1, 24), (40, 2000, 2, 16), (60, 330, 1, 61)]


@pytest.mark.parametrize("shape", PLAIN + GENERAL)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("full", [True, False])
def test_step(shape, dtype, full):
    scan.test_step(shape, dtype, full)


@pytest.mark.parametrize("C,N", [(128, 16), (64, 32), (32, 64)])
def test_step_repeated_and_missing_slots(C, N):
    """As in the scan's own tests, over more rows than a block has: slots named by rows of one block and of several."""
    rows = 2500
    t = scan.make(1, rows, C, 1, N, "f32", seed=6)
    s = {k: t[k][0] for k in ("x", "dt", "Bm", "Cm", "z")}
    pool = torch.randn(rows, C, N, device="cuda")
    before = pool.clone()
    idx = torch.randperm(rows, generator=torch.Generator().manual_seed(C)).to(torch.int32)
    again = [3, 4, 9, 700, 701, 2499]
    idx[again] = idx[2].clone()
    idx[[5, 1200]] = torch.tensor([-1, rows], dtype=torch.int32)
    y = torch.full((rows, C), 7.0, device="cuda")
    g.ssm_step(s["x"], s["dt"], t["A"], s["Bm"], s["Cm"], pool, D=t["D"], z=s["z"], dt_bias=t["dt_bias"], y=y, idx=idx.cuda())
    for first in (2, 6, 1000, 2498):
        at = [2] + again if first == 2 else [first]
        slot = idx[first].item()
        one = {k: t[k][:, at] for k in ("x", "dt", "Bm", "Cm", "z")}
        ref = R.scan(one["x"], one["dt"], t["A"], one["Bm"], one["Cm"], t["D"], one["z"], t["dt_bias"], True, None, before[slot][None])
        f = R.scan_factor(len(at), N, C)
        R.check(y[at], ref["y"][0], ref["y_m"][0], f, "y")
        R.check(pool[slot], ref["h"][0], ref["h_m"][0], f, "h")
    assert (y[[5, 1200]] == 7).all()
    left = torch.ones(rows, dtype=torch.bool)
    left[idx[(idx >= 0) & (idx < rows)].long()] = False
    assert torch.equal(pool[left.cuda()], before[left.cuda()])


# more rows than the blocks that run at once (warps with a row each up to 256 columns)
ROWS = [(9700, 96), (5001, 257), (2501, 1153), (1301, 2048), (701, 4096), (451, 5000)]


@pytest.mark.parametrize("rows,C", ROWS)
@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("parts,center", [("all", True), ("rms", False), ("pre", False)])
def test_norms_of_several_rows_a_block(rows, C, types, parts, center):
    norm.test_forward(rows, C, types, parts, center)
    norm.test_backward(rows, C, types, parts)


@pytest.mark.parametrize("shape", [(1, 400, 40, 1, 24), (2, 333, 36, 2, 32), (1, 400, 40, 1, 40), (1, 290, 18, 1, 64), (1, 400, 33, 1, 3)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pieces_of_sequences(shape, dtype):
    scan.test_prompt(shape, dtype, True)
    scan.test_gradients(shape, dtype, True)


def lengths(S, seed, most):
    r = torch.Generator().manual_seed(seed)
    n = torch.randint(0, most + 1, (S,), generator=r)
    n[torch.randint(0, S, (S // 4,), generator=r)] = 0
    cu = [3] + (3 + n.cumsum(0)).tolist()
    return cu, cu[-1] + 5


@pytest.mark.parametrize("S,most,C,G,N", [(3, 40, 40, 2, 24), (3, 30, 24, 1, 64), (4, 200, 40, 1, 32), (33, 20, 40, 2, 16), (40, 12, 18, 1, 40),
                                          (32, 12, 40, 1, 16), (150, 3, 33, 1, 12)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_scans(S, most, C, G, N, dtype):
    """Up to 32 sequences are taken longest first, more as they come; some hold no token. Tokens outside stay out."""
    cu, L = lengths(S, S + N, most)
    t = scan.make(1, L, C, G, N, dtype, seqs=S, seed=2)
    a, b = cu[0], cu[-1]
    for k in ("x", "dt", "Bm", "Cm", "z", "dy"):
        t[k][:, :a] = float("nan")
        t[k][:, b:] = float("nan")
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ref = scan.reference(t, cu=cu, grads=True)
    y, h = torch.full_like(t["x"], 7.0), torch.empty_like(t["h0"])
    _, hsave = g.ssm_forward_save(*scan.args(t), **scan.opts(t, cu=c, y=y, h=h))
    out = [torch.full_like(v, 7.0) for v in (t["x"], t["dt"], t["A"], t["Bm"], t["Cm"], t["D"], t["z"], t["dt_bias"], t["h0"])]
    got = g.ssm_backward(*scan.args(t), t["dy"], hsave, **scan.opts(t, cu=c, dh=t["dh"], out=out))
    f = scan.factor(t, cu) + L
    inside = torch.zeros(1, L, dtype=torch.bool)
    inside[:, a:b] = True
    for name, v, r, m in (("y", y, ref["y"], ref["y_m"]), *((n, v, ref[n], ref[n + "_m"]) for n, v in zip(scan.GRADS, got))):
        if name in ("y", "dx", "ddt", "dB", "dC", "dz"):
            assert (v.cpu()[~inside] == 7).all(), f"{name}: tokens outside were written"
            v, r, m = v.cpu()[inside], r[inside], m[inside]
        R.check(v, r, m, f, name)
    R.check(h, ref["h"], ref["h_m"], f, "h")


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_convolutions_of_several_runs_a_block(cut, dtype):
    """Few channels and many tokens: a block of the backward pass takes several runs one after the other."""
    L, C = 30000, 8
    cu = None
    if cut:
        cu, L = lengths(60, 1, 1000)
    t = conv.make(1, L, C, 4, dtype, seqs=60 if cut else None, seed=7)
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    ref = R.conv(t["x"], t["w"], t["bias"], True, cu, t["state0"], t["dy"], t["dstate"])
    state = torch.empty_like(t["dstate"])
    y = g.conv_forward(t["x"], t["w"], t["bias"], cu=c, state0=t["state0"], state=state)
    got = g.conv_backward(t["x"], t["w"], t["bias"], t["dy"], cu=c, state0=t["state0"], dstate=t["dstate"])
    s = slice(0, L) if cu is None else slice(cu[0], cu[-1])
    assert torch.equal(R.f64(state), ref["state"])
    R.check(y[:, s], ref["y"][:, s], ref["y_m"][:, s], conv.F, "y")
    R.check(got[0][:, s], ref["dx"][:, s], ref["dx_m"][:, s], conv.F, "dx")
    for name, v in zip(("dw", "db", "ds"), got[1:]):
        R.check(v, ref[name], ref[name + "_m"], conv.F + L, name)
