"""Host-side checks of the token-sequence calls (no GPU needed): what they refuse is refused before
anything is launched. Pointers are made up; no call here gets past its checks."""
import ctypes

import pytest
import torch

import linear_spatial_propagation_gspn_b200 as g
from linear_spatial_propagation_gspn_b200 import seq

P = 0x10000


def conv(**kw):
    return seq.ConvDesc(*{**dict(B=2, L=8, C=16, K=4, S=0, dtype=0, silu=1, x_row=128, x_tok=16), **kw}.values())


def ssm(**kw):
    base = dict(B=2, L=8, C=16, G=1, N=16, S=0, dtype=0, softplus=1, x_row=128, x_tok=16, dt_row=128, dt_tok=16, z_row=128, z_tok=16,
                b_row=128, b_tok=16, c_row=128, c_tok=16)
    return seq.SsmDesc(*{**base, **kw}.values())


def norm(**kw):
    return seq.NormDesc(*{**dict(rows=4, C=16, dtype=0, res_dtype=0, center=0, eps=1e-5, y_row=16, gate_row=16, r_row=16), **kw}.values())


def call(name, d, args):
    return getattr(g.lib(), name)(ctypes.byref(d), *args)


# every call with made-up pointers; the positions of the ones that may not be null
CALLS = {
    "gspn_conv_forward": (conv, [P, P, P, None, P, P, P, None], (0, 1, 5)),
    "gspn_conv_backward": (conv, [P, P, P, None, P, P, P, P, P, P, P, P, 1 << 20, None], (0, 1, 5, 7, 8, 11)),
    "gspn_conv_step": (lambda **k: conv(**{**dict(L=1), **k}), [P, P, P, P, 4, P, P, None], (0, 1, 5, 6)),
    "gspn_ssm_forward": (ssm, [P, P, P, P, P, P, P, P, None, P, P, P, P, P, 1 << 20, None], (0, 1, 2, 3, 4, 10)),
    "gspn_ssm_backward": (ssm, [P, P, P, P, P, P, P, P, None, P, P, P, P, P, P, P, P, P, P, P, P, P, 1 << 24, None],
                          (0, 1, 2, 3, 4, 9, 10, 12, 13, 14, 15, 16, 18, 21)),
    "gspn_ssm_step": (lambda **k: ssm(**{**dict(L=1), **k}), [P, P, P, P, P, P, P, P, P, 4, P, P, None], (0, 1, 2, 3, 4, 10, 11)),
    "gspn_norm_forward": (norm, [P, P, P, P, P, P, P, P, P, P, None], (0, 8)),
    "gspn_norm_backward": (norm, [P] * 18 + [1 << 24, None], (0, 9, 17)),
}
BAD = {
    conv: [dict(B=0), dict(L=-1), dict(C=0), dict(K=1), dict(K=5), dict(S=-1), dict(S=3), dict(dtype=2), dict(silu=2), dict(x_tok=-1)],
    ssm: [dict(B=0), dict(L=-1), dict(C=0), dict(G=0), dict(G=3), dict(N=0), dict(S=-1), dict(S=2), dict(dtype=2), dict(softplus=3),
          dict(b_tok=-16)],
    norm: [dict(rows=-1), dict(C=0), dict(dtype=5), dict(dtype=0, res_dtype=1), dict(center=2), dict(eps=-1.0), dict(eps=float("nan")),
           dict(r_row=-1)],
}


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_descriptors(name):
    make, args, _ = CALLS[name]
    kind = {"conv": conv, "ssm_": ssm, "norm": norm}[name[5:9]]
    for bad in BAD[kind]:
        d = make(**bad)
        assert call(name, d, args) == g.GSPN_ERR_INVALID_ARG, (name, bad)
        assert getattr(g.lib(), name.rsplit("_", 1)[0] + "_workspace_size")(ctypes.byref(d), 1) == 0, (name, bad)


@pytest.mark.parametrize("name", list(CALLS))
def test_null_and_misaligned(name):
    make, args, needed = CALLS[name]
    for i in needed:
        a = list(args)
        a[i] = None
        assert call(name, make(), a) == g.GSPN_ERR_INVALID_ARG, (name, i)
    for i, v in enumerate(args[:-1]):
        if v == P:
            a = list(args)
            a[i] = P + 2
            assert call(name, make(), a) == g.GSPN_ERR_ALIGNMENT, (name, i)


def test_optional_parts_that_go_together():
    make, args, _ = CALLS["gspn_ssm_backward"]
    a = list(args)
    a[18] = None                                                    # dz without its place
    assert call("gspn_ssm_backward", make(), a) == g.GSPN_ERR_INVALID_ARG
    a = list(args)
    a[6] = None                                                     # dz, but no z
    assert call("gspn_ssm_backward", make(), a) == g.GSPN_ERR_INVALID_ARG
    for name in ("gspn_conv_forward", "gspn_ssm_forward"):          # cu goes with S
        make, args, _ = CALLS[name]
        a = list(args)
        a[3 if "conv" in name else 8] = P
        assert call(name, make(), a) == g.GSPN_ERR_INVALID_ARG
        assert call(name, make(B=1, S=2), args) == g.GSPN_ERR_INVALID_ARG
    make, args, _ = CALLS["gspn_norm_forward"]
    for i in (2, 6, 9):                                             # b_post without w_post; w_pre and o
        a = list(args)
        a[i] = None
        assert call("gspn_norm_forward", make(), a) == g.GSPN_ERR_INVALID_ARG, i
    make, args, _ = CALLS["gspn_norm_backward"]
    for i in (1, 2, 4, 5, 6, 8):
        a = list(args)
        a[i] = None
        assert call("gspn_norm_backward", make(), a) == g.GSPN_ERR_INVALID_ARG, i


def test_workspaces():
    L = g.lib()
    for name, make, i in (("conv", conv, 12), ("ssm", ssm, 22), ("norm", norm, 18)):
        d = make()
        n = getattr(L, f"gspn_{name}_workspace_size")(ctypes.byref(d), 1)
        assert n > 256
        _, args, _ = CALLS[f"gspn_{name}_backward"]
        a = list(args)
        a[i] = n - 1
        assert call(f"gspn_{name}_backward", d, a) == g.GSPN_ERR_WORKSPACE
    d = ssm(B=1, L=100000, C=32)                                    # cut into pieces: the forward pass needs one too
    n = L.gspn_ssm_workspace_size(ctypes.byref(d), 0)
    assert n > 256
    a = list(CALLS["gspn_ssm_forward"][1])
    a[14] = n - 1
    assert call("gspn_ssm_forward", d, a) == g.GSPN_ERR_WORKSPACE
    a[13] = None
    assert call("gspn_ssm_forward", d, a) == g.GSPN_ERR_INVALID_ARG


def test_what_is_too_large():
    assert call("gspn_ssm_forward", ssm(N=65), CALLS["gspn_ssm_forward"][1]) == g.GSPN_ERR_UNSUPPORTED
    assert call("gspn_ssm_step", ssm(L=1, N=65), CALLS["gspn_ssm_step"][1]) == g.GSPN_ERR_UNSUPPORTED
    assert call("gspn_ssm_forward", ssm(B=4, L=1 << 29), CALLS["gspn_ssm_forward"][1]) == g.GSPN_ERR_UNSUPPORTED
    assert call("gspn_conv_forward", conv(B=4, L=1 << 29), CALLS["gspn_conv_forward"][1]) == g.GSPN_ERR_UNSUPPORTED
    a = list(CALLS["gspn_conv_step"][1])
    a[4] = 1 << 20
    assert call("gspn_conv_step", conv(B=65536, L=1), a) == g.GSPN_ERR_UNSUPPORTED
    assert call("gspn_norm_forward", norm(C=16385), CALLS["gspn_norm_forward"][1]) == g.GSPN_ERR_UNSUPPORTED
    # five column sums of a wide row
    assert call("gspn_norm_backward", norm(C=16384), CALLS["gspn_norm_backward"][1]) == g.GSPN_ERR_UNSUPPORTED


def test_slots():
    for name in ("gspn_conv_step", "gspn_ssm_step"):
        make, args, _ = CALLS[name]
        i = args.index(4)
        a = list(args)
        a[i] = 0
        assert call(name, make(), a) == g.GSPN_ERR_INVALID_ARG
        a[i], a[i - 1] = 1, None                                    # two rows, one slot, no index
        assert call(name, make(), a) == g.GSPN_ERR_INVALID_ARG
        assert call(name, make(L=2), args) == g.GSPN_ERR_INVALID_ARG


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    for f in (lambda: g.conv_forward(x, w), lambda: g.norm_forward(x), lambda: g.conv_step(x[0], w, None, torch.zeros(4, 3, 8)),
              lambda: g.ssm_forward(x, x, torch.zeros(8, 2), torch.zeros(1, 4, 1, 2), torch.zeros(1, 4, 1, 2))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        g.conv_forward(None, w)


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    x, w = z(2, 4, 8), z(8, 4)
    A, B = z(8, 2), z(2, 4, 1, 2)
    i32 = dict(dtype=torch.int32)
    bad = [
        (ValueError, lambda: g.conv_forward(x[0], w)), (ValueError, lambda: g.conv_forward(x, z(4, 8))),
        (TypeError, lambda: g.conv_forward(x, w.bfloat16())), (TypeError, lambda: g.conv_forward(x.half(), w)),
        (ValueError, lambda: g.conv_forward(x.transpose(1, 2), z(4, 4))), (ValueError, lambda: g.conv_forward(x, w, cu=z(3, **i32))),
        (TypeError, lambda: g.conv_forward(x[:1], w, cu=z(3))), (ValueError, lambda: g.conv_forward(x, w, state0=z(2, 4, 8))),
        (g.GspnError, lambda: g.conv_forward(x, z(8, 5))), (ValueError, lambda: g.conv_step(x[0], w, None, z(3, 3, 8))),
        (TypeError, lambda: g.conv_step(x[0], w, None, z(4, 3, 8), idx=z(4).long())), (ValueError, lambda: g.conv_backward(x, w, None, x[:1])),
        (ValueError, lambda: g.ssm_forward(x, x, A, B, z(2, 4, 1, 3))), (ValueError, lambda: g.ssm_forward(x, x, A, z(2, 4, 3, 2), B)),
        (ValueError, lambda: g.ssm_forward(x, x, A, B, B, h0=z(1, 8, 2))), (TypeError, lambda: g.ssm_forward(x, x, A, B, B, D=z(8).bfloat16())),
        (ValueError, lambda: g.ssm_forward(x, x[:, :3], A, B, B)), (g.GspnError, lambda: g.ssm_forward(x, x, z(8, 65), z(2, 4, 1, 65), z(2, 4, 1, 65))),
        (ValueError, lambda: g.ssm_backward(x, x, A, B, B, x, z(3))), (ValueError, lambda: g.ssm_step(x[0], x[0], A, B[0], B[0], z(3, 8, 2))),
        (ValueError, lambda: g.norm_forward(x, x, b_pre=z(8))), (TypeError, lambda: g.norm_forward(x.bfloat16(), x.half())),
        (ValueError, lambda: g.norm_forward(x, x[:1])), (ValueError, lambda: g.norm_backward(x, x, None, x)),
        (ValueError, lambda: g.norm_forward(x.transpose(0, 1).transpose(1, 2))),
    ]
    for k, (kind, f) in enumerate(bad):
        with pytest.raises(kind):
            f()
            pytest.fail(f"call {k} was taken")


@pytest.mark.gpu
def test_an_error_of_the_device_is_raised_and_the_call_not_made_again():
    """A step that reached the device with an error is not repeated by the path that explains refusals. The entry
    point is a stand-in on the host that only counts."""
    x, w, state = torch.ones(2, 64, device="cuda"), torch.ones(64, 4, device="cuda"), torch.zeros(2, 3, 64, device="cuda")
    g.conv_step(x, w, None, state.clone())
    fast = pytest.importorskip("linear_spatial_propagation_gspn_b200._seq_fast")
    real = {n: ctypes.cast(getattr(g.lib(), n), ctypes.c_void_p).value for n in seq.SIGNATURES}
    calls = []
    fake = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * 5, ctypes.c_int, *[ctypes.c_void_p] * 3)(
        lambda *a: calls.append(a) or g.GSPN_ERR_CUDA)
    fast.init({**real, "gspn_conv_step": ctypes.cast(fake, ctypes.c_void_p).value})
    try:
        with pytest.raises(g.GspnError) as e:
            g.conv_step(x, w, None, state)
    finally:
        fast.init(real)
    assert e.value.status == g.GSPN_ERR_CUDA and len(calls) == 1 and not state.any()
    g.conv_step(x, w, None, state)
    assert torch.equal(state.sum(1), torch.ones(2, 64, device="cuda"))


@pytest.mark.gpu
def test_flags_that_are_no_truth():
    x, w = torch.ones(2, 64, device="cuda"), torch.ones(64, 4, device="cuda")
    state = torch.zeros(2, 3, 64, device="cuda")
    with pytest.raises((RuntimeError, ValueError)):
        g.conv_step(x, w, None, state, silu=torch.ones(3))
    assert not state.any()
    assert torch.equal(g.conv_step(x, w, None, state.clone(), silu=1), g.conv_step(x, w, None, state.clone(), silu=True))


WRITES = ("conv_forward", "conv_backward", "conv_step", "ssm_forward", "ssm_forward_save", "ssm_backward", "ssm_step", "norm_forward")


@pytest.mark.gpu
@pytest.mark.parametrize("named", [False, True])
@pytest.mark.parametrize("name", WRITES)
def test_what_a_call_writes_is_known_to_autograd(name, named):
    """Every tensor of the caller's that a call writes to counts as changed in place, on the path without the
    interpreter and on the one that checks (a named stream); what it only reads does not."""
    z = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    B, L, C, N = 2, 5, 8, 4
    x, w, bias, A, D = z(B, L, C), z(C, 4), z(C), -z(C, N), z(C)
    bc, state, h, v = z(B, L, 1, N), z(B, 3, C), z(B, C, N), z(B, L, C)
    kw = dict(stream=torch.cuda.current_stream()) if named else {}
    save = g.ssm_forward_save(x, x, A, bc, bc)[1]
    out = [z(*t.shape) for t in ((x, w, bias, state) if name == "conv_backward" else (x, x, A, bc, bc, D, x, D, h))]
    y, s1, h1, step = z(B, L, C), z(B, 3, C), z(B, C, N), z(B, C)
    call, written = {
        "conv_forward": (lambda: g.conv_forward(x, w, bias, state0=state, state=s1, y=y, **kw), [s1, y]),
        "conv_backward": (lambda: g.conv_backward(x, w, bias, v, state0=state, out=out, **kw), out),
        "conv_step": (lambda: g.conv_step(x[:, 0], w, bias, s1, y=step, **kw), [s1, step]),
        "ssm_forward": (lambda: g.ssm_forward(x, x, A, bc, bc, D=D, z=v, h0=h, h=h1, y=y, **kw), [h1, y]),
        "ssm_forward_save": (lambda: g.ssm_forward_save(x, x, A, bc, bc, D=D, z=v, h0=h, h=h1, y=y, **kw), [h1, y]),
        "ssm_backward": (lambda: g.ssm_backward(x, x, A, bc, bc, v, save, D=D, z=v, dt_bias=D, h0=h, out=out, **kw), out),
        "ssm_step": (lambda: g.ssm_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], h1, D=D, y=step, **kw), [h1, step]),
        "norm_forward": (lambda: g.norm_forward(x, v, w_pre=D, r_out=y, o=out[0], **kw), [y, out[0]]),
    }[name]
    read = [t for t in (x, w, bias, A, D, bc, state, h, v, save)]
    before = [t._version for t in written], [t._version for t in read]
    call()
    assert [t._version for t in written] == [n + 1 for n in before[0]]
    assert [t._version for t in read] == before[1]


@pytest.mark.gpu
@pytest.mark.parametrize("named", [False, True])
@pytest.mark.parametrize("op", ["conv", "scan"])
def test_a_state_moved_on_before_its_gradient_is_refused(op, named):
    """The differentiable calls keep the state that a sequence starts from; a step that moves it on in place before
    the backward pass must not end in gradients of another state."""
    B, L, C, N = 2, 6, 8, 4
    x = torch.randn(B, L, C, device="cuda", requires_grad=True)
    kw = dict(stream=torch.cuda.current_stream()) if named else {}
    if op == "conv":
        w, state = torch.randn(C, 4, device="cuda"), torch.randn(B, 3, C, device="cuda")
        y = g.causal_conv(x, w, state0=state)
        g.conv_step(x.detach()[:, 0], w, None, state, **kw)
    else:
        A, bc, state = -torch.rand(C, N, device="cuda"), torch.randn(B, L, 1, N, device="cuda"), torch.randn(B, C, N, device="cuda")
        y = g.selective_scan(x, x, A, bc, bc, h0=state)
        d = x.detach()
        g.ssm_step(d[:, 0], d[:, 0], A, bc[:, 0], bc[:, 0], state, **kw)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.gpu
def test_states_of_inference_tensors_are_written():
    """Tensors made in inference mode have no count of changes; calls write to them all the same."""
    with torch.inference_mode():
        x, w, state = torch.ones(2, 8, device="cuda"), torch.ones(8, 4, device="cuda"), torch.zeros(2, 3, 8, device="cuda")
        for kw in ({}, dict(stream=torch.cuda.current_stream())):
            g.conv_step(x, w, None, state, **kw)
    assert torch.equal(state.sum(1), torch.full((2, 8), 2.0, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_batch_of_no_rows(dtype):
    """Prompts, gradients and tokens of no rows, as the norms take them: empty outputs, states as they were, zero
    gradients of the parameters. Shapes are checked as ever."""
    e = lambda *s: torch.empty(0, *s, dtype=dtype, device="cuda")  # noqa: E731
    f = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    C, N, K = 8, 4, 4
    x, bc, w, bias, A, s0, h0 = e(5, C), e(5, 1, N), f(C, K), f(C), -f(C, N), e(K - 1, C), f(0, C, N)
    assert g.conv_forward(x, w, bias, state0=s0, state=s0).shape == x.shape
    dx, dw, db, ds = g.conv_backward(x, w, bias, x, state0=s0)
    assert dx.shape == x.shape and ds.shape == s0.shape and not dw.any() and not db.any() and dw.shape == w.shape
    y, save = g.ssm_forward_save(x, x, A, bc, bc, D=bias, z=x, dt_bias=bias, h0=h0)
    assert y.shape == g.ssm_forward(x, x, A, bc, bc).shape == x.shape
    got = g.ssm_backward(x, x, A, bc, bc, x, save, D=bias, z=x, dt_bias=bias, h0=h0)
    assert [t.shape for t in got] == [t.shape for t in (x, x, A, bc, bc, bias, x, bias, h0)]
    assert not any(got[i].any() for i in (2, 5, 7))
    pool, states, idx = f(3, K - 1, C).to(dtype), f(3, C, N), torch.empty(0, dtype=torch.int32, device="cuda")
    for i in (None, idx):
        assert g.conv_step(e(C), w, None, pool, idx=i).shape == g.ssm_step(e(C), e(C), A, e(1, N), e(1, N), states, idx=i).shape == (0, C)
    assert (pool == 1).all() and (states == 1).all()
    leaf = [t.clone().requires_grad_(True) for t in (x, w, A)]
    (g.causal_conv(leaf[0], leaf[1]).sum() + g.selective_scan(leaf[0], x, leaf[2], bc, bc).sum()).backward()
    assert not any(t.grad.any() for t in leaf)
    with pytest.raises(ValueError):
        g.conv_forward(x, f(C + 1, K))
    with pytest.raises(ValueError):
        g.ssm_backward(x, x, A, bc, bc, x, f(8))


@pytest.mark.gpu
def test_what_is_no_tensor_is_named():
    """A list, a number or nothing where a tensor has to be: a TypeError that names the argument."""
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    x, w, A, B, h, st = z(2, 4, 8), z(8, 4), z(8, 2), z(2, 4, 1, 2), z(2, 8, 2), z(2, 3, 8)
    bad = [
        ("w", lambda: g.conv_forward(x, None)), ("bias", lambda: g.conv_forward(x, w, 1.0)), ("cu", lambda: g.conv_forward(x[:1], w, cu=[0, 4])),
        ("state0", lambda: g.conv_forward(x, w, state0=0)), ("dy", lambda: g.conv_backward(x, w, None, None)),
        ("w", lambda: g.conv_step(x[:, 0], [1], None, st)), ("state", lambda: g.conv_step(x[:, 0], w, None, None)),
        ("idx", lambda: g.conv_step(x[:, 0], w, None, st, idx=[0, 1])), ("Bm", lambda: g.ssm_forward(x, x, A, None, B)),
        ("Cm", lambda: g.ssm_forward(x, x, A, B, None)), ("A", lambda: g.ssm_forward(x, x, 1, B, B)), ("dt", lambda: g.ssm_forward(x, None, A, B, B)),
        ("hsave", lambda: g.ssm_backward(x, x, A, B, B, x, None)), ("h", lambda: g.ssm_step(x[:, 0], x[:, 0], A, B[:, 0], B[:, 0], None)),
        ("Cm", lambda: g.ssm_step(x[:, 0], x[:, 0], A, B[:, 0], None, h)), ("r", lambda: g.norm_forward(x, 1)),
        ("w_pre", lambda: g.norm_forward(x, x, w_pre=[1])), ("r_out", lambda: g.norm_backward(x, 2, None, x, w_pre=z(8))),
        ("w", lambda: g.causal_conv(x, None, return_state=True)), ("A", lambda: g.selective_scan(x, x, None, B, B, return_state=True)),
        ("x", lambda: g.causal_conv(None, w)), ("x", lambda: g.selective_scan(None, x, A, B, B)),
    ]
    for name, f in bad:
        with pytest.raises(TypeError, match=f"^{name} must be a torch.Tensor"):
            f()
    for f in (lambda: g.conv_step(x[:, 0], w, None, st[0]), lambda: g.ssm_step(x[:, 0], x[:, 0], A, B[:, 0], B[:, 0], h[0])):
        with pytest.raises(ValueError):
            f()
