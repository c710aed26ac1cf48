"""Token-sequence operators of libgspn (``include/gspn_seq.h`` has the full contract): a short
causal convolution, a selective state space scan and the norms around a block.

Argument marshalling only, as in the package's other calls: the work runs in the CUDA kernels of
``libgspn.so``. Activations are (B, L, C) tensors with channels side by side, fp32 or bf16; tokens
and rows may have any stride, so slices of a wider projection are taken as they are. Parameters,
scan states and parameter gradients are fp32.

``cu`` packs several sequences into one row: int32, (S + 1,), on the device, non-decreasing;
sequence q is tokens cu[q] .. cu[q+1]-1 of x[0]. Tokens in no sequence are left as they were in an
output that the caller passes, and hold nothing meaningful in one that is allocated here (the
autograd functions give zeros there).

Every call runs on x's device, on ``stream`` (default: that device's current one), and what it
allocates belongs to that stream. A tensor of the caller's that a call writes to counts as changed in
place: autograd refuses a backward pass that had kept it. A batch of no rows is taken: nothing is launched, and
gradients of parameters are zero.
"""
from __future__ import annotations

import ctypes
import functools

import torch

_VP, _SZ, _I, _LL, _F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_longlong, ctypes.c_float


class ConvDesc(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("B", "L", "C", "K", "S", "dtype", "silu")] + [("x_row", _LL), ("x_tok", _LL)]


class SsmDesc(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("B", "L", "C", "G", "N", "S", "dtype", "softplus")] + [
        (n, _LL) for n in ("x_row", "x_tok", "dt_row", "dt_tok", "z_row", "z_tok", "b_row", "b_tok", "c_row", "c_tok")]


class NormDesc(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("rows", "C", "dtype", "res_dtype", "center")] + [("eps", _F)] + [
        (n, _LL) for n in ("y_row", "gate_row", "r_row")]


_CP, _SP, _NP = (ctypes.POINTER(d) for d in (ConvDesc, SsmDesc, NormDesc))
SIGNATURES = {
    "gspn_conv_workspace_size": (_SZ, [_CP, _I]),
    "gspn_conv_forward": (_I, [_CP] + [_VP] * 8),
    "gspn_conv_backward": (_I, [_CP] + [_VP] * 12 + [_SZ, _VP]),
    "gspn_conv_step": (_I, [_CP] + [_VP] * 4 + [_I] + [_VP] * 3),
    "gspn_ssm_workspace_size": (_SZ, [_SP, _I]),
    "gspn_ssm_hsave_size": (_SZ, [_SP]),
    "gspn_ssm_forward": (_I, [_SP] + [_VP] * 14 + [_SZ, _VP]),
    "gspn_ssm_backward": (_I, [_SP] + [_VP] * 22 + [_SZ, _VP]),
    "gspn_ssm_step": (_I, [_SP] + [_VP] * 9 + [_I] + [_VP] * 3),
    "gspn_norm_workspace_size": (_SZ, [_NP, _I]),
    "gspn_norm_forward": (_I, [_NP] + [_VP] * 11),
    "gspn_norm_backward": (_I, [_NP] + [_VP] * 18 + [_SZ, _VP]),
}


def _pkg():
    import linear_spatial_propagation_gspn_b200 as g

    return g


@functools.lru_cache(maxsize=None)
def _fn(name):
    return getattr(_pkg().lib(), name)


def _ok(status, what):
    if status:
        raise _pkg().GspnError(status, what)


def _decline(*args):
    return None


class _Fast:
    """The calls of csrc/seq_binding.cpp: each makes the whole call, or returns None for the checks here to
    say why not. Looked up once, when the library is first needed; without the module (a tree that was
    built before it) every call goes through the checks here."""

    def __getattr__(self, name):
        fns = dict.fromkeys(("conv_forward", "conv_backward", "conv_step", "ssm_forward", "ssm_backward", "ssm_step", "norm_forward",
                             "norm_backward"), _decline)
        if name not in fns:
            raise AttributeError(name)
        L = _pkg().lib()
        try:
            from . import _seq_fast

            _seq_fast.init({n: ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in SIGNATURES})
            fns = {n: getattr(_seq_fast, n) for n in fns}
        except ImportError:
            pass
        self.__dict__.update(fns)
        return fns[name]


_fast = _Fast()


# Descriptors by their values: building one costs more than a small call's launch.
@functools.lru_cache(maxsize=1024)
def _desc(kind, *values):
    d = kind(*values)
    return d, ctypes.byref(d)


@functools.lru_cache(maxsize=1024)
def _size(name, device, kind, values, *more):
    n = int(_fn(name)(_desc(kind, *values)[1], *more))
    if n == 0:
        raise _pkg().GspnError(_pkg().GSPN_ERR_UNSUPPORTED, name)
    return n


def _workspace(name, x, kind, values, backward):
    n = _size(name, x.device.index, kind, values, backward)
    if n <= 256:
        return None, 0
    return torch.empty(n, dtype=torch.uint8, device=x.device), n


def _ptr(t):
    return None if t is None else t.data_ptr()


def _wrote(*ts):
    """Tells autograd that a call wrote to these tensors of the caller's (through their pointers, which it cannot
    see): a graph that kept one of them for its backward pass then refuses it, as after any in-place operation."""
    for t in ts:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _on_device(fn):
    """Runs fn(x, ...) on x's device, and on ``stream`` where one is given."""

    @functools.wraps(fn)
    def call(x, *args, stream=None, **kw):
        if not isinstance(x, torch.Tensor):
            raise TypeError("the first argument must be a torch.Tensor")
        if x.device.type != "cuda":
            raise ValueError("tensors must be CUDA tensors")
        if stream is None:
            if x.device.index == torch.cuda.current_device():
                return fn(x, *args, **kw)
            with torch.cuda.device(x.device):
                return fn(x, *args, **kw)
        if stream.device != x.device:
            raise ValueError(f"the stream is on {stream.device}, x on {x.device}")
        with torch.cuda.stream(stream):
            return fn(x, *args, **kw)

    return call


def _no_rows(x, *sums):
    """True for a batch of no rows, which is no call of the library's: what it would add up (sums) is zero, and the
    rest has no elements."""
    if x.shape[0]:
        return False
    for t in sums:
        if t is not None:
            t.zero_()
    return True


def _stream(x):
    return torch.cuda.current_stream(x.device).cuda_stream


def _code(t):
    if t == torch.float32:
        return 0
    if t == torch.bfloat16:
        return 1
    raise TypeError(f"unsupported dtype {t} (float32 or bfloat16)")


def _tensor(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


def _axes(name, t, form, n):
    if _tensor(name, t).dim() != n:
        raise ValueError(f"{name} must be {form}")
    return t.shape


def _is(name, t, shape, dtype, device, contiguous=True):
    _tensor(name, t)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _opt(name, t, shape, dtype, device):
    return None if t is None else _is(name, t, shape, dtype, device)


def _tokens(name, t, shape, dtype, device):
    """(row stride, token stride) of a (B, L, C) or (B, C) input whose channels stand side by side, or of
    a (B, L, G, N) one whose G x N do."""
    _is(name, t, shape, dtype, device, contiguous=False)
    st, inner = t.stride(), 1
    for i in range(len(shape) - 1, 1 if len(shape) > 2 else 0, -1):
        if shape[i] != 1 and st[i] != inner:
            raise ValueError(f"{name}: the elements of a token must stand side by side")
        inner *= shape[i]
    row, tok = st[0], (st[1] if len(shape) > 2 else 0)
    # the stride of an axis of one says nothing
    return (row if shape[0] > 1 else 0), (tok if len(shape) > 2 and shape[1] > 1 else 0)


def _packed(cu, x):
    if cu is None:
        return 0, x.shape[0]
    if _tensor("cu", cu).dim() != 1 or cu.shape[0] < 2:
        raise ValueError("cu must hold the S + 1 borders of the sequences")
    _is("cu", cu, cu.shape, torch.int32, x.device)
    if x.shape[0] != 1:
        raise ValueError("packed sequences stand in one row: x must be (1, L, C)")
    return cu.shape[0] - 1, cu.shape[0] - 1


def _slots(idx, state, rows, device):
    if idx is None:
        if state.shape[0] < rows:
            raise ValueError(f"{rows} rows, but {state.shape[0]} slots")
        return None
    return _is("idx", idx, (rows,), torch.int32, device)


# ------------------------------------------------------------------------------- convolution
def _conv_args(x, w, bias, silu, cu):
    B, L, C = _axes("x", x, "(B, L, C)", 3)
    K = _axes("w", w, "(C, K)", 2)[1]
    dev = x.device
    _is("w", w, (C, K), torch.float32, dev)
    _opt("bias", bias, (C,), torch.float32, dev)
    S, n = _packed(cu, x)
    values = (B, L, C, K, S, _code(x.dtype), int(bool(silu)), *_tokens("x", x, x.shape, x.dtype, dev))
    return values, (n, K - 1, C)


def conv_forward(x, w, bias=None, silu=True, cu=None, state0=None, y=None, state=None, stream=None):
    """y_t = act(bias + sum_k w[:, k] x_{t-K+1+k}), act = silu or nothing. x: (B, L, C); w: (C, K), K = 2..4;
    state0: (S or B, K-1, C), what lies before each sequence, oldest first (default zeros); state, of
    the same shape, receives the last K-1 inputs of each and may be state0."""
    if stream is None:
        done = _fast.conv_forward(x, w, bias, cu, state0, y, state, silu)
        if done is not None:
            return done
    return _conv_forward(x, w, bias, silu, cu, state0, y, state, stream=stream)


@_on_device
def _conv_forward(x, w, bias, silu, cu, state0, y, state):
    values, ss = _conv_args(x, w, bias, silu, cu)
    dev, dt = x.device, x.dtype
    _opt("state0", state0, ss, dt, dev)
    _opt("state", state, ss, dt, dev)
    given = y
    y = torch.empty(x.shape, dtype=dt, device=dev) if y is None else _is("y", y, x.shape, dt, dev)
    if _no_rows(x):
        return y
    _ok(_fn("gspn_conv_forward")(_desc(ConvDesc, *values)[1], x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(cu), _ptr(state0),
                                 y.data_ptr(), _ptr(state), _stream(x)), "gspn_conv_forward")
    _wrote(given, state)
    return y


def conv_backward(x, w, bias, dy, silu=True, cu=None, state0=None, dstate=None, out=None, stream=None):
    """Gradients (dx, dw, dbias, dstate0) of sum(dy y) + sum(dstate state); None for what was not given.
    out: tensors to write them to, in that order."""
    if stream is None and out is None:
        done = _fast.conv_backward(x, w, bias, cu, state0, dy, dstate, silu)
        if done is not None:
            return done
    return _conv_backward(x, w, bias, dy, silu, cu, state0, dstate, out, stream=stream)


@_on_device
def _conv_backward(x, w, bias, dy, silu, cu, state0, dstate, out):
    values, ss = _conv_args(x, w, bias, silu, cu)
    dev, dt = x.device, x.dtype
    _is("dy", dy, x.shape, dt, dev)
    _opt("state0", state0, ss, dt, dev)
    _opt("dstate", dstate, ss, dt, dev)
    given = out or ()
    if out is None:
        out = (torch.empty(x.shape, dtype=dt, device=dev), torch.empty_like(w), None if bias is None else torch.empty_like(bias),
               None if state0 is None else torch.empty_like(state0))
    dx, dw, db, ds = out
    _is("dx", dx, x.shape, dt, dev)
    _is("dw", dw, w.shape, torch.float32, dev)
    _opt("dbias", db, (x.shape[2],), torch.float32, dev)
    _opt("dstate0", ds, ss, dt, dev)
    if _no_rows(x, dw, db):
        return dx, dw, db, ds
    ws, n = _workspace("gspn_conv_workspace_size", x, ConvDesc, values, 1)
    _ok(_fn("gspn_conv_backward")(_desc(ConvDesc, *values)[1], x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(cu), _ptr(state0),
                                  dy.data_ptr(), _ptr(dstate), dx.data_ptr(), dw.data_ptr(), _ptr(db), _ptr(ds), _ptr(ws), n,
                                  _stream(x)), "gspn_conv_backward")
    _wrote(*given)
    return dx, dw, db, ds


def conv_step(x, w, bias, state, idx=None, silu=True, y=None, stream=None):
    """One token for each row. x: (B, C); state: (slots, K-1, C), moved on in place; idx: (B,) int32, each
    row's slot (default: its number). A row whose index is no slot is skipped; rows that name the
    same slot take their tokens in row order."""
    if stream is None:
        done = _fast.conv_step(x, w, bias, state, idx, y, silu)
        if done is not None:
            return done
    return _conv_step(x, w, bias, state, idx, silu, y, stream=stream)


@_on_device
def _conv_step(x, w, bias, state, idx, silu, y):
    (B, C), K = _axes("x", x, "(B, C)", 2), _axes("w", w, "(C, K)", 2)[1]
    _axes("state", state, "(slots, K-1, C)", 3)
    dev, dt = x.device, x.dtype
    _is("w", w, (C, K), torch.float32, dev)
    _opt("bias", bias, (C,), torch.float32, dev)
    _is("state", state, (state.shape[0], K - 1, C), dt, dev)
    _slots(idx, state, B, dev)
    row, _ = _tokens("x", x, x.shape, dt, dev)
    given = y
    y = torch.empty((B, C), dtype=dt, device=dev) if y is None else _is("y", y, (B, C), dt, dev)
    if _no_rows(x):
        return y
    _ok(_fn("gspn_conv_step")(_desc(ConvDesc, B, 1, C, K, 0, _code(dt), int(bool(silu)), row, 0)[1], x.data_ptr(), w.data_ptr(),
                              _ptr(bias), _ptr(idx), state.shape[0], state.data_ptr(), y.data_ptr(), _stream(x)),
        "gspn_conv_step")
    _wrote(state, given)
    return y


# ------------------------------------------------------------------------------ selective scan
def _ssm_args(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, cu):
    B, L, C = _axes("x", x, "(B, L, C)", 3)
    G, N = _axes("Bm", Bm, "(B, L, G, N)", 4)[2:]
    dev, ty, f = x.device, x.dtype, torch.float32
    if G < 1 or C % G:
        raise ValueError(f"{G} groups do not divide {C} channels")
    _is("A", A, (C, N), f, dev)
    _opt("D", D, (C,), f, dev)
    _opt("dt_bias", dt_bias, (C,), f, dev)
    S, n = _packed(cu, x)
    bc = (B, L, G, N)
    strides = (*_tokens("x", x, x.shape, ty, dev), *_tokens("dt", dt, x.shape, ty, dev),
               *((0, 0) if z is None else _tokens("z", z, x.shape, ty, dev)),
               *_tokens("Bm", Bm, bc, ty, dev), *_tokens("Cm", Cm, bc, ty, dev))
    return (B, L, C, G, N, S, _code(ty), int(bool(softplus)), *strides), (n, C, N)


def _ssm_run(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, cu, h0, y, h, save):
    values, ss = _ssm_args(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, cu)
    dev = x.device
    _opt("h0", h0, ss, torch.float32, dev)
    _opt("h", h, ss, torch.float32, dev)
    given = y
    y = torch.empty(x.shape, dtype=x.dtype, device=dev) if y is None else _is("y", y, x.shape, x.dtype, dev)
    if _no_rows(x):
        return y, torch.empty(0, dtype=torch.float32, device=dev) if save else None
    hsave = None
    if save:
        hsave = torch.empty(_size("gspn_ssm_hsave_size", dev.index, SsmDesc, values) // 4, dtype=torch.float32, device=dev)
    ws, n = _workspace("gspn_ssm_workspace_size", x, SsmDesc, values, 0)
    _ok(_fn("gspn_ssm_forward")(_desc(SsmDesc, *values)[1], x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(),
                                _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(cu), _ptr(h0), y.data_ptr(), _ptr(h), _ptr(hsave), _ptr(ws),
                                n, _stream(x)), "gspn_ssm_forward")
    _wrote(given, h)
    return y, hsave


def ssm_forward(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=True, cu=None, h0=None, y=None, h=None,
                stream=None):
    """h_t = exp(d_t A) h_{t-1} + d_t x_t B_t, y_t = (C_t h_t + D x_t) silu(z_t), with d = dt + dt_bias taken
    through softplus unless softplus is false. x, dt, z: (B, L, C); Bm, Cm: (B, L, G, N), G dividing C;
    A: (C, N), N <= 64; D, dt_bias: (C,). h0: (S or B, C, N) fp32, the states before the sequences
    (default zeros); h, of the same shape, receives the ones behind them and may be h0."""
    if stream is None:
        done = _fast.ssm_forward(x, dt, A, Bm, Cm, D, z, dt_bias, cu, h0, y, h, softplus, False)
        if done is not None:
            return done
    return _ssm_forward(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, cu, h0, y, h, stream=stream)


@_on_device
def _ssm_forward(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, cu, h0, y, h):
    return _ssm_run(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, cu, h0, y, h, False)[0]


def ssm_forward_save(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=True, cu=None, h0=None, y=None, h=None,
                     stream=None):
    """Training forward: y as ssm_forward, and the states (a flat fp32 tensor) that ssm_backward starts from."""
    if stream is None:
        done = _fast.ssm_forward(x, dt, A, Bm, Cm, D, z, dt_bias, cu, h0, y, h, softplus, True)
        if done is not None:
            return done
    return _ssm_forward_save(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, cu, h0, y, h, stream=stream)


@_on_device
def _ssm_forward_save(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, cu, h0, y, h):
    return _ssm_run(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, cu, h0, y, h, True)


def ssm_backward(x, dt, A, Bm, Cm, dy, hsave, D=None, z=None, dt_bias=None, softplus=True, cu=None, h0=None, dh=None, out=None,
                 stream=None):
    """Gradients (dx, ddt, dA, dBm, dCm, dD, dz, ddt_bias, dh0) of sum(dy y) + sum(dh h), None for what was not
    given; hsave from ssm_forward_save on the same inputs. out: tensors to write them to, in that order."""
    if stream is None and out is None:
        done = _fast.ssm_backward(x, dt, A, Bm, Cm, dy, hsave, D, z, dt_bias, cu, h0, dh, softplus)
        if done is not None:
            return done
    return _ssm_backward(x, dt, A, Bm, Cm, dy, hsave, D, z, dt_bias, softplus, cu, h0, dh, out, stream=stream)


@_on_device
def _ssm_backward(x, dt, A, Bm, Cm, dy, hsave, D, z, dt_bias, softplus, cu, h0, dh, out):
    values, ss = _ssm_args(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, cu)
    dev, ty, f = x.device, x.dtype, torch.float32
    _is("dy", dy, x.shape, ty, dev)
    _is("hsave", hsave, (_size("gspn_ssm_hsave_size", dev.index, SsmDesc, values) // 4 if x.shape[0] else 0,), f, dev)
    _opt("h0", h0, ss, f, dev)
    _opt("dh", dh, ss, f, dev)

    def like(t, shape, dtype):
        return None if t is None else torch.empty(shape, dtype=dtype, device=dev)

    given = out or ()
    if out is None:
        out = (like(x, x.shape, ty), like(x, x.shape, ty), like(A, A.shape, f), like(Bm, Bm.shape, ty), like(Cm, Cm.shape, ty),
               like(D, (x.shape[2],), f), like(z, x.shape, ty), like(dt_bias, (x.shape[2],), f), like(h0, ss, f))
    dx, ddt, dA, dB, dC, dD, dz, dbias, dh0 = out
    for name, t, like_t, dtype in (("dx", dx, x, ty), ("ddt", ddt, x, ty), ("dA", dA, A, f), ("dBm", dB, Bm, ty), ("dCm", dC, Cm, ty)):
        _is(name, t, like_t.shape, dtype, dev)
    _opt("dD", dD, (x.shape[2],), f, dev)
    _opt("dz", dz, x.shape, ty, dev)
    _opt("ddt_bias", dbias, (x.shape[2],), f, dev)
    _opt("dh0", dh0, ss, f, dev)
    if _no_rows(x, dA, dD, dbias):
        return dx, ddt, dA, dB, dC, dD, dz, dbias, dh0
    n = _size("gspn_ssm_workspace_size", dev.index, SsmDesc, values, 1)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _ok(_fn("gspn_ssm_backward")(_desc(SsmDesc, *values)[1], x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(),
                                 _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(cu), hsave.data_ptr(), dy.data_ptr(), _ptr(dh),
                                 dx.data_ptr(), ddt.data_ptr(), dA.data_ptr(), dB.data_ptr(), dC.data_ptr(), _ptr(dD), _ptr(dz),
                                 _ptr(dbias), _ptr(dh0), ws.data_ptr(), n, _stream(x)), "gspn_ssm_backward")
    _wrote(*given)
    return dx, ddt, dA, dB, dC, dD, dz, dbias, dh0


def ssm_step(x, dt, A, Bm, Cm, h, D=None, z=None, dt_bias=None, softplus=True, idx=None, y=None, stream=None):
    """One token for each row. x, dt, z: (B, C); Bm, Cm: (B, G, N); h: (slots, C, N) fp32, moved on in place;
    idx as for conv_step."""
    if stream is None:
        done = _fast.ssm_step(x, dt, A, Bm, Cm, h, D, z, dt_bias, idx, y, softplus)
        if done is not None:
            return done
    return _ssm_step(x, dt, A, Bm, Cm, h, D, z, dt_bias, softplus, idx, y, stream=stream)


@_on_device
def _ssm_step(x, dt, A, Bm, Cm, h, D, z, dt_bias, softplus, idx, y):
    (B, C), (G, N) = _axes("x", x, "(B, C)", 2), _axes("Bm", Bm, "(B, G, N)", 3)[1:]
    _axes("h", h, "(slots, C, N)", 3)
    dev, ty, f = x.device, x.dtype, torch.float32
    if G < 1 or C % G:
        raise ValueError(f"{G} groups do not divide {C} channels")
    _is("A", A, (C, N), f, dev)
    _opt("D", D, (C,), f, dev)
    _opt("dt_bias", dt_bias, (C,), f, dev)
    _is("h", h, (h.shape[0], C, N), f, dev)
    _slots(idx, h, B, dev)
    xr, dr = _tokens("x", x, x.shape, ty, dev)[0], _tokens("dt", dt, x.shape, ty, dev)[0]
    zr = 0 if z is None else _tokens("z", z, x.shape, ty, dev)[0]
    br, cr = (_tokens(n, _tensor(n, t).unsqueeze(1), (B, 1, G, N), ty, dev)[0] for n, t in (("Bm", Bm), ("Cm", Cm)))
    given = y
    y = torch.empty((B, C), dtype=ty, device=dev) if y is None else _is("y", y, (B, C), ty, dev)
    if _no_rows(x):
        return y
    desc = _desc(SsmDesc, B, 1, C, G, N, 0, _code(ty), int(bool(softplus)), xr, 0, dr, 0, zr, 0, br, 0, cr, 0)[1]
    _ok(_fn("gspn_ssm_step")(desc, x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(), _ptr(D), _ptr(z),
                             _ptr(dt_bias), _ptr(idx), h.shape[0], h.data_ptr(), y.data_ptr(), _stream(x)), "gspn_ssm_step")
    _wrote(h, given)
    return y


# ------------------------------------------------------------------------- norms around a block
def _rows(name, t, shape, dtypes, device):
    """Stride between the rows of a (..., C) tensor that is one run of rows."""
    if _tensor(name, t).device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    C = shape[-1]
    if t.is_contiguous():
        return C
    st = t.stride()
    if C != 1 and st[-1] != 1:
        raise ValueError(f"{name}: the elements of a row must stand side by side")
    row, inner = None, None                       # leading axes must be one run of rows
    for i in range(len(shape) - 2, -1, -1):
        if shape[i] == 1:
            continue
        if row is None:
            row, inner = st[i], st[i] * shape[i]
        elif st[i] == inner:
            inner *= shape[i]
        else:
            raise ValueError(f"{name}: its rows must be evenly spaced")
    return C if row is None else row


def _norm_args(y, gate, w_post, b_post, scale, r, w_pre, b_pre, eps, center, res_dtype):
    if y.dim() < 1:
        raise ValueError("y must be (..., C)")
    C, dev = y.shape[-1], y.device
    for name, t in (("w_post", w_post), ("b_post", b_post), ("scale", scale), ("w_pre", w_pre), ("b_pre", b_pre)):
        if t is not None:
            _is(name, t, (C,), torch.float32, dev)
    if (b_post is not None and w_post is None) or (b_pre is not None and w_pre is None):
        raise ValueError("a norm's bias needs its weight")
    dts = (y.dtype,)
    rows = 1
    for s in y.shape[:-1]:
        rows *= s
    return (rows, C, _code(y.dtype), _code(res_dtype), int(bool(center)), float(eps), _rows("y", y, y.shape, dts, dev),
            0 if gate is None else _rows("gate", gate, y.shape, dts, dev),
            0 if r is None else _rows("r", r, y.shape, (y.dtype, torch.float32), dev))


def norm_forward(y, r=None, gate=None, w_post=None, b_post=None, scale=None, w_pre=None, b_pre=None, eps=1e-5, center=False,
                 r_out=None, o=None, stream=None):
    """(r_out, o): r_out = r + scale * (norm(y silu(gate)) w_post + b_post) and o = norm(r_out) w_pre + b_pre, the end
    of one block and the beginning of the next in one pass. norm(v) = v / sqrt(mean(v^2) + eps), of
    v - mean(v) if center. y, gate: (..., C); r of y's dtype or fp32, and r_out with it. Whatever is None
    is left out (no w_post or w_pre: no norm there; no w_pre: o is None; no r: r_out has y's dtype)."""
    if stream is None:
        done = _fast.norm_forward(y, r, gate, w_post, b_post, scale, w_pre, b_pre, r_out, o, eps, center)
        if done is not None:
            return done
    return _norm_forward(y, r, gate, w_post, b_post, scale, w_pre, b_pre, eps, center, r_out, o, stream=stream)


@_on_device
def _norm_forward(y, r, gate, w_post, b_post, scale, w_pre, b_pre, eps, center, r_out, o):
    rt = y.dtype if r is None else _tensor("r", r).dtype
    values = _norm_args(y, gate, w_post, b_post, scale, r, w_pre, b_pre, eps, center, rt)
    dev, given = y.device, (r_out, o if w_pre is not None else None)
    r_out = torch.empty(y.shape, dtype=rt, device=dev) if r_out is None else _is("r_out", r_out, y.shape, rt, dev)
    if w_pre is None:
        o = None
    else:
        o = torch.empty(y.shape, dtype=y.dtype, device=dev) if o is None else _is("o", o, y.shape, y.dtype, dev)
    _ok(_fn("gspn_norm_forward")(_desc(NormDesc, *values)[1], y.data_ptr(), _ptr(gate), _ptr(w_post), _ptr(b_post), _ptr(scale),
                                 _ptr(r), _ptr(w_pre), _ptr(b_pre), r_out.data_ptr(), _ptr(o), _stream(y)), "gspn_norm_forward")
    _wrote(*given)
    return r_out, o


def norm_backward(y, r_out, dr, do, gate=None, w_post=None, b_post=None, scale=None, w_pre=None, b_pre=None, eps=1e-5,
                  center=False, stream=None):
    """Gradients (dy, dr_in, dgate, dw_post, db_post, dscale, dw_pre, db_pre) of sum(dr r_out) + sum(do o), None for what
    was not given. r_out is norm_forward's; dr_in is the gradient of its r (of r_out's dtype). dr may be
    None (the stream behind the block is not used); do goes with w_pre, and without it r_out may be None."""
    if stream is None:
        done = _fast.norm_backward(y, r_out, dr, do, gate, w_post, b_post, scale, w_pre, b_pre, eps, center)
        if done is not None:
            return done
    return _norm_backward(y, r_out, dr, do, gate, w_post, b_post, scale, w_pre, b_pre, eps, center, stream=stream)


@_on_device
def _norm_backward(y, r_out, dr, do, gate, w_post, b_post, scale, w_pre, b_pre, eps, center):
    if (w_pre is None) != (do is None):
        raise ValueError("do goes with w_pre")
    if r_out is None and dr is None or r_out is None and w_pre is not None:
        raise ValueError("r_out (or, without w_pre, dr) must be given")
    rt = (_tensor("dr", dr) if r_out is None else _tensor("r_out", r_out)).dtype
    values = _norm_args(y, gate, w_post, b_post, scale, r_out, w_pre, b_pre, eps, center, rt)
    dev, ty = y.device, y.dtype
    _opt("dr", dr, y.shape, rt, dev)
    _opt("do", do, y.shape, ty, dev)

    def like(t, dtype=None):
        return None if t is None else torch.empty(t.shape, dtype=dtype or t.dtype, device=dev)

    dy, dgate = like(y), like(gate)
    dr_in = torch.empty(y.shape, dtype=rt, device=dev)
    sums = tuple(like(t) for t in (w_post, b_post, scale, w_pre, b_pre))
    n = _size("gspn_norm_workspace_size", dev.index, NormDesc, values, 1)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)

    def run(*wanted):
        return _fn("gspn_norm_backward")(_desc(NormDesc, *values)[1], y.data_ptr(), _ptr(gate), _ptr(w_post), _ptr(b_post), _ptr(scale),
                                         _ptr(r_out), _ptr(w_pre), _ptr(dr), _ptr(do), dy.data_ptr(), dr_in.data_ptr(), _ptr(dgate),
                                         *map(_ptr, wanted), ws.data_ptr(), n, _stream(y))

    status = run(*sums)
    if status == _pkg().GSPN_ERR_UNSUPPORTED and sum(t is not None for t in sums) > 3:
        # Column sums of so wide rows fit three at a time: the other norm's in a second pass, which writes the rows'
        # gradients again, the same ones.
        status = run(*sums[:3], None, None) or run(None, None, None, *sums[3:])
    _ok(status, "gspn_norm_backward")
    return (dy, dr_in, dgate, *sums)


# ------------------------------------------------------------------------------------ autograd
def _fresh(t, cu):
    """An output for autograd: tokens outside every packed sequence have to read as zero."""
    return None if t is None else (torch.empty if cu is None else torch.zeros)(t.shape, dtype=t.dtype, device=t.device)


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, silu, cu, state0, return_state):
        S, n = _packed(cu, x) if _tensor("x", x).dim() == 3 else (0, 0)
        state = torch.empty((n, _axes("w", w, "(C, K)", 2)[1] - 1, x.shape[-1]), dtype=x.dtype, device=x.device) if return_state else None
        y = conv_forward(x, w, bias, silu=silu, cu=cu, state0=state0, y=_fresh(x, cu), state=state)
        ctx.save_for_backward(x, w, bias, cu, state0)
        ctx.silu = silu
        return (y, state) if return_state else y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dstate=None):
        x, w, bias, cu, state0 = ctx.saved_tensors
        out = (_fresh(x, cu), torch.empty_like(w), None if bias is None else torch.empty_like(bias),
               None if state0 is None else torch.empty_like(state0))
        dx, dw, db, ds = conv_backward(x, w, bias, dy.contiguous(), silu=ctx.silu, cu=cu, state0=state0,
                                       dstate=None if dstate is None else dstate.contiguous(), out=out)
        return dx, dw, db, None, None, ds, None


def causal_conv(x, w, bias=None, silu=True, cu=None, state0=None, return_state=False):
    """Differentiable conv_forward; with return_state, (y, state)."""
    return _CausalConv.apply(x, w, bias, silu, cu, state0, return_state)


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, Bm, Cm, D, z, dt_bias, softplus, cu, h0, return_state, grad):
        S, n = _packed(cu, x) if _tensor("x", x).dim() == 3 else (0, 0)
        h = torch.empty((n, *_axes("A", A, "(C, N)", 2)), dtype=torch.float32, device=x.device) if return_state else None
        kw = dict(D=D, z=z, dt_bias=dt_bias, softplus=softplus, cu=cu, h0=h0, y=_fresh(x, cu), h=h)
        ctx.softplus = softplus
        if grad and any(ctx.needs_input_grad):
            y, hsave = ssm_forward_save(x, dt, A, Bm, Cm, **kw)
            ctx.save_for_backward(x, dt, A, Bm, Cm, D, z, dt_bias, cu, h0, hsave)
        else:
            y = ssm_forward(x, dt, A, Bm, Cm, **kw)
        return (y, h) if return_state else y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh=None):
        x, dt, A, Bm, Cm, D, z, dt_bias, cu, h0, hsave = ctx.saved_tensors
        like = lambda t: None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)  # noqa: E731
        out = (_fresh(x, cu), _fresh(x, cu), like(A), _fresh(Bm, cu), _fresh(Cm, cu), like(D), _fresh(z, cu), like(dt_bias), like(h0))
        g = ssm_backward(x, dt, A, Bm, Cm, dy.contiguous(), hsave, D=D, z=z, dt_bias=dt_bias, softplus=ctx.softplus, cu=cu,
                         h0=h0, dh=None if dh is None else dh.contiguous(), out=out)
        return (*g[:8], None, None, g[8], None, None)


def selective_scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=True, cu=None, h0=None, return_state=False):
    """Differentiable ssm_forward; with return_state, (y, h)."""
    # needs_input_grad tells what the inputs ask for, under no_grad too
    return _SelectiveScan.apply(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, cu, h0, return_state, torch.is_grad_enabled())


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, r, gate, w_post, b_post, scale, w_pre, b_pre, eps, center):
        r_out, o = norm_forward(y, r, gate=gate, w_post=w_post, b_post=b_post, scale=scale, w_pre=w_pre, b_pre=b_pre, eps=eps,
                                center=center)
        ctx.save_for_backward(y, gate, w_post, b_post, scale, w_pre, b_pre, r_out)
        ctx.eps, ctx.center, ctx.has_r = eps, center, r is not None
        ctx.set_materialize_grads(False)
        return r_out if o is None else (r_out, o)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dr, do=None):
        y, gate, w_post, b_post, scale, w_pre, b_pre, r_out = ctx.saved_tensors
        if dr is None and do is None:
            return (None,) * 10
        if w_pre is not None and do is None:
            do = torch.zeros(y.shape, dtype=y.dtype, device=y.device)
        g = norm_backward(y, r_out, None if dr is None else dr.contiguous(), None if do is None else do.contiguous(), gate=gate,
                          w_post=w_post, b_post=b_post, scale=scale, w_pre=w_pre, b_pre=b_pre, eps=ctx.eps, center=ctx.center)
        dy, dr_in, dgate, *sums = g
        return (dy, dr_in if ctx.has_r else None, dgate, *sums, None, None)


def block_norm(y, r=None, gate=None, w_post=None, b_post=None, scale=None, w_pre=None, b_pre=None, eps=1e-5, center=False):
    """Differentiable norm_forward: (r_out, o), with o None without w_pre."""
    out = _BlockNorm.apply(y, r, gate, w_post, b_post, scale, w_pre, b_pre, eps, center)
    return out if w_pre is not None else (out, None)
