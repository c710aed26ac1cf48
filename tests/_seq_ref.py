"""Plain 64-bit forms of the token-sequence operators, their gradients by formula, and bounds on the
rounding errors of an fp32 evaluation.

Bounds. u = 2^-24 is half a step of fp32. An output is a sum of products; with every term replaced by
its magnitude the same formulas give M, the sum of magnitudes. A product of f rounded factors, each
within k u of its value, is off by at most f k u (to first order), and adding n terms adds n u, so the
fp32 error is at most (k f + n) u M. Rounding the result to the storage type t adds
finfo(t).eps / 2 of its value. The k of each operator is derived where it is used.
"""
import torch

U = 2.0 ** -24
F64 = torch.float64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().cpu().to(F64)


def check(got, ref, mag, factor, what, dtype=None):
    """|got - ref| <= half a step of got's type + factor u mag, elementwise; got and ref share their shape."""
    dtype = dtype or got.dtype
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)}, expected {tuple(ref.shape)}"
    g = f64(got)
    # the last rounding is of the computed value, not of ref: the half step covers both to first order
    tol = half_step(dtype) * ref.abs() * (1 + 2.0 ** -7) + factor * U * mag + 1e-37
    bad = ~((g - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off; worst "
                           f"{((g - ref).abs() / tol).nan_to_num(9e9).max():.2f} times its bound")


def spans(B, L, cu):
    """(row, first token, end) of every sequence."""
    if cu is None:
        return [(b, 0, L) for b in range(B)]
    cu = [min(max(int(v), 0), L) for v in cu]
    return [(0, a, max(a, b)) for a, b in zip(cu, cu[1:])]


def sigmoid(v):
    return torch.sigmoid(v)


def silu(v):
    return v * torch.sigmoid(v)


def slope(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


# ------------------------------------------------------------------------------------ convolution
def conv(x, w, bias, act, cu, state0, dy=None, dstate=None):
    """dict of y, state and, with dy, dx, dw, db, ds; and the same names with '_m' for magnitudes."""
    x, w, bias, state0, dy, dstate = map(f64, (x, w, bias, state0, dy, dstate))
    B, L, C = x.shape
    K = w.shape[1]
    sp = spans(B, L, cu)
    out = dict(y=torch.zeros_like(x), y_m=torch.zeros_like(x), state=torch.zeros(len(sp), K - 1, C, dtype=F64))
    if dy is not None:
        for n, like in (("dx", x), ("dw", w), ("db", w[:, 0]), ("ds", out["state"])):
            out[n], out[n + "_m"] = torch.zeros_like(like), torch.zeros_like(like)
    for q, (r, a, b) in enumerate(sp):
        n = b - a
        before = torch.zeros(K - 1, C, dtype=F64) if state0 is None else state0[q]
        line = torch.cat([before, x[r, a:b]])
        out["state"][q] = line[n:]
        u = torch.zeros(n, C, dtype=F64) if bias is None else bias.expand(n, C).clone()
        um = u.abs()
        for k in range(K):
            u = u + w[:, k] * line[k:k + n]
            um = um + (w[:, k] * line[k:k + n]).abs()
        out["y"][r, a:b] = silu(u) if act else u
        out["y_m"][r, a:b] = 1.1 * um if act else um           # |silu'| < 1.1 carries u's error; |silu(u)| <= |u|
        if dy is None:
            continue
        g = dy[r, a:b]
        du = g * slope(u) if act else g
        dum = g.abs() * (1.1 + um) if act else g.abs()         # |silu''| <= 1/2: u's error moves the slope by as much
        dl, dlm = torch.zeros_like(line), torch.zeros_like(line)
        for k in range(K):
            dl[k:k + n] += w[:, k] * du
            dlm[k:k + n] += w[:, k].abs() * dum
            out["dw"][:, k] += (du * line[k:k + n]).sum(0)
            out["dw_m"][:, k] += (dum * line[k:k + n].abs()).sum(0)
        out["db"] += du.sum(0)
        out["db_m"] += dum.sum(0)
        if dstate is not None:
            dl[n:] += dstate[q]
            dlm[n:] += dstate[q].abs()
        out["dx"][r, a:b], out["dx_m"][r, a:b] = dl[K - 1:], dlm[K - 1:]
        out["ds"][q], out["ds_m"][q] = dl[:K - 1], dlm[:K - 1]
    return out


# --------------------------------------------------------------------------------- selective scan
def softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def scan(x, dt, A, Bm, Cm, D, z, dt_bias, sp_on, cu, h0, dy=None, dh=None):
    """dict of y, h and, with dy, the gradients dx ddt dA dB dC dD dz dbias dh0; '_m' for magnitudes."""
    x, dt, A, Bm, Cm, D, z, dt_bias, h0, dy, dh = map(f64, (x, dt, A, Bm, Cm, D, z, dt_bias, h0, dy, dh))
    B, L, C = x.shape
    G, N = Bm.shape[2:]
    wide = lambda v: v.repeat_interleave(C // G, dim=0)  # noqa: E731   (G, N) -> (C, N)
    narrow = lambda v: v.reshape(G, C // G, N).sum(1)    # noqa: E731
    v = dt if dt_bias is None else dt + dt_bias
    d = softplus(v) if sp_on else v
    dv = sigmoid(v) if sp_on else torch.ones_like(v)
    D0 = torch.zeros(C, dtype=F64) if D is None else D
    sps = spans(B, L, cu)
    o = {n: torch.zeros_like(x) for n in ("y", "y_m")}
    o["h"] = torch.zeros(len(sps), C, N, dtype=F64)
    o["h_m"] = torch.zeros_like(o["h"])
    if dy is not None:
        for n, like in (("dx", x), ("ddt", x), ("dz", x), ("dA", A), ("dB", Bm), ("dC", Cm), ("dD", D0), ("dbias", D0), ("dh0", o["h"])):
            o[n], o[n + "_m"] = torch.zeros_like(like), torch.zeros_like(like)
    for q, (r, first, end) in enumerate(sps):
        h = torch.zeros(C, N, dtype=F64) if h0 is None else h0[q]
        m = h.abs()
        hs, ms = [h], [m]
        for t in range(first, end):
            a = torch.exp(d[r, t, :, None] * A)
            b = (d[r, t] * x[r, t])[:, None] * wide(Bm[r, t])
            h, m = a * h + b, a * m + b.abs()
            hs.append(h)
            ms.append(m)
            s = silu(z[r, t]) if z is not None else 1.0
            sm = z[r, t].abs() if z is not None else 1.0
            o["y"][r, t] = ((h * wide(Cm[r, t])).sum(1) + D0 * x[r, t]) * s
            o["y_m"][r, t] = ((m * wide(Cm[r, t]).abs()).sum(1) + (D0 * x[r, t]).abs()) * sm
        o["h"][q], o["h_m"][q] = h, m
        if dy is None:
            continue
        ag = torch.zeros(C, N, dtype=F64) if dh is None else dh[q]
        am = ag.abs()
        for i in range(end - first, 0, -1):
            t = first + i - 1
            Bw, Cw, xt, dt_ = wide(Bm[r, t]), wide(Cm[r, t]), x[r, t], d[r, t]
            a = torch.exp(dt_[:, None] * A)
            g0 = dy[r, t]
            rr, rm = (g0, g0.abs()) if z is None else (g0 * silu(z[r, t]), (g0 * z[r, t]).abs())
            if z is not None:
                y0 = (hs[i] * Cw).sum(1) + D0 * xt
                ym = (ms[i] * Cw.abs()).sum(1) + (D0 * xt).abs()
                o["dz"][r, t], o["dz_m"][r, t] = g0 * y0 * slope(z[r, t]), g0.abs() * ym * 1.1
            g, gm = Cw * rr[:, None] + ag, Cw.abs() * rm[:, None] + am
            o["dC"][r, t], o["dC_m"][r, t] = narrow(rr[:, None] * hs[i]), narrow(rm[:, None] * ms[i])
            dx_ = dt_ * xt
            o["dB"][r, t], o["dB_m"][r, t] = narrow(g * dx_[:, None]), narrow(gm * dx_.abs()[:, None])
            thr, thm = (g * Bw).sum(1), (gm * Bw.abs()).sum(1)
            ag, am = a * g, a * gm
            e, em = ag * hs[i - 1], am * ms[i - 1]
            o["dA"] += e * dt_[:, None]
            o["dA_m"] += em * dt_.abs()[:, None]
            dd, dm = (e * A).sum(1) + thr * xt, (em * A.abs()).sum(1) + thm * xt.abs()
            o["ddt"][r, t], o["ddt_m"][r, t] = dd * dv[r, t], dm * dv[r, t]
            o["dx"][r, t], o["dx_m"][r, t] = thr * dt_ + D0 * rr, thm * dt_.abs() + D0.abs() * rm
            o["dD"] += rr * xt
            o["dD_m"] += rm * xt.abs()
            o["dbias"] += dd * dv[r, t]
            o["dbias_m"] += dm * dv[r, t]
        o["dh0"][q], o["dh0_m"][q] = ag, am
    return o


def scan_factor(T, N, C_group):
    """Per token the decay exp(d A) is off by: d, 12 u (softplus: exponential, quotient, seven-term series);
    times |d A|, which is under 4 in these tests: 48 u with the product's and the exponent scaling's
    roundings 8 u; the exponential itself 4 u; two more for the update: k = 64 for each of T tokens.
    Sums over N states, over a group's channels and over T tokens add their counts, gates and slopes 32."""
    return 64 * T + N + C_group + T + 64


# ------------------------------------------------------------------------------------------- norm
def norm(y, r, gate, w_post, b_post, scale, w_pre, b_pre, eps, center, r_given=None, dr=None, do=None):
    """dict of r_out, o and, with r_given (the stream as saved), the gradients; 64 bits."""
    y, r, gate, w_post, b_post, scale, w_pre, b_pre, r_given, dr, do = map(
        f64, (y, r, gate, w_post, b_post, scale, w_pre, b_pre, r_given, dr, do))

    def unit(v):
        c = v - v.mean(-1, keepdim=True) if center else v
        k = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
        return c * k, k

    def back(g, u, k):
        g2 = g - u * (g * u).mean(-1, keepdim=True)
        return (g2 - g.mean(-1, keepdim=True) if center else g2) * k

    m = y if gate is None else y * silu(gate)
    v, um, km = m, None, None
    if w_post is not None:
        um, km = unit(m)
        v = um * w_post + (0 if b_post is None else b_post)
    sv = v if scale is None else v * scale
    o = dict(r_out=sv if r is None else r + sv)
    if w_pre is not None:
        o["o"] = unit(o["r_out"])[0] * w_pre + (0 if b_pre is None else b_pre)
    if r_given is None and dr is None:
        return o
    d = torch.zeros_like(y) if dr is None else dr
    flat = lambda t: t.reshape(-1, t.shape[-1]).sum(0)  # noqa: E731
    if w_pre is not None:
        u, k = unit(r_given)
        o["dw_pre"], o["db_pre"] = flat(do * u), flat(do)
        o["dw_pre_m"], o["db_pre_m"] = flat((do * u).abs()), flat(do.abs())
        d = d + back(do * w_pre, u, k)
    o["dr_in"] = d
    if scale is not None:
        o["dscale"], o["dscale_m"] = flat(d * v), flat((d * v).abs())
    g = d if scale is None else d * scale
    if w_post is not None:
        o["dw_post"], o["db_post"] = flat(g * um), flat(g)
        o["dw_post_m"], o["db_post_m"] = flat((g * um).abs()), flat(g.abs())
        g = back(g * w_post, um, km)
    if gate is not None:
        o["dgate"] = g * y * slope(gate)
        g = g * silu(gate)
    o["dy"] = g
    return o
