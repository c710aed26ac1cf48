"""Cases of the token-sequence operators: the short causal convolution, the selective state space
scan and the norms around a block, in their plain form and as calls of the library.

Sizes: 192, 96 and 1152 channels are the ones of this repository's workloads; the others are
generic powers of two and odd numbers beside them. State width 16 throughout unless a case is there
to have another one.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one user being answered: a single token of one row through the scan, latency alone
        dict(name="scan step, 1 row", op="scan", pass_="step", rows=1, C=1152, G=1, N=16, dtype="bf16", slots=4),
        # a full serving batch: a token for each of 256 rows, states scattered over a larger pool
        dict(name="scan step, 256 rows", op="scan", pass_="step", rows=256, C=4096, G=1, N=16, dtype="bf16", slots=320),
        # a later piece of one prompt, odd length, few channels: starts from a state and leaves one
        dict(name="scan prompt, f32 odd", op="scan", pass_="prompt", B=1, L=333, C=192, G=1, N=16, dtype="f32", seqs=0, gate=True, state=True),
        # prompts of several users packed behind one another, lengths far apart
        dict(name="scan prompt, packed", op="scan", pass_="prompt", B=1, L=8192, C=2048, G=1, N=16, dtype="bf16", seqs=9, gate=True, state=True),
        # one long document read in one go
        dict(name="scan prompt, long", op="scan", pass_="prompt", B=1, L=16384, C=4096, G=1, N=16, dtype="bf16", seqs=0, gate=True, state=True),
        # the scan in a training step, forward and gradients, at a usual batch
        dict(name="scan train, bf16", op="scan", pass_="train", B=4, L=2048, C=2048, G=1, N=16, dtype="bf16", seqs=0, gate=True, state=False),
        # the same in full precision with two groups, a wider state and odd sizes
        dict(name="scan train, f32 odd", op="scan", pass_="train", B=3, L=577, C=202, G=2, N=24, dtype="f32", seqs=0, gate=True, state=False),
        # the convolution before the scan, over packed prompts
        dict(name="conv prompt, packed", op="conv", pass_="prompt", B=1, L=8192, C=4096, K=4, dtype="bf16", seqs=9, state=True),
        # the convolution for a token of each row of a serving batch
        dict(name="conv step, 256 rows", op="conv", pass_="step", rows=256, C=4096, K=4, dtype="bf16", slots=320),
        # gradients of the convolution in a training step
        dict(name="conv train, bf16", op="conv", pass_="train", B=4, L=2048, C=2048, K=4, dtype="bf16", seqs=0, state=False),
        # the end of a block and the norm before the next one, a long prompt, fp32 residual stream
        dict(name="norm forward", op="norm", pass_="forward", rows=8192, C=4096, dtype="bf16", res="f32", gate=True, post=True, center=False),
        # its gradients in a training step, an odd width, centred norms
        dict(name="norm backward, odd", op="norm", pass_="backward", rows=8190, C=1153, dtype="bf16", res="bf16", gate=True, post=True, center=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "conv", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        c = dict(op=op, pass_=rng.choice(["forward", "backward"]), rows=_log(rng, 1, 8192), C=_log(rng, 96, 4096), dtype=dtype,
                 res=rng.choice([dtype, "f32"]), gate=rng.random() < 0.7, post=rng.random() < 0.7, center=rng.random() < 0.3)
        if rng.random() < 0.5:
            c["C"] = max(8, c["C"] // 8 * 8)
        return c
    C = _log(rng, 64, 4096)
    if rng.random() < 0.6:
        C = max(32, C // 32 * 32)
    what = rng.choice(["step", "prompt", "train"])
    if op == "conv":
        K = rng.choice([2, 3, 4, 4])
        if what == "step":
            rows = _log(rng, 1, 256)
            return dict(op=op, pass_=what, rows=rows, C=C, K=K, dtype=dtype, slots=rows + rng.randrange(1, 64))
        B, L = _batch(rng, C, 1 << 25 if what == "prompt" else 1 << 24)
        seqs = rng.randrange(1, 10) if B == 1 and rng.random() < 0.6 else 0
        return dict(op=op, pass_=what, B=B, L=L, C=C, K=K, dtype=dtype, seqs=seqs, state=rng.random() < 0.5)
    N = rng.choice([16, 16, 16, 8, 12, 32])
    G = rng.choice([1, 1, 2])
    C = C // G * G
    if what == "step":
        rows = _log(rng, 1, 256)
        return dict(op=op, pass_=what, rows=rows, C=C, G=G, N=N, dtype=dtype, slots=rows + rng.randrange(1, 64))
    B, L = _batch(rng, C * N // 16 + 1, 1 << 26 if what == "prompt" else 1 << 23)
    seqs = rng.randrange(1, 10) if B == 1 and rng.random() < 0.6 else 0
    return dict(op=op, pass_=what, B=B, L=L, C=C, G=G, N=N, dtype=dtype, seqs=seqs, gate=rng.random() < 0.7, state=rng.random() < 0.5)


def _batch(rng, C, most):
    """Rows and tokens: 1 to 8 rows, 1 to 16384 tokens, no more than `most` elements in all."""
    B = rng.choice([1, 1, 1, 2, 3, 4, 8])
    return B, max(1, min(_log(rng, 1, 16384), most // (B * C)))


# ----------------------------------------------------------------------------------------- inputs
def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _lengths(total, seqs, seed):
    """`seqs` lengths that add up to `total`, far apart."""
    r = random.Random(seed)
    cuts = sorted(r.randrange(0, total + 1) for _ in range(seqs - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _cu(case, seed):
    if not case["seqs"]:
        return None
    at = [0]
    for n in _lengths(case["L"], case["seqs"], seed):
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _slots(case, seed):
    r = random.Random(seed)
    return torch.tensor(r.sample(range(case["slots"]), case["rows"]), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _type(case["dtype"])

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=g, device="cuda")

    s = dict(case=dict(case))
    C = case["C"]
    if case["op"] == "norm":
        R, f = case["rows"], torch.float32
        rt = _type(case["res"])
        s.update(y=normal(R, C), gate=normal(R, C) if case["gate"] else None,
                 w_post=uniform(0.5, 1.5, C) if case["post"] else None, scale=uniform(0.1, 1.0, C), w_pre=uniform(0.5, 1.5, C),
                 b_post=normal(C, std=0.1, dtype=f) if case["post"] and case["center"] else None,
                 b_pre=normal(C, std=0.1, dtype=f) if case["center"] else None)
        s["r"] = normal(R, C, std=2.0, dtype=rt)
        if case["pass_"] == "backward":  # r is then the stream behind the block, as the forward pass left it
            s.update(do=normal(R, C), dr=normal(R, C, dtype=rt))
        return s
    step = case["pass_"] == "step"
    lead = (case["rows"],) if step else (case["B"], case["L"])
    if case["op"] == "conv":
        K = case["K"]
        s.update(x=normal(*lead, C), w=uniform(-1.0, 1.0, C, K) / math.sqrt(K), bias=uniform(-0.5, 0.5, C))
        if step:
            s.update(state=normal(case["slots"], K - 1, C), idx=_slots(case, seed))
            return s
        s["cu"] = _cu(case, seed)
        S = case["seqs"] or case["B"]
        s["state0"] = normal(S, K - 1, C) if case["state"] else None
        if case["pass_"] == "train":
            s["dy"] = normal(*lead, C)
        elif case["state"]:
            s["state"] = torch.empty(S, K - 1, C, dtype=dt, device="cuda")
        return s
    G, N = case["G"], case["N"]
    # rates 1 .. N and steps log-uniform in [1e-3, 1e-1], the usual start of such a model
    step_size = torch.exp(uniform(math.log(1e-3), math.log(1e-1), C))
    s.update(x=normal(*lead, C), dt=normal(*lead, C, std=0.5), A=-(torch.arange(1, N + 1, device="cuda") * uniform(0.8, 1.2, C, N)),
             Bm=normal(*lead, G, N), Cm=normal(*lead, G, N), D=uniform(0.5, 1.5, C), dt_bias=torch.log(torch.expm1(step_size)),
             z=normal(*lead, C) if case.get("gate", True) else None)
    if step:
        s.update(h=normal(case["slots"], C, N, std=0.5, dtype=torch.float32), idx=_slots(case, seed))
        return s
    s["cu"] = _cu(case, seed)
    S = case["seqs"] or case["B"]
    s["h0"] = normal(S, C, N, std=0.5, dtype=torch.float32) if case["state"] else None
    if case["pass_"] == "train":
        s["dy"] = normal(*lead, C)
    elif case["state"]:
        s["h"] = torch.empty(S, C, N, device="cuda")
    return s


# -------------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if case["op"] == "norm":
        return _norm_forward(s, case) if case["pass_"] == "forward" else _norm_backward(s, case)
    if case["op"] == "conv":
        return dict(step=_conv_step, prompt=_conv_prompt, train=_conv_train)[case["pass_"]](s, case)
    return dict(step=_scan_step, prompt=_scan_prompt, train=_scan_train)[case["pass_"]](s, case)


def _own(s, case):
    import linear_spatial_propagation_gspn_b200 as g

    if case["op"] == "norm":
        if case["pass_"] == "forward":
            return g.norm_forward(s["y"], s["r"], gate=s["gate"], w_post=s["w_post"], b_post=s["b_post"], scale=s["scale"],
                                  w_pre=s["w_pre"], b_pre=s["b_pre"], center=case["center"])
        return g.norm_backward(s["y"], s["r"], s["dr"], s["do"], gate=s["gate"], w_post=s["w_post"], b_post=s["b_post"],
                               scale=s["scale"], w_pre=s["w_pre"], b_pre=s["b_pre"], center=case["center"])
    if case["op"] == "conv":
        if case["pass_"] == "step":
            return g.conv_step(s["x"], s["w"], s["bias"], s["state"], idx=s["idx"]), s["state"]
        if case["pass_"] == "prompt":
            y = g.conv_forward(s["x"], s["w"], s["bias"], cu=s["cu"], state0=s["state0"], state=s.get("state"))
            return y, s.get("state")
        y = g.conv_forward(s["x"], s["w"], s["bias"], cu=s["cu"], state0=s["state0"])
        return y, g.conv_backward(s["x"], s["w"], s["bias"], s["dy"], cu=s["cu"], state0=s["state0"])
    if case["pass_"] == "step":
        y = g.ssm_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["h"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"], idx=s["idx"])
        return y, s["h"]
    if case["pass_"] == "prompt":
        y = g.ssm_forward(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"], cu=s["cu"],
                          h0=s["h0"], h=s.get("h"))
        return y, s.get("h")
    y, hsave = g.ssm_forward_save(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"], cu=s["cu"],
                                  h0=s["h0"])
    return y, g.ssm_backward(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], hsave, D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                             cu=s["cu"], h0=s["h0"])


# ---- plain forms: elementary operations in 32 bits, rounded once at the end
def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _silu_slope(v):
    p = 1.0 / (1.0 + torch.exp(-v))
    return p * (1.0 + v * (1.0 - p))


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-v.abs()))


def _places(s, case):
    """For each token: its sequence, its place in it, and the sequence's length (all B x L)."""
    B, L = case["B"], case["L"]
    t = torch.arange(L, device="cuda")
    if s["cu"] is None:
        return torch.arange(B, device="cuda")[:, None].expand(B, L), t.expand(B, L), torch.full((B, L), L, device="cuda")
    cu = s["cu"].long()
    q = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return q[None], (t - cu[q])[None], (cu[q + 1] - cu[q])[None]


def _taps(s, case):
    """x at every token and the K - 1 before it, B x L x C x K; what lies before a sequence is its state, or zero."""
    x, K, L = s["x"].float(), case["K"], case["L"]
    seq, place, _ = _places(s, case)
    back = K - 1 - torch.arange(K, device="cuda")
    at = torch.arange(L, device="cuda")[:, None] - back                       # L x K
    taken = x[:, at.clamp(min=0)]                                             # B x L x K x C
    inside = (place[..., None] >= back)[..., None]
    if s["state0"] is None:
        before = torch.zeros((), device="cuda")
    else:
        before = s["state0"].float()[seq[..., None], (K - 1 + place[..., None] - back).clamp(0, K - 2)]
    return torch.where(inside, taken, before).transpose(2, 3)


def _last_inputs(s, case):
    """The last K - 1 inputs of every sequence, S x (K - 1) x C."""
    x, K, L = s["x"], case["K"], case["L"]
    if s["cu"] is None:
        first = torch.arange(case["B"], device="cuda") * L
        n = torch.full_like(first, L)
    else:
        first = s["cu"][:-1].long()
        n = s["cu"][1:].long() - first
    place = n[:, None] + torch.arange(-(K - 1), 0, device="cuda")             # S x (K - 1)
    flat = x.reshape(-1, case["C"])
    taken = flat[(first[:, None] + place.clamp(min=0)).clamp(max=flat.shape[0] - 1)]
    before = s["state0"][torch.arange(len(first), device="cuda")[:, None], (K - 1 + place).clamp(0, K - 2)]
    return torch.where((place >= 0)[..., None], taken, before)


def _conv_prompt(s, case):
    u = (_taps(s, case) * s["w"]).sum(-1) + s["bias"]
    y = _silu(u).to(s["x"].dtype)
    if not case["state"]:
        return y, None
    s["state"].copy_(_last_inputs(s, case))
    return y, s["state"]


def _conv_train(s, case):
    K, dtype = case["K"], s["x"].dtype
    taps = _taps(s, case)
    u = (taps * s["w"]).sum(-1) + s["bias"]
    du = s["dy"].float() * _silu_slope(u)
    dw = (du[..., None] * taps).sum((0, 1))
    db = du.sum((0, 1))
    seq, place, n = _places(s, case)
    ahead = torch.arange(K, device="cuda")                                    # x_t meets u_{t + ahead} through w_{K-1-ahead}
    at = torch.arange(case["L"], device="cuda")[:, None] + ahead
    met = du[:, at.clamp(max=case["L"] - 1)] * (place[..., None] + ahead < n[..., None])[..., None]
    dx = (met * s["w"].flip(1).t()).sum(2)
    d0 = None
    if s["state0"] is not None:
        # state row j stands K-1-j places before the sequence; u at place p takes it through tap j-p
        c = du[..., None] * s["w"]                                            # B x L x C x K
        row = place[..., None] + torch.arange(K, device="cuda")               # the state row that tap k of this token reads
        use = row < K - 1
        d0 = torch.zeros(s["state0"].shape, device="cuda")
        b, t, k = torch.nonzero(use, as_tuple=True)
        d0.index_put_((seq[b, t], row[b, t, k]), c.transpose(2, 3)[b, t, k], accumulate=True)
        d0 = d0.to(dtype)
    y = _silu(u).to(dtype)
    return y, (dx.to(dtype), dw, db, d0)


def _conv_step(s, case):
    idx = s["idx"].long()
    seen = torch.cat([s["state"][idx], s["x"][:, None]], 1)                   # rows x K x C
    u = (seen.float() * s["w"].t()).sum(1) + s["bias"]
    s["state"][idx] = seen[:, 1:]
    return _silu(u).to(s["x"].dtype), s["state"]


def _wide(v, case):
    """B or C of each channel: ... x G x N -> ... x C x N."""
    return v.float().unsqueeze(-2).expand(*v.shape[:-1], case["C"] // case["G"], case["N"]).flatten(-3, -2)


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0, by doubling: after each round a pair covers twice as many tokens."""
    reach, L = 1, a.shape[1]
    while reach < L:
        b = torch.cat([b[:, :reach], torch.addcmul(b[:, reach:], a[:, reach:], b[:, :-reach])], 1)
        if 2 * reach < L:
            a = torch.cat([a[:, :reach], a[:, reach:] * a[:, :-reach]], 1)
        reach *= 2
    return b


def _scan_states(s, case):
    d = _softplus(s["dt"].float() + s["dt_bias"])
    a = torch.exp(d[..., None] * s["A"])
    x = s["x"].float()
    b = (d * x)[..., None] * _wide(s["Bm"], case)
    seq, place, _ = _places(s, case)
    new = (place == 0)[..., None, None]
    if s["h0"] is not None:
        b = torch.where(new, b + a * s["h0"][seq[:, :1]] if s["cu"] is None else b + a * s["h0"][seq[0]][None], b)
    carried = torch.where(new, torch.zeros((), device="cuda"), a)
    return d, x, a, _scan(carried, b), place, seq


def _scan_prompt(s, case):
    d, x, a, h, _, _ = _scan_states(s, case)
    y = (h * _wide(s["Cm"], case)).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    y = y.to(s["x"].dtype)
    if not case["state"]:
        return y, None
    if s["cu"] is None:
        s["h"].copy_(h[:, -1])
    else:
        last = s["cu"][1:].long() - 1
        s["h"].copy_(torch.where((s["cu"][1:] > s["cu"][:-1])[:, None, None], h[0, last.clamp(min=0)], s["h0"]))
    return y, s["h"]


def _scan_train(s, case):
    dtype, G, C = s["x"].dtype, case["G"], case["C"]
    d, x, a, h, place, seq = _scan_states(s, case)
    Bw, Cw = _wide(s["Bm"], case), _wide(s["Cm"], case)
    y0 = (h * Cw).sum(-1) + s["D"] * x
    dy = s["dy"].float()
    out, dz = y0, None
    if s["z"] is not None:
        z = s["z"].float()
        out, dz = y0 * _silu(z), (dy * y0 * _silu_slope(z)).to(dtype)
        dy = dy * _silu(z)
    new = (place == 0)[..., None, None]
    # the state before each token
    prior = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    start = torch.zeros((), device="cuda") if s["h0"] is None else (s["h0"][:, None] if s["cu"] is None else s["h0"][seq[0]][None])
    prior = torch.where(new, start, prior)
    # g_t = C_t dy_t + a_{t+1} g_{t+1}, the same scan run backwards
    passed = torch.cat([torch.where(new, torch.zeros((), device="cuda"), a)[:, 1:], torch.zeros_like(a[:, :1])], 1)
    grad = _scan(passed.flip(1), (dy[..., None] * Cw).flip(1)).flip(1)
    dCm = (dy[..., None] * h).unflatten(2, (G, C // G)).sum(3)
    dBm = (grad * (d * x)[..., None]).unflatten(2, (G, C // G)).sum(3)
    through = (grad * Bw).sum(-1)                                             # gradient of d x
    da = grad * prior * a
    dA = (da * d[..., None]).sum((0, 1))
    dd = (da * s["A"]).sum(-1) + through * x
    v = s["dt"].float() + s["dt_bias"]
    ddt = dd / (1.0 + torch.exp(-v))
    dx = through * d + dy * s["D"]
    dh0 = None
    if s["h0"] is not None:
        first = a * grad
        if s["cu"] is None:
            dh0 = first[:, 0]
        else:
            at = s["cu"][:-1].long().clamp(max=case["L"] - 1)
            dh0 = torch.where((s["cu"][1:] > s["cu"][:-1])[:, None, None], first[0, at], torch.zeros((), device="cuda"))
    return out.to(dtype), (dx.to(dtype), ddt.to(dtype), dA, dBm.to(dtype), dCm.to(dtype), (dy * x).sum((0, 1)), dz, ddt.sum((0, 1)), dh0)


def _scan_step(s, case):
    idx = s["idx"].long()
    d = _softplus(s["dt"].float() + s["dt_bias"])
    x = s["x"].float()
    h = torch.exp(d[..., None] * s["A"]) * s["h"][idx] + (d * x)[..., None] * _wide(s["Bm"], case)
    y = (h * _wide(s["Cm"], case)).sum(-1) + s["D"] * x
    s["h"][idx] = h
    return (y * _silu(s["z"].float())).to(s["x"].dtype), s["h"]


EPS = 1e-5


def _unit(v, center):
    """The normalised rows and one over their spread."""
    if center:
        v = v - v.mean(-1, keepdim=True)
    k = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    return v * k, k


def _unit_back(g, unit, k, center):
    g = g - unit * (g * unit).mean(-1, keepdim=True)
    if center:
        g = g - g.mean(-1, keepdim=True)
    return g * k


def _norm_forward(s, case):
    v = s["y"].float()
    if s["gate"] is not None:
        v = v * _silu(s["gate"].float())
    if s["w_post"] is not None:
        v = _unit(v, case["center"])[0] * s["w_post"]
        v = v if s["b_post"] is None else v + s["b_post"]
    r = s["r"].float() + s["scale"] * v
    o = _unit(r, case["center"])[0] * s["w_pre"]
    o = o if s["b_pre"] is None else o + s["b_pre"]
    return r.to(s["r"].dtype), o.to(s["y"].dtype)


def _norm_backward(s, case):
    c = case["center"]
    do = s["do"].float()
    unit, k = _unit(s["r"].float(), c)
    dr = s["dr"].float() + _unit_back(do * s["w_pre"], unit, k, c)
    dw_pre, db_pre = (do * unit).sum(0), do.sum(0)
    y = s["y"].float()
    m = y if s["gate"] is None else y * _silu(s["gate"].float())
    v, dv, dw_post, db_post = m, dr * s["scale"], None, None
    if s["w_post"] is not None:
        unit, k = _unit(m, c)
        v = unit * s["w_post"]
        v = v if s["b_post"] is None else v + s["b_post"]
        dw_post, db_post = (dv * unit).sum(0), dv.sum(0)
        dv = _unit_back(dv * s["w_post"], unit, k, c)
    dscale = (dr * v).sum(0)
    dgate = None
    if s["gate"] is not None:
        z = s["gate"].float()
        dgate = (dv * y * _silu_slope(z)).to(s["y"].dtype)
        dv = dv * _silu(z)
    return (dv.to(s["y"].dtype), dr.to(s["r"].dtype), dgate, dw_post, db_post if s["b_post"] is not None else None, dscale, dw_pre,
            db_pre if s["b_pre"] is not None else None)


# ------------------------------------------------------------------------------------------ work
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    C = case["C"]
    if case["op"] == "norm":
        n, r = case["rows"] * C, 4 if case["res"] == "f32" else 2
        gate = 1 if case["gate"] else 0
        if case["pass_"] == "forward":
            return dict(bytes=n * (2 * e + gate * e + 2 * r), flops=n * 14)
        return dict(bytes=n * (3 * e + 2 * gate * e + 3 * r), flops=n * 40)
    if case["op"] == "conv":
        K = case["K"]
        if case["pass_"] == "step":
            n = case["rows"] * C
            return dict(bytes=n * e * (2 + 2 * (K - 1)) + C * (K + 1) * 4, flops=n * (2 * K + 4))
        n = case["B"] * case["L"] * C
        if case["pass_"] == "prompt":
            return dict(bytes=2 * n * e, flops=n * (2 * K + 4))
        return dict(bytes=4 * n * e, flops=n * (6 * K + 10))                  # x, dy read; y, dx written
    N, G = case["N"], case["G"]
    z = 1 if case.get("gate", True) else 0
    if case["pass_"] == "step":
        n = case["rows"] * C
        return dict(bytes=n * (8 * N + e * (3 + z)) + C * (N + 2) * 4 + case["rows"] * 2 * G * N * e, flops=n * (7 * N + 20))
    n, bc = case["B"] * case["L"] * C, case["B"] * case["L"] * 2 * G * N
    if case["pass_"] == "prompt":
        return dict(bytes=(n * (3 + z) + bc) * e, flops=n * (7 * N + 20))
    return dict(bytes=(n * (3 + z) + bc + n * (3 + 2 * z) + bc) * e, flops=n * (27 * N + 60))


# ----------------------------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions in 64 bits: a loop over tokens or taps, gradients by differentiating it."""
    s = prepare(case, seed)
    t = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    return dict(norm=_exact_norm, conv=_exact_conv, scan=_exact_scan)[case["op"]](t, case)


def _leaf(t, *names):
    for n in names:
        if t.get(n) is not None:
            t[n] = t[n].clone().requires_grad_(True)
    return [t[n] for n in names if t.get(n) is not None]


def _grads(of, t, names):
    there = [n for n in names if t.get(n) is not None]
    got = dict(zip(there, torch.autograd.grad(of, [t[n] for n in there])))
    return tuple(got.get(n) for n in names)


def _exact_norm(t, case):
    def norm(v, w, b):
        if w is None:
            return v
        if case["center"]:
            v = v - v.sum(-1, keepdim=True) / v.shape[-1]
        v = v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS) * w
        return v if b is None else v + b

    def added(t):
        v = t["y"] if t["gate"] is None else t["y"] * t["gate"] * torch.sigmoid(t["gate"])
        return t["scale"] * norm(v, t["w_post"], t["b_post"])

    if case["pass_"] == "forward":
        r = t["r"] + added(t)
        return r, norm(r, t["w_pre"], t["b_pre"])
    # the stream behind the block is given; what was before it does not matter to any gradient
    _leaf(t, "y", "gate", "w_post", "b_post", "scale", "w_pre", "b_pre", "r")
    o = (norm(t["r"], t["w_pre"], t["b_pre"]) * t["do"]).sum()
    dr, dw_pre, db_pre = _grads(o, t, ("r", "w_pre", "b_pre"))
    dr = dr + t["dr"]
    dy, dgate, dw_post, db_post, dscale = _grads((added(t) * dr).sum(), t, ("y", "gate", "w_post", "b_post", "scale"))
    return dy, dr, dgate, dw_post, db_post, dscale, dw_pre, db_pre


def _bounds(t, case):
    """(row, first token, behind the last token) of every sequence."""
    if t["cu"] is None:
        return [(b, 0, case["L"]) for b in range(case["B"])]
    cu = t["cu"].tolist()
    return [(0, a, b) for a, b in zip(cu, cu[1:])]


def _exact_conv(t, case):
    K = case["K"]
    if case["pass_"] == "step":
        i = t["idx"].long()
        u = t["bias"] + t["w"][:, K - 1] * t["x"]
        for k in range(K - 1):
            u = u + t["w"][:, k] * t["state"][i, k]
        state = t["state"].clone()
        for k in range(K - 1):
            state[i, k] = t["x"] if k == K - 2 else t["state"][i, k + 1]
        return u * torch.sigmoid(u), state
    train = case["pass_"] == "train"
    if train:
        _leaf(t, "x", "w", "bias", "state0")
    y, last = torch.zeros_like(t["x"]).detach(), []
    rows = [[] for _ in range(case["B"])]
    for q, (b, first, end) in enumerate(_bounds(t, case)):
        before = torch.zeros(K - 1, case["C"], dtype=torch.float64, device="cuda") if t["state0"] is None else t["state0"][q]
        line = torch.cat([before, t["x"][b, first:end]], 0)
        u = t["bias"].expand(end - first, -1)
        for k in range(K):
            u = u + t["w"][:, k] * line[k:k + end - first]
        rows[b].append(u * torch.sigmoid(u))
        last.append(line[end - first:])
    y = torch.stack([torch.cat(r, 0) for r in rows])
    if train:
        return y.detach(), _grads((y * t["dy"]).sum(), t, ("x", "w", "bias", "state0"))
    return y, torch.stack(last) if case["state"] else None


def _exact_scan(t, case):
    G, C, N = case["G"], case["C"], case["N"]
    group = torch.arange(C, device="cuda") // (C // G)

    def token(h, x, dt, B, Cm, z):
        d = torch.where(dt + t["dt_bias"] > 30, dt + t["dt_bias"], torch.log1p(torch.exp((dt + t["dt_bias"]).clamp(max=30))))
        h = torch.exp(d[..., None] * t["A"]) * h + d[..., None] * B[..., group, :] * x[..., None]
        y = torch.einsum("...cn,...cn->...c", h, Cm[..., group, :]) + t["D"] * x
        return h, y if z is None else y * z * torch.sigmoid(z)

    if case["pass_"] == "step":
        i = t["idx"].long()
        h, y = token(t["h"][i], t["x"], t["dt"], t["Bm"], t["Cm"], t["z"])
        state = t["h"].clone()
        state[i] = h
        return y, state
    train = case["pass_"] == "train"
    if case["L"] > 20000 or train and case["B"] * case["L"] * C * N > 3 << 27:
        return None
    if train:
        _leaf(t, "x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0")
    starts = {(0, a): q for q, (_, a, b) in enumerate(_bounds(t, case)) if b > a} if t["cu"] is not None else {}
    S = case["seqs"] or case["B"]
    none = torch.zeros(S, C, N, dtype=torch.float64, device="cuda")
    h0 = none if t["h0"] is None else t["h0"]
    final = list(h0.unbind(0)) if t["cu"] is not None else None
    h, ys, q = h0 if t["cu"] is None else None, [], None
    x, dt, Bm, Cm = t["x"].unbind(1), t["dt"].unbind(1), t["Bm"].unbind(1), t["Cm"].unbind(1)
    z = [None] * case["L"] if t["z"] is None else t["z"].unbind(1)
    for k in range(case["L"]):
        if (0, k) in starts:
            if q is not None:
                final[q] = h[0]
            q = starts[0, k]
            h = h0[q][None]
        h, y = token(h, x[k], dt[k], Bm[k], Cm[k], z[k])
        ys.append(y)
    if q is not None:
        final[q] = h[0]
    y = torch.stack(ys, 1)
    if train:
        return y.detach(), _grads((y * t["dy"]).sum(), t, ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0"))
    if not case["state"]:
        return y, None
    return y, h if t["cu"] is None else torch.stack(final)
