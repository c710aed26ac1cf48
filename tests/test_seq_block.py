"""The token-sequence operators together, as a block of a model runs them: norm, convolution, scan, norm;
a training pass, a prompt with tokens after it, captured graphs, several streams.

Every operator's results are checked against its 64-bit form on the inputs that the run gave it, with
the bounds that its own tests use, so that no bound has to cover what other operators round.
"""
import pytest
import torch

import _seq_ref as R
import linear_spatial_propagation_gspn_b200 as g

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
K, N, G = 4, 16, 2


class Block:
    """y, r (B, L, C) -> the next stream and the next block's input. The projections are products with one
    vector each: they make the branches' gradients meet, and are not the operators' own."""

    def __init__(self, C, dtype, seed=0):
        r = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=r).cuda()  # noqa: E731
        self.C, self.dtype = C, dtype
        self.p = dict(w_post=1 + 0.3 * n(C), b_post=n(C), scale=1 + 0.3 * n(C), w_pre=1 + 0.3 * n(C), b_pre=n(C), w_next=1 + 0.3 * n(C),
                      conv_w=0.5 * n(C, K), conv_b=0.1 * n(C), A=-(0.2 + n(C, N).abs()), D=n(C), dt_bias=n(C) - 3,
                      px=1 + 0.1 * n(C), pz=1 + 0.1 * n(C), pdt=0.1 * n(C))

    def __call__(self, y, r, p=None, cu=None, keep=lambda name, v: v):
        p, C = p or self.p, self.C
        r1, o = g.block_norm(y, r, w_post=p["w_post"], b_post=p["b_post"], scale=p["scale"], w_pre=p["w_pre"], b_pre=p["b_pre"],
                             center=True)
        r1, o = keep("r1", r1), keep("o", o)
        x = keep("x", (o * p["px"]).to(self.dtype))
        z = keep("z", (o * p["pz"]).to(self.dtype))
        dt = keep("dt", (o * p["pdt"]).to(self.dtype))
        bc = keep("bc", o[..., :2 * G * N])                      # side by side in the norm's rows
        Bm, Cm = bc[..., :G * N].unflatten(-1, (G, N)), bc[..., G * N:].unflatten(-1, (G, N))
        u = keep("u", g.causal_conv(x, p["conv_w"], p["conv_b"], cu=cu))
        v = keep("v", g.selective_scan(u, dt, p["A"], Bm, Cm, p["D"], z, p["dt_bias"], cu=cu))
        r2, o2 = g.block_norm(v, r1, scale=p["scale"], w_pre=p["w_next"])
        return keep("r2", r2), keep("o2", o2)


def bands(t):
    return t["bc"][..., :G * N].unflatten(-1, (G, N)), t["bc"][..., G * N:].unflatten(-1, (G, N))


def rms(v):
    return v.pow(2).mean(-1, keepdim=True).sqrt()


def check_unit(got, v, w, b, center, what):
    """got = norm(v) w + b. As for the operator alone: 96 u of a normalised row's size times its weight; taking
    the mean off leaves errors of the size of the row's values, however little is left of them."""
    v = R.f64(v)
    c = v - v.mean(-1, keepdim=True) if center else v
    ref = R.norm(v, None, None, w, b, None, None, None, 1e-5, center)["r_out"]
    size = (1 + v.abs() / rms(v)) * rms(v) / rms(c) * (1 + rms(v) / rms(c)) * R.f64(w).abs()
    R.check(got, ref, size + (0 if b is None else R.f64(b).abs()) + ref.abs(), 96, what)


def check_norms(p, y, r, t):
    v = R.f64(y)
    c = v - v.mean(-1, keepdim=True)
    ref = R.norm(y, r, None, p["w_post"], p["b_post"], p["scale"], None, None, 1e-5, True)["r_out"]
    size = (1 + v.abs() / rms(v)) * rms(v) / rms(c) * (1 + rms(v) / rms(c)) * R.f64(p["w_post"]).abs() + R.f64(p["b_post"]).abs()
    R.check(t["r1"], ref, size * R.f64(p["scale"]).abs() + ref.abs(), 96, "r1")
    check_unit(t["o"], t["r1"], p["w_pre"], p["b_pre"], True, "o")
    ref = R.norm(t["v"], t["r1"], None, None, None, p["scale"], None, None, 1e-5, False)["r_out"]
    R.check(t["r2"], ref, R.f64(t["v"]).abs() * R.f64(p["scale"]).abs() + ref.abs(), 4, "r2")
    check_unit(t["o2"], t["r2"], p["w_next"], None, False, "o2")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,C,cu", [(2, 37, 72, None), (1, 90, 66, [0, 1, 1, 40, 83]), (3, 1, 64, None)])
def test_training_pass(B, L, C, cu, dtype):
    block = Block(C, DT[dtype])
    gen = torch.Generator().manual_seed(1)
    n = lambda: torch.randn(B, L, C, generator=gen).cuda()  # noqa: E731
    y, r, dr, do = n().to(DT[dtype]), n(), n(), n().to(DT[dtype])
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    p = {k: v.clone().requires_grad_(True) for k, v in block.p.items()}
    y.requires_grad_(True), r.requires_grad_(True)
    t = {}

    def keep(name, v):
        v.retain_grad()
        t[name] = v
        return v

    r2, o2 = block(y, r, p, c, keep)
    torch.autograd.backward([r2, o2], [dr, do])
    gr = {k: v.grad for k, v in t.items()}
    check_norms(p, y, r, t)
    conv = R.conv(t["x"], p["conv_w"], p["conv_b"], True, cu, None, gr["u"])
    end = L if cu is None else cu[-1]
    # as in the convolution's own tests: 48 u a product, one more for every token of a sum
    R.check(t["u"][:, :end], conv["y"][:, :end], conv["y_m"][:, :end], 48, "u")
    R.check(gr["x"][:, :end], conv["dx"][:, :end], conv["dx_m"][:, :end], 48, "dx")
    R.check(p["conv_w"].grad, conv["dw"], conv["dw_m"], 48 + B * L, "conv dw")
    R.check(p["conv_b"].grad, conv["db"], conv["db_m"], 48 + B * L, "conv db")
    Bm, Cm = bands(t)
    scan = R.scan(t["u"], t["dt"], p["A"], Bm, Cm, p["D"], t["z"], p["dt_bias"], True, cu, None, gr["v"])
    f = R.scan_factor(L if cu is None else max(b - a for a, b in zip(cu, cu[1:])), N, C // G)
    R.check(t["v"], scan["y"], scan["y_m"], f, "v")
    for name, got in (("dx", gr["u"]), ("ddt", gr["dt"]), ("dz", gr["z"])):
        R.check(got, scan[name], scan[name + "_m"], f, name)
    both = torch.cat([scan["dB"].flatten(2), scan["dC"].flatten(2)], -1)
    R.check(gr["bc"], both, torch.cat([scan["dB_m"].flatten(2), scan["dC_m"].flatten(2)], -1), f, "dB, dC")
    for name, got in (("dA", p["A"]), ("dD", p["D"]), ("dbias", p["dt_bias"])):
        R.check(got.grad, scan[name], scan[name + "_m"], f + B * L, name)
    # the branches meet: o's gradient is the projections' sum, each term and each sum rounded to its type
    parts = [R.f64(gr[k]) * R.f64(p[q]) for k, q in (("x", "px"), ("z", "pz"), ("dt", "pdt"))]
    parts.append(torch.nn.functional.pad(R.f64(gr["bc"]), (0, C - 2 * G * N)))
    mag = sum(v.abs() for v in parts)
    R.check(gr["o"], sum(parts), mag * 8 * R.half_step(DT[dtype]) / R.U, 1, "do")
    # the first norm's gradients: 96 u for each norm that they go through, of the row's largest gradient times
    # how far values reach over what the mean leaves of them
    nrm = R.norm(y, None, None, p["w_post"], p["b_post"], p["scale"], p["w_pre"], p["b_pre"], 1e-5, True, t["r1"], gr["r1"], gr["o"])
    reach = 1.0
    for q in (R.f64(y), R.f64(t["r1"])):
        reach *= 1 + (q.abs().max(-1, keepdim=True).values / rms(q - q.mean(-1, keepdim=True))).max().item()
    for name, got in (("dr_in", r), ("dy", y)):
        R.check(got.grad, nrm[name], nrm[name].abs() + nrm[name].abs().max(-1, keepdim=True).values, 8 * 96 * reach, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_then_tokens(dtype):
    """Packed prompts (one without tokens), states into slots, then tokens of some of the rows: each sequence's
    outputs are those of the whole sequence."""
    C, cu, steps = 72, [0, 13, 13, 40], 5
    block, S = Block(C, DT[dtype], seed=2), 3
    p = block.p
    gen = torch.Generator().manual_seed(3)
    L = cu[-1]
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    conv_pool = torch.zeros(5, K - 1, C, dtype=DT[dtype], device="cuda")
    scan_pool = torch.zeros(5, C, N, device="cuda")
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    seen = [dict(x=[], u=[], dt=[], Bm=[], Cm=[], z=[], v=[]) for _ in range(S)]

    def project(y, r):
        r1, o = g.norm_forward(y, r, w_post=p["w_post"], b_post=p["b_post"], scale=p["scale"], w_pre=p["w_pre"], b_pre=p["b_pre"],
                               center=True)
        bc = o[..., :2 * G * N]
        return r1, dict(x=(o * p["px"]).to(o.dtype), z=(o * p["pz"]).to(o.dtype), dt=(o * p["pdt"]).to(o.dtype),
                        Bm=bc[..., :G * N].unflatten(-1, (G, N)), Cm=bc[..., G * N:].unflatten(-1, (G, N)))

    y, r = torch.randn(1, L, C, generator=gen).cuda().to(DT[dtype]), torch.randn(1, L, C, generator=gen).cuda()
    r1, t = project(y, r)
    state, h = torch.empty(S, K - 1, C, dtype=DT[dtype], device="cuda"), torch.empty(S, C, N, device="cuda")
    t["u"] = g.conv_forward(t["x"], p["conv_w"], p["conv_b"], cu=c, state=state)
    t["v"] = g.ssm_forward(t["u"], t["dt"], p["A"], t["Bm"], t["Cm"], D=p["D"], z=t["z"], dt_bias=p["dt_bias"], cu=c, h=h)
    conv_pool[slots.long()], scan_pool[slots.long()] = state, h
    for q in range(S):
        for k, v in seen[q].items():
            v.append(t[k][0, cu[q]:cu[q + 1]])
    for i in range(steps):
        rows = [0, 1, 2] if i % 2 else [2, 1]
        idx = slots[rows].contiguous()
        y, r = torch.randn(len(rows), C, generator=gen).cuda().to(DT[dtype]), torch.randn(len(rows), C, generator=gen).cuda()
        r1, t = project(y, r)
        t["u"] = g.conv_step(t["x"], p["conv_w"], p["conv_b"], conv_pool, idx=idx)
        t["v"] = g.ssm_step(t["u"], t["dt"], p["A"], t["Bm"], t["Cm"], scan_pool, D=p["D"], z=t["z"], dt_bias=p["dt_bias"], idx=idx)
        for j, q in enumerate(rows):
            for k, v in seen[q].items():
                v.append(t[k][j:j + 1])
    for q in range(S):
        s = {k: torch.cat(v)[None] for k, v in seen[q].items()}
        conv = R.conv(s["x"], p["conv_w"], p["conv_b"], True, None, None)
        R.check(s["u"], conv["y"], conv["y_m"], 48, f"u of {q}")
        assert torch.equal(R.f64(conv_pool[slots[q].item()]), conv["state"][0])
        ref = R.scan(s["u"], s["dt"], p["A"], s["Bm"], s["Cm"], p["D"], s["z"], p["dt_bias"], True, None, None)
        f = R.scan_factor(s["u"].shape[1], N, C // G)
        R.check(s["v"], ref["y"], ref["y_m"], f, f"v of {q}")
        R.check(scan_pool[slots[q].item()], ref["h"][0], ref["h_m"][0], f, f"h of {q}")
    assert not scan_pool[[1, 3]].any() and not conv_pool[[1, 3]].any()


def raw(t, p, cu=None):
    """Forward, backward and a token of all three operators by the calls without autograd."""
    r1, o = g.norm_forward(t["y"], t["r"], gate=t["gate"], w_post=p["w_post"], scale=p["scale"], w_pre=p["w_pre"])
    u = g.conv_forward(o, p["conv_w"], p["conv_b"], cu=cu)
    bc = o[..., :2 * G * N]
    Bm, Cm = bc[..., :G * N].unflatten(-1, (G, N)), bc[..., G * N:].unflatten(-1, (G, N))
    kw = dict(D=p["D"], z=t["gate"], dt_bias=p["dt_bias"], cu=cu)
    v, save = g.ssm_forward_save(u, o, p["A"], Bm, Cm, **kw)
    v2 = g.ssm_forward(u, o, p["A"], Bm, Cm, **kw)
    grads = list(g.ssm_backward(u, o, p["A"], Bm, Cm, v, save, **kw))
    grads += g.conv_backward(o, p["conv_w"], p["conv_b"], grads[0], cu=cu)
    grads += g.norm_backward(t["y"], r1, gate=t["gate"], w_post=p["w_post"], scale=p["scale"], w_pre=p["w_pre"], dr=t["r"], do=grads[-4])
    s = g.conv_step(o[:, -1], p["conv_w"], p["conv_b"], t["conv"])
    s = g.ssm_step(s, o[:, -1], p["A"], Bm[:, -1], Cm[:, -1], t["h"], D=p["D"], z=t["gate"][:, -1], dt_bias=p["dt_bias"])
    return [x for x in [r1, o, u, v, v2, s, *grads] if x is not None]


def fresh(B, L, C, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(y=n(B, L, C).to(dtype).cuda(), gate=n(B, L, C).to(dtype).cuda(), r=n(B, L, C).cuda(), conv=n(B, K - 1, C).to(dtype).cuda(),
                h=n(B, C, N).cuda())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_and_replayed(dtype):
    """Two graphs of everything, replayed on new inputs, one after the other and beside each other: the same
    bits as the calls themselves (no sum's order depends on the run)."""
    B, L, C = 2, 300, 72                                          # long enough for pieces
    p = Block(C, DT[dtype]).p
    graphs = []
    for seed in (0, 1):
        t = fresh(B, L, C, DT[dtype], seed)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            raw(t, p)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = raw(t, p)
        graphs.append((graph, t, out))
    for turn in range(2):
        want = []
        for i, (_, t, _) in enumerate(graphs):
            new = fresh(B, L, C, DT[dtype], 10 + 2 * turn + i)
            for k, v in t.items():
                v.copy_(new[k])
            want.append((raw(new, p), new))
        torch.cuda.synchronize()
        if turn:
            for graph, _, _ in graphs:
                with torch.cuda.stream(torch.cuda.Stream()):
                    graph.replay()
        else:
            for graph, _, _ in graphs:
                graph.replay()
        torch.cuda.synchronize()
        for (_, t, out), (ref, after) in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, ref))
            assert torch.equal(t["h"], after["h"]) and torch.equal(t["conv"], after["conv"])


def test_captured_training_pass():
    """The differentiable forms inside a graph: leaves of the capture's own."""
    B, L, C = 2, 40, 64
    block = Block(C, torch.float32)
    data = [torch.randn(B, L, C, device="cuda") for _ in range(2)]

    def run():
        p = {k: v.detach().requires_grad_(True) for k, v in block.p.items()}
        y, r = (v.detach().requires_grad_(True) for v in data)
        r2, o2 = block(y, r, p)
        return torch.autograd.grad([r2, o2], [y, r, *p.values()], [data[0], data[1]])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for v in data:
        v.normal_()
    graph.replay()
    got = [v.clone() for v in out]
    assert all(torch.equal(a, b) for a, b in zip(got, run()))


@pytest.mark.parametrize("named", [True, False])
def test_two_streams_at_once(named):
    """Calls that run beside each other, on a stream named in the call or on the current one, after inputs that
    the stream itself still has to make."""
    B, L, C = 1, 700, 72
    p = Block(C, torch.bfloat16).p
    ts = [fresh(B, L, C, torch.bfloat16, 20 + i) for i in range(2)]
    want = [raw({k: v.clone() for k, v in t.items()}, p) for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got.clear()
        for t, s in zip(ts, streams):
            with torch.cuda.stream(s):
                mine = {k: v.clone() for k, v in t.items()}
            if not named:
                with torch.cuda.stream(s):
                    got.append(raw(mine, p))
                continue
            r1, o = g.norm_forward(mine["y"], mine["r"], gate=mine["gate"], w_post=p["w_post"], scale=p["scale"], w_pre=p["w_pre"], stream=s)
            u = g.conv_forward(o, p["conv_w"], p["conv_b"], stream=s)
            got.append([r1, o, u])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(TypeError):
        g.conv_forward(ts[0]["y"].cpu().numpy(), p["conv_w"])
