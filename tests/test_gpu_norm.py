"""GPU parity of the row norm, its gradients and the delta-rule layer with the
float64 oracle, through the C ABI.

Tolerances, |got - ref| <= r |ref| + s max|ref|: r half a step of the type
(bf16 2^-8, float32 2^-24).  s: a row's sum of D squares is off by sqrt(D)
2^-24 at random, 8 times that for the largest row; the products and the
sigmoid of an element add about 16 roundings, and its exponential is good to
2^-21: s = (8 sqrt(D) + 16 + 8) 2^-24, and sqrt(rows) in the place of sqrt(D)
for dw, which is a sum over the rows."""
import numpy as np
import pytest
import torch

import learned_linear_attention_b200 as T
from oracle import delta_recurrent, row_norm, row_norm_backward
from test_gpu_delta import HALF, TYPES, Problem, leave_an_error, near, tol

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(rows, D, dt, w, gate, res, seed=0):
    r = np.random.default_rng([rows, D, seed])
    on = lambda x: torch.from_numpy(x).to(TYPES[dt]).cuda()  # noqa: E731
    return dict(x=on(r.standard_normal((rows, D))), w=torch.from_numpy(1 + 0.1 * r.standard_normal(D)).float().cuda() if w else None,
                z=on(2 * r.standard_normal((rows, D))) if gate != "none" else None,
                res=on(r.standard_normal((rows, D))) if res else None, dout=on(r.standard_normal((rows, D))))


def host(t):
    return None if t is None else t.double().cpu().numpy()


def check(p, rows, D, dt, kind, gate, eps=1e-6, scale=0.7):
    d = T.make_norm_desc(rows, D, kind=kind, gate=gate, eps=eps, scale=scale, dtype=dt)
    eps, scale = d.eps, d.scale      # as float32 holds them
    out = torch.full_like(p["x"], float("nan"))
    T.ttt_norm_fwd(d, p["x"], p["w"], p["z"], p["res"], out)
    kw = dict(kind=kind, gate=gate, eps=eps, scale=scale)
    s = (8 * np.sqrt(D) + 24) * U
    near(out, row_norm(host(p["x"]), host(p["w"]), host(p["z"]), host(p["res"]), **kw), HALF[dt], s, "out")
    nan = lambda t: None if t is None else torch.full_like(t, float("nan"))  # noqa: E731
    dx, dw, dz = nan(p["x"]), nan(p["w"]), nan(p["z"])
    ws = T.alloc_workspace(T.ttt_norm_bwd_workspace_bytes(d))
    T.ttt_norm_bwd(d, p["x"], p["w"], p["z"], p["dout"], dx, dw, dz, ws)
    ref = row_norm_backward(host(p["x"]), host(p["dout"]), host(p["w"]), host(p["z"]), **kw)
    for name, a, b, m in (("dx", dx, ref[0], D), ("dw", dw, ref[1], rows), ("dz", dz, ref[2], D)):
        if b is None:
            assert a is None
        else:
            near(a, b, HALF["f32" if name == "dw" else dt], (8 * np.sqrt(m) + 32) * U, name)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", [(1, 8), (7, 16), (515, 40), (33, 64), (1000, 128), (3, 264), (65, 1024), (5, 1032), (4, 8192)])
@pytest.mark.parametrize("kind,gate,w,res", [("rms", "silu", True, True), ("l2", "none", False, False), ("rms", "none", True, False),
                                             ("l2", "sigmoid", True, True)])
def test_against_oracle(cuda_device, rows, D, dt, kind, gate, w, res):
    check(make(rows, D, dt, w, gate, res), rows, D, dt, kind, gate)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [248, 256, 264, 504, 512, 520, 1016, 1032, 2056, 4104])
def test_widths_around_the_borders_of_a_rows_threads(cuda_device, D, dt):
    check(make(301, D, dt, True, "silu", True), 301, D, dt, "rms", "silu")


def test_many_rows(cuda_device):
    check(make(20011, 128, "bf16", True, "silu", True), 20011, 128, "bf16", "rms", "silu")


@pytest.mark.parametrize("kind", ["rms", "l2"])
def test_zero_and_tiny_rows(cuda_device, kind):
    """Rows of zeros and rows shorter than eps: finite, and the L2 factor 1/eps is a constant there."""
    p = make(6, 16, "f32", True, "none", False)
    p["x"][1] = 0
    p["x"][4] *= 1e-5
    check(p, 6, 16, "f32", kind, "none", eps=1e-2)


def test_large_gates_saturate(cuda_device):
    p = make(4, 16, "f32", False, "silu", False)
    p["z"][0] = 200.0
    p["z"][1] = -200.0
    d = T.make_norm_desc(4, 16, gate="silu", dtype="f32")
    out = torch.empty_like(p["x"])
    T.ttt_norm_fwd(d, p["x"], None, p["z"], None, out)
    assert bool(torch.isfinite(out).all()) and bool((out[1] == 0).all())


@pytest.mark.parametrize("onto", ["x", "z", "res"])
def test_in_place(cuda_device, onto):
    p = make(300, 128, "bf16", True, "silu", True)
    d = T.make_norm_desc(300, 128, gate="silu")
    want = torch.empty_like(p["x"])
    T.ttt_norm_fwd(d, p["x"], p["w"], p["z"], p["res"], want)
    T.ttt_norm_fwd(d, p["x"], p["w"], p["z"], p["res"], p[onto])
    assert torch.equal(p[onto], want)


def test_gradients_in_place_and_same_bits(cuda_device):
    p = make(5000, 128, "bf16", True, "silu", False)
    d = T.make_norm_desc(5000, 128, gate="silu")
    ws = T.alloc_workspace(T.ttt_norm_bwd_workspace_bytes(d))
    outs = []
    for _ in range(2):
        g = [torch.empty_like(p[n]) for n in ("x", "w", "z")]
        T.ttt_norm_bwd(d, p["x"], p["w"], p["z"], p["dout"], *g, ws)
        outs.append(g)
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    x, z = p["x"].clone(), p["z"].clone()
    dw = torch.empty_like(p["w"])
    T.ttt_norm_bwd(d, x, p["w"], z, p["dout"], x, dw, z, ws)
    assert all(torch.equal(a, b) for a, b in zip((x, dw, z), outs[0]))


def test_no_rows(cuda_device):
    d = T.make_norm_desc(0, 64, gate="none")
    dw = torch.full((64,), float("nan"), device="cuda")
    w = torch.ones(64, device="cuda")
    T.ttt_norm_bwd(d, None, w, None, None, None, dw, None, T.alloc_workspace(T.ttt_norm_bwd_workspace_bytes(d)))
    assert bool((dw == 0).all())


# ------------------------------------------------------------------ the layer
@pytest.mark.parametrize("dt,dk,dv,N", [("f32", 24, 40, 70), ("bf16", 64, 64, 200), ("bf16", 128, 128, 129)])
@pytest.mark.parametrize("full", [True, False])
def test_layer(cuda_device, dt, dk, dv, N, full):
    """Norm, delta rule, gated norm and residual as one call, and as the calls it stands for (bit for bit)."""
    p = Problem(2, 2, N, dk, dv, dt)
    x = p.dev
    x["q"] *= 3
    x["k"] *= 0.5
    w = 1 + 0.1 * torch.randn(dv, device="cuda") if full else None
    z, res = (torch.randn_like(x["v"]), torch.randn_like(x["v"])) if full else (None, None)
    d, S, out = p.desc(), p.S0.clone(), torch.full_like(x["v"], float("nan"))
    ws = T.alloc_workspace(T.ttt_delta_layer_workspace_bytes(d))
    T.ttt_delta_layer_fwd(d, 1e-5, 0.5, x["q"], x["k"], x["v"], x["g"], x["beta"], w, z, res, S, out, ws)
    assert T.ttt_check_device_status(ws) == T.TTT_OK
    # the calls one by one
    rows = 4 * N
    qn, kn, o, y = (torch.empty_like(t) for t in (x["q"], x["k"], x["v"], x["v"]))
    dn = T.make_norm_desc(rows, dk, kind="l2", dtype=dt)
    T.ttt_norm_fwd(dn, x["q"], None, None, None, qn)
    T.ttt_norm_fwd(dn, x["k"], None, None, None, kn)
    S2 = p.S0.clone()
    ws2 = T.alloc_workspace(T.ttt_delta_workspace_bytes(d))
    T.ttt_delta_fwd(d, qn, kn, x["v"], x["g"], x["beta"], S2, o, ws2)
    dy = T.make_norm_desc(rows, dv, gate="silu" if full else "none", eps=1e-5, scale=0.5, dtype=dt)
    T.ttt_norm_fwd(dy, o, w, z, res, y)
    assert torch.equal(out, y) and torch.equal(S, S2)
    # and against the oracle on the rounded unit keys
    unit = row_norm(host(x["k"]), kind="l2")
    near(kn, unit, HALF[dt], (8 * np.sqrt(dk) + 24) * U)
    ref, Sr = delta_recurrent(host(qn), host(kn), host(x["v"]), host(x["g"]), host(x["beta"]), host(p.S0))
    near(S, Sr, HALF["f32"], tol(dt, dk, dv, N))
    near(o, ref, HALF[dt], tol(dt, dk, dv, N))


def test_training_step_of_the_layer(cuda_device):
    """The gradients of norm -> delta rule -> gated norm, chained through the
    three backward calls, against differences of the oracle's chain in float64."""
    B, H, N, d = 1, 2, 40, 16
    p = Problem(B, H, N, d, d, "f32")
    x, rows = p.dev, B * H * N
    w, z = 1 + 0.1 * torch.randn(d, device="cuda"), torch.randn_like(x["v"])
    dy = torch.randn_like(x["v"])
    dn = T.make_norm_desc(rows, d, kind="l2", dtype="f32")
    do = T.make_norm_desc(rows, d, gate="silu", dtype="f32")
    kn, o = torch.empty_like(x["k"]), torch.empty_like(x["v"])
    T.ttt_norm_fwd(dn, x["k"], None, None, None, kn)
    S = p.S0.clone()
    desc = p.desc()
    T.ttt_delta_fwd(desc, x["q"], kn, x["v"], x["g"], x["beta"], S, o, T.alloc_workspace(T.ttt_delta_workspace_bytes(desc)))
    gw, gz, go = torch.empty_like(w), torch.empty_like(z), torch.empty_like(o)
    T.ttt_norm_bwd(do, o, w, z, dy, go, gw, gz, T.alloc_workspace(T.ttt_norm_bwd_workspace_bytes(do)))
    g = p.new_grads()
    T.ttt_delta_bwd(desc, x["q"], kn, x["v"], x["g"], x["beta"], p.S0, go, None, *g,
                    T.alloc_workspace(T.ttt_delta_bwd_workspace_bytes(desc)))
    gk = torch.empty_like(kn)
    T.ttt_norm_bwd(dn, x["k"], None, None, g[1], gk, None, None, T.alloc_workspace(T.ttt_norm_bwd_workspace_bytes(dn)))
    at = {n: host(t) for n, t in dict(q=x["q"], k=x["k"], v=x["v"], g=x["g"], beta=x["beta"], S0=p.S0, w=w, z=z).items()}
    up = host(dy)

    def loss(a):
        out, _ = delta_recurrent(a["q"], row_norm(a["k"], kind="l2"), a["v"], a["g"], a["beta"], a["S0"])
        return (up * row_norm(out, a["w"], a["z"], gate="silu", eps=float(do.eps))).sum()

    grads = dict(q=g[0], k=gk, v=g[2], g=g[3], beta=g[4], S0=g[5], w=gw, z=gz)
    r = np.random.default_rng(11)
    for n, got in grads.items():
        dirn = r.standard_normal(at[n].shape)
        h = 1e-5
        lo, hi = dict(at), dict(at)
        lo[n], hi[n] = at[n] - h * dirn, at[n] + h * dirn
        diff = (loss(hi) - loss(lo)) / (2 * h)
        # the sum of |d_i g_i| over n entries, each off by the float32 chain's 2e-5 at most
        assert abs(diff - (host(got) * dirn).sum()) <= 2e-5 * np.abs(host(got) * dirn).sum() + 1e-7, n


def test_an_earlier_error_is_not_this_calls(cuda_device):
    p = make(50, 64, "f32", True, "silu", False)
    d = T.make_norm_desc(50, 64, gate="silu", dtype="f32")
    ws, outs = T.alloc_workspace(T.ttt_norm_bwd_workspace_bytes(d)), []
    for error in (False, True):
        g = [torch.empty_like(p[n]) for n in ("x", "x", "w", "z")]
        if error:
            leave_an_error()
        T.ttt_norm_fwd(d, p["x"], p["w"], p["z"], None, g[0])
        if error:
            leave_an_error()
        T.ttt_norm_bwd(d, p["x"], p["w"], p["z"], p["dout"], *g[1:], ws)
        outs.append(g)
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_float32_gates_have_float32_precision(cuda_device):
    """Rows of ones gated by z in [-80, 80], each value against its own size.  The
    exponential is good to 2 ulp (2^-23 each), 1 + e rounds once, the quotient is
    good to 2 ulp, and r, the norm's and the gate's products round seven times:
    (4 + 1 + 4 + 7) 2^-24."""
    z = torch.linspace(-80, 80, 1 << 16, device="cuda").view(-1, 128)
    x, out = torch.ones_like(z), torch.empty_like(z)
    d = T.make_norm_desc(len(z), 128, gate="sigmoid", dtype="f32")
    T.ttt_norm_fwd(d, x, None, z, None, out)
    ref = row_norm(host(x), None, host(z), gate="sigmoid", eps=d.eps)
    assert (np.abs(host(out) - ref) / ref).max() <= 16 * U


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind,eps", [("rms", 1e-6), ("l2", 1e-6), ("l2", 1.1754944e-38)])
def test_rows_at_the_ends_of_the_range(cuda_device, dt, kind, eps):
    """A row whose squares' sum is infinite has r = 0; a row of zeros stays zero
    with the smallest eps.  Rows beside them are as without them."""
    p = make(5, 64, dt, True, "silu", True)
    d = T.make_norm_desc(5, 64, kind=kind, gate="silu", eps=eps, dtype=dt)
    ws = T.alloc_workspace(T.ttt_norm_bwd_workspace_bytes(d))

    def run():
        out, dx, dz, dw = torch.empty_like(p["x"]), torch.empty_like(p["x"]), torch.empty_like(p["x"]), torch.empty_like(p["w"])
        T.ttt_norm_fwd(d, p["x"], p["w"], p["z"], p["res"], out)
        T.ttt_norm_bwd(d, p["x"], p["w"], p["z"], p["dout"], dx, dw, dz, ws)
        return out, dx, dz, dw

    want = run()
    p["x"][1], p["x"][3] = 2e19, 0
    out, dx, dz, dw = run()
    for r in (1, 3):
        assert torch.equal(out[r], p["res"][r])
        assert bool((dz[r] == 0).all())
    assert bool((dx[1] == 0).all()) and bool(torch.isfinite(dw).all())
    for a, b in zip((out, dx, dz), want):
        assert torch.equal(a[[0, 2, 4]], b[[0, 2, 4]])
