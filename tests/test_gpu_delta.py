"""GPU parity of the gated delta rule (sequence, gradients, single tokens) with
the float64 oracle, through the C ABI.

Tolerances, |got - ref| <= r |ref| + s max|ref|:
  r  half a step of the output's type (bf16 2^-8, float32 2^-24);
  s  the sums.  Float32 path: a token's e and u are sums over dk products,
     each rounded to 2^-24 of the running sum, and unit keys with
     0 <= beta <= 1 make every step a contraction, so the errors of the N
     tokens add up as independent ones at most: sqrt(dk N) 2^-24, times 8 for
     the largest of many.  Tensor-core path: every derived operand is bf16 hi +
     lo, off by at most 2^-17, of which a value's chain meets five (T, W, U, S,
     and the partner's); dk or 128 products average them, and tokens add up
     over the memory of the decay, so 8 * 5 * 2^-17 bounds the largest.
"""
import ctypes

import numpy as np
import pytest
import torch

import learned_linear_attention_b200 as T
from oracle import delta_backward, delta_recurrent

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def tensor_cores(dt, dk, dv):
    return dt == "bf16" and dk == dv and dk in (64, 128)


def tol(dt, dk, dv, N):
    return 8 * 5 * 2.0 ** -17 if tensor_cores(dt, dk, dv) else 8 * np.sqrt(dk * max(N, 1)) * 2.0 ** -24


def near(got, ref, r, s, what=""):
    got = got.detach().double().cpu().numpy() if torch.is_tensor(got) else np.asarray(got)
    ref = np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, what
    assert np.isfinite(got).all(), what
    if ref.size == 0:
        return
    over = np.abs(got - ref) - (r * np.abs(ref) + s * np.abs(ref).max())
    assert over.max() <= 0, f"{what}: {np.abs(got - ref).max():.3e} of {np.abs(ref).max():.3e}, over by {over.max():.3e}"


class Problem:
    """Inputs of one call: float64 copies hold the exact values given to the device."""

    def __init__(self, B, H, N, dk, dv, dt, decay=True, start=True, seed=0, g_of=None, beta_of=None):
        r = np.random.default_rng([B, H, N, dk, dv, seed])
        self.shape, self.dt, self.decay = (B, H, N, dk, dv), dt, decay
        k = r.standard_normal((2, B, H, N, dk))
        k /= np.maximum(np.linalg.norm(k, axis=-1, keepdims=True), 1e-30)
        g = -np.log1p(np.exp(1.5 * r.standard_normal((B, H, N)) - 4)) if g_of is None else g_of(r, (B, H, N))
        beta = 1 / (1 + np.exp(-r.standard_normal((B, H, N)))) if beta_of is None else beta_of(r, (B, H, N))
        raw = dict(q=k[0], k=k[1], v=r.standard_normal((B, H, N, dv)), g=g, beta=beta,
                   dout=r.standard_normal((B, H, N, dv)))
        self.dev = {n: torch.from_numpy(np.ascontiguousarray(x)).to(TYPES[dt]).cuda() for n, x in raw.items()}
        self.S0 = torch.from_numpy(0.3 * r.standard_normal((B, H, dk, dv))).float().cuda() if start else None
        self.dS = torch.from_numpy(0.3 * r.standard_normal((B, H, dk, dv))).float().cuda() if start else None
        if not decay:
            self.dev["g"] = None

    def host(self, n):
        x = self.dev.get(n) if n in self.dev else getattr(self, n)
        return None if x is None else x.double().cpu().numpy()

    def desc(self, out=None, N=None, scale=0.0):
        B, H, n, dk, dv = self.shape
        return T.make_delta_desc(B, H, n if N is None else N, dk, dv, scale=scale, in_dtype=self.dt,
                                 out_dtype=out or self.dt)

    def fwd(self, out=None, scale=0.0, stream=None, ws=None):
        B, H, N, dk, dv = self.shape
        d = self.desc(out, scale=scale)
        S = torch.zeros(B, H, dk, dv, device="cuda") if self.S0 is None else self.S0.clone()
        o = torch.full((B, H, N, dv), float("nan"), dtype=TYPES[out or self.dt], device="cuda")
        ws = T.alloc_workspace(T.ttt_delta_workspace_bytes(d)) if ws is None else ws
        x = self.dev
        T.ttt_delta_fwd(d, x["q"], x["k"], x["v"], x["g"], x["beta"], S, o, ws, stream=stream)
        assert T.ttt_check_device_status(ws, stream) == T.TTT_OK
        return o, S

    def new_grads(self):
        B, H, N, dk, dv = self.shape
        full = lambda *s, t=TYPES[self.dt]: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
        return [full(B, H, N, dk), full(B, H, N, dk), full(B, H, N, dv), full(B, H, N) if self.decay else None,
                full(B, H, N), full(B, H, dk, dv, t=torch.float32)]

    def bwd(self, scale=0.0):
        d, x, outs = self.desc(scale=scale), self.dev, self.new_grads()
        ws = T.alloc_workspace(T.ttt_delta_bwd_workspace_bytes(d))
        T.ttt_delta_bwd(d, x["q"], x["k"], x["v"], x["g"], x["beta"], self.S0, x["dout"], self.dS, *outs, ws)
        assert T.ttt_check_device_status(ws) == T.TTT_OK
        return outs

    def check_fwd(self, got, out=None, scale=0.0):
        B, H, N, dk, dv = self.shape
        ref, S = delta_recurrent(*(self.host(n) for n in ("q", "k", "v", "g", "beta")), self.host("S0"), scale)
        s = tol(self.dt, dk, dv, N)
        near(got[0], ref, HALF[out or self.dt], s, "out")
        near(got[1], S, HALF["f32"], s, "S")

    def check_bwd(self, got, scale=0.0):
        B, H, N, dk, dv = self.shape
        ref = delta_backward(*(self.host(n) for n in ("q", "k", "v", "g", "beta", "dout", "S0", "dS")), scale)
        # the gradients meet the forward's errors and the reverse pass's: twice s
        s = 2 * tol(self.dt, dk, dv, N)
        for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), got, ref):
            if b is None:
                assert a is None
            elif b.size:
                near(a, b, HALF["f32" if name == "dS0" else self.dt], s, name)


SHAPES = [(1, 1, 1, 64, 64), (1, 2, 1, 128, 128), (2, 3, 77, 24, 40), (1, 2, 130, 64, 64), (2, 1, 128, 128, 128),
          (1, 1, 300, 128, 128), (1, 3, 257, 64, 64), (1, 1, 64, 1, 1), (1, 1, 33, 128, 3), (1, 2, 50, 5, 128)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(cuda_device, shape, dt):
    p = Problem(*shape, dt)
    p.check_fwd(p.fwd())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(cuda_device, shape, dt):
    p = Problem(*shape, dt)
    p.check_bwd(p.bwd())


@pytest.mark.parametrize("dt,dk,dv", [("f32", 16, 24), ("bf16", 64, 64), ("bf16", 128, 128)])
@pytest.mark.parametrize("decay", [True, False])
@pytest.mark.parametrize("start", [True, False])
def test_without_decay_and_without_states(cuda_device, dt, dk, dv, decay, start):
    p = Problem(1, 2, 200, dk, dv, dt, decay=decay, start=start)
    p.check_fwd(p.fwd())
    p.check_bwd(p.bwd())


@pytest.mark.parametrize("dt,dk,dv", [("f32", 16, 24), ("bf16", 64, 64), ("bf16", 32, 48)])
def test_other_output_type_and_scale(cuda_device, dt, dk, dv):
    p = Problem(1, 2, 150, dk, dv, dt)
    other = "f32" if dt == "bf16" else "bf16"
    p.check_fwd(p.fwd(out=other, scale=0.5), out=other, scale=0.5)
    p.check_bwd(p.bwd(scale=0.5), scale=0.5)


GATES = {
    # a state cleared in the middle of a tile, at its first token, and twice in a row
    "cleared": dict(g_of=lambda r, s: np.where(np.isin(np.arange(s[-1]), [0, 40, 41, 128, 190]), -np.inf,
                                               -0.1 * np.abs(r.standard_normal(s)))),
    # decays so strong that products over a tile leave float32's range
    "strong": dict(g_of=lambda r, s: -20 * np.abs(r.standard_normal(s))),
    "full steps": dict(beta_of=lambda r, s: np.ones(s)),
    # tokens that write nothing, and some with no decay either: padding
    "no steps": dict(beta_of=lambda r, s: np.where(r.uniform(size=s) < 0.7, 0.0, r.uniform(size=s)),
                     g_of=lambda r, s: np.where(r.uniform(size=s) < 0.5, 0.0, -0.05)),
    "beta to two": dict(beta_of=lambda r, s: 2 * r.uniform(size=s) * 0.95),
}


@pytest.mark.parametrize("dt,dk,dv", [("f32", 16, 24), ("bf16", 64, 64), ("bf16", 128, 128)])
@pytest.mark.parametrize("gates", sorted(GATES))
def test_gates(cuda_device, gates, dt, dk, dv):
    p = Problem(1, 2, 260, dk, dv, dt, **GATES[gates])
    p.check_fwd(p.fwd())
    p.check_bwd(p.bwd())


@pytest.mark.parametrize("d,N", [(64, 65), (64, 128), (64, 130), (64, 200), (128, 45), (128, 129)])
@pytest.mark.parametrize("gates", [None] + sorted(GATES))
def test_short_sequences_of_many_heads(cuda_device, gates, d, N):
    """Enough heads for the chunk form at every one of these lengths."""
    p = Problem(2, 10240 // d // 2, N, d, d, "bf16", **GATES.get(gates, {}))
    p.check_fwd(p.fwd())
    p.check_bwd(p.bwd())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [283, 385, 500])
def test_gates_in_the_chunk_form(cuda_device, d, N):
    """One head: longer sequences than the token form takes."""
    for gates in sorted(GATES):
        p = Problem(1, 1, N, d, d, "bf16", **GATES[gates])
        p.check_fwd(p.fwd())
        p.check_bwd(p.bwd())


@pytest.mark.parametrize("d", [64, 128])
def test_equal_keys(cuda_device, d):
    """Every key the same, full steps, no decay: (I + A) is the all-ones triangle,
    whose inverse is bidiagonal; its powers are not bounded, its inverse is."""
    p = Problem(1, 2, 256, d, d, "bf16", decay=False, beta_of=lambda r, s: np.ones(s))
    k = torch.zeros(d)
    k[: d // 16] = (16 / d) ** 0.5      # exact in bf16 for these sizes (0.5, and 2^-1.5 rounded)
    p.dev["k"] = k.to(torch.bfloat16).cuda().expand(p.dev["k"].shape).contiguous()
    p.check_fwd(p.fwd())
    p.check_bwd(p.bwd())


@pytest.mark.parametrize("dt,d,cut", [("bf16", 64, 100), ("bf16", 128, 128), ("f32", 40, 33)])
def test_two_calls_continue_a_sequence(cuda_device, dt, d, cut):
    p = Problem(2, 2, 300, d, d, dt)
    ref, _ = delta_recurrent(*(p.host(n) for n in ("q", "k", "v", "g", "beta")), p.host("S0"))
    S, outs = p.S0.clone(), []
    for a, b in ((0, cut), (cut, 300)):
        x = {n: p.dev[n][:, :, a:b].contiguous() for n in ("q", "k", "v", "g", "beta")}
        o = torch.full((2, 2, b - a, d), float("nan"), dtype=TYPES[dt], device="cuda")
        desc = p.desc(N=b - a)
        ws = T.alloc_workspace(T.ttt_delta_workspace_bytes(desc))
        T.ttt_delta_fwd(desc, x["q"], x["k"], x["v"], x["g"], x["beta"], S, o, ws)
        assert T.ttt_check_device_status(ws) == T.TTT_OK
        outs.append(o)
    near(torch.cat(outs, 2), ref, HALF[dt], tol(dt, d, d, 300))


@pytest.mark.parametrize("d", [64, 128])
def test_long_sequence(cuda_device, d):
    """Few heads over a long odd sequence (the form that splits it)."""
    p = Problem(1, 2, 5003, d, d, "bf16")
    p.check_fwd(p.fwd())
    p.check_bwd(p.bwd())


@pytest.mark.parametrize("d,N", [(64, 2700), (128, 2600)])
def test_many_heads_are_the_heads_one_by_one(cuda_device, d, N):
    """64 heads go over the sequence in several slabs that share the workspace in
    turn (their lengths go by the number of heads), one head in one: the same bits."""
    p = Problem(1, 1, N, d, d, "bf16", seed=5)
    B, H = 2, 32
    r = torch.Generator(device="cuda").manual_seed(7)
    shift = torch.randint(0, N, (B * H,), generator=r, device="cuda").tolist()
    many = {n: torch.stack([t[0, 0].roll(s, 0) for s in shift]).view(B, H, *t.shape[2:]) for n, t in p.dev.items()}
    S = torch.randn(B, H, d, d, generator=r, device="cuda")
    one = [0, 31, 63]
    S_one = [S.view(-1, d, d)[i].clone() for i in one]
    o = torch.full_like(many["v"], float("nan"))
    desc = T.make_delta_desc(B, H, N, d, d)
    ws = T.alloc_workspace(T.ttt_delta_workspace_bytes(desc))
    T.ttt_delta_fwd(desc, many["q"], many["k"], many["v"], many["g"], many["beta"], S, o, ws)
    assert T.ttt_check_device_status(ws) == T.TTT_OK
    desc = T.make_delta_desc(1, 1, N, d, d)
    ws = T.alloc_workspace(T.ttt_delta_workspace_bytes(desc))
    for i, s in zip(one, S_one):
        x = {n: t.flatten(0, 1)[i].clone() for n, t in many.items()}   # (aligned)
        got = torch.empty_like(x["v"])
        T.ttt_delta_fwd(desc, x["q"], x["k"], x["v"], x["g"], x["beta"], s, got, ws)
        assert torch.equal(got, o.flatten(0, 1)[i]) and torch.equal(s, S.view(-1, d, d)[i])


@pytest.mark.parametrize("d,N", [(64, 70), (128, 33), (64, 1)])
def test_many_short_sequences(cuda_device, d, N):
    """So many heads that less than one chunk of each goes to the tensor cores (one token does not)."""
    p = Problem(8, 20, N, d, d, "bf16")
    p.check_fwd(p.fwd())
    p.check_bwd(p.bwd())


@pytest.mark.parametrize("dt,d,first", [("f32", 24, 189), ("bf16", 40, 189), ("bf16", 64, 128), ("bf16", 128, 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_value_stays_behind(cuda_device, dt, d, first, bad):
    """NaN or infinity in token 189 of one head: nothing before it changes (on
    tensor cores, nothing before its chunk), nor any other head."""
    p = Problem(1, 2, 300, d, d, dt)
    want = p.fwd()
    p.dev["v"][0, 1, 189, 3] = bad
    got = p.fwd()
    assert torch.equal(got[0][0, 0], want[0][0, 0]) and torch.equal(got[1][0, 0], want[1][0, 0])
    assert torch.equal(got[0][0, 1, :first], want[0][0, 1, :first])
    assert not torch.isfinite(got[0][0, 1, 189:]).all() and not torch.isfinite(got[1][0, 1]).all()


def test_empty_sequence(cuda_device):
    for dt, d in (("f32", 24), ("bf16", 64)):
        p = Problem(1, 2, 0, d, d, dt)
        assert torch.equal(p.fwd()[1], p.S0)
        assert torch.equal(p.bwd()[-1], p.dS)


@pytest.mark.parametrize("d", [64, 128])
def test_same_bits_twice_and_after_another_call(cuda_device, d):
    p, other = Problem(2, 3, 333, d, d, "bf16"), Problem(1, 5, 700, d, d, "bf16", seed=3)
    ws = T.alloc_workspace(max(T.ttt_delta_workspace_bytes(x.desc()) for x in (p, other)))
    a = p.fwd(ws=ws)
    other.fwd(ws=ws)
    b = p.fwd(ws=ws)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert all(torch.equal(x, y) for x, y in zip(p.bwd(), p.bwd()))


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("bf16", 40), ("f32", 24)])
def test_tensors_aligned_to_16_bytes_only(cuda_device, dt, d):
    """Every tensor and the workspace 16 bytes behind a 256-byte boundary: the same bits."""
    p = Problem(1, 2, 200, d, d, dt)
    want_f, want_b = p.fwd(), p.bwd()

    def shifted(t):
        n = t.numel() * t.element_size()
        raw = torch.zeros(n + 512, dtype=torch.uint8, device="cuda")
        off = -raw.data_ptr() % 256 + 16
        out = raw[off:off + n].view(t.dtype).view(t.shape)
        out.copy_(t)
        return out

    desc, x = p.desc(), {n: shifted(t) for n, t in p.dev.items()}
    S, S0, dS, o = shifted(p.S0), shifted(p.S0), shifted(p.dS), shifted(torch.zeros_like(p.dev["v"]))
    g = [shifted(t) for t in p.new_grads()]
    nf, nb = T.ttt_delta_workspace_bytes(desc), T.ttt_delta_bwd_workspace_bytes(desc)
    wf, wb = (shifted(torch.zeros(n, dtype=torch.uint8, device="cuda")) for n in (nf, nb))
    T.ttt_delta_fwd(desc, x["q"], x["k"], x["v"], x["g"], x["beta"], S, o, wf)
    T.ttt_delta_bwd(desc, x["q"], x["k"], x["v"], x["g"], x["beta"], S0, x["dout"], dS, *g, wb)
    assert T.ttt_check_device_status(wf) == T.TTT_OK and T.ttt_check_device_status(wb) == T.TTT_OK
    assert torch.equal(o, want_f[0]) and torch.equal(S, want_f[1])
    assert all(torch.equal(a, b) for a, b in zip(g, want_b))


@pytest.mark.parametrize("dt,d", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_captured_calls_replay(cuda_device, dt, d):
    """Forward, backward and step in one graph on another stream; replays on new
    inputs in the same buffers."""
    p = Problem(1, 2, 200, d, d, dt)
    want_f, want_b = p.fwd(), p.bwd()
    desc, x = p.desc(), p.dev
    S, o, g = p.S0.clone(), torch.empty_like(x["v"]), p.new_grads()
    ws = T.alloc_workspace(T.ttt_delta_workspace_bytes(desc))
    wb = T.alloc_workspace(T.ttt_delta_bwd_workspace_bytes(desc))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        graph.capture_begin()
        S.copy_(p.S0)
        T.ttt_delta_fwd(desc, x["q"], x["k"], x["v"], x["g"], x["beta"], S, o, ws)
        T.ttt_delta_bwd(desc, x["q"], x["k"], x["v"], x["g"], x["beta"], p.S0, x["dout"], p.dS, *g, wb)
        graph.capture_end()
    torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want_f[0]) and torch.equal(S, want_f[1])
    assert all(torch.equal(a, b) for a, b in zip(g, want_b))
    new = Problem(1, 2, 200, d, d, dt, seed=9)
    for n in x:
        x[n].copy_(new.dev[n])
    p.S0.copy_(new.S0)
    p.dS.copy_(new.dS)
    graph.replay()
    torch.cuda.synchronize()
    new.check_fwd((o, S))
    new.check_bwd(g)


def test_two_streams_at_once(cuda_device):
    ps = [Problem(2, 4, 400, d, d, "bf16", seed=d) for d in (64, 128)]
    want = [p.fwd() for p in ps]
    streams, got = [torch.cuda.Stream() for _ in ps], []
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for p, s in zip(ps, streams):
            with torch.cuda.stream(s):
                got.append(p.fwd())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))


# ------------------------------------------------------------------ single tokens
def step_ref(x, slots, S, n_slots):
    """Rows in order on a float64 pool."""
    S = S.copy()
    B, H, dk = x["k"].shape
    out = np.full(x["v"].shape, 7.0)
    for b in range(B):
        at = int(slots[b])
        if 0 <= at < n_slots:
            g = None if x["g"] is None else x["g"][b][None, :, None]
            o, s = delta_recurrent(x["q"][b][None, :, None], x["k"][b][None, :, None], x["v"][b][None, :, None], g,
                                   x["beta"][b][None, :, None], S[at][None])
            S[at], out[b] = s[0], o[0, :, 0]
    return out, S


@pytest.mark.parametrize("dt,dk,dv,B,H", [("f32", 24, 40, 5, 3), ("bf16", 64, 64, 1, 1), ("bf16", 128, 128, 9, 4),
                                          ("bf16", 128, 128, 70, 16), ("f32", 128, 128, 3, 2), ("bf16", 7, 5, 4, 2),
                                          ("f32", 1, 1, 2, 1), ("bf16", 128, 67, 3, 2), ("bf16", 128, 36, 300, 2)])
@pytest.mark.parametrize("kind", ["none", "spread", "idle and shared"])
@pytest.mark.parametrize("decay", [True, False])
def test_step(cuda_device, dt, dk, dv, B, H, kind, decay):
    r = np.random.default_rng([dk, dv, B])
    p = Problem(B, H, 1, dk, dv, dt, decay=decay)
    x = {n: None if t is None else t[:, :, 0].contiguous() for n, t in p.dev.items()}
    n_slots = B + 3
    if kind == "none":
        slots, idx = None, np.arange(B)
    elif kind == "spread":
        idx = r.permutation(n_slots)[:B]
    else:   # negative and too large slots, and rows that share one
        idx = r.integers(-2, max(2, B // 2), B)
        idx[r.integers(B)] = n_slots
    if kind != "none":
        slots = torch.from_numpy(idx.astype(np.int32)).cuda()
    pool = torch.from_numpy(0.3 * r.standard_normal((n_slots, H, dk, dv))).float().cuda()
    want = step_ref({n: None if t is None else t.double().cpu().numpy() for n, t in x.items()}, idx,
                    pool.double().cpu().numpy(), n_slots)
    out = torch.full((B, H, dv), 7.0, dtype=TYPES[dt], device="cuda")
    T.ttt_delta_step(p.desc(N=1), x["q"], x["k"], x["v"], x["g"], x["beta"], slots, n_slots, pool, out)
    s = 8 * np.sqrt(dk * B) * 2.0 ** -24     # a state may take as many as B tokens
    near(out, want[0], HALF[dt], s, "out")
    near(pool, want[1], HALF["f32"], s, "S")
    used = np.isin(np.arange(n_slots), idx)
    assert np.array_equal(pool.cpu().numpy()[~used], want[1][~used].astype(np.float32))


def test_large_pool_offsets(cuda_device):
    """States beyond 2^32 bytes and 2^31 elements from the pool's start."""
    H, d, n = 16, 128, 8400            # 8400 * 16 * 128 * 128 = 2.2e9 elements, 8.8 GB
    pool = torch.empty(n, H, d, d, device="cuda")
    p = Problem(2, H, 1, d, d, "bf16")
    x = {m: t[:, :, 0].contiguous() for m, t in p.dev.items()}
    idx = np.array([n - 1, 4200])
    pool[torch.from_numpy(idx).cuda()] = 0.25
    pool[0] = 5.0
    host = np.full((2, H, d, d), 0.25)
    want = step_ref({m: t.double().cpu().numpy() for m, t in x.items()}, np.array([0, 1]), host, 2)
    out = torch.empty(2, H, d, dtype=torch.bfloat16, device="cuda")
    T.ttt_delta_step(p.desc(N=1), x["q"], x["k"], x["v"], x["g"], x["beta"],
                     torch.from_numpy(idx.astype(np.int32)).cuda(), n, pool, out)
    near(out, want[0], HALF["bf16"], 8 * np.sqrt(d) * 2.0 ** -24)
    near(pool[torch.from_numpy(idx).cuda()], want[1], HALF["f32"], 8 * np.sqrt(d) * 2.0 ** -24)
    assert bool((pool[0] == 5.0).all())


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("f32", 24)])
def test_prefill_then_single_tokens(cuda_device, dt, d):
    """A prompt through the sequence form, then tokens one by one on its state,
    read as one sequence."""
    p = Problem(2, 3, 150, d, d, dt)
    ref, Sref = delta_recurrent(*(p.host(n) for n in ("q", "k", "v", "g", "beta")), p.host("S0"))
    cut, S = 141, p.S0.clone()
    x = {n: t[:, :, :cut].contiguous() for n, t in p.dev.items()}
    out = torch.empty(2, 3, cut, d, dtype=TYPES[dt], device="cuda")
    desc = p.desc(N=cut)
    ws = T.alloc_workspace(T.ttt_delta_workspace_bytes(desc))
    T.ttt_delta_fwd(desc, x["q"], x["k"], x["v"], x["g"], x["beta"], S, out, ws)
    outs = [out]
    for t in range(cut, 150):
        x = {n: y[:, :, t].contiguous() for n, y in p.dev.items()}
        o = torch.empty(2, 3, d, dtype=TYPES[dt], device="cuda")
        T.ttt_delta_step(p.desc(N=1), x["q"], x["k"], x["v"], x["g"], x["beta"], None, 2, S, o)
        outs.append(o[:, :, None])
    s = tol(dt, d, d, 150)
    near(torch.cat(outs, 2), ref, HALF[dt], s)
    near(S, Sref, HALF["f32"], s)


# ------------------------------------------------------------------ refusals with a device
def test_memory_of_the_host_is_refused(cuda_device):
    p = Problem(1, 1, 4, 16, 16, "f32")
    d, x, S = p.desc(), p.dev, p.S0.clone()
    ws, out = T.alloc_workspace(T.ttt_delta_workspace_bytes(d)), torch.empty_like(x["v"])
    assert T.ttt_delta_fwd(d, x["q"].cpu(), x["k"], x["v"], x["g"], x["beta"], S, out, ws, check=False) == T.TTT_ERR_ARG
    assert T.ttt_delta_fwd(d, x["q"], x["k"], x["v"], x["g"], x["beta"], S, x["v"], ws, check=False) == T.TTT_ERR_ARG
    assert T.ttt_delta_fwd(d, x["q"], x["k"], x["v"], x["g"], x["beta"], S, out, ws, check=False) == T.TTT_OK


# ------------------------------------------------------------------ gradients of strong decays
DECAYS = {"-4": -4.0, "-8": -8.0, "-12": -12.0, "-16": -16.0, "-30": -30.0,
          # strong decays among weak ones, where terms of the weak ones are e^30 times larger
          "mixed": np.array([-0.02, -0.02, -0.02, -4, -8, -12, -16, -30])}


def check_decay_gradient(p, got):
    """dg_t = a_t <Y, S_{t-1}> is as small as its own decay a_t = exp(g_t), so it
    is compared as dg_t / a_t: no term of another token's size may enter it.
    Tolerance: the gradients' one of check_bwd, r for the type's rounding."""
    B, H, N, dk, dv = p.shape
    ref = delta_backward(*(p.host(n) for n in ("q", "k", "v", "g", "beta", "dout", "S0", "dS")))[3]
    a = np.exp(p.host("g"))
    near(got[3].double().cpu().numpy() / a, ref / a, HALF[p.dt], 2 * tol(p.dt, dk, dv, N), "dg / a")


def strong(dt, N, d, decay, B=1, H=2):
    return Problem(B, H, N, *d, dt, g_of=lambda r, s: r.choice(np.atleast_1d(DECAYS[decay]), s))


@pytest.mark.parametrize("dt,N,d", [("f32", 32, (64, 64)), ("f32", 75, (24, 40)), ("bf16", 100, (128, 128)),
                                    ("f32", 150, (5, 3))])
@pytest.mark.parametrize("decay", list(DECAYS))
def test_gradients_of_strong_decays_token_form(cuda_device, dt, N, d, decay):
    p = strong(dt, N, d, decay)
    got = p.bwd()
    p.check_bwd(got)
    check_decay_gradient(p, got)


@pytest.mark.parametrize("d,N,B,H", [(64, 400, 1, 2), (128, 300, 1, 2), (64, 130, 4, 40), (128, 45, 4, 20)])
@pytest.mark.parametrize("decay", list(DECAYS))
def test_gradients_of_strong_decays_chunk_form(cuda_device, d, N, B, H, decay):
    p = strong("bf16", N, (d, d), decay, B, H)
    got = p.bwd()
    p.check_bwd(got)
    check_decay_gradient(p, got)


# ------------------------------------------------------------------ errors of earlier calls
def leave_an_error():
    """A refused memset of an earlier call stays the library runtime's last
    error (the state is host memory)."""
    d = T.make_linear_desc(1, 1, 4, 8, 8, 4, in_dtype="f32", out_dtype="f32")
    T.load().ttt_linear_state_init(ctypes.byref(d), None, torch.zeros(1, 1, 8, 8).data_ptr(), None)


@pytest.mark.parametrize("dt,d", [("f32", 24), ("bf16", 64)])
def test_an_earlier_error_is_not_this_calls(cuda_device, dt, d):
    """A pending error of another call: the work is done once and reported as done."""
    p = Problem(2, 2, 200, d, d, dt)
    want_f, want_b = p.fwd(), p.bwd()
    leave_an_error()
    got = p.fwd()
    leave_an_error()
    grads = p.bwd()
    assert all(torch.equal(a, b) for a, b in zip(want_f + tuple(want_b), got + tuple(grads)))
    x = {n: t[:, :, 0].contiguous() for n, t in p.dev.items()}
    pools, outs = [p.S0.clone(), p.S0.clone()], []
    for S, error in zip(pools, (False, True)):
        if error:
            leave_an_error()
        outs.append(torch.empty_like(x["v"]))
        T.ttt_delta_step(p.desc(N=1), x["q"], x["k"], x["v"], x["g"], x["beta"], None, 2, S, outs[-1])
    assert torch.equal(*pools) and torch.equal(*outs)


@pytest.mark.parametrize("dt,dk,dv,N,B,H", [("f32", 3, 2, 2, 7, 10001), ("bf16", 8, 8, 1, 1, 65537)])
def test_more_heads_than_a_grid_dimension(cuda_device, dt, dk, dv, N, B, H):
    """The chunk gradients go over the heads in slices of 65,535."""
    p = Problem(B, H, N, dk, dv, dt)
    p.check_fwd(p.fwd())
    p.check_bwd(p.bwd())


# ------------------------------------------------------------------ the precision of each form
def in_chunks(p, backward):
    """Whether the call runs on tensor cores (the workspaces of the two forms differ)."""
    B, H, N, dk, dv = p.shape
    if not backward:
        return T.ttt_delta_workspace_bytes(p.desc()) > T.TTT_STATUS_BYTES
    f32 = T.make_delta_desc(B, H, N, dk, dv, in_dtype="f32", out_dtype="f32")
    return T.ttt_delta_bwd_workspace_bytes(p.desc()) != T.ttt_delta_bwd_workspace_bytes(f32)


def norm_near(got, ref, limit, what):
    got = got.detach().double().cpu().numpy()
    err = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert err <= limit, f"{what}: {err:.2e} of the norm, limit {limit:.1e}"


@pytest.mark.parametrize("N,B,H", [(1, 1, 2), (77, 1, 2), (128, 1, 2), (20, 3, 16)])
@pytest.mark.parametrize("d", [64, 128])
def test_short_bf16_sequences_have_the_float32_bounds(cuda_device, d, N, B, H):
    """bf16 heads of 64 and 128 that go token by token: float32 throughout, so
    the bounds of the float32 path, and the inputs' type for what is rounded to it."""
    p = Problem(B, H, N, d, d, "bf16")
    assert not in_chunks(p, False) and not in_chunks(p, True)
    s = 8 * np.sqrt(d * N) * 2.0 ** -24
    ref, S = delta_recurrent(*(p.host(n) for n in ("q", "k", "v", "g", "beta")), p.host("S0"))
    for out in ("f32", "bf16"):
        o, S_end = p.fwd(out=out)
        near(o, ref, HALF[out], s, "out")
        near(S_end, S, HALF["f32"], s, "S")
    want = delta_backward(*(p.host(n) for n in ("q", "k", "v", "g", "beta", "dout", "S0", "dS")))
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), p.bwd(), want):
        near(a, b, HALF["f32" if name == "dS0" else "bf16"], 2 * s, name)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("decay", [True, False])
@pytest.mark.parametrize("start", [True, False])
def test_states_and_float32_outputs_of_the_chunk_form(cuda_device, d, decay, start):
    """Norm-wise limits of the float32 results on tensor cores.

    An operand hi + lo is off by at most 2^-18 (two roundings of 2^-9 each), 0.4
    of that in the mean square, and the lo lo left out of a product of two pairs
    is as much: 2.4e-6 a product, norm-wise, as terms of either sign add up.
    Without decay the state goes through three in turn (T gam K, rho W, M S: 3.7e-6)
    in every chunk, of which the contraction I + M keeps less with every further
    one: twice to three times that, 1e-5.  Outputs join W S0, P U and Q S0 to it:
    1.5e-5.  With decays of 0.05 a token the mean chunk keeps e^-7 of the state
    before it, so S and dS0 are H and Hb, whose operands have three planes (2^-26):
    what is left is T diag(beta) above (its diagonal is exact, and the rest is a
    third of it in norm: 5e-7), the decays' exponentials (2^-22, 2.4e-7) and the
    truncated sum of 128 terms (2^-24 each): 2e-6.  Two planes would leave 2^-18.
    """
    p = Problem(1, 2, 1024, d, d, "bf16", decay=decay, start=start)
    assert in_chunks(p, False) and in_chunks(p, True)
    ref, S = delta_recurrent(*(p.host(n) for n in ("q", "k", "v", "g", "beta")), p.host("S0"))
    o, S_end = p.fwd(out="f32")
    dS0 = p.bwd()[-1]
    want = delta_backward(*(p.host(n) for n in ("q", "k", "v", "g", "beta", "dout", "S0", "dS")))[-1]
    norm_near(S_end, S, 2e-6 if decay else 1e-5, "S")
    norm_near(dS0, want, 2e-6 if decay else 1e-5, "dS0")
    norm_near(o, ref, 1.5e-5, "out")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("start", [True, False])
def test_float32_outputs_of_the_chunk_form_with_decay(cuda_device, d, start):
    """P and U in three planes (2^-26 an operand, products down to 2^-27 kept), so the
    outputs are off by what two planes of S0 (2^-18, 0.4 in the mean square: 1.5e-6 of
    Q S0, which the decay makes a third of the outputs in norm: 5e-7) and of T diag(beta)
    (5e-7) leave, the exponentials' 2^-22 and the sums: 2e-6.  Two planes of P or U
    would leave 2.5e-6 more."""
    p = Problem(1, 2, 1024, d, d, "bf16", start=start)
    assert in_chunks(p, False)
    ref, _ = delta_recurrent(*(p.host(n) for n in ("q", "k", "v", "g", "beta")), p.host("S0"))
    norm_near(p.fwd(out="f32")[0], ref, 2e-6, "out")


@pytest.mark.parametrize("d,N", [(64, 2048), (128, 1024)])
def test_gradients_of_the_chunk_form_round_as_their_float32_values_do(cuda_device, d, N):
    """A bf16 result whose error before rounding is s of the norm falls on the other
    side of a border than the exact value with probability 0.8 s sum_e P(e) 2^(7-e)
    over its binades e: normal values are in a binade e < 0 with probability 0.8 2^e,
    so each of the dozen down to s adds 100, 960 s in all.  What two planes leave in
    them, by operand: dq 7e-7 of S0 and 6e-7 of T diag(beta), s = 1.0e-6; dv 9e-7 of
    X1 and 6e-7 of T, 1.1e-6; dk 9e-7 of X1 and 7e-7 each of Mk, Y and dU's other
    terms, 1.5e-6: 1.0e-3, 1.1e-3 and 1.5e-3 of the values, and a quarter more as the
    limit.  Two planes of U, Mq or dU leave 2.5e-6 more: 2.6e-3 and above."""
    p = Problem(1, 2, N, d, d, "bf16")
    assert in_chunks(p, True)
    want = delta_backward(*(p.host(n) for n in ("q", "k", "v", "g", "beta", "dout", "S0", "dS")))
    for name, a, b in zip(("dq", "dk", "dv"), p.bwd(), want):
        other = (a.cpu() != torch.from_numpy(b).to(torch.bfloat16)).double().mean().item()
        assert other <= {"dq": 1.4e-3, "dk": 1.9e-3, "dv": 1.4e-3}[name], f"{name}: {other:.2e} of the values"


@pytest.mark.parametrize("B,H,N", [(1, 2, 400), (4, 20, 130)])
@pytest.mark.parametrize("start", [True, False])
def test_chunk_form_gradients_without_decay(cuda_device, B, H, N, start):
    for d in (64, 128):
        p = Problem(B, H, N, d, d, "bf16", decay=False, start=start)
        assert in_chunks(p, True)
        p.check_bwd(p.bwd())


def test_gradients_on_two_streams_at_once(cuda_device):
    """Calls of either size and form side by side, each with its own workspace: the same bits."""
    ps = [Problem(2, 4, N, d, d, dt, seed=N) for d, N, dt in ((64, 700, "bf16"), (128, 500, "bf16"), (32, 200, "f32"))]
    want = [p.bwd() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    outs = [p.new_grads() for p in ps]
    wss = [T.alloc_workspace(T.ttt_delta_bwd_workspace_bytes(p.desc())) for p in ps]
    torch.cuda.synchronize()
    for _ in range(4):
        for p, s, g, ws in zip(ps, streams, outs, wss):
            x = p.dev
            T.ttt_delta_bwd(p.desc(), x["q"], x["k"], x["v"], x["g"], x["beta"], p.S0, x["dout"], p.dS, *g, ws, stream=s)
    torch.cuda.synchronize()
    assert all(T.ttt_check_device_status(ws) == T.TTT_OK for ws in wss)
    assert all(torch.equal(a, b) for w, g in zip(want, outs) for a, b in zip(w, g))
