"""Pins of the gated delta rule and row norm oracles against facts that are
not their code: closed forms, the linear layer's oracle, and differences."""
import numpy as np
import pytest

from oracle import (delta_backward, delta_recurrent, row_norm, row_norm_backward,
                    ttt_linear_recurrent)


def _problem(seed, B=1, H=2, N=7, dk=5, dv=3):
    r = np.random.default_rng(seed)
    q, k = r.standard_normal((2, B, H, N, dk))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return dict(q=q, k=k, v=r.standard_normal((B, H, N, dv)),
                g=-np.abs(r.standard_normal((B, H, N))) * 0.5,
                beta=r.uniform(0, 1, (B, H, N)), S0=r.standard_normal((B, H, dk, dv)),
                dout=r.standard_normal((B, H, N, dv)), dS_end=r.standard_normal((B, H, dk, dv)))


def test_full_step_writes_the_value():
    """beta = 1 with a unit key: the key reads back its value exactly."""
    p = _problem(1)
    out, S = delta_recurrent(p["k"], p["k"], p["v"], p["g"], np.ones(p["beta"].shape), p["S0"], 1.0)
    assert np.allclose(out, p["v"], atol=1e-12)


def test_orthogonal_keys_without_decay_are_the_linear_layer():
    """With orthogonal keys and no start state the prediction S^T k is zero, so
    the squared and the inner-product loss take the same steps."""
    p = _problem(2, N=5)
    k = np.broadcast_to(np.eye(5), (1, 2, 5, 5))
    out, S = delta_recurrent(p["q"][:, :, :5], k, p["v"][:, :, :5], None, p["beta"][:, :, :5], None, 1.0)
    ref, Sr = ttt_linear_recurrent(p["q"][:, :, :5], k, p["v"][:, :, :5], p["beta"][:, :, :5])
    assert np.allclose(out, ref, atol=1e-12) and np.allclose(S, Sr, atol=1e-12)


def test_cleared_state_forgets():
    p = _problem(3)
    g = p["g"].copy()
    g[:, :, 4] = -np.inf
    a, Sa = delta_recurrent(p["q"], p["k"], p["v"], g, p["beta"], p["S0"])
    b, Sb = delta_recurrent(*(p[n][:, :, 4:] for n in "qkv"), p["g"][:, :, 4:], p["beta"][:, :, 4:])
    assert np.allclose(a[:, :, 4:], b, atol=1e-12) and np.allclose(Sa, Sb, atol=1e-12)


@pytest.mark.parametrize("decay", [True, False])
def test_gradients_are_differences(decay):
    p = _problem(4)
    names = ["q", "k", "v", "beta", "S0"] + (["g"] if decay else [])

    def loss(x):
        out, S = delta_recurrent(x["q"], x["k"], x["v"], x["g"] if decay else None, x["beta"], x["S0"])
        return (out * p["dout"]).sum() + (S * p["dS_end"]).sum()

    got = delta_backward(p["q"], p["k"], p["v"], p["g"] if decay else None, p["beta"], p["dout"],
                         p["S0"], p["dS_end"])
    got = dict(zip(("q", "k", "v", "g", "beta", "S0"), got))
    r = np.random.default_rng(5)
    for n in names:
        d = r.standard_normal(p[n].shape)
        lo, hi = dict(p), dict(p)
        h = 1e-5
        lo[n], hi[n] = p[n] - h * d, p[n] + h * d
        assert abs((loss(hi) - loss(lo)) / (2 * h) - (got[n] * d).sum()) < 1e-6, n


@pytest.mark.parametrize("kind", ["rms", "l2"])
@pytest.mark.parametrize("gate", ["none", "silu", "sigmoid"])
def test_norm_gradients_are_differences(kind, gate):
    r = np.random.default_rng(6)
    x, z, dout = r.standard_normal((3, 4, 6))
    w = r.standard_normal(6)
    kw = dict(kind=kind, gate=gate, scale=0.7)
    got = row_norm_backward(x, dout, w, z, **kw)

    def f(x, w, z):
        return (dout * row_norm(x, w, z, **kw)).sum()

    h = 1e-6
    for i, a in enumerate((x, w, z)):
        if i == 2 and gate == "none":
            assert got[2] is None
            continue
        d = r.standard_normal(a.shape)
        lo, hi = [x, w, z], [x, w, z]
        lo[i], hi[i] = a - h * d, a + h * d
        assert abs((f(*hi) - f(*lo)) / (2 * h) - (got[i] * d).sum()) < 1e-7


def test_norm_makes_unit_rows():
    x = np.random.default_rng(7).standard_normal((5, 8))
    assert np.allclose(np.linalg.norm(row_norm(x, kind="l2"), axis=-1), 1)
    assert np.allclose((row_norm(x, eps=1e-30) ** 2).mean(-1), 1)
