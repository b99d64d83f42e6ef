"""Delta rule and row norm without a GPU: struct layouts, workspace sizes and
the refusals that the host makes before anything is enqueued."""
import ctypes
import os
import subprocess

import pytest

import learned_linear_attention_b200 as T
from learned_linear_attention_b200 import _lib

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ttt.h")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from learned_linear_attention_b200 import build
        build.build()
    return T.load()


def test_structs_match_c_layout(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', 'int main(void){']
    for cls in (T.ttt_delta_desc, T.ttt_norm_desc):
        s = cls.__name__
        lines.append(f'printf("{s} %zu\\n", sizeof({s}));')
        lines += [f'printf("{s}.{f[0]} %zu\\n", offsetof({s}, {f[0]}));' for f in cls._fields_]
    (tmp_path / "l.c").write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-o", str(tmp_path / "l"), str(tmp_path / "l.c")], check=True)
    out = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout
    got = dict(line.split() for line in out.splitlines())
    for cls in (T.ttt_delta_desc, T.ttt_norm_desc):
        assert int(got[cls.__name__]) == ctypes.sizeof(cls)
        for f in cls._fields_:
            assert int(got[f"{cls.__name__}.{f[0]}"]) == getattr(cls, f[0]).offset


# addresses far apart, so that nothing overlaps; never dereferenced on the host
def _far(**over):
    names = ("q", "k", "v", "g", "beta", "S", "out", "ws", "dout", "dS_end", "dq", "dk", "dv", "dg",
             "dbeta", "dS0", "slots", "x", "w", "z", "res", "dx", "dw", "dz")
    p = {n: (i + 1) << 40 for i, n in enumerate(names)}
    p.update(over)
    return p


def _fwd(d, ws_bytes=1 << 39, **over):
    p = _far(**over)
    return T.load().ttt_delta_fwd(ctypes.byref(d), *(p[n] for n in ("q", "k", "v", "g", "beta", "S", "out", "ws")),
                                  ws_bytes, None)


def _bwd(d, ws_bytes=1 << 39, **over):
    p = _far(**over)
    names = ("q", "k", "v", "g", "beta", "S", "dout", "dS_end", "dq", "dk", "dv", "dg", "dbeta", "dS0", "ws")
    return T.load().ttt_delta_bwd(ctypes.byref(d), *(p[n] for n in names), ws_bytes, None)


def _step(d, n_slots=64, **over):
    p = _far(**over)
    return T.load().ttt_delta_step(ctypes.byref(d), *(p[n] for n in ("q", "k", "v", "g", "beta", "slots")),
                                   n_slots, p["S"], p["out"], None)


def _norm(d, **over):
    p = _far(**over)
    return T.load().ttt_norm_fwd(ctypes.byref(d), *(p[n] for n in ("x", "w", "z", "res", "out")), None)


def _norm_bwd(d, ws_bytes=1 << 39, **over):
    p = _far(**over)
    return T.load().ttt_norm_bwd(ctypes.byref(d), *(p[n] for n in ("x", "w", "z", "dout", "dx", "dw", "dz", "ws")),
                                 ws_bytes, None)


def test_delta_refuses_sizes_that_wrap():
    """Tokens whose byte counts would pass 64 bits are refused, not wrapped to a small workspace."""
    d = T.make_delta_desc(1 << 16, (1 << 15) - 1, (1 << 31) - 1, 128, 128)
    n = ctypes.c_size_t(0)
    for fn in ("ttt_delta_workspace_bytes", "ttt_delta_bwd_workspace_bytes", "ttt_delta_layer_workspace_bytes"):
        assert getattr(T.load(), fn)(ctypes.byref(d), ctypes.byref(n)) == T.TTT_ERR_SHAPE, fn
    assert _fwd(d) == _bwd(d) == T.TTT_ERR_SHAPE
    # the largest that pass: 64-bit sizes, larger than their tensors
    d = T.make_delta_desc(1, 1, (1 << 31) - 1, 128, 128)
    for fn in ("ttt_delta_bwd_workspace_bytes", "ttt_delta_layer_workspace_bytes"):
        assert getattr(T.load(), fn)(ctypes.byref(d), ctypes.byref(n)) == T.TTT_OK
        assert n.value > ((1 << 31) - 1) * 128 * 2


@pytest.mark.parametrize("call", [_fwd, _bwd, _step])
def test_delta_descriptor_refusals(call):
    N = 1 if call is _step else 8
    mk = lambda **kw: T.make_delta_desc(**{**dict(B=2, H=2, N=N, dk=64, dv=64), **kw})  # noqa: E731
    assert call(mk(B=0)) == T.TTT_ERR_SHAPE
    assert call(mk(H=0)) == T.TTT_ERR_SHAPE
    assert call(mk(N=-1)) == T.TTT_ERR_SHAPE
    assert call(mk(dk=0)) == T.TTT_ERR_SHAPE
    assert call(mk(dk=129)) == T.TTT_ERR_UNSUPPORTED
    assert call(mk(dv=136)) == T.TTT_ERR_UNSUPPORTED
    assert call(mk(B=1 << 16, H=1 << 15)) == T.TTT_ERR_SHAPE
    assert call(mk(scale=float("nan"))) == T.TTT_ERR_ARG
    for f in ("in_dtype", "out_dtype"):
        d = mk()
        setattr(d, f, 2)
        assert call(d) == T.TTT_ERR_DTYPE
    for n in ("q", "k", "v", "beta"):
        assert call(mk(), **{n: 0}) == T.TTT_ERR_ARG, n
        assert call(mk(), **{n: (9 << 44) + 8}) == T.TTT_ERR_ALIGN, n


def test_delta_fwd_refusals():
    d = T.make_delta_desc(1, 2, 8, 64, 64)
    assert _fwd(d, ws_bytes=T.ttt_delta_workspace_bytes(d) - 1) == T.TTT_ERR_WORKSPACE
    assert _fwd(d, S=0) == T.TTT_ERR_ARG
    assert _fwd(d, ws=0) == T.TTT_ERR_ARG
    assert _fwd(d, out=0) == T.TTT_ERR_ARG
    # overlapping ranges: out on v, out in the middle of q, the state on the workspace
    assert _fwd(d, out=3 << 40) == T.TTT_ERR_ARG
    assert _fwd(d, out=(1 << 40) + 256) == T.TTT_ERR_ARG
    assert _fwd(d, S=8 << 40) == T.TTT_ERR_ARG
    # N = 0: nothing to do
    assert _fwd(T.make_delta_desc(1, 2, 0, 64, 64)) == T.TTT_OK


def test_delta_bwd_refusals():
    d = T.make_delta_desc(1, 2, 8, 64, 64)
    assert _bwd(d, ws_bytes=T.ttt_delta_bwd_workspace_bytes(d) - 1) == T.TTT_ERR_WORKSPACE
    for n in ("dq", "dk", "dv", "dbeta", "dS0", "dout"):
        assert _bwd(d, **{n: 0}) == T.TTT_ERR_ARG, n
    assert _bwd(d, g=0) == T.TTT_ERR_ARG      # dg without g
    assert _bwd(d, dg=0) == T.TTT_ERR_ARG     # g without dg
    assert _bwd(d, dq=1 << 40) == T.TTT_ERR_ARG     # dq on q
    assert _bwd(d, dq=12 << 40) == T.TTT_ERR_ARG    # dq on dk


def test_delta_step_refusals():
    d = T.make_delta_desc(4, 2, 1, 64, 64)
    assert _step(T.make_delta_desc(4, 2, 2, 64, 64)) == T.TTT_ERR_SHAPE
    assert _step(T.make_delta_desc(4, 2, 0, 64, 64)) == T.TTT_ERR_SHAPE
    assert _step(d, n_slots=0) == T.TTT_ERR_SHAPE
    assert _step(d, n_slots=3, slots=0) == T.TTT_ERR_SHAPE   # row 3 would have no state
    assert _step(d, S=0) == T.TTT_ERR_ARG
    assert _step(d, out=6 << 40) == T.TTT_ERR_ARG


def test_norm_refusals():
    mk = lambda **kw: T.make_norm_desc(**{**dict(rows=5, D=64, gate="silu"), **kw})  # noqa: E731
    for call in (_norm, _norm_bwd):
        assert call(mk(rows=-1)) == T.TTT_ERR_SHAPE
        assert call(mk(D=0)) == T.TTT_ERR_SHAPE
        assert call(mk(D=8200)) == T.TTT_ERR_UNSUPPORTED
        assert call(mk(D=68)) == T.TTT_ERR_ALIGN
        assert call(mk(rows=1 << 50)) == T.TTT_ERR_SHAPE
        assert call(mk(eps=0.0)) == T.TTT_ERR_ARG
        assert call(mk(eps=float("nan"))) == T.TTT_ERR_ARG
        assert call(mk(scale=float("nan"))) == T.TTT_ERR_ARG
        for f in ("kind", "gate"):
            d = mk()
            setattr(d, f, 3)
            assert call(d) == T.TTT_ERR_ARG
        d = mk()
        d.dtype = 2
        assert call(d) == T.TTT_ERR_DTYPE
        assert call(mk(), x=0) == T.TTT_ERR_ARG
        assert call(mk(), z=0) == T.TTT_ERR_ARG
        assert call(mk(gate="none")) == T.TTT_ERR_ARG     # z without a gate
        assert call(mk(), x=(9 << 44) + 4) == T.TTT_ERR_ALIGN
    d = mk()
    assert _norm(d, out=(18 << 40) + 128) == T.TTT_ERR_ARG   # out across x
    assert _norm(mk(rows=0)) == T.TTT_OK
    assert _norm_bwd(d, ws_bytes=T.ttt_norm_bwd_workspace_bytes(d) - 1) == T.TTT_ERR_WORKSPACE
    assert _norm_bwd(d, dw=0) == T.TTT_ERR_ARG
    assert _norm_bwd(d, w=0) == T.TTT_ERR_ARG
    assert _norm_bwd(d, dz=0) == T.TTT_ERR_ARG
    assert _norm_bwd(d, dx=24 << 40) == T.TTT_ERR_ARG        # dx on dz


def test_layer_refusals():
    def call(d, ws_bytes=1 << 39, eps=1e-6, **over):
        p = _far(**over)
        names = ("q", "k", "v", "g", "beta", "w", "z", "res", "S", "out", "ws")
        return T.load().ttt_delta_layer_fwd(ctypes.byref(d), eps, 1.0, *(p[n] for n in names), ws_bytes, None)
    d = T.make_delta_desc(1, 2, 8, 64, 64)
    need = T.ttt_delta_layer_workspace_bytes(d)
    assert need >= T.ttt_delta_workspace_bytes(d) + 3 * 2 * 8 * 64 * 2
    assert call(d, ws_bytes=need - 1) == T.TTT_ERR_WORKSPACE
    assert call(d, eps=0.0) == T.TTT_ERR_ARG
    assert call(d, q=0) == T.TTT_ERR_ARG
    assert call(d, out=3 << 40) == T.TTT_ERR_ARG
    assert call(T.make_delta_desc(1, 2, 8, 60, 64)) == T.TTT_ERR_ALIGN
    assert call(T.make_delta_desc(1, 2, 8, 64, 64, out_dtype="f32")) == T.TTT_ERR_DTYPE
    assert call(T.make_delta_desc(1, 2, 0, 64, 64)) == T.TTT_OK


def _bytes(fn, d):
    n = ctypes.c_size_t(0)
    assert getattr(T.load(), fn)(ctypes.byref(d), ctypes.byref(n)) == T.TTT_OK
    return n.value


def test_workspace_of_the_longest_sequences():
    """Tiles of 32 and chunks of 128 tokens are counted without a sum that passes
    2^31: the sizes follow the layouts' formulas up to the largest N."""
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    for N in [(1 << 31) - i for i in (1, 2, 31, 32, 33, 100, 127, 128, 129, 200)]:
        # token by token: e and du of every token, two states a tile
        tiles = -(-N // 32)
        for dk, dv in ((1, 1), (3, 2)):
            want = 256 + 2 * up(4 * N * dv) + 2 * up(4 * tiles * dk * dv)
            assert _bytes("ttt_delta_bwd_workspace_bytes", T.make_delta_desc(1, 1, N, dk, dv)) == want
        for D in (64, 128):
            d, chunks, slices = T.make_delta_desc(1, 1, N, D, D), -(-N // 128), D // 64
            pair, mat = 2 * 128 * D * 2, 4 * D * D
            # W, Ut, Y; U in three planes; T; M, H, Hb and two border states; sums of tokens and chunks
            want = 512 + up(4 * chunks) + 3 * up(pair * chunks) + up(pair * chunks // 2 * 3) + up(chunks * 2 * 128 * 128 * 2) + 5 * up(mat * chunks)
            want += 4 * up(4 * slices * N) + up(4 * N) + up(4 * slices * chunks)
            assert _bytes("ttt_delta_bwd_workspace_bytes", d) == want
            # forward: at most three slabs, at least one chunk in six
            one = 4 + 2 * pair + 3 * mat
            assert chunks / 6 * one <= _bytes("ttt_delta_workspace_bytes", d) <= (chunks + 8) * one + 4096
            assert _bytes("ttt_delta_layer_workspace_bytes", d) >= _bytes("ttt_delta_workspace_bytes", d) + 3 * N * D * 2


def test_norm_refuses_an_eps_whose_inverse_is_infinite():
    """A row of zeros has the factor 1 / eps: with eps below 1.2e-38 it would be 0 times infinity."""
    for eps in (1e-40, 1.4e-45, 1.1754942e-38):
        for call in (_norm, _norm_bwd):
            assert call(T.make_norm_desc(5, 64, kind="l2", gate="silu", eps=eps)) == T.TTT_ERR_ARG
        # (rms: the mean of squares is added to it; nothing but the pointers is wrong here)
        assert _norm(T.make_norm_desc(5, 64, gate="silu", eps=eps), x=0) == T.TTT_ERR_ARG
        assert _norm(T.make_norm_desc(0, 64, gate="silu", eps=eps)) == T.TTT_OK
    assert _norm(T.make_norm_desc(0, 64, kind="l2", gate="silu", eps=1.1754944e-38)) == T.TTT_OK
