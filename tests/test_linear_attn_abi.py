"""Linear attention and rotary positions without a GPU: what the C ABI refuses before any CUDA
call, the workspace rule, the binding's marshalling and checks, the rotary plans."""
import contextlib
import ctypes
import math

import numpy as np
import pytest
import torch

from test_sequence_modeling_b200 import _lib as L
from test_sequence_modeling_b200 import ttt

# Fake, never-dereferenced device addresses.
A, STEP = 0x100000, 1 << 32


@pytest.fixture(scope="module")
def lib():
    from test_sequence_modeling_b200.build import build
    build()
    return L.load()


def _at(i):
    return A + i * STEP


def fwd(lib, **kw):
    a = dict(Q=_at(0), K=_at(1), V=_at(2), dt=L.TTT_BF16, g=_at(3), S0=_at(4), n=_at(5), scale=0.125, B=2, H=3, T=2000,
             d=64, Z=_at(6), S=_at(7), ws=_at(8), wsn=1 << 30)
    a.update(kw)
    return lib.ttt_linear_attn_fwd(a["Q"], a["K"], a["V"], a["dt"], a["g"], a["S0"], a["n"], a["scale"], a["B"], a["H"],
                                   a["T"], a["d"], a["Z"], a["S"], a["ws"], a["wsn"], None)


def bwd(lib, **kw):
    a = dict(Q=_at(0), K=_at(1), V=_at(2), dt=L.TTT_BF16, g=_at(3), S0=_at(4), n=_at(5), scale=0.125, dZ=_at(9),
             dST=_at(10), B=2, H=3, T=2000, d=64, dQ=_at(11), dK=_at(12), Z=_at(6), S=_at(7), ws=_at(8), wsn=1 << 30)
    a.update(kw)
    return lib.ttt_linear_attn_bwd(a["Q"], a["K"], a["V"], a["dt"], a["g"], a["S0"], a["n"], a["scale"], a["dZ"],
                                   a["dST"], a["B"], a["H"], a["T"], a["d"], a["dQ"], a["dK"], a["Z"], a["S"], a["ws"],
                                   a["wsn"], None)


@pytest.mark.parametrize("fn", [fwd, bwd])
def test_sequences_refuse_on_the_host(lib, fn):
    n0 = lib.ttt_launch_count()
    assert fn(lib, dt=7) == L.TTT_ERR_ARG
    assert fn(lib, B=-1) == L.TTT_ERR_ARG
    assert fn(lib, H=-1) == L.TTT_ERR_ARG
    assert fn(lib, T=-1) == L.TTT_ERR_ARG
    assert fn(lib, d=0) == L.TTT_ERR_ARG
    assert fn(lib, scale=float("nan")) == L.TTT_ERR_ARG
    assert fn(lib, scale=float("inf")) == L.TTT_ERR_ARG
    assert fn(lib, d=128) == L.TTT_ERR_UNSUPPORTED
    assert fn(lib, B=1 << 20, H=1 << 10, T=1 << 10) == L.TTT_ERR_UNSUPPORTED
    assert fn(lib, B=1 << 15, H=1 << 15) == L.TTT_ERR_UNSUPPORTED
    for p in ("Q", "K", "V", "g", "Z"):
        assert fn(lib, **{p: None}) == L.TTT_ERR_ARG, p
    for p in ("Q", "K", "V", "g", "Z", "S0", "n", "S", "ws"):
        assert fn(lib, **{p: _at(20) + 4}) == L.TTT_ERR_ALIGN, p
    assert fn(lib, Z=_at(2) + 64) == L.TTT_ERR_ARG            # over V
    assert fn(lib, S=_at(4)) == L.TTT_ERR_ARG                 # the states in place
    assert fn(lib, ws=_at(6) + 1024) == L.TTT_ERR_ARG         # workspace over an output
    assert fn(lib, ws=None) == L.TTT_ERR_ARG                  # few units: the sequences are cut
    need = lib.ttt_linear_attn_workspace_bytes(2, 3, 2000, 64, int(fn is bwd))
    assert need > 0 and fn(lib, wsn=need - 1) == L.TTT_ERR_ARG
    assert fn(lib, B=0) == L.TTT_OK and fn(lib, H=0) == L.TTT_OK
    assert lib.ttt_launch_count() == n0, "a refused call launched a kernel"


def test_backward_refuses_its_own_arguments(lib):
    for p in ("dZ", "dQ", "dK"):
        assert bwd(lib, **{p: None}) == L.TTT_ERR_ARG, p
    assert bwd(lib, dST=_at(20) + 8) == L.TTT_ERR_ALIGN
    assert bwd(lib, dQ=_at(9)) == L.TTT_ERR_ARG
    assert bwd(lib, dQ=_at(12)) == L.TTT_ERR_ARG


def test_workspace_rule(lib):
    size = lib.ttt_linear_attn_workspace_bytes
    state, counters = 64 * 64 * 4, 608  # a state; the CTAs' counters (1 + 148 ints, rounded to 16 bytes)
    # One chunk of 128 tokens, or nothing: nothing to share or cut; nor with whole rounds of units on 148 SMs
    # (two at a time for the CUDA-core kernel).
    for B, H, T in ((16, 12, 128), (1, 1, 128), (0, 3, 4096), (3, 3, 0), (296, 1, 1 << 20), (37, 16, 300)):
        assert size(B, H, T, 64, 0) == 0 and size(B, H, T, 64, 1) == 0, (B, H, T)
    # More units (of all passes) than SMs: 148 states to hand on and the counters (or, for the CUDA-core
    # kernel, the segments of a last round, if more).
    for B, H, T in ((16, 12, 2048), (149, 1, 129), (16, 32, 8192)):
        assert size(B, H, T, 64, 0) >= 148 * state + counters, (B, H, T)
    for B, H, T in ((16, 12, 2048), (50, 1, 129), (16, 32, 8192)):
        assert size(B, H, T, 64, 1) >= 148 * state + counters, (B, H, T)
    # Fewer: none, or two to 64 segments a unit.
    for B, H, T in ((1, 1, 2000), (1, 32, 32768), (1, 1, 1 << 30), (6, 8, 1999), (1, 12, 4096)):
        n, odd = divmod(size(B, H, T, 64, 0), B * H * state)
        assert odd == 0 and 2 <= n <= 64, (B, H, T, n)
        n, odd = divmod(size(B, H, T, 64, 1), 2 * B * H * state)
        assert odd == 0 and n <= 64 and n != 1, (B, H, T, n)
    assert size(-1, 2, 3, 64, 0) == 0 and size(1, 2, 3000, 32, 0) == 0


def decode(lib, **kw):
    a = dict(q=_at(0), k=_at(1), v=_at(2), dt=L.TTT_F32, g=_at(3), scale=1.0, S=_at(4), p=_at(5), f=_at(6), rot=64,
             il=0, m=1.0, B=2, H=3, d=64, z=_at(7))
    a.update(kw)
    return lib.ttt_linear_attn_decode(a["q"], a["k"], a["v"], a["dt"], a["g"], a["scale"], a["S"], a["p"], a["f"],
                                      a["rot"], a["il"], a["m"], a["B"], a["H"], a["d"], a["z"], None)


def test_decode_refuses_on_the_host(lib):
    n0 = lib.ttt_launch_count()
    for bad in (dict(dt=2), dict(B=-1), dict(d=-64), dict(scale=float("inf")), dict(rot=65), dict(rot=66), dict(rot=-2),
                dict(il=2), dict(m=float("nan")), dict(q=None), dict(g=None), dict(S=None), dict(z=None), dict(p=None),
                dict(f=None), dict(z=_at(4)), dict(S=_at(1)), dict(z=_at(0))):
        assert decode(lib, **bad) == L.TTT_ERR_ARG, bad
    assert decode(lib, d=32, rot=32) == L.TTT_ERR_UNSUPPORTED
    for p in ("q", "k", "v", "g", "S", "z", "p", "f"):
        assert decode(lib, **{p: _at(20) + 8}) == L.TTT_ERR_ALIGN, p
    assert decode(lib, B=0) == L.TTT_OK
    assert lib.ttt_launch_count() == n0


def rope(lib, **kw):
    a = dict(Q=_at(0), K=_at(1), dt=L.TTT_BF16, p=_at(2), first=0, f=_at(3), rot=64, il=0, m=1.0, inv=0, B=2, Hq=4, Hk=2,
             T=5, d=64, sq=None, sk=None, Qo=_at(4), Ko=_at(5))
    a.update(kw)
    s = [None if x is None else (ctypes.c_longlong * 3)(*x) for x in (a["sq"], a["sk"])]
    return lib.ttt_rope(a["Q"], a["K"], a["dt"], a["p"], a["first"], a["f"], a["rot"], a["il"], a["m"], a["inv"], a["B"],
                        a["Hq"], a["Hk"], a["T"], a["d"], s[0], s[1], a["Qo"], a["Ko"], None)


def test_rope_refuses_on_the_host(lib):
    n0 = lib.ttt_launch_count()
    for bad in (dict(dt=3), dict(B=-1), dict(Hq=-1), dict(T=-2), dict(d=0), dict(rot=3), dict(rot=66), dict(il=-1),
                dict(inv=2), dict(m=float("inf")), dict(Q=None), dict(K=None), dict(f=None), dict(Qo=None), dict(Ko=None),
                dict(Qo=_at(1)), dict(Ko=_at(4)), dict(Qo=_at(0)), dict(sq=(-64, 64, 64)),
                dict(sq=(1 << 60, 1 << 60, 64)), dict(p=None, first=0x7fffffff),
                # The K rows that the strides reach lie under Q's output.
                dict(sk=(64, 64, (STEP * 3 // 2) // 4))):
        assert rope(lib, **bad) == L.TTT_ERR_ARG, bad
    assert rope(lib, d=128) == L.TTT_ERR_UNSUPPORTED
    assert rope(lib, B=1 << 20, T=1 << 20) == L.TTT_ERR_UNSUPPORTED
    for p in ("Q", "K", "p", "f", "Qo", "Ko"):
        assert rope(lib, **{p: _at(20) + 8}) == L.TTT_ERR_ALIGN, p
    assert rope(lib, sq=(64 * 20, 64, 65)) == L.TTT_ERR_ALIGN
    for empty in (dict(B=0), dict(T=0), dict(Hq=0, Hk=0)):
        assert rope(lib, **empty) == L.TTT_OK
    assert lib.ttt_launch_count() == n0


# ---- the binding ------------------------------------------------------------------------

class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name not in L.SIGNATURES:
            raise AttributeError(name)

        def call(*args):
            assert len(args) == len(L.SIGNATURES[name][1]), (name, len(args))
            self.calls.append((name, args))
            return 4096 if name.endswith("workspace_bytes") else L.TTT_OK
        return call

    def names(self):
        return [n for n, _ in self.calls if not n.endswith("workspace_bytes")]

    def args(self, name):
        return [a for n, a in self.calls if n == name][-1]


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder()

    def any_device(t, name, dtype=None):
        if not isinstance(t, torch.Tensor) or (dtype is not None and t.dtype != dtype):
            raise TypeError(name)
        if not t.is_contiguous():
            raise ValueError(name)
        return t

    monkeypatch.setattr(ttt, "_cuda", any_device)
    monkeypatch.setattr(ttt, "_rope_rows", lambda t, name: t)
    monkeypatch.setattr(L, "load", lambda *a, **k: r)
    monkeypatch.setattr(ttt, "_stream", lambda s, d: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    return r


B, H, T, d = 2, 3, 32, 64


def _qkv(dt=torch.bfloat16):
    return [torch.zeros(B, H, T, d, dtype=dt) for _ in range(3)]


def test_binding_passes_every_argument(rec):
    Q, K, V = _qkv()
    g, S0, n = torch.zeros(H), torch.zeros(B, H, d, d), torch.zeros(B, dtype=torch.int32)
    Z, S = ttt.ttt_linear_attn_fwd(Q, K, V, g, scale=0.5, S0=S0, lengths=n)
    assert Z.dtype == torch.bfloat16 and Z.shape == Q.shape and S.dtype == torch.float32 and S.shape == S0.shape
    a = rec.args("ttt_linear_attn_fwd")
    assert a[3] == L.TTT_BF16 and a[4:8] == (g.data_ptr(), S0.data_ptr(), n.data_ptr(), 0.5)
    assert a[8:12] == (B, H, T, d) and a[12] == Z.data_ptr() and a[13] == S.data_ptr() and a[15] == 4096
    ttt.ttt_linear_attn_fwd(*_qkv(torch.float32), g)
    a = rec.args("ttt_linear_attn_fwd")
    assert a[3] == L.TTT_F32 and a[5] is None and a[6] is None and a[7] == 0.125
    out = ttt.ttt_linear_attn_bwd(Q, K, V, g, torch.zeros_like(Q), dS_T=S0)
    assert sorted(out) == ["dK", "dQ", "dS0", "dV"] and out["dK"].dtype == torch.bfloat16
    assert out["dS0"].dtype == torch.float32
    assert rec.args("ttt_linear_attn_bwd")[9:14] == (S0.data_ptr(), B, H, T, d)
    plan = ttt.Rope(torch.zeros(20), 1.5, True)
    pos = torch.zeros(B, dtype=torch.int32)
    q = torch.zeros(B, H, d)
    z = ttt.ttt_linear_attn_decode(q, q, q, g, S0, rope=plan, positions=pos)
    a = rec.args("ttt_linear_attn_decode")
    assert a[7:15] == (pos.data_ptr(), plan.inv_freq.data_ptr(), 40, 1, 1.5, B, H, d) and a[15] == z.data_ptr()
    ttt.ttt_linear_attn_decode(q, q, q, g, S0)
    assert rec.args("ttt_linear_attn_decode")[7:12] == (None, None, 0, 0, 1.0)


def test_a_rope_argument_turns_before_and_turns_back(rec):
    Q, K, V = _qkv()
    plan, pos = ttt.Rope(torch.zeros(32)), torch.zeros(B, T, dtype=torch.int32)
    ttt.ttt_linear_attn_fwd(Q, K, V, torch.zeros(H), rope=plan, positions=pos)
    assert rec.names() == ["ttt_rope", "ttt_linear_attn_fwd"]
    assert rec.args("ttt_rope")[3] == pos.data_ptr() and rec.args("ttt_rope")[9] == 0
    rec.calls.clear()
    ttt.ttt_linear_attn_bwd(Q, K, V, torch.zeros(H), torch.zeros_like(Q), rope=plan)
    assert rec.names() == ["ttt_rope", "ttt_linear_attn_bwd", "ttt_rope"]
    assert rec.args("ttt_rope")[3] is None and rec.args("ttt_rope")[9] == 1


def test_rope_binding_takes_strided_rows(rec):
    joint = torch.zeros(B, T, 2, H, d)
    Q, K = joint[:, :, 0].transpose(1, 2), joint[:, :, 1, :2].transpose(1, 2)
    Qo, Ko = ttt.ttt_rope(Q, K, ttt.Rope(torch.zeros(16)), first_position=5)
    assert Qo.is_contiguous() and Qo.shape == Q.shape and Ko.shape == (B, 2, T, d)
    a = rec.args("ttt_rope")
    assert list(a[15]) == list(Q.stride()[:3]) and list(a[16]) == list(K.stride()[:3])
    assert a[4] == 5 and a[6] == 32 and a[10:15] == (B, H, 2, T, d)
    Qo, Ko = ttt.ttt_rope(Q, None, ttt.Rope(torch.zeros(16)))
    assert Ko is None and rec.args("ttt_rope")[12] == 0


@pytest.mark.parametrize("case", ["decay", "S0", "lengths", "lengths type", "dZ", "dZ type", "positions alone", "Z", "mixed types",
                                  "K rows", "positions", "decode S", "decode rope alone", "K_out", "inv_freq", "strided V"])
def test_binding_refuses_before_any_call(rec, case):
    Q, K, V = _qkv()
    g = torch.zeros(H)
    q = torch.zeros(B, H, d)
    plan = ttt.Rope(torch.zeros(32))
    with pytest.raises((ValueError, TypeError)):
        if case == "decay":
            ttt.ttt_linear_attn_fwd(Q, K, V, torch.zeros(H + 1))
        elif case == "S0":
            ttt.ttt_linear_attn_fwd(Q, K, V, g, S0=torch.zeros(H, d, d))
        elif case == "lengths":
            ttt.ttt_linear_attn_fwd(Q, K, V, g, lengths=torch.zeros(B + 1, dtype=torch.int32))
        elif case == "lengths type":
            ttt.ttt_linear_attn_fwd(Q, K, V, g, lengths=torch.zeros(B, dtype=torch.int64))
        elif case == "dZ":
            ttt.ttt_linear_attn_bwd(Q, K, V, g, torch.zeros(B, H, T - 1, d, dtype=Q.dtype))
        elif case == "dZ type":
            ttt.ttt_linear_attn_bwd(Q, K, V, g, torch.zeros(B, H, T, d))
        elif case == "positions alone":
            ttt.ttt_linear_attn_fwd(Q, K, V, g, positions=torch.zeros(B, T, dtype=torch.int32))
        elif case == "Z":
            ttt.ttt_linear_attn_fwd(Q, K, V, g, Z=torch.zeros(B, H, T, d))
        elif case == "mixed types":
            ttt.ttt_linear_attn_fwd(Q, K.float(), V, g)
        elif case == "K rows":
            ttt.ttt_rope(Q, K[:, :, 1:], plan)
        elif case == "positions":
            ttt.ttt_rope(Q, K, plan, positions=torch.zeros(B, dtype=torch.int32))
        elif case == "decode S":
            ttt.ttt_linear_attn_decode(q, q, q, g, torch.zeros(H, d, d))
        elif case == "decode rope alone":
            ttt.ttt_linear_attn_decode(q, q, q, g, torch.zeros(B, H, d, d), rope=plan)
        elif case == "K_out":
            ttt.ttt_rope(Q, None, plan, K_out=Q)
        elif case == "inv_freq":
            ttt.Rope(torch.zeros(4, 8))
        else:
            ttt.ttt_linear_attn_fwd(Q, K, torch.zeros(B, T, H, d, dtype=Q.dtype).transpose(1, 2), g)
    assert rec.names() == []


def test_tensors_off_the_gpu_are_refused():
    Q, K, V = _qkv()
    with pytest.raises(ValueError, match="CUDA"):
        ttt.ttt_linear_attn_fwd(Q, K, V, torch.zeros(H))
    with pytest.raises(ValueError, match="CUDA"):
        ttt.Rope(torch.zeros(4))


# ---- rotary plans -----------------------------------------------------------------------

def test_rope_frequencies():
    f, m = ttt.rope_frequencies(64)
    i = np.arange(32)
    assert m == 1.0 and f.dtype == torch.float32
    assert np.allclose(f.numpy(), 10000.0 ** (-i / 32.0), rtol=2 ** -23)
    lin, m = ttt.rope_frequencies(64, scaling="linear", factor=4.0)
    assert m == 1.0 and np.allclose(lin.numpy(), f.numpy() / 4, rtol=2 ** -23)
    ntk, m = ttt.rope_frequencies(64, scaling="ntk", factor=4.0)
    assert m == 1.0 and ntk[0] == 1.0 and math.isclose(ntk[-1], float(f[-1]) / 4, rel_tol=1e-6)
    yarn, m = ttt.rope_frequencies(64, scaling="yarn", factor=4.0, original_length=4096)
    assert math.isclose(m, 0.1 * math.log(4.0) + 1.0)
    turns = 4096 * f.numpy() / (2 * math.pi)
    assert np.allclose(yarn.numpy()[turns > 40], f.numpy()[turns > 40], rtol=2 ** -22)
    assert np.allclose(yarn.numpy()[turns < 0.8], f.numpy()[turns < 0.8] / 4, rtol=2 ** -22)
    ratio = yarn.numpy() / f.numpy()
    assert np.all(np.diff(ratio) <= 1e-6) and np.all(ratio >= 0.25 - 1e-6)
    for bad in (dict(rotary=3), dict(rotary=0), dict(rotary=64, base=1.0), dict(rotary=64, factor=0.5),
                dict(rotary=64, scaling="no"), dict(rotary=64, scaling="yarn", factor=2.0),
                dict(rotary=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            ttt.rope_frequencies(**bad)
