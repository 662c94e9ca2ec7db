"""Linear attention however its work is dealt out: whole units, sequences cut into segments (a pass for the
segments' states, a scan, the outputs) and chunks shared by all SMs (states handed on), each against the fp64
oracle over every kind of decay, with empty segments and sequences, between canaries, without the optional
states, and bit by bit on whole numbers that every rounding on the way holds exactly."""
import numpy as np
import pytest
import torch

import test_sequence_modeling_b200 as ttt
from linear_attn_helpers import D, DECAYS, TYPES, bounds, check, device, make, reference
from test_sequence_modeling_b200 import _lib as L

pytestmark = pytest.mark.gpu

# B, H, T and, for bf16, the launches of a forward and of a backward: 3 where the sequences are cut.
PLANS = {"whole": (1, 3, 70, 1, 1), "cut": (2, 2, 1500, 3, 3), "cut, segments of two chunks": (5, 2, 1900, 3, 3),
         "shared": (5, 30, 130, 1, 1), "shared, ragged": (6, 25, 200, 1, 1), "backward shared": (6, 9, 300, 1, 1)}


def run_fwd(x, **kw):
    Z, S = ttt.ttt_linear_attn_fwd(x["Q"], x["K"], x["V"], x["log_decay"], scale=x["scale"], S0=x["S0"],
                                   lengths=x["lengths"], **kw)
    return {"Z": Z, "S": S}


def run_bwd(x, **kw):
    return ttt.ttt_linear_attn_bwd(x["Q"], x["K"], x["V"], x["log_decay"], x["dZ"], scale=x["scale"], S0=x["S0"],
                                   dS_T=x["dS_T"], lengths=x["lengths"], **kw)


RUNS = (("fwd", run_fwd), ("bwd", run_bwd))


def _ends(B, T):
    """Full, empty, one token, a segment's edge and ragged ones."""
    rng = np.random.default_rng(6)
    n = rng.integers(0, T + 1, B)
    some = [T, 0, 1, min(T, 128), min(T, 257), T - 1]
    n[:min(B, 6)] = some[:B]
    return n


@pytest.mark.parametrize("plan", list(PLANS))
def test_launches(plan):
    B, H, T, fwd, bwd = PLANS[plan]
    x = device(make(B, H, T, "bf16", back=True), "bf16")
    for run, want in ((run_fwd, fwd), (run_bwd, bwd)):
        before = ttt.launch_count()
        run(x)
        assert ttt.launch_count() - before == want


def test_a_cut_that_gains_nothing_is_not_taken():
    """32 units of 64 chunks: the forward is cut (64 us against 105), the backward, 117 us whole and 125 in
    three, is not."""
    x = device(make(1, 32, 8192, "bf16", back=True), "bf16")
    for run, want in ((run_fwd, 3), (run_bwd, 1)):
        before = ttt.launch_count()
        run(x)
        assert ttt.launch_count() - before == want


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", list(DECAYS))
@pytest.mark.parametrize("plan", [p for p in PLANS if p != "whole"])
def test_decays(plan, decay, dtype):
    B, H, T = PLANS[plan][:3]
    for lengths in (None, _ends(B, T)):
        c = make(B, H, T, dtype, decay, True, lengths=lengths, back=True)
        x = device(c, dtype)
        for fn, run in RUNS:
            ref = reference(c, fn)
            check(run(x), ref, bounds(c, fn, dtype, ref))
    assert ttt.last_device_status() == 0


@pytest.mark.parametrize("size", [(1, 1, 0), (2, 3, 1), (1, 2, 63), (2, 1, 64), (1, 2, 129), (2, 2, 1500), (50, 3, 130),
                                  (100, 3, 200)], ids=str)
@pytest.mark.parametrize("padded", [False, True])
def test_bf16_on_the_cuda_cores(size, padded):
    B, H, T = size
    c = make(*size, "bf16", "slow", True, lengths=_ends(B, T) if padded and T else None, back=True)
    x = device(c, "bf16")
    prev = ttt.set_path(ttt.TTT_PATH_SIMT)
    try:
        for fn, run in RUNS:
            ref = reference(c, fn)
            check(run(x), ref, bounds(c, fn, "bf16", ref))
    finally:
        ttt.set_path(prev)


@pytest.mark.parametrize("plan", list(PLANS))
def test_tensor_core_path_setting(plan):
    """TTT_PATH_TC runs what AUTO runs for bf16 and refuses fp32 before any launch."""
    B, H, T = PLANS[plan][:3]
    c = make(B, H, T, "bf16", "slow", True, back=True)
    x = device(c, "bf16")
    want = {**run_fwd(x), **run_bwd(x)}
    prev = ttt.set_path(ttt.TTT_PATH_TC)
    try:
        got = {**run_fwd(x), **run_bwd(x)}
        before = ttt.launch_count()
        f = {n: t.float() if n in ("Q", "K", "V", "dZ") else t for n, t in x.items()}
        for run in (run_fwd, run_bwd):
            with pytest.raises(ttt.TTTError):
                run(f)
        assert ttt.launch_count() == before
    finally:
        ttt.set_path(prev)
    for n in want:
        assert torch.equal(got[n], want[n]), n


# ---- canaries ---------------------------------------------------------------------------

class Guarded:
    """Buffers inside larger ones whose rims have to keep what they hold."""
    PAD = 4096

    def __init__(self):
        self.rims = []

    def __call__(self, shape, dtype, fill=7):
        n = int(np.prod(shape))
        whole = torch.full((n + 2 * self.PAD,), fill, dtype=dtype, device="cuda")
        self.rims.append((whole, n, fill))
        return whole[self.PAD:self.PAD + n].view(*shape)

    def intact(self):
        torch.cuda.synchronize()
        return all(bool((w[:self.PAD] == f).all()) and bool((w[self.PAD + n:] == f).all()) for w, n, f in self.rims)


def _abi(x, fn, outs, states, ws):
    """The C entry points themselves: outputs where the test wants them, states left out as NULL."""
    lib = L.load()
    B, H, T, d = x["Q"].shape
    p = {n: (t.data_ptr() if isinstance(t, torch.Tensor) else None) for n, t in {**x, **outs}.items()}
    dt = L.TTT_BF16 if x["Q"].dtype == torch.bfloat16 else L.TTT_F32
    stream = torch.cuda.current_stream().cuda_stream
    S0 = p["S0"] if states else None
    if fn == "fwd":
        return lib.ttt_linear_attn_fwd(p["Q"], p["K"], p["V"], dt, p["log_decay"], S0, p["lengths"], x["scale"], B, H, T,
                                       d, p["Z"], p.get("S"), ws.data_ptr(), ws.numel(), stream)
    return lib.ttt_linear_attn_bwd(p["Q"], p["K"], p["V"], dt, p["log_decay"], S0, p["lengths"], x["scale"], p["dZ"],
                                   p["dS_T"] if states else None, B, H, T, d, p["dQ"], p["dK"], p["dV"], p.get("dS0"),
                                   ws.data_ptr(), ws.numel(), stream)


NAMES = {"fwd": ("Z", "S"), "bwd": ("dQ", "dK", "dV", "dS0")}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("plan", list(PLANS))
@pytest.mark.parametrize("padded", [False, True])
def test_every_output_and_the_workspace_between_canaries(plan, dtype, padded):
    B, H, T = PLANS[plan][:3]
    x = device(make(B, H, T, dtype, "slow", True, lengths=_ends(B, T) if padded else None, back=True), dtype)
    for fn, run in RUNS:
        g = Guarded()
        outs = {n: g((B, H, D, D) if n in ("S", "dS0") else (B, H, T, D),
                     torch.float32 if n in ("S", "dS0") else TYPES[dtype]) for n in NAMES[fn]}
        need = ttt.linear_attn_workspace_bytes((B, H, T, D), fn == "bwd")
        ws = g((max(need, 1),), torch.uint8, 5)
        assert _abi(x, fn, outs, True, ws) == L.TTT_OK
        assert g.intact(), fn
        want = run(x)
        for n in want:
            assert torch.equal(outs[n], want[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("plan", list(PLANS))
def test_states_may_be_left_out(plan, dtype):
    """S_out and dS0 NULL with and without S0 and dS_T: the other outputs are those with all of them."""
    B, H, T = PLANS[plan][:3]
    x = device(make(B, H, T, dtype, "slow", True, lengths=_ends(B, T), back=True), dtype)
    for states in (True, False):
        given = x if states else {**x, "S0": None, "dS_T": None}
        for fn, run in RUNS:
            want = run(given)
            outs = {n: torch.empty_like(x["Q"]) for n in NAMES[fn] if n not in ("S", "dS0")}
            need = ttt.linear_attn_workspace_bytes((B, H, T, D), fn == "bwd")
            ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
            assert _abi(x, fn, outs, states, ws) == L.TTT_OK
            torch.cuda.synchronize()
            for n in outs:
                assert torch.equal(outs[n], want[n]), (n, states)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_and_rope_between_canaries(dtype):
    for B, H in ((1, 1), (3, 5), (37, 4)):
        g = Guarded()
        q, k, v = (torch.randn(B, H, D, device="cuda").to(TYPES[dtype]) for _ in range(3))
        S, z = g((B, H, D, D), torch.float32), g((B, H, D), TYPES[dtype])
        S.normal_()
        S1 = S.clone()
        pos = torch.arange(B, dtype=torch.int32, device="cuda")
        decay = torch.full((H,), -0.1, device="cuda")
        plan = ttt.Rope.build(40, interleaved=True)
        ttt.ttt_linear_attn_decode(q, k, v, decay, S, rope=plan, positions=pos, z=z)
        assert g.intact()
        assert torch.equal(z, ttt.ttt_linear_attn_decode(q, k, v, decay, S1, rope=plan, positions=pos))
        assert torch.equal(S, S1)
    for rotary in (64, 40, 14, 0):
        for interleaved in (False, True):
            for B, Hq, Hk, T in ((1, 1, 1, 1), (3, 5, 2, 21), (2, 33, 1, 130)):
                g = Guarded()
                Q, K = (torch.randn(B, h, T, D, device="cuda").to(TYPES[dtype]) for h in (Hq, Hk))
                plan = ttt.Rope(torch.rand(rotary // 2, device="cuda"), interleaved=interleaved)
                Qo, Ko = g(Q.shape, Q.dtype), g(K.shape, K.dtype)
                ttt.ttt_rope(Q, K, plan, first_position=3, Q_out=Qo, K_out=Ko)
                assert g.intact()
                for got, want in zip((Qo, Ko), ttt.ttt_rope(Q, K, plan, first_position=3)):
                    assert torch.equal(got, want)


# ---- whole numbers ------------------------------------------------------------------------

def _onehot(rng, B, H, T, signed):
    at = torch.from_numpy(rng.integers(0, D, (B, H, T))).cuda()
    sign = torch.from_numpy(rng.choice([-1, 1], (B, H, T)) if signed else np.ones((B, H, T), np.int64)).cuda()
    return at, sign


def _dense(hot, alive, dtype):
    at, sign = hot
    x = torch.zeros(*at.shape, D, dtype=dtype, device="cuda")
    return x.scatter_(3, at[..., None], (sign * alive)[..., None].to(dtype))


def _sums(x, y, w, alive, reverse):
    """sum over s <= t (reverse: s >= t) of (x_t . y_s) w_s for one-hot x, y, w: whole numbers, row by row."""
    W = _dense(w, alive, torch.int32)
    if reverse:
        W = W.flip(2)
    out = torch.zeros_like(W)
    for r in range(D):
        hit = torch.where(y[0] == r, y[1], 0).to(torch.int32)
        run = torch.cumsum(W * (hit.flip(2) if reverse else hit)[..., None], 2, dtype=torch.int32)
        run = run.flip(2) if reverse else run
        out += torch.where(((x[0] == r) & (alive > 0))[..., None], run * x[1][..., None].to(torch.int32), 0)
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(1, 9, 32768), (1, 3, 5000), (16, 12, 2048), (40, 5, 1000), (9, 1, 9000)], ids=str)
@pytest.mark.parametrize("padded", [False, True])
def test_whole_numbers_exactly(dtype, size, padded):
    """Undecayed sequences of one-hot rows: every product and sum is a whole number that bf16 holds exactly
    (<= 256, checked), so the results are equal bit by bit and one lost, doubled or misplaced token shows
    however long the sequence."""
    B, H, T = size
    rng = np.random.default_rng([3, B, H, T])
    lengths = torch.from_numpy(_ends(B, T).astype(np.int32)).cuda() if padded else None
    if padded and B == 1:
        lengths[0] = T - 77
    alive = torch.ones(B, H, T, dtype=torch.int64, device="cuda")
    if padded:
        alive *= torch.arange(T, device="cuda") < lengths.long()[:, None, None]
    hot = {n: _onehot(rng, B, H, T, signed=n in ("V", "dZ")) for n in ("Q", "K", "V", "dZ")}
    x = {n: _dense(h, torch.ones_like(alive), TYPES[dtype]) for n, h in hot.items()}
    x.update(log_decay=torch.zeros(H, device="cuda"), scale=1.0, S0=None, dS_T=None, lengths=lengths)
    q, k, v, dz = (hot[n] for n in ("Q", "K", "V", "dZ"))
    want = {"Z": _sums(q, k, v, alive, False), "dQ": _sums(dz, v, k, alive, False),
            "dK": _sums(v, dz, q, alive, True), "dV": _sums(k, q, dz, alive, True)}
    full = {n: _dense(h, alive, torch.float64) for n, h in hot.items()}
    want["S"] = full["K"].transpose(2, 3) @ full["V"]
    want["dS0"] = full["Q"].transpose(2, 3) @ full["dZ"]
    got = {**run_fwd(x), **run_bwd(x)}
    for n, w in want.items():
        assert 0 < w.abs().max() <= 256, n
        assert torch.equal(got[n].double(), w.double()), n
    assert ttt.last_device_status() == 0
