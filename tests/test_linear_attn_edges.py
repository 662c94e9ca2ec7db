"""Linear attention and rotary positions: empty and one-sided calls, heads that share rows, calls in graphs and on a
workspace of the caller's, and tensors whose offsets pass 32 bits."""
import numpy as np
import pytest
import torch

import test_sequence_modeling_b200 as ttt
from linear_attn_helpers import D, TYPES, bounds, check, device, make, reference
from test_linear_attn_plans import PLANS, run_bwd, run_fwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("plan", list(PLANS))
def test_a_batch_of_empty_sequences(plan, dtype):
    """Nothing is read: zeros for the rows, the states as they came."""
    B, H, T = PLANS[plan][:3]
    x = device(make(B, H, T, dtype, "slow", True, lengths=[0] * B, back=True), dtype)
    for n in ("Q", "K", "V", "dZ"):
        x[n].fill_(float("nan"))
    got = {**run_fwd(x), **run_bwd(x)}
    for n in ("Z", "dQ", "dK", "dV"):
        assert not got[n].any(), n
    assert torch.equal(got["S"], x["S0"]) and torch.equal(got["dS0"], x["dS_T"])
    x.update(S0=None, dS_T=None)
    got = {**run_fwd(x), **run_bwd(x)}
    assert not got["S"].any() and not got["dS0"].any()
    assert ttt.last_device_status() == 0


@pytest.mark.parametrize("B,H,T", [(0, 3, 5), (2, 0, 5), (2, 3, 0)])
def test_sizes_of_zero(B, H, T):
    x = {n: torch.empty(B, H, T, D, device="cuda", dtype=torch.bfloat16) for n in ("Q", "K", "V", "dZ")}
    x.update(log_decay=torch.zeros(H, device="cuda"), scale=1.0, S0=None, dS_T=None, lengths=None)
    got = {**run_fwd(x), **run_bwd(x)}
    assert got["Z"].shape == (B, H, T, D) and got["S"].shape == (B, H, D, D) and not got["S"].any()
    Qo, Ko = ttt.ttt_rope(x["Q"], x["K"], ttt.Rope.build(64))
    assert Qo.shape == Ko.shape == (B, H, T, D)
    if T:
        z = ttt.ttt_linear_attn_decode(*(x[n][:, :, 0].contiguous() for n in "QKV"), x["log_decay"], got["S"])
        assert z.shape == (B, H, D)
    assert ttt.last_device_status() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_of_heads_that_share_rows(interleaved):
    """Expanded inputs: a stride of zero over heads, and over sequences."""
    plan = ttt.Rope.build(48, interleaved=interleaved)
    one = torch.randn(3, 1, 40, D, device="cuda").bfloat16()
    row = torch.randn(1, 5, 40, D, device="cuda").bfloat16()
    pos = torch.arange(120, dtype=torch.int32, device="cuda").view(3, 40)
    Qo, Ko = ttt.ttt_rope(row.expand(3, 5, 40, D), one.expand(3, 4, 40, D), plan, positions=pos)
    Qw, Kw = ttt.ttt_rope(row.expand(3, 5, 40, D).contiguous(), one.expand(3, 4, 40, D).contiguous(), plan, positions=pos)
    assert torch.equal(Qo, Qw) and torch.equal(Ko, Kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_captured_and_replayed(dtype):
    """A graph of one token, replayed for each: inputs and positions written in place, the state carried on."""
    B, H, n = 3, 5, 6
    c = make(B, H, n, dtype, "slow", True)
    x, plan = device(c, dtype), ttt.Rope.build(64)
    q, k, v = (x[m][:, :, 0].contiguous() for m in "QKV")
    at = torch.zeros(B, dtype=torch.int32, device="cuda")
    S, z = x["S0"].clone(), torch.empty_like(q)
    want_S = x["S0"].clone()
    want = []
    for t in range(n):
        want.append(ttt.ttt_linear_attn_decode(*(x[m][:, :, t].contiguous() for m in "QKV"), x["log_decay"], want_S, rope=plan,
                                               positions=torch.full((B,), 100 + t, dtype=torch.int32, device="cuda")))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ttt.ttt_linear_attn_decode(q, k, v, x["log_decay"], S, rope=plan, positions=at, z=z)
    for t in range(n):
        for to, m in ((q, "Q"), (k, "K"), (v, "V")):
            to.copy_(x[m][:, :, t])
        at.fill_(100 + t)
        graph.replay()
        assert torch.equal(z, want[t]), t
    assert torch.equal(S, want_S)


@pytest.mark.parametrize("plan", ["cut", "shared, ragged"])
def test_one_workspace_for_calls_in_turn(plan):
    """Forward and backward, eager and in two graphs, on one uncleared workspace on one stream."""
    B, H, T = PLANS[plan][:3]
    x = device(make(B, H, T, "bf16", "slow", True, back=True), "bf16")
    want = {**run_fwd(x), **run_bwd(x)}
    need = max(ttt.linear_attn_workspace_bytes((B, H, T, D), b) for b in (False, True))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g, run in zip(graphs, (run_fwd, run_bwd)):
        with torch.cuda.graph(g):
            outs.append(run(x, workspace=ws))
    for _ in range(3):
        got = {**run_fwd(x, workspace=ws), **run_bwd(x, workspace=ws)}
        for g in graphs:
            g.replay()
        for results in (got, {**outs[0], **outs[1]}):
            for n in want:
                assert torch.equal(results[n], want[n]), n
    assert ttt.last_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_state_in_two_steps_is_the_same_on_every_plan(dtype):
    """A cut call continues a whole one and is continued by a shared one's form: against the oracle at the end."""
    c = make(2, 2, 1700, dtype, "slow", True)
    x = device(c, dtype)
    S, Z = x["S0"], []
    for lo, hi in ((0, 1500), (1500, 1501), (1501, 1700)):
        part = [x[n][:, :, lo:hi].contiguous() for n in "QKV"]
        z, S = ttt.ttt_linear_attn_fwd(*part, x["log_decay"], scale=x["scale"], S0=S)
        Z.append(z)
    ref = reference(c, "fwd")
    check({"Z": torch.cat(Z, 2), "S": S}, ref, bounds(c, "fwd", dtype, ref))


# ---- beyond 32 bits -----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_beyond_32_bits(dtype):
    """922 x 37 units of 1024 tokens: 2.2e9 values a tensor.  What lies behind the 2^31st value is what a call on
    that part alone gives, bit by bit: 8 x 37 units, which are whole in either call, and the last 2 x 37, which
    the CUDA-core kernel cuts alike in both."""
    B, H, T = 922, 37, 1024
    assert 911 * H * T * D > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(5)
    x = {n: torch.randn(B, H, T, D, device="cuda", dtype=TYPES[dtype], generator=g) for n in ("Q", "K", "V", "dZ")}
    x.update(log_decay=torch.linspace(-0.2, 0.0, H, device="cuda"), scale=0.125, S0=None, dS_T=None,
             lengths=torch.randint(0, T + 1, (B,), device="cuda", generator=g).int())
    for run in (run_fwd, run_bwd):
        got = run(x)
        for lo, hi in ((911, 919), (920, 922)):
            part = {n: t[lo:hi] if n in ("Q", "K", "V", "dZ") else t for n, t in x.items()}
            part["lengths"] = x["lengths"][lo:hi].clone()
            want = run(part)
            for n in want:
                assert torch.equal(got[n][lo:hi], want[n]), (n, lo)
        del got, want, part
    plan = ttt.Rope.build(64)
    rows = x["Q"].view(B, T, H, D).transpose(1, 2)  # as out of a projection
    got, _ = ttt.ttt_rope(rows, None, plan, first_position=7)
    want, _ = ttt.ttt_rope(rows[911:], None, plan, first_position=7)
    assert torch.equal(got[911:], want)
    assert ttt.last_device_status() == 0


def test_decode_offsets_beyond_32_bits():
    B, H = 16400, 32
    assert B * H * D * D > 2 ** 31
    q, k, v = (torch.randn(B, H, D, device="cuda").bfloat16() for _ in range(3))
    S = torch.randn(B, H, D, D, device="cuda")
    tail = S[-3:].clone()
    decay = torch.linspace(-0.2, 0.0, H, device="cuda")
    z = ttt.ttt_linear_attn_decode(q, k, v, decay, S)
    want = ttt.ttt_linear_attn_decode(*(t[-3:].clone() for t in (q, k, v)), decay, tail)
    assert torch.equal(z[-3:], want) and torch.equal(S[-3:], tail)
