"""GPU parity of linear attention with a decay for each head (forward, backward, single-token
step) and of rotary positions with the fp64 oracle; bounds from counted roundings."""
import numpy as np
import pytest
import torch

import test_sequence_modeling_b200 as ttt
from linear_attn_helpers import D, DECAYS, TYPES, U, U32, bounds, check, device, make, reference
from oracle import linear_attn as O
from test_sequence_modeling_b200 import _lib as L

pytestmark = pytest.mark.gpu


def run_fwd(x, **kw):
    Z, S = ttt.ttt_linear_attn_fwd(x["Q"], x["K"], x["V"], x["log_decay"], scale=x["scale"], S0=x["S0"],
                                   lengths=x["lengths"], **kw)
    return {"Z": Z, "S": S}


def run_bwd(x, **kw):
    return ttt.ttt_linear_attn_bwd(x["Q"], x["K"], x["V"], x["log_decay"], x["dZ"], scale=x["scale"], S0=x["S0"],
                                   dS_T=x["dS_T"], lengths=x["lengths"], **kw)


# Lengths about every edge: a chunk of 64 or 128 tokens, a segment's least length (512), one token,
# none; few units (cut into segments) and many.
SIZES = [(1, 1, 0), (2, 3, 1), (1, 2, 2), (2, 2, 63), (1, 3, 64), (2, 1, 65), (1, 2, 127), (1, 2, 128), (2, 1, 129),
         (1, 1, 192), (1, 2, 300), (1, 1, 512), (1, 2, 513), (1, 1, 1100), (50, 3, 130)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(dtype, size):
    c = make(*size, dtype, "slow", state=True)
    ref = reference(c, "fwd")
    check(run_fwd(device(c, dtype)), ref, bounds(c, "fwd", dtype, ref))
    assert ttt.last_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(dtype, size):
    c = make(*size, dtype, "slow", state=True, back=True)
    ref = reference(c, "bwd")
    check(run_bwd(device(c, dtype)), ref, bounds(c, "bwd", dtype, ref))
    assert ttt.last_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", list(DECAYS))
@pytest.mark.parametrize("state", [False, True])
def test_decays(dtype, decay, state):
    c = make(2, 4, 700, dtype, decay, state, back=True, lengths=[700, 333])
    x = device(c, dtype)
    for fn, run in (("fwd", run_fwd), ("bwd", run_bwd)):
        ref = reference(c, fn)
        check(run(x), ref, bounds(c, fn, dtype, ref))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [70, 1300])
def test_ends_of_padded_sequences(dtype, T):
    """Rows behind the ends hold NaN and infinities and are not used; lengths outside [0, T] count
    as the nearer end; an empty sequence hands its state on."""
    lengths = [T, 0, 1, T - 1, T // 2 + 1, T + 5, -3]
    c = make(7, 2, T, dtype, "slow", True, lengths=lengths, back=True)
    x = device(c, dtype)
    for n in ("Q", "K", "V", "dZ"):
        for b, end in enumerate(lengths):
            x[n][b, :, min(max(end, 0), T):] = float("nan") if b % 2 else float("inf")
    for fn, run in (("fwd", run_fwd), ("bwd", run_bwd)):
        ref = reference(c, fn)
        got = run(x)
        check(got, ref, bounds(c, fn, dtype, ref))
        for n in got:
            if n in ("S", "dS0"):
                assert torch.equal(got[n][1], x["S0" if fn == "fwd" else "dS_T"][1])
            else:
                for b, end in enumerate(lengths):
                    assert not got[n][b, :, min(max(end, 0), T):].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_sequence_in_parts(dtype):
    """The state of one part continues the next: prompt, prompt, then single tokens."""
    c = make(2, 3, 150, dtype, "slope")
    x = device(c, dtype)
    ref = reference(c, "fwd")
    cuts = [0, 90, 140]
    S, Z = None, []
    for lo, hi in zip(cuts, cuts[1:]):
        part = [x[n][:, :, lo:hi].contiguous() for n in "QKV"]
        z, S = ttt.ttt_linear_attn_fwd(*part, x["log_decay"], scale=x["scale"], S0=S)
        Z.append(z)
    for t in range(140, 150):
        q, k, v = (x[n][:, :, t].contiguous() for n in "QKV")
        Z.append(ttt.ttt_linear_attn_decode(q, k, v, x["log_decay"], S, scale=x["scale"])[:, :, None])
    check({"Z": torch.cat(Z, 2), "S": S}, ref, bounds(c, "fwd", dtype, ref))


def test_gradient_is_the_difference():
    """fp32 calls on both sides: the loss is quadratic at most along one input, so the central
    difference is off by rounding alone: <= 2 U32 sum|dZ| A / h for the two losses."""
    c = make(1, 2, 40, "f32", "slope", True, back=True)
    x = device(c, "f32")
    grad = run_bwd(x)
    rng = np.random.default_rng(3)
    h = 0.25

    def loss():
        r = run_fwd(x)
        return float((r["Z"].double() * x["dZ"].double()).sum() + (r["S"].double() * x["dS_T"].double()).sum())

    ref = reference(c, "fwd")
    b = bounds(c, "fwd", "f32", ref)
    for n in ("Q", "K", "V", "S0"):
        way = torch.from_numpy(rng.integers(-1, 2, c[n].shape)).float().cuda()
        keep = x[n].clone()
        x[n] = keep + h * way
        up = loss()
        x[n] = keep - h * way
        down = loss()
        x[n] = keep
        # Inputs within 1 + h / |x| of the bound's: doubled for both sides, and again for them.
        off = 4 * ((b["Z"] * np.abs(c["dZ"])).sum() + (b["S"] * np.abs(c["dS_T"])).sum()) / (2 * h)
        off += float((grad["d" + n].double() * way.double()).abs().sum()) * 1000 * U32
        assert abs((up - down) / (2 * h) - float((grad["d" + n].double() * way.double()).sum())) <= off, n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rotary,interleaved", [(0, False), (64, False), (64, True), (40, False), (20, True), (2, False)])
def test_decode(dtype, rotary, interleaved):
    Bn, H = 3, 5
    c = make(Bn, H, 4, dtype, "slow", True)
    x = device(c, dtype)
    plan = ttt.Rope.build(rotary, interleaved=interleaved) if rotary else None
    pos = np.array([[0, 1, 2, 3], [7, 100000, 8, 2 ** 31 - 1], [-5, 4, -2 ** 31, 77]])
    ref_c = dict(c)
    if rotary:
        f = plan.inv_freq.double().cpu().numpy()
        ref_c["Q"], ref_c["K"] = (O.rope(c[n], pos, f, 1.0, interleaved) for n in "QK")
    S = x["S0"].clone()
    S_ref = c["S0"]
    for t in range(4):
        q, k, v = (x[n][:, :, t].contiguous() for n in "QKV")
        p = torch.from_numpy(pos[:, t].astype(np.int32)).cuda() if rotary else None
        z = ttt.ttt_linear_attn_decode(q, k, v, x["log_decay"], S, scale=x["scale"], rope=plan, positions=p)
        one = {n: ref_c[n][:, :, t:t + 1] for n in "QKV"}
        Z, S_ref = O.forward(one["Q"], one["K"], one["V"], c["log_decay"], c["scale"], S_ref)
        A, _ = O.forward(*(np.abs(one[n]) for n in "QKV"), c["log_decay"], c["scale"], np.abs(S_ref))
        # Four additions and four scalings of the state so far, gamma (4), the turn of q and of k: each
        # within 8 roundings of |x| + |partner|, at most 2^(1/2) 8 more, and the sum over 64 rows.
        bz = 130 * U32 * (A + 12) + U[dtype] * np.abs(Z)
        bS = 40 * U32 * (np.abs(S_ref) + 40)
        assert np.all(np.abs(z.double().cpu().numpy() - Z[:, :, 0]) <= bz[:, :, 0])
        assert np.all(np.abs(S.double().cpu().numpy() - S_ref) <= bS)


def test_decode_many_units_are_each_their_own():
    c = make(40, 7, 1, "bf16", "slow", True)
    x = device(c, "bf16")
    S = x["S0"].clone()
    z = ttt.ttt_linear_attn_decode(*(x[n][:, :, 0].contiguous() for n in "QKV"), x["log_decay"], S, scale=x["scale"])
    ref = reference(c, "fwd")
    check({"Z": z[:, :, None], "S": S}, ref, bounds(c, "fwd", "bf16", ref))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rotary", [64, 48, 40, 20, 14, 2, 0])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(dtype, rotary, interleaved, inverse):
    rng = np.random.default_rng(5)
    Bn, T = 3, 21
    joint = torch.from_numpy(rng.standard_normal((Bn, T, 7, D))).to(TYPES[dtype]).cuda()
    Q, K = joint[:, :, :5].transpose(1, 2), joint[:, :, 5:].transpose(1, 2)
    f = torch.from_numpy((10000.0 ** (-2.0 * np.arange(rotary // 2) / max(rotary, 1))).astype(np.float32)).cuda()
    plan = ttt.Rope(f, mscale=1.25, interleaved=interleaved)
    pos = np.concatenate([rng.integers(-100, 100, (Bn, 7)), rng.integers(0, 2 ** 31, (Bn, 7)),
                          rng.integers(-2 ** 31, 0, (Bn, 7))], 1)
    Qo, Ko = ttt.ttt_rope(Q, K, plan, positions=torch.from_numpy(pos.astype(np.int32)).cuda(), inverse=inverse)
    for got, x in ((Qo, Q), (Ko, K)):
        x = x.double().cpu().numpy()
        ref = O.rope(x, pos, f.double().cpu().numpy(), 1.25, interleaved, inverse)
        # cos and sin: the angle in fp64 (2^31 x 2^-53 of a turn and less), sincosf within 4 half
        # steps, two more for the correction and one for mscale; two products, one sum: 12 half
        # steps of mscale (|x| + |partner|), at most 2 max over the row; rounded once.
        most = 2 * 1.25 * np.abs(x).max(-1, keepdims=True)
        bound = 12 * U32 * most + U[dtype] * np.abs(ref)
        g = got.double().cpu().numpy()
        assert np.all(np.abs(g - ref) <= bound), float((np.abs(g - ref) - bound).max())
        assert np.array_equal(g[..., rotary:], x[..., rotary:])


@pytest.mark.parametrize("B,H,T", [(1, 1, 1), (300, 4, 1), (2, 3, 1000), (1, 70, 33)])
def test_rope_sizes_and_first_position(B, H, T):
    x = torch.randn(B, H, T, D, device="cuda", dtype=torch.bfloat16)
    plan = ttt.Rope.build(64)
    Qo, Ko = ttt.ttt_rope(x, None, plan, first_position=11)
    pos = np.broadcast_to(11 + np.arange(T), (B, T))
    ref = O.rope(x.double().cpu().numpy(), pos, plan.inv_freq.double().cpu().numpy())
    assert Ko is None
    # Angles below 1100 in the oracle's fp64; as in test_rope with mscale 1.
    most = 2 * np.abs(x.double().cpu().numpy()).max(-1, keepdims=True)
    assert np.all(np.abs(Qo.double().cpu().numpy() - ref) <= 12 * U32 * most + U["bf16"] * np.abs(ref))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_and_attention_together(dtype):
    """As they are used: Q, K out of a joint projection, turned and attended, the gradient brought
    back through the turn, the prompt's state decoded on."""
    Bn, H, T = 2, 3, 90
    c = make(Bn, H, T, dtype, "slow", back=True, lengths=[T, 50])
    x = device(c, dtype)
    plan = ttt.Rope.build(32, interleaved=True, scaling="yarn", factor=4.0, original_length=64)
    f = plan.inv_freq.double().cpu().numpy()
    joint = torch.stack([x["Q"].transpose(1, 2), x["K"].transpose(1, 2)], 2)
    Q, K = joint[:, :, 0].transpose(1, 2), joint[:, :, 1].transpose(1, 2)
    pos = np.broadcast_to(np.arange(T), (Bn, T))
    turned = dict(c)
    for n in "QK":
        # The turned rows as the call rounds them: what the attention gets.
        turned[n] = ttt.ttt_rope(x[n], None, plan)[0].double().cpu().numpy()
    ref = reference(turned, "fwd")
    Z, S = ttt.ttt_linear_attn_fwd(Q, K, x["V"], x["log_decay"], scale=x["scale"], lengths=x["lengths"], rope=plan)
    check({"Z": Z, "S": S}, ref, bounds(turned, "fwd", dtype, ref))
    ref = reference(turned, "bwd")
    b = bounds(turned, "bwd", dtype, ref)
    got = ttt.ttt_linear_attn_bwd(Q, K, x["V"], x["log_decay"], x["dZ"], scale=x["scale"], lengths=x["lengths"],
                                  rope=plan)
    for n in ("dQ", "dK"):
        ref[n] = O.rope(ref[n], pos, f, plan.mscale, True, inverse=True)
        # The turn carries errors of a row at most mscale x sqrt(2) of its largest, and rounds once more.
        b[n] = plan.mscale * 1.5 * b[n].max(-1, keepdims=True) + (U[dtype] + 24 * U32) * (np.abs(ref[n]) + 2 * np.abs(
            ref[n]).max(-1, keepdims=True))
    check(got, ref, b)
    # Decode on from each sequence's own end.
    q, k, v = (torch.randn(Bn, H, D, device="cuda").to(TYPES[dtype]) for _ in range(3))
    S1 = S.clone()
    z = ttt.ttt_linear_attn_decode(q, k, v, x["log_decay"], S1, scale=x["scale"], rope=plan, positions=x["lengths"])
    at = x["lengths"].cpu().numpy()[:, None]
    qr, kr = (O.rope(t.double().cpu().numpy()[:, :, None], at, f, plan.mscale, True) for t in (q, k))
    Zr, Sr = O.forward(qr, kr, v.double().cpu().numpy()[:, :, None], c["log_decay"], c["scale"], S.double().cpu().numpy())
    assert np.abs(S1.double().cpu().numpy() - Sr).max() <= 40 * U32 * (np.abs(Sr).max() + 40)
    A = np.abs(c["scale"]) * np.einsum("bhti,bhij->bhtj", np.abs(qr), np.abs(Sr))
    assert np.all(np.abs(z.double().cpu().numpy() - Zr[:, :, 0]) <= (130 * U32 * (A + 12) + U[dtype] * np.abs(Zr))[:, :, 0])


@pytest.mark.parametrize("size", [(1, 32, 8192), (160, 1, 1000), (3, 7, 5000)], ids=str)
@pytest.mark.parametrize("decay", ["slow", "slope"])
def test_many_chunks_and_segments_on_both_paths(size, decay):
    """bf16 on the tensor cores against the CUDA-core kernels in fp32 on the same values: U A for the
    rounded operand and U |value| for the output (see bounds), with A from the same kernels on
    absolute values, and each doubled for the reference's own roundings (far below them)."""
    c = make(*size, "bf16", decay, True, back=True, seed=4)
    x = device(c, "bf16")
    exact = {n: (t.float() if isinstance(t, torch.Tensor) and t.dtype == torch.bfloat16 else t) for n, t in x.items()}
    mags = {n: (t.abs() if isinstance(t, torch.Tensor) and n != "log_decay" else t) for n, t in exact.items()}
    for run in (run_fwd, run_bwd):
        for _ in range(3):
            got = run(x)
            want, mag = run(exact), run(mags)
            for n, t in got.items():
                u = 600 * U32 if n in ("S", "dS0") else U["bf16"] * (1 + 2.0 ** -6)
                bound = u * mag[n] + (0 if n in ("S", "dS0") else U["bf16"] * (1 + 2.0 ** -6) * want[n].abs())
                over = (t.float() - want[n]).abs() - bound
                assert bool((over <= 1e-30).all()), (n, float(over.max()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,T", [(64, 7, 70), (64, 7, 300), (9, 40, 513)])
def test_padded_batches_of_many_sequences(dtype, B, H, T):
    """Many units an SM, among them empty ones, one after another: the pipelines run on over them."""
    rng = np.random.default_rng(8)
    lengths = rng.integers(0, T + 1, B)
    lengths[rng.permutation(B)[: B // 2]] = 0
    lengths[:4] = (T, 0, 0, 0)
    c = make(B, H, T, dtype, "slow", True, lengths=lengths, back=True)
    x = device(c, dtype)
    for fn, run in (("fwd", run_fwd), ("bwd", run_bwd)):
        ref = reference(c, fn)
        check(run(x), ref, bounds(c, fn, dtype, ref))
    assert ttt.last_device_status() == 0


def test_an_expired_wait_is_reported():
    """Every CTA's first wait runs out (nothing arrives there): the calls come back, the status says so once,
    and the next calls are right."""
    c = make(6, 30, 300, "bf16", "slow", True, back=True, lengths=[300, 0, 7, 128, 299, 1])
    x = device(c, "bf16")
    want = {**run_fwd(x), **run_bwd(x)}
    ttt.debug_inject_timeout(True)
    try:
        run_fwd(x), run_bwd(x)
        assert ttt.last_device_status() == ttt.TTT_ERR_TIMEOUT
    finally:
        ttt.debug_inject_timeout(False)
    assert ttt.last_device_status() == 0
    got = {**run_fwd(x), **run_bwd(x)}
    for n in want:
        assert torch.equal(got[n], want[n]), n
    assert ttt.last_device_status() == 0


# ---- calls a user makes that the sizes do not show ------------------------------------------

def test_results_do_not_change_between_calls():
    c = make(1, 3, 1500, "bf16", "slow", True, back=True)
    x = device(c, "bf16")
    first, again = {**run_fwd(x), **run_bwd(x)}, {**run_fwd(x), **run_bwd(x)}
    for n in first:
        assert torch.equal(first[n], again[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_streams_at_once(dtype):
    cs = [make(1, 2, 1400, dtype, "slow", True, back=True, seed=s) for s in (1, 2)]
    xs = [device(c, dtype) for c in cs]
    want = [{**run_fwd(x), **run_bwd(x)} for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, (x, s) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(s):
                got[i] = {**run_fwd(x), **run_bwd(x)}
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for n in w:
            assert torch.equal(g[n], w[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_stream_argument(dtype):
    """A call on a stream of its own that is behind: what the call allocated for itself stays its own
    while the current stream allocates and writes."""
    c = make(1, 4, 2000, dtype, "slow", True, back=True)
    x, plan = device(c, dtype), ttt.Rope.build(64)
    assert ttt.linear_attn_workspace_bytes((1, 4, 2000, D)) > 0
    want = {**run_fwd(x, rope=plan), **run_bwd(x, rope=plan)}
    q, k, v = (x[n][:, :, 0].contiguous() for n in "QKV")
    at = torch.tensor([5], dtype=torch.int32, device="cuda")
    S_want = x["S0"].clone()
    z_want = ttt.ttt_linear_attn_decode(q, k, v, x["log_decay"], S_want, rope=plan, positions=at)
    S = x["S0"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # ~10 ms
    got = {**run_fwd(x, rope=plan, stream=side), **run_bwd(x, rope=plan, stream=side)}
    z = ttt.ttt_linear_attn_decode(q, k, v, x["log_decay"], S, rope=plan, positions=at, stream=side)
    waste = [torch.full((1 << n,), 0x40, dtype=torch.uint8, device="cuda") for n in range(9, 24) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    assert len(waste) == 60 and torch.equal(z, z_want) and torch.equal(S, S_want)
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_states_handed_on_in_two_streams_and_graphs():
    """More units than SMs: two calls at once and two graphs that replay side by side, each with the
    workspace that it allocated."""
    cs = [make(40, 5, 700, "bf16", "slow", True, back=True, seed=s) for s in (1, 2)]
    xs = [device(c, "bf16") for c in cs]
    want = [{**run_fwd(x), **run_bwd(x)} for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, (x, s) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(s):
                got[i] = {**run_fwd(x), **run_bwd(x)}
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in xs], []
    for x, g in zip(xs, graphs):
        with torch.cuda.graph(g):
            outs.append({**run_fwd(x), **run_bwd(x)})
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for results in (got, outs):
        for g, w in zip(results, want):
            for n in w:
                assert torch.equal(g[n], w[n]), n
    assert ttt.last_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_thousands_of_short_sequences(dtype):
    """Dozens of segments a CTA, of a chunk or none."""
    lengths = [(7 * i) % 42 for i in range(1400)]
    c = make(1400, 5, 41, dtype, "slow", lengths=lengths, back=True)
    x = device(c, dtype)
    for fn, run in (("fwd", run_fwd), ("bwd", run_bwd)):
        ref = reference(c, fn)
        check(run(x), ref, bounds(c, fn, dtype, ref))
    assert ttt.last_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_and_replayed(dtype):
    c, c2 = (make(2, 2, 900, dtype, "slow", True, back=True, lengths=[900, 400], seed=s) for s in (1, 2))
    x, new = device(c, dtype), device(c2, dtype)
    plan = ttt.Rope.build(64)
    run_fwd(x), run_bwd(x)  # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = {**run_fwd(x, rope=plan), **run_bwd(x, rope=plan)}
    for n, t in new.items():
        if isinstance(t, torch.Tensor):
            x[n].copy_(t)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    want = {**run_fwd(new, rope=plan), **run_bwd(new, rope=plan)}
    for n in want:
        assert torch.equal(out[n], want[n]), n


def test_outputs_keep_within_their_rows():
    """Canaries about every output, at sizes that end inside a tile."""
    for dtype in ("f32", "bf16"):
        for B, H, T in ((1, 1, 1), (2, 1, 70), (1, 3, 700)):
            c = make(B, H, T, dtype, "slow", True)
            x = device(c, dtype)
            pad = 4096
            zbuf = torch.full((B * H * T * D + 2 * pad,), 7.0, dtype=TYPES[dtype], device="cuda")
            sbuf = torch.full((B * H * D * D + 2 * pad,), 7.0, device="cuda")
            Z = zbuf[pad:-pad].view(B, H, T, D)
            S = sbuf[pad:-pad].view(B, H, D, D)
            need = ttt.linear_attn_workspace_bytes((B, H, T, D))
            ws = torch.full((need + 2 * pad,), 5, dtype=torch.uint8, device="cuda")
            run_fwd(x, Z=Z, S_out=S, workspace=ws[pad:pad + need])
            torch.cuda.synchronize()
            for buf in (zbuf, sbuf):
                assert bool((buf[:pad] == 7).all()) and bool((buf[-pad:] == 7).all())
            assert bool((ws[:pad] == 5).all()) and bool((ws[pad + need:] == 5).all())
            want = run_fwd(x)
            assert torch.equal(Z, want["Z"]) and torch.equal(S, want["S"])


def test_state_outputs_may_be_left_out():
    lib = L.load()
    c = make(1, 2, 600, "bf16", "slow", back=True)
    x = device(c, "bf16")
    want = {**run_fwd(x), **run_bwd(x)}
    out = {n: torch.empty_like(x["Q"]) for n in ("Z", "dQ", "dK", "dV")}
    n = lib.ttt_linear_attn_workspace_bytes(1, 2, 600, 64, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    p = {k: v.data_ptr() for k, v in {**x, **out}.items() if isinstance(v, torch.Tensor)}
    assert lib.ttt_linear_attn_fwd(p["Q"], p["K"], p["V"], L.TTT_BF16, p["log_decay"], None, None, x["scale"], 1, 2, 600,
                                   64, p["Z"], None, ws.data_ptr(), n, s) == L.TTT_OK
    assert lib.ttt_linear_attn_bwd(p["Q"], p["K"], p["V"], L.TTT_BF16, p["log_decay"], None, None, x["scale"], p["dZ"],
                                   None, 1, 2, 600, 64, p["dQ"], p["dK"], p["dV"], None, ws.data_ptr(), n, s) == L.TTT_OK
    torch.cuda.synchronize()
    for k in out:
        assert torch.equal(out[k], want[k]), k


def test_bf16_path_setting():
    """TTT_PATH_SIMT takes the CUDA-core kernels for bf16 too, TTT_PATH_TC refuses what has no
    tensor-core kernel; both within the same bounds."""
    c = make(2, 2, 300, "bf16", "slow", True, back=True)
    x = device(c, "bf16")
    prev = ttt.set_path(ttt.TTT_PATH_SIMT)
    try:
        for fn, run in (("fwd", run_fwd), ("bwd", run_bwd)):
            ref = reference(c, fn)
            check(run(x), ref, bounds(c, fn, "bf16", ref))
    finally:
        ttt.set_path(prev)
