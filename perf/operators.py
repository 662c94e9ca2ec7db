"""What is measured of the linear attention and rotary operators: cases, plain forms and 64-bit values.

Linear attention with a decay for each head, state S [d, d] per (batch, head), gamma = exp(log_decay[head]):
    S_t = gamma S_{t-1} + k_t^T v_t,    z_t = scale q_t S_t
over whole sequences (forward and backward) and for one token (decode).  Rotary positions turn the pairs of
a row of Q and K by position x frequency.  The sizes are this repository's workloads (d = 64; B = 16, H = 12,
T = 2048; B = 16, H = 32, T = 8192; B = 1, H = 32, T = 32768; decode with 512 sequences of 32 heads) and ragged ones.
"""
import math

import torch

own = False

D = 64      # the head dimension of the library
CHUNK = 64  # tokens a chunk of the plain form

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------------------

def _attn(name, op, B, H, T, dtype, decay, state, ragged):
    return {"name": name, "op": op, "B": B, "H": H, "T": T, "dtype": dtype, "decay": decay, "state": state,
            "ragged": ragged}


def _decode(name, B, H, dtype, rotary, interleaved):
    return {"name": name, "op": "decode", "B": B, "H": H, "dtype": dtype, "decay": "slow", "rotary": rotary,
            "interleaved": interleaved}


def _rope(name, B, H, T, dtype, rotary, interleaved, scaling, inverse, first):
    return {"name": name, "op": "rope", "B": B, "H": H, "T": T, "dtype": dtype, "rotary": rotary,
            "interleaved": interleaved, "scaling": scaling, "inverse": inverse, "first": first}


def listed():
    return [
        # One short prompt of a small model: the call's latency is what a user waits for.
        _attn("fwd_prompt37", "fwd", 1, 12, 37, "bf16", "slow", False, False),
        # Training forward, 12 heads.
        _attn("fwd_B16H12T2048", "fwd", 16, 12, 2048, "bf16", "slow", False, False),
        # Training forward at the library's headline size: the largest case.
        _attn("fwd_B16H32T8192", "fwd", 16, 32, 8192, "bf16", "slope", False, False),
        # One long document, continued from the state of an earlier part: few heads, a long axis.
        _attn("fwd_B1H32T32768", "fwd", 1, 32, 32768, "bf16", "slow", True, False),
        # A padded batch of prompts of unlike lengths, in 32 bits, an odd padded length.
        _attn("fwd_f32_ragged", "fwd", 6, 8, 1999, "f32", "slope", True, True),
        # Training backward, 12 heads.
        _attn("bwd_B16H12T2048", "bwd", 16, 12, 2048, "bf16", "slow", False, False),
        # Backward of one long document with the gradient of its final state.
        _attn("bwd_B1H32T32768", "bwd", 1, 32, 32768, "bf16", "slope", True, False),
        # Backward of a small ragged batch in 32 bits, without decay.
        _attn("bwd_f32_ragged", "bwd", 3, 5, 777, "f32", "none", True, True),
        # One token of one sequence: latency.
        _decode("decode_B1H32", 1, 32, "bf16", 64, False),
        # One token of each of 512 sequences: the states do not fit any cache.
        _decode("decode_B512H32", 512, 32, "bf16", 64, False),
        # Q and K of a training step, out of a joint projection.
        _rope("rope_B16H32T2048", 16, 32, 2048, "bf16", 64, False, "none", False, 0),
        # A chunk of a long context, part of the head, neighbouring pairs, stretched frequencies; the gradient's way.
        _rope("rope_inverse_far", 2, 12, 1001, "f32", 40, True, "yarn", True, 200000),
    ]


def _nameless(case):
    return {k: v for k, v in case.items() if k != "name"}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "bwd", "decode", "rope"])
    if kind in ("fwd", "bwd"):
        T = _log_int(rng, 1, 32768)
        most = (2 << 20) if kind == "fwd" else (1 << 20)  # head-tokens
        H = rng.choice([1, 3, 4, 5, 8, 12, 16, 20, 32])
        B = _log_int(rng, 1, max(1, min(64, most // (H * T))))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return _nameless(_attn("", kind, B, H, T, dtype, rng.choice(["slow", "slope", "none"]), rng.random() < 0.5,
                               B > 1 and rng.random() < 0.5))
    if kind == "decode":
        return _nameless(_decode("", _log_int(rng, 1, 512), rng.choice([1, 5, 12, 32]), rng.choice(["bf16", "f32"]),
                                 rng.choice([0, 16, 32, 40, 64]), rng.random() < 0.5))
    T = _log_int(rng, 1, 32768)
    H = rng.choice([1, 5, 12, 32])
    B = _log_int(rng, 1, max(1, min(64, (1 << 20) // (H * T))))
    return _nameless(_rope("", B, H, T, rng.choice(["bf16", "f32"]), rng.choice([16, 20, 32, 40, 64]), rng.random() < 0.5,
                           rng.choice(["none", "linear", "yarn"]), rng.random() < 0.5, rng.choice([0, 7, 100000])))


# ---- inputs --------------------------------------------------------------------------------------------

def _log_decay(kind, H, device):
    h = torch.arange(H, dtype=torch.float64, device=device)
    if kind == "none":
        g = torch.zeros_like(h)
    elif kind == "slow":   # decay factors 1 - 2^-5 .. 1 - 2^-12 over the heads
        g = torch.log1p(-torch.exp2(-5.0 - 7.0 * h / max(1, H - 1)))
    else:                  # geometric slopes over the heads
        g = -torch.exp2(-8.0 * (h + 1) / H)
    return g.float()


def _inv_freq(rotary, scaling, device):
    """Frequencies 10000^(-2i/rotary) and the factor on the rotated values; "linear": every position divided by 8;
    "yarn": only the pairs that turn less than 32 times over the first 4096 positions, fully below one turn."""
    i = torch.arange(rotary // 2, dtype=torch.float64, device=device)
    f = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=device), -2.0 * i / rotary)
    if scaling == "linear":
        return (f / 8.0).float(), 1.0
    if scaling == "yarn":
        def at(turns):
            return rotary * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
        low, high = max(math.floor(at(32)), 0), min(math.ceil(at(1)), rotary - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        return (f / 8.0 * ramp + f * (1 - ramp)).float(), 0.1 * math.log(8.0) + 1.0
    return f.float(), 1.0


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = _TYPES[case["dtype"]]
    B, H = case["B"], case["H"]

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    s = {"case": case, "scale": D ** -0.5}
    if case["op"] == "rope":
        T = case["T"]
        # The joint projection's output [B, T, 2, H, d]; Q and K are views of it.
        joint = normal(B, T, 2, H, D)
        s["Q"], s["K"] = joint[:, :, 0].transpose(1, 2), joint[:, :, 1].transpose(1, 2)
        s["inv_freq"], s["mscale"] = _inv_freq(case["rotary"], case["scaling"], dev)
        # Each sequence at its own place.
        start = torch.randint(0, 50, (B, 1), generator=gen, device=dev) + case["first"]
        s["positions"] = (start + torch.arange(T, device=dev)).to(torch.int32)
        return s
    s["log_decay"] = _log_decay(case["decay"], H, dev)
    if case["op"] == "decode":
        s["q"], s["k"], s["v"] = (normal(B, H, D) for _ in range(3))
        s["S"] = normal(B, H, D, D, dtype=torch.float32, std=4.0)
        s["rotary"] = case["rotary"]
        if case["rotary"]:
            s["inv_freq"], s["mscale"] = _inv_freq(case["rotary"], "none", dev)
            s["positions"] = torch.randint(0, 32768, (B,), generator=gen, device=dev).to(torch.int32)
        return s
    T = case["T"]
    s["Q"], s["K"], s["V"] = (normal(B, H, T, D) for _ in range(3))
    s["S0"] = normal(B, H, D, D, dtype=torch.float32, std=4.0) if case["state"] else None
    s["lengths"] = None
    if case["ragged"]:
        n = torch.randint(0, T + 1, (B,), generator=gen, device=dev).to(torch.int32)
        n[0] = T
        s["lengths"] = n
    if case["op"] == "bwd":
        s["dZ"] = normal(B, H, T, D)
        s["dS_T"] = normal(B, H, D, D, dtype=torch.float32) if case["state"] else None
    return s


# ---- plain forms ---------------------------------------------------------------------------------------

def _powers(log_decay, n):
    """exp(log_decay * n) as [H, *n.shape] in 32 bits (the exponent in 64)."""
    g = log_decay.double().reshape(-1, *([1] * n.dim()))
    return torch.exp(g * n.double()).float()


def _alive(x, lengths):
    """x [B, H, T, d] in 32 bits with the rows from lengths[b] on as zeros."""
    x = x.float()
    if lengths is None:
        return x
    t = torch.arange(x.shape[2], device=x.device)
    return torch.where((t < lengths.reshape(-1, 1)).reshape(x.shape[0], 1, -1, 1), x, torch.zeros((), device=x.device))


def _chunks(x):
    B, H, T, d = x.shape
    N = -(-T // CHUNK)
    pad = x.new_zeros(B, H, N * CHUNK - T, d)
    return torch.cat([x, pad], 2).reshape(B, H, N, CHUNK, d)


def _attention(q, k, v, log_decay, S0):
    """sum_{s <= t} gamma^(t-s) (q_t . k_s) v_s + gamma^(t+1) q_t S0 for 32-bit [B, H, T, d] inputs."""
    B, H, T, d = q.shape
    q, k, v = _chunks(q), _chunks(k), _chunks(v)
    N = q.shape[2]
    t = torch.arange(CHUNK, device=q.device)
    gap = t.reshape(-1, 1) - t
    low = torch.where(gap >= 0, _powers(log_decay, gap.clamp(min=0)), torch.zeros((), device=q.device))
    inner = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * low[:, None], v)
    own_part = torch.matmul((k * _powers(log_decay, CHUNK - 1 - t)[:, None, :, None]).transpose(-1, -2), v)
    n = torch.arange(N, device=q.device)
    before = n.reshape(-1, 1) - 1 - n
    carry = torch.where(before >= 0, _powers(log_decay, CHUNK * before.clamp(min=0)), torch.zeros((), device=q.device))
    S = torch.matmul(carry, own_part.reshape(B, H, N, d * d)).reshape(B, H, N, d, d)
    if S0 is not None:
        S = S + _powers(log_decay, CHUNK * n)[:, :, None, None] * S0[:, :, None]
    z = inner + torch.matmul(q, S) * _powers(log_decay, t + 1)[:, None, :, None]
    return z.reshape(B, H, N * CHUNK, d)[:, :, :T]


def _final_state(k, v, log_decay, n, S0):
    """sum_{s < n} gamma^(n-1-s) k_s^T v_s + gamma^n S0, n [B] the sequences' lengths (rows behind them are zeros)."""
    B, H, T, d = k.shape
    left = (n.reshape(-1, 1) - 1 - torch.arange(T, device=k.device)).clamp(min=0)
    w = _powers(log_decay, left).transpose(0, 1)  # [B, H, T]
    S = torch.matmul((k * w[..., None]).transpose(-1, -2), v)
    if S0 is not None:
        S = S + _powers(log_decay, n).transpose(0, 1)[..., None, None] * S0
    return S


def _lengths_of(s):
    B, T = s["case"]["B"], s["case"]["T"]
    if s["lengths"] is not None:
        return s["lengths"].long()
    return torch.full((B,), T, device=s["Q"].device)


def _plain_fwd(s):
    q, k, v = (_alive(s[x], s["lengths"]) for x in "QKV")
    g, n = s["log_decay"], _lengths_of(s)
    Z = _attention(q, k, v, g, s["S0"]) * s["scale"]
    return {"Z": _alive(Z, s["lengths"]).to(s["Q"].dtype), "S": _final_state(k, v, g, n, s["S0"])}


def _from_the_end(x, n):
    """Row t of each sequence to row n - 1 - t (rows behind the end are zeros and stay so)."""
    at = n.reshape(-1, 1) - 1 - torch.arange(x.shape[2], device=x.device)
    y = torch.gather(x, 2, at.clamp(min=0).reshape(x.shape[0], 1, -1, 1).expand_as(x))
    return torch.where((at >= 0).reshape(x.shape[0], 1, -1, 1), y, torch.zeros((), device=x.device))


def _plain_bwd(s):
    dt, g, n, scale = s["Q"].dtype, s["log_decay"], _lengths_of(s), s["scale"]
    q, k, v, dz = (_alive(s[x], s["lengths"]) for x in ("Q", "K", "V", "dZ"))
    St = None if s["S0"] is None else s["S0"].transpose(-1, -2)
    dq = _alive(_attention(dz, v, k, g, St) * scale, s["lengths"])
    # The reverse pass is the forward over the sequences read from their ends; a row's own token counts the final
    # state's cotangent with gamma^(n-1-t), one power less than the forward's gamma^(t+1).
    qr, kr, vr, dzr = (_from_the_end(x, n) for x in (q, k, v, dz))
    dk, dv = _attention(vr, dzr, qr * scale, g, None), _attention(kr, qr * scale, dzr, g, None)
    if s["dS_T"] is not None:
        w = _powers(g, torch.arange(q.shape[2], device=q.device))[None, :, :, None]
        dk = dk + w * torch.matmul(vr, s["dS_T"].transpose(-1, -2))
        dv = dv + w * torch.matmul(kr, s["dS_T"])
    dk, dv = (_from_the_end(_alive(x, s["lengths"]), n) for x in (dk, dv))
    w = _powers(g, torch.arange(q.shape[2], device=q.device) + 1)[None, :, :, None]
    dS0 = torch.matmul((q * (w * scale)).transpose(-1, -2), dz)
    if s["dS_T"] is not None:
        dS0 = dS0 + _powers(g, n).transpose(0, 1)[..., None, None] * s["dS_T"]
    return {"dQ": dq.to(dt), "dK": dk.to(dt), "dV": dv.to(dt), "dS0": dS0}


def _turn(x, positions, inv_freq, mscale, interleaved, inverse):
    """x [..., d] in 32 bits turned by positions (shaped to x's leading axes) x inv_freq."""
    half = inv_freq.numel()
    angle = positions.double()[..., None] * inv_freq.double() * (-1.0 if inverse else 1.0)
    c, sn = (torch.cos(angle) * mscale).float(), (torch.sin(angle) * mscale).float()
    x = x.float()
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * c - b * sn, a * sn + b * c], -1).reshape(r.shape)
    else:
        a, b = r[..., :half], r[..., half:]
        y = torch.cat([a * c - b * sn, a * sn + b * c], -1)
    return torch.cat([y, rest], -1)


def _plain_rope(s):
    c = s["case"]
    p = s["positions"][:, None, :]
    return {x: _turn(s[x], p, s["inv_freq"], s["mscale"], c["interleaved"], c["inverse"]).to(s[x].dtype).contiguous()
            for x in "QK"}


def _plain_decode(s):
    q, k, v = (s[x].float() for x in "qkv")
    if s["rotary"]:
        p = s["positions"][:, None]
        q, k = (_turn(x, p, s["inv_freq"], s["mscale"], s["case"]["interleaved"], False) for x in (q, k))
    S = s["S"] * torch.exp(s["log_decay"])[:, None, None] + k[..., :, None] * v[..., None, :]
    s["S"].copy_(S)
    z = torch.matmul(q[..., None, :], S)[..., 0, :] * s["scale"]
    return {"z": z.to(s["q"].dtype), "S": s["S"]}


# ---- one pass ------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "rope": _plain_rope, "decode": _plain_decode}[op](s)
    import test_sequence_modeling_b200 as ttt
    if op == "fwd":
        Z, S = ttt.ttt_linear_attn_fwd(s["Q"], s["K"], s["V"], s["log_decay"], scale=s["scale"], S0=s["S0"],
                                       lengths=s["lengths"])
        return {"Z": Z, "S": S}
    if op == "bwd":
        return ttt.ttt_linear_attn_bwd(s["Q"], s["K"], s["V"], s["log_decay"], s["dZ"], scale=s["scale"], S0=s["S0"],
                                       dS_T=s["dS_T"], lengths=s["lengths"])
    if op == "rope":
        c = s["case"]
        plan = ttt.Rope(s["inv_freq"], mscale=s["mscale"], interleaved=c["interleaved"])
        Q, K = ttt.ttt_rope(s["Q"], s["K"], plan, positions=s["positions"], inverse=c["inverse"])
        return {"Q": Q, "K": K}
    plan = ttt.Rope(s["inv_freq"], mscale=s["mscale"], interleaved=s["case"]["interleaved"]) if s["rotary"] else None
    z = ttt.ttt_linear_attn_decode(s["q"], s["k"], s["v"], s["log_decay"], s["S"], scale=s["scale"], rope=plan,
                                   positions=s["positions"] if s["rotary"] else None)
    return {"z": z, "S": s["S"]}


def work(case):
    B, H, op = case["B"], case["H"], case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    state = B * H * D * D * 4
    if op == "decode":
        rot = case["rotary"]
        turned = 4 * B + 2 * rot if rot else 0
        return {"bytes": 2 * state + 4 * B * H * D * e + 4 * H + turned,
                "flops": B * H * (5 * D * D + (6 * rot if rot else 0))}
    rows = B * H * case["T"]
    if op == "rope":
        return {"bytes": 4 * rows * D * e + 4 * B * case["T"] + 2 * case["rotary"], "flops": 2 * rows * 3 * case["rotary"]}
    # Half of a padded batch's rows are behind the ends on the average: written (zeros), not read.
    read = rows * (0.5 + 0.5 / B) if case["ragged"] else rows
    states = (2 if op == "bwd" and case["state"] else 1 if case["state"] else 0) + 1
    inputs, outputs, products = (3, 1, 4) if op == "fwd" else (4, 3, 10)
    return {"bytes": (inputs * read + outputs * rows) * D * e + states * state + 4 * H,
            "flops": read * products * D * D}


# ---- the definition in 64 bits -------------------------------------------------------------------------

def _exact_turn(x, positions, inv_freq, mscale, interleaved, inverse):
    """Pairs as complex numbers, each times mscale e^(+-i position frequency)."""
    half = inv_freq.numel()
    phase = torch.polar(torch.full((), float(mscale), dtype=torch.float64, device=x.device).expand(positions.shape + (half,)),
                        positions.double()[..., None] * inv_freq.double())
    if inverse:
        phase = phase.conj()
    y = x.double().clone()
    if interleaved:
        a, b = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    else:
        a, b = slice(0, half), slice(half, 2 * half)
    w = torch.complex(y[..., a], y[..., b]) * phase
    y[..., a], y[..., b] = w.real, w.imag
    return y


def exact(case, seed):
    """The recursions token by token in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        p = s["positions"][:, None, :]
        return {x: _exact_turn(s[x], p, s["inv_freq"], s["mscale"], case["interleaved"], case["inverse"]) for x in "QK"}
    gamma = torch.exp(s["log_decay"].double())[None, :, None, None]
    scale = s["scale"]
    if op == "decode":
        q, k, v = (s[x].double() for x in "qkv")
        if s["rotary"]:
            p = s["positions"][:, None]
            q, k = (_exact_turn(x, p, s["inv_freq"], s["mscale"], case["interleaved"], False) for x in (q, k))
        S = s["S"].double() * gamma + k.unsqueeze(-1) * v.unsqueeze(-2)
        return {"z": (q.unsqueeze(-1) * S).sum(-2) * scale, "S": S}
    B, H, T = case["B"], case["H"], case["T"]
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device=s["Q"].device)
    live = (torch.arange(T, device=n.device)[:, None] < n[None, :]).double()[:, :, None, None, None]  # [T, B, 1, 1, 1]
    q, k, v = (s[x].double() for x in "QKV")
    S = torch.zeros(B, H, D, D, dtype=torch.float64, device=q.device) if s["S0"] is None else s["S0"].double()
    S = S.clone()
    if op == "fwd":
        Z = torch.empty_like(q)
        for t in range(T):
            m = live[t] if case["ragged"] else 1.0
            keep = 1.0 + m * (gamma - 1.0) if case["ragged"] else gamma
            S.mul_(keep).addcmul_(k[:, :, t, :, None] * m, v[:, :, t, None, :])
            Z[:, :, t] = torch.matmul(q[:, :, t, None, :], S)[:, :, 0] * (m[..., 0] * scale if case["ragged"] else scale)
        return {"Z": Z, "S": S}
    dz = s["dZ"].double()
    dQ, dK, dV = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    for t in range(T):
        m = live[t] if case["ragged"] else 1.0
        keep = 1.0 + m * (gamma - 1.0) if case["ragged"] else gamma
        S.mul_(keep).addcmul_(k[:, :, t, :, None] * m, v[:, :, t, None, :])
        dQ[:, :, t] = torch.matmul(S, dz[:, :, t, :, None])[..., 0] * (m[..., 0] * scale if case["ragged"] else scale)
    G = torch.zeros_like(S) if s["dS_T"] is None else s["dS_T"].double().clone()
    for t in range(T - 1, -1, -1):
        m = live[t] if case["ragged"] else 1.0
        G.addcmul_(q[:, :, t, :, None] * m, dz[:, :, t, None, :], value=scale)
        dK[:, :, t] = torch.matmul(G, v[:, :, t, :, None])[..., 0] * (m[..., 0] if case["ragged"] else 1.0)
        dV[:, :, t] = torch.matmul(k[:, :, t, None, :], G)[:, :, 0] * (m[..., 0] if case["ragged"] else 1.0)
        G.mul_(1.0 + m * (gamma - 1.0) if case["ragged"] else gamma)
    return {"dQ": dQ, "dK": dK, "dV": dV, "dS0": G}
