"""Shared by the tests of linear attention and rotary positions: seeded inputs, the fp64 oracle
and the error bounds."""
from __future__ import annotations

import numpy as np
import torch

from oracle import linear_attn as O

D = 64
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# A rounding is off by at most half a step of the type, relative to the value.
U32 = torch.finfo(torch.float32).eps / 2
U = {"f32": U32, "bf16": torch.finfo(torch.bfloat16).eps / 2}

DECAYS = {
    "none": lambda H: np.zeros(H),
    "slow": lambda H: np.log1p(-np.exp2(-5.0 - 7.0 * np.arange(H) / max(1, H - 1))),
    "slope": lambda H: -np.exp2(-8.0 * (np.arange(H) + 1) / H),
    "strong": lambda H: -3.0 - 40.0 * np.arange(H),   # gamma^2 already vanishes, gamma^n underflows
    "nothing": lambda H: np.full(H, -np.inf),         # gamma = 0
}


def make(B, H, T, dtype, decay="slow", state=False, lengths=None, seed=0, back=False):
    """Host inputs in float64 that the type holds exactly: a dict of numpy arrays."""
    rng = np.random.default_rng([seed, B, H, T])

    def exact(*shape, t=TYPES[dtype], std=1.0):
        x = torch.from_numpy(rng.standard_normal(shape) * std)
        return x.to(t).double().numpy()

    c = {"log_decay": DECAYS[decay](H).astype(np.float32), "scale": float(np.float32(0.125))}
    for n in "QKV":
        c[n] = exact(B, H, T, D)
    c["S0"] = exact(B, H, D, D, t=torch.float32, std=4.0) if state else None
    c["lengths"] = None if lengths is None else np.asarray(lengths, np.int32)
    if back:
        c["dZ"] = exact(B, H, T, D)
        c["dS_T"] = exact(B, H, D, D, t=torch.float32) if state else None
    return c


def device(c, dtype):
    d = {"scale": c["scale"], "log_decay": torch.from_numpy(c["log_decay"]).cuda()}
    for n in ("Q", "K", "V", "dZ"):
        if n in c:
            d[n] = torch.from_numpy(c[n]).to(TYPES[dtype]).cuda()
    for n in ("S0", "dS_T"):
        d[n] = torch.from_numpy(c[n]).float().cuda() if c.get(n) is not None else None
    d["lengths"] = torch.from_numpy(c["lengths"]).cuda() if c["lengths"] is not None else None
    return d


def _magnitude(c, fn, *extra):
    """The oracle on absolute values: what every rounding of a product or a sum is relative to."""
    a = {n: (np.abs(c[n]) if c.get(n) is not None else None) for n in ("Q", "K", "V", "S0", "dZ", "dS_T")}
    if fn == "fwd":
        Z, S = O.forward(a["Q"], a["K"], a["V"], c["log_decay"], abs(c["scale"]), a["S0"], c["lengths"])
        return {"Z": Z, "S": S}
    return O.backward(a["Q"], a["K"], a["V"], c["log_decay"], abs(c["scale"]), a["dZ"], a["S0"], a["dS_T"], c["lengths"])


def reference(c, fn):
    if fn == "fwd":
        Z, S = O.forward(c["Q"], c["K"], c["V"], c["log_decay"], c["scale"], c["S0"], c["lengths"])
        return {"Z": Z, "S": S}
    return O.backward(c["Q"], c["K"], c["V"], c["log_decay"], c["scale"], c["dZ"], c["S0"], c["dS_T"], c["lengths"])


def bounds(c, fn, dtype, ref):
    """Largest error of each output, element by element.  With A the same sum over absolute
    values, each rounding on the way costs at most its half step times A, and the roundings
    that one summand passes are counted:
      fp32: two dot products over d = 64 (64 + 64), the sum over a chunk (128) for the chunk's
      own part; a state's summand enters by a chunk's sum (128) and passes one scaling and
      one addition a chunk of at least 64 tokens, twice if the sequence is cut (its segment's
      sum, then the scan), and a power of gamma: expf is within 2 half steps x 2 of the exact
      value and its argument, rounded once, is off by |n g| half steps, which counts only where
      gamma^n >= e^-104 (fp32 holds nothing below): 104 + 4.  Together at most
      64 + 64 + 128 + 128 + 4 ceil(T / 64) + 2 (104 + 4) + 8 roundings.
      bf16: a summand of an output passes one operand rounded to bf16, the masked products or
      the state (one half step of bf16 times A), and the output is rounded once (one half step
      times the value).  The states themselves pass no rounding to bf16: the decayed rows that
      enter them are three bf16 numbers, all of fp32."""
    A = _magnitude(c, fn)
    T = c["Q"].shape[2]
    n = 64 + 64 + 128 + 128 + 4 * -(-T // 64) + 2 * 108 + 8
    out = {}
    for name, a in A.items():
        state = name in ("S", "dS0")
        b = n * U32 * a
        if dtype == "bf16":
            if not state:
                b = b + U["bf16"] * a + U["bf16"] * np.abs(ref[name]) * (1 + U["bf16"])
                b = b + U["bf16"] ** 2 * a  # both on one summand
        elif not state:
            b = b + U32 * np.abs(ref[name])
        # What underflows: gamma^n below the smallest fp32 value counts as zero.
        out[name] = b + 1e-37
    return out


def check(got, ref, bound):
    for name, r in ref.items():
        g = got[name].double().cpu().numpy()
        assert g.shape == r.shape, name
        assert np.all(np.isfinite(g)), name
        over = np.abs(g - r) - bound[name]
        assert over.max(initial=-1.0) <= 0, (name, float(over.max()), np.unravel_index(over.argmax(), over.shape))
