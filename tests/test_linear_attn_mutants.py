"""Planted mistakes: chunked linear attention in fp64 with one thing wrong each, the way a kernel over chunks and
segments could have it wrong, has to exceed the element-wise bounds that the GPU tests use, in both types.  No GPU."""
import numpy as np
import pytest

from linear_attn_helpers import bounds, make, reference

CHUNK = 128


def _pass(x, y, w, C, g, a, c, e, n, reverse, wrong):
    """One pass over a unit's n tokens in chunks (the roles of csrc/linear_attn.cuh), with `wrong` in it."""
    out = np.zeros_like(x)
    starts = list(range(0, n, CHUNK))
    for s0 in (starts[::-1] if reverse else starts):
        m = min(CHUNK, n - s0)
        t = np.arange(m)
        X, Y, W = (r[s0:s0 + m] for r in (x, y, w))
        gap = (t - t[:, None]) if reverse else (t[:, None] - t)
        least = 1 if wrong == "the token itself left out" else 0
        mask = np.where(gap >= least, np.exp(g * np.maximum(gap, 0)), 0.0)
        if wrong == "the mask turned around":
            mask = mask.T
        if wrong == "no decay inside a chunk":
            mask = (gap >= 0).astype(float)
        f = np.exp(g * ((m - 1 - t) if reverse else (t + 1)))
        h = np.exp(g * ((t + 1) if reverse else (m - 1 - t)))
        if wrong == "the state's decay off by one":
            f = f * np.exp(-g)
        if wrong == "the chunk's part decayed once too often":
            h = h * np.exp(g)
        if wrong == "a row lost from the chunk's part":
            h[0] = 0.0
        o = a * ((X @ Y.T) * mask) @ W
        if wrong != "the carried state left out":
            o = o + c * f[:, None] * (X @ (C.T if wrong == "the state transposed" else C))
        out[s0:s0 + m] = o
        full = CHUNK if wrong == "a ragged chunk decayed as a full one" else m
        C = np.exp(g * full) * C + e * (h[:, None] * Y).T @ W
        if wrong == "the state not handed on after the first chunks" and s0 == CHUNK:
            C = np.zeros_like(C)
    return out, C


def _all(c, fn, wrong=None):
    B, H, T, D = c["Q"].shape
    names = ("Z", "S") if fn == "fwd" else ("dQ", "dK", "dV", "dS0")
    out = {n: np.zeros((B, H, D, D) if n in ("S", "dS0") else (B, H, T, D)) for n in names}
    s = c["scale"]
    for b in range(B):
        n = T if c["lengths"] is None else int(c["lengths"][b])
        if wrong == "a sequence's last token cut off":
            n = max(n - 1, 0)
        if wrong == "lengths not used":
            n = T
        for h in range(H):
            g = float(c["log_decay"][(h + 1) % H if wrong == "the next head's decay" else h])
            S0 = np.zeros((D, D)) if wrong == "S0 left out" else c["S0"][b, h]
            q, k, v = (c[x][b, h] for x in "QKV")
            sc = 1.0 if wrong == "no scale" else s
            if fn == "fwd":
                out["Z"][b, h], out["S"][b, h] = _pass(q, k, v, S0, g, sc, sc, 1.0, n, False, wrong)
                continue
            G0 = np.zeros((D, D)) if wrong == "dS_T left out" else c["dS_T"][b, h]
            dz = c["dZ"][b, h]
            out["dQ"][b, h] = _pass(dz, v, k, S0.T, g, sc, sc, 1.0, n, False, wrong)[0]
            out["dK"][b, h] = _pass(v, dz, q, G0.T, g, sc, 1.0, sc, n, True, wrong)[0]
            out["dV"][b, h], out["dS0"][b, h] = _pass(k, q, dz, G0, g, sc, 1.0, sc, n, True, wrong)
    return out


def _case(dtype):
    return make(2, 2, 300, dtype, "slow", True, lengths=[300, 170], back=True)


def _over(got, ref, bound):
    return {n for n in ref if np.any(np.abs(got[n] - ref[n]) > bound[n])}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fn", ["fwd", "bwd"])
def test_without_a_mistake_all_is_within(fn, dtype):
    c = _case(dtype)
    ref = reference(c, fn)
    assert _over(_all(c, fn), ref, bounds(c, fn, dtype, ref)) == set()


# The outputs that each mistake has to show in, in either type.  (A state's part that is off by a factor e^g, 3 % in
# the head that forgets fastest, is within a bf16 output's half step of the sum of absolute values, 2^-8: it shows
# in the states, which pass no rounding to bf16.)
MISTAKES = {
    "the token itself left out": {"Z", "dQ", "dK", "dV"},
    "the mask turned around": {"Z", "dQ", "dK", "dV"},
    "no decay inside a chunk": {"Z", "dQ", "dK", "dV"},
    "the state's decay off by one": {"Z", "dQ", "dK", "dV"},
    "the chunk's part decayed once too often": {"S", "dS0"},
    "a row lost from the chunk's part": {"Z", "S", "dQ", "dK", "dV", "dS0"},
    "the carried state left out": {"Z", "dQ", "dK", "dV"},
    "the state transposed": {"Z", "dQ", "dK", "dV"},
    "a ragged chunk decayed as a full one": {"S", "dK", "dV", "dS0"},
    "the state not handed on after the first chunks": {"Z", "S", "dQ", "dK", "dV", "dS0"},
    "a sequence's last token cut off": {"Z", "S", "dQ", "dK", "dV", "dS0"},
    "lengths not used": {"Z", "S", "dQ", "dK", "dV", "dS0"},
    "the next head's decay": {"Z", "S", "dQ", "dK", "dV", "dS0"},
    "S0 left out": {"Z", "S", "dQ"},
    "dS_T left out": {"dK", "dV", "dS0"},
    "no scale": {"Z", "dQ", "dK", "dV", "dS0"},
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wrong", list(MISTAKES))
def test_a_mistake_is_seen(wrong, dtype):
    c = _case(dtype)
    for fn in ("fwd", "bwd"):
        ref = reference(c, fn)
        want = MISTAKES[wrong] & set(ref)
        assert _over(_all(c, fn, wrong), ref, bounds(c, fn, dtype, ref)) >= want
