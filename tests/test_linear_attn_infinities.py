"""Infinities among the tokens: what the formulas make of one is an infinity in the state, of the formulas' sign,
on every path; the rest of the results stays what it was."""
import numpy as np
import pytest
import torch

import test_sequence_modeling_b200 as ttt
from linear_attn_helpers import bounds, device, make, reference

pytestmark = pytest.mark.gpu

T = 300  # chunks of 64 and of 128 tokens, the last one ragged


def _same(got, ref, bound, name):
    """Infinities of the same sign in the same places, the finite values within their bound."""
    g = got.double().cpu().numpy()
    inf = np.isinf(ref)
    assert inf.any() and not np.isnan(ref).any(), name
    assert np.array_equal(g[inf], ref[inf]), (name, g[inf][:4], ref[inf][:4])
    assert np.all(np.abs(g[~inf] - ref[~inf]) <= bound[~inf]), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", ["none", "slow"])
@pytest.mark.parametrize("size", [(2, 2, T), (1, 1, 1500), (60, 3, T)], ids=str)
@pytest.mark.parametrize("which", ["K", "V"])
def test_forward(dtype, decay, size, which):
    """One in K: its row of the state, and every output from there on.  One in V: its column of the state; its
    column of the outputs from there on is not finite (the formulas' order of sums decides between an infinity
    and NaN), the other columns are untouched."""
    c = make(*size, dtype, decay, True)
    ref, plain = {}, reference(c, "fwd")
    b = bounds(c, "fwd", dtype, plain)
    B, H, n = size
    at = [(0, H - 1, 5, 7, np.inf), (B - 1, 0, 130, 33, -np.inf), (B - 1, H - 1, n - 1, 63, np.inf)]
    if size[0] * size[1] == 1:
        at = at[1:2]
    x = device(c, dtype)
    S = plain["S"].copy()
    for bi, h, t, j, value in at:
        x[which][bi, h, t, j] = float(value)
        if which == "K":
            S[bi, h, j] = value * np.sign(c["V"][bi, h, t])
        else:
            S[bi, h, :, j] = value * np.sign(c["K"][bi, h, t])
    Z, got = ttt.ttt_linear_attn_fwd(x["Q"], x["K"], x["V"], x["log_decay"], scale=x["scale"], S0=x["S0"])
    _same(got, S, b["S"], "S")
    Z = Z.double().cpu().numpy()
    free = np.ones(Z.shape, bool)  # untouched values
    for bi, h, t, j, value in at:
        if which == "K":
            free[bi, h, t:] = False
            sign = value * np.sign(c["Q"][bi, h, t:, j])[:, None] * np.sign(c["V"][bi, h, t])
            assert np.array_equal(Z[bi, h, t:], sign), (bi, h, t)
        else:
            free[bi, h, :, j] = False
            assert not np.isfinite(Z[bi, h, t:, j]).any()
    assert np.all((np.abs(Z - plain["Z"]) <= b["Z"])[free])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(2, 2, T), (1, 1, 1500), (60, 3, T)], ids=str)
def test_backward(dtype, size):
    """One in Q: its row of dS0 (G = scale q^T dz is carried in reverse), as the forward's K."""
    c = make(*size, dtype, "slow", True, back=True)
    plain = reference(c, "bwd")
    b = bounds(c, "bwd", dtype, plain)
    x = device(c, dtype)
    bi, h, t, j = size[0] - 1, size[1] - 1, 140, 9
    x["Q"][bi, h, t, j] = float("-inf")
    want = plain["dS0"].copy()
    want[bi, h, j] = -np.inf * np.sign(c["dZ"][bi, h, t])
    out = ttt.ttt_linear_attn_bwd(x["Q"], x["K"], x["V"], x["log_decay"], x["dZ"], scale=x["scale"], S0=x["S0"],
                                  dS_T=x["dS_T"])
    _same(out["dS0"], want, b["dS0"], "dS0")
