"""The fp64 oracle of linear attention and rotary positions against closed forms, autograd and
differences, and the chunk algebra of the CUDA path in fp64.  No GPU."""
import numpy as np
import pytest
import torch

from linear_attn_helpers import D, make, reference
from oracle import linear_attn as O


@pytest.mark.parametrize("decay", ["none", "slow", "slope", "strong", "nothing"])
@pytest.mark.parametrize("state", [False, True])
def test_forward_is_the_masked_product(decay, state):
    c = make(2, 3, 21, "f32", decay, state)
    Z, S = O.forward(c["Q"], c["K"], c["V"], c["log_decay"], c["scale"], c["S0"])
    g = c["log_decay"].astype(np.float64)
    t = np.arange(21)
    gap = t[:, None] - t
    with np.errstate(invalid="ignore"):
        power = np.where(gap == 0, 1.0, np.exp(g[:, None, None] * np.maximum(gap, 1)))
        first = np.exp(g[:, None] * (t + 1))
        last = np.where(t[::-1] == 0, 1.0, np.exp(g[:, None] * np.maximum(t[::-1], 1)))
    P = np.where(gap >= 0, np.einsum("bhti,bhsi->bhts", c["Q"], c["K"]) * power, 0.0)
    want = c["scale"] * np.einsum("bhts,bhsj->bhtj", P, c["V"])
    wantS = np.einsum("bhti,bhtj->bhij", c["K"] * last[None, :, :, None], c["V"])
    if state:
        want += c["scale"] * np.einsum("bhti,bhij->bhtj", c["Q"], c["S0"]) * first[None, :, :, None]
        wantS += first[None, :, -1, None, None] * c["S0"]
    assert np.allclose(Z, want, rtol=1e-12, atol=1e-12)
    assert np.allclose(S, wantS, rtol=1e-12, atol=1e-12)


def test_lengths_cut_each_sequence():
    c = make(4, 2, 9, "f32", "slow", True, lengths=[9, 4, 0, 1], back=True)
    c["Q"][1, :, 4:] = np.nan
    ref, grad = reference(c, "fwd"), reference(c, "bwd")
    for b, n in enumerate([9, 4, 0, 1]):
        one = {x: c[x][b:b + 1, :, :n] for x in ("Q", "K", "V", "dZ")}
        Z, S = O.forward(one["Q"], one["K"], one["V"], c["log_decay"], c["scale"], c["S0"][b:b + 1])
        assert np.array_equal(ref["Z"][b:b + 1, :, :n], Z) and np.array_equal(ref["S"][b:b + 1], S)
        assert np.all(ref["Z"][b, :, n:] == 0) and np.all(grad["dV"][b, :, n:] == 0)
        if n == 0:
            assert np.array_equal(grad["dS0"][b], c["dS_T"][b])


@pytest.mark.parametrize("decay", ["none", "slope", "nothing"])
def test_backward_is_autograd(decay):
    c = make(2, 2, 11, "f32", decay, True, lengths=[11, 6], back=True)
    x = {n: torch.tensor(c[n], requires_grad=True) for n in ("Q", "K", "V", "S0")}
    gamma = torch.exp(torch.tensor(c["log_decay"].astype(np.float64)))
    loss = 0.0
    for b, n in enumerate([11, 6]):
        S = x["S0"][b]
        for t in range(n):
            S = gamma[:, None, None] * S + x["K"][b, :, t, :, None] * x["V"][b, :, t, None, :]
            z = c["scale"] * torch.einsum("hi,hij->hj", x["Q"][b, :, t], S)
            loss = loss + (z * torch.tensor(c["dZ"][b, :, t])).sum()
        loss = loss + (S * torch.tensor(c["dS_T"][b])).sum()
    loss.backward()
    grad = reference(c, "bwd")
    for n in ("Q", "K", "V", "S0"):
        assert np.allclose(grad["d" + n], x[n].grad.numpy(), rtol=1e-11, atol=1e-11), n


def test_backward_is_the_difference():
    c = make(1, 2, 7, "f32", "slope", True, back=True)
    grad = reference(c, "bwd")

    def loss():
        r = reference(c, "fwd")
        return (r["Z"] * c["dZ"]).sum() + (r["S"] * c["dS_T"]).sum()

    rng = np.random.default_rng(1)
    for n in ("Q", "K", "V", "S0"):
        way = rng.standard_normal(c[n].shape)
        x, h = c[n].copy(), 1e-4
        c[n] = x + h * way
        up = loss()
        c[n] = x - h * way
        down = loss()
        c[n] = x
        # L is at most quadratic along Q, K, V or S0 alone: the central difference is exact but
        # for rounding, about 1e-16 |L| / h.
        assert abs((up - down) / (2 * h) - (grad["d" + n] * way).sum()) < 1e-8 * abs(up), n


@pytest.mark.parametrize("n", [128, 5])
def test_the_passes_chunk_algebra_in_64_bits(n):
    """The roles of csrc/linear_attn.cuh: one chunk rule, forward or reverse, gives Z, dQ, dK, dV
    and the states."""
    c = make(1, 2, n, "f32", "slow", True, back=True)
    g = c["log_decay"].astype(np.float64)[:, None]
    t = np.arange(n)
    ref, grad = reference(c, "fwd"), reference(c, "bwd")

    def chunk(x, y, w, C, a, cc, e, reverse):
        gap = (t - t[:, None]) if reverse else (t[:, None] - t)
        m = np.where(gap >= 0, np.exp(g[..., None] * np.maximum(gap, 0)), 0.0)
        f = np.exp(g * ((n - 1 - t) if reverse else (t + 1)))
        h = np.exp(g * ((t + 1) if reverse else (n - 1 - t)))
        out = a * np.einsum("bhts,bhsj->bhtj", np.einsum("bhti,bhsi->bhts", x, y) * m, w)
        out += cc * f[None, :, :, None] * np.einsum("bhti,bhij->bhtj", x, C)
        return out, np.exp(g * n)[None, :, :, None] * C + e * np.einsum("bhsi,bhsj->bhij", h[None, :, :, None] * y, w)

    Q, K, V, dZ, S, G, s = c["Q"], c["K"], c["V"], c["dZ"], c["S0"], c["dS_T"], c["scale"]
    turn = lambda X: X.swapaxes(-1, -2)  # noqa: E731
    Z, S1 = chunk(Q, K, V, S, s, s, 1.0, False)
    assert np.allclose(Z, ref["Z"], rtol=1e-11, atol=1e-11) and np.allclose(S1, ref["S"], rtol=1e-11, atol=1e-11)
    assert np.allclose(chunk(dZ, V, K, turn(S), s, s, 1.0, False)[0], grad["dQ"], rtol=1e-11, atol=1e-10)
    assert np.allclose(chunk(V, dZ, Q, turn(G), s, 1.0, s, True)[0], grad["dK"], rtol=1e-11, atol=1e-10)
    dV, dS0 = chunk(K, Q, dZ, G, s, 1.0, s, True)
    assert np.allclose(dV, grad["dV"], rtol=1e-11, atol=1e-10) and np.allclose(dS0, grad["dS0"], rtol=1e-11, atol=1e-10)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [64, 20, 2])
def test_rope_turns_and_turns_back(interleaved, rotary):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 5, D))
    f = 10000.0 ** (-2.0 * np.arange(rotary // 2) / rotary)
    pos = rng.integers(-1000, 100000, (2, 5))
    y = O.rope(x, pos, f, 1.5, interleaved)
    back = O.rope(y, pos, f, 1.5, interleaved, inverse=True)
    want = x.copy()
    want[..., :rotary] *= 2.25
    assert np.allclose(back, want, atol=1e-12) and np.array_equal(y[..., rotary:], x[..., rotary:])
    # Products of turned rows go by the distance of the positions.
    q, k = rng.standard_normal((2, 1, 1, 1, D))
    a = (O.rope(q, [[7]], f, 1.0, interleaved) * O.rope(k, [[3]], f, 1.0, interleaved)).sum()
    b = (O.rope(q, [[1007]], f, 1.0, interleaved) * O.rope(k, [[1003]], f, 1.0, interleaved)).sum()
    assert abs(a - b) < 1e-10
    # The gradient of <u, rope(x)> is the inverse turn of u.
    u = rng.standard_normal(x.shape)
    assert abs((u * O.rope(x, pos, f, 1.5, interleaved)).sum() -
               (O.rope(u, pos, f, 1.5, interleaved, inverse=True) * x).sum()) < 1e-9
