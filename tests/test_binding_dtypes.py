"""What the binding allocates for a call has the type that the library writes, whatever torch's default
type is: a buffer of a narrower one would be written past its end.  No GPU."""
import pytest
import torch

from test_binding import rec  # noqa: F401 (the recorder fixture)
from test_sequence_modeling_b200 import ttt

B, H, T, d, b, h = 2, 3, 32, 64, 16, 256


@pytest.fixture(params=[torch.bfloat16, torch.float64], ids=["bf16", "f64"])
def default_type(request):
    before = torch.get_default_dtype()
    torch.set_default_dtype(request.param)
    yield
    torch.set_default_dtype(before)


def _z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def _calls():
    x = [_z(B, H, T, d, dtype=torch.bfloat16) for _ in range(3)]
    q = [_z(B, H, d, dtype=torch.bfloat16) for _ in range(3)]
    e, W, g = _z(B, H, T), _z(H, d, d), _z(H, d)
    W1, W2, dZ = _z(H, d, h), _z(H, h, d), _z(B, H, T, d)
    e1, s1, s2, st = _z(B, H), _z(B, H, d, h), _z(B, H, h, d), _z(B, H, d, d)
    return {
        "linear_fwd": lambda: ttt.ttt_linear_fwd(*x, e, W, b),
        "linear_ln_fwd": lambda: ttt.ttt_linear_ln_fwd(*x, e, W, g, g, b),
        "mlp_fwd": lambda: ttt.ttt_mlp_fwd(*x, e, W1, W2, g, g, b),
        "linear_bwd": lambda: ttt.ttt_linear_bwd(*x, e, W, dZ, b),
        "linear_ln_bwd": lambda: ttt.ttt_linear_bwd(*x, e, W, dZ, b, gamma=g, beta=g),
        "linear_ln_bwd_noalloc": lambda: ttt.ttt_linear_ln_bwd_noalloc(*x, e, W, dZ, b, g, g),
        "mlp_bwd": lambda: ttt.ttt_mlp_bwd(*x, e, W1, W2, g, g, dZ, b),
        "linear_momentum_fwd": lambda: ttt.ttt_linear_momentum_fwd(*x, e, e, e, W, b),
        "mlp_momentum_fwd": lambda: ttt.ttt_mlp_momentum_fwd(*x, e, e, e, W1, W2, g, g, b),
        "linear_decode": lambda: ttt.ttt_linear_decode(*q, e1, st, st.clone(), b, 3),
        "mlp_decode": lambda: ttt.ttt_mlp_decode(*q, e1, s1, s2, s1.clone(), s2.clone(), g, g, b, 3),
    }


def _tensors(out):
    if isinstance(out, torch.Tensor):
        return {"": out}
    return out if isinstance(out, dict) else dict(enumerate(out))


@pytest.mark.parametrize("name", list(_calls()))
def test_outputs_are_fp32(rec, default_type, name):  # noqa: F811
    for n, t in _tensors(_calls()[name]()).items():
        assert t.dtype == torch.float32, (name, n)


def test_linear_attention_outputs(rec, default_type, monkeypatch):  # noqa: F811
    monkeypatch.setattr(ttt, "linear_attn_workspace_bytes", lambda shape, backward=False: 64)
    x = [_z(B, H, T, d, dtype=torch.bfloat16) for _ in range(4)]
    Z, S = ttt.ttt_linear_attn_fwd(*x[:3], _z(H))
    assert Z.dtype == torch.bfloat16 and S.dtype == torch.float32
    out = ttt.ttt_linear_attn_bwd(*x[:3], _z(H), x[3])
    assert {n: t.dtype for n, t in out.items()} == {
        "dQ": torch.bfloat16, "dK": torch.bfloat16, "dV": torch.bfloat16, "dS0": torch.float32}
    f, _ = ttt.rope_frequencies(64)
    assert f.dtype == torch.float32
