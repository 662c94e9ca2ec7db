"""The path setting of the linear attention entry points, without a GPU."""
import pytest

from test_linear_attn_abi import bwd, fwd, lib  # noqa: F401 (lib: the built library)
from test_sequence_modeling_b200 import _lib as L


@pytest.mark.parametrize("fn", [fwd, bwd])
def test_tensor_core_path_refuses_fp32(lib, fn):  # noqa: F811
    """TTT_PATH_TC: no tensor-core kernel takes fp32 inputs."""
    n0 = lib.ttt_launch_count()
    prev = lib.ttt_set_path(L.TTT_PATH_TC)
    try:
        for T in (1, 128, 2000):
            assert fn(lib, dt=L.TTT_F32, T=T) == L.TTT_ERR_UNSUPPORTED
        assert fn(lib, dt=L.TTT_F32, B=0) == L.TTT_OK
        # What is wrong by itself stays an argument error.
        assert fn(lib, dt=L.TTT_F32, scale=float("nan")) == L.TTT_ERR_ARG
        assert fn(lib, Z=None) == L.TTT_ERR_ARG
    finally:
        lib.ttt_set_path(prev)
    assert lib.ttt_launch_count() == n0
