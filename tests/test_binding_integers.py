"""Whole numbers that a call hands to the library as C ints: what an int cannot hold is refused, not
wrapped.  No GPU."""
import numpy as np
import pytest
import torch

import test_linear_attn_abi as abi
from test_linear_attn_abi import rec  # noqa: F401 (the recorder fixture)
from test_sequence_modeling_b200 import ttt

B, H, T, d = 2, 3, 8, 64


@pytest.mark.parametrize("first", [2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1, 1.5, float("nan"), float("inf")])
def test_first_position_outside_an_int_is_refused(rec, first):  # noqa: F811
    x = torch.zeros(B, H, T, d)
    with pytest.raises((ValueError, OverflowError)):
        ttt.ttt_rope(x, None, ttt.Rope(torch.zeros(32)), first_position=first)
    assert rec.names() == []


@pytest.mark.parametrize("first", [0, 5, 5.0, -7, -2 ** 31, 2 ** 31 - T, np.int64(9)])
def test_first_position_arrives_as_given(rec, first):  # noqa: F811
    ttt.ttt_rope(torch.zeros(B, H, T, d), None, ttt.Rope(torch.zeros(32)), first_position=first)
    assert rec.args("ttt_rope")[4] == first


def test_first_position_is_not_looked_at_beside_positions(rec):  # noqa: F811
    ttt.ttt_rope(torch.zeros(B, H, T, d), None, ttt.Rope(torch.zeros(32)), first_position=2 ** 40,
                 positions=torch.zeros(B, T, dtype=torch.int32))
    assert rec.names() == ["ttt_rope"]


def test_last_position_is_the_librarys_check():
    """2**31 - T is the last first_position of T tokens; the library refuses the next one on the host."""
    from test_sequence_modeling_b200.build import build
    build()
    lib = abi.L.load()
    assert abi.rope(lib, p=None, T=T, first=2 ** 31 - T + 1) == abi.L.TTT_ERR_ARG
