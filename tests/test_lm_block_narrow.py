"""The norms between blocks: rows of 129 to 256 columns, which half a wave holds."""

import pytest
import test_lm_block as block

SHAPES = [(1, 130, 0), (9, 200, 3), (8, 256, 0), (4000, 256, 0), (2500, 249, 1), (37, 257, 0), (5001, 144, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("t,r,p", block.KINDS)
@pytest.mark.parametrize("n,D,gap", SHAPES)
def test_rows_of_half_a_wave(n, D, gap, t, r, p, monkeypatch):
    monkeypatch.setattr(block, "CASES", SHAPES)
    block.test_forward_and_gradients(n, D, gap, t, r, p)
