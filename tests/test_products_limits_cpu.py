"""Limits of the grouped products, the output layer with its loss and the
4-bit weights that show without a device: every call below returns before any
HIP call."""
import pytest

from fp32_sgemm_tuning_amd import capi

AL = 0x10000                        # a fake device address, aligned; never dereferenced


@pytest.mark.parametrize("M", range(1, 9))
@pytest.mark.parametrize("N", [17_180_000, 1 << 25, 1 << 26, 1 << 28, 1 << 30])
def test_pieces_of_a_large_vocabulary_fit_a_descriptor(M, N):
    """P [M, piece] is the transposed operand of dW: its descriptor spans up to
    63 rows of it and 256 columns, which must end below the 2^31 that stands
    for "out of range".  (The workspace bounds the piece's columns from above.)"""
    columns = capi.sgemm_lowp_xent_workspace(M, N, 8, AL, 8, AL, 8, 1) // (2 * M)
    assert 2 * (63 * columns + 256) <= 1 << 31
