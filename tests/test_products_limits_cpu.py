"""Limits of the grouped products, the output layer with its loss and the
4-bit weights that show without a device: every call below returns before any
HIP call."""
import pytest

from fp32_sgemm_tuning_amd import capi
from w4_forms import FORMS, SHAPES

AL = 0x10000                        # a fake device address, aligned; never dereferenced


@pytest.mark.parametrize("M", range(1, 9))
@pytest.mark.parametrize("N", [17_180_000, 1 << 25, 1 << 26, 1 << 28, 1 << 30])
def test_pieces_of_a_large_vocabulary_fit_a_descriptor(M, N):
    """P [M, piece] is the transposed operand of dW: its descriptor spans up to
    63 rows of it and 256 columns, which must end below the 2^31 that stands
    for "out of range".  (The workspace bounds the piece's columns from above.)"""
    columns = capi.sgemm_lowp_xent_workspace(M, N, 8, AL, 8, AL, 8, 1) // (2 * M)
    assert 2 * (63 * columns + 256) <= 1 << 31


@pytest.mark.parametrize("form,M,N", SHAPES)
def test_form_of_a_4bit_product(form, M, N):
    """The shapes the 4-bit products are tested on take every launch form."""
    assert capi.sgemm_w4_select_form(M, N) == form


def test_forms_of_4bit_products():
    assert {f for f, _, _ in SHAPES} == set(FORMS)
    seen = {capi.sgemm_w4_select_form(M, N) for M in (1, 16, 17, 64, 65, 100, 128, 256, 1000, 4096)
            for N in (1, 100, 3200, 4096, 6400, 8192, 12800, 14336, 50000)}
    assert seen == set(FORMS)
    for bad in ((-1, 5), (5, -1)):
        assert capi.sgemm_w4_select_form(*bad) == capi.SGEMM_STATUS_INVALID_DIM
