"""Checks on the gfx950 assembly of the 8-bit products (CPU only: hipcc
cross-compiles), as test_products_asm.py makes them for the 16-bit ones."""
import pytest

from test_kernel_asm import _device_asm, _kernels, _waits_after_direct_loads, _waterfall_loops

UNIT = "sgemm_i8.hip"
# kernels that stream tiles with direct-to-LDS loads, and how many of them there are
STREAMED = {"i8_tile_kernel": 5, "i8_wide_kernel": 1, "i8_share_kernel": 1}


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    return _device_asm({"": (UNIT, []), "poison": (UNIT, ["-DSGEMM_LDS_POISON=1"])}, tmp_path_factory.mktemp("i8_asm"))


def streamed(asm, build=""):
    return [(name, key, lines) for name, lines in _kernels(asm[build]) for key in STREAMED if key in name]


def test_every_streaming_kernel_is_looked_at(asm):
    for build in asm:
        names = [key for _, key, _ in streamed(asm, build)]
        assert {key: names.count(key) for key in STREAMED} == STREAMED


def test_integers_are_multiplied_by_matrix_instructions(asm):
    for name, _, lines in streamed(asm):
        assert any("v_mfma_i32_16x16x64_i8" in x for x in lines), name


def test_no_waterfall_loops(asm):
    bad = {name: n for name, _, lines in streamed(asm) if (n := _waterfall_loops(lines))}
    assert not bad, bad


def test_loads_stay_in_flight(asm):
    waits = _waits_after_direct_loads(asm[""])
    assert waits
    bad = {name: v for name, v in waits.items() if v[1] > max(4, v[0] // 4)}
    assert not bad, bad


def test_no_kernel_spills(asm):
    for name, lines in _kernels(asm[""]):
        assert not any("scratch_" in x for x in lines), name


def test_race_check_build_poisons_the_stages(asm):
    def writes(build):
        return {name: sum("ds_write" in x for x in lines) for name, _, lines in streamed(asm, build)}
    plain, poisoned = writes(""), writes("poison")
    assert set(plain) == set(poisoned)
    bad = {name: (plain[name], poisoned[name]) for name in plain if poisoned[name] <= plain[name]}
    assert not bad, bad
