"""Checks on the gfx950 assembly of the grouped products, the output layer and
the 4-bit weights (CPU only: hipcc cross-compiles), as test_kernel_asm.py makes
them for the lean kernels: direct-to-LDS loads stay in flight, buffer descriptors
in scalar registers, and the race-check build poisons the stages that it should.
"""
import pytest

from test_kernel_asm import _device_asm, _kernels, _waits_after_direct_loads, _waterfall_loops

POISON = ["-DSGEMM_LDS_POISON=1"]
UNITS = ("sgemm_group.hip", "sgemm_xent.hip", "sgemm_w4.hip")
# kernels that stream tiles with direct-to-LDS loads, and how many of them there are
STREAMED = {"group_rows_kernel": 16, "group_mixed_kernel": 8, "group_k_kernel": 12, "xent_mixed_kernel": 6, "xent_rows_kernel": 4,
            "xent_dx_kernel": 6, "w4_tile_kernel": 48}


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    return _device_asm({**{u: (u, []) for u in UNITS}, **{"poison:" + u: (u, POISON) for u in UNITS}},
                       tmp_path_factory.mktemp("products_asm"))


def streamed(asm, prefix=""):
    """(name, its entry in STREAMED, lines) of every kernel that streams tiles."""
    for unit in UNITS:
        for name, lines in _kernels(asm[prefix + unit]):
            for key in STREAMED:
                if key in name:
                    yield name, key, lines


def test_every_streaming_kernel_is_looked_at(asm):
    for prefix in ("", "poison:"):
        names = [key for _, key, _ in streamed(asm, prefix)]
        assert {key: names.count(key) for key in STREAMED} == STREAMED


def test_no_waterfall_loops(asm):
    bad = {name: n for name, _, lines in streamed(asm) if (n := _waterfall_loops(lines))}
    assert not bad, bad


def test_loads_stay_in_flight(asm):
    """Direct loads that a wait for all loads follows before the next: the K
    loop waits once per tile, behind its last direct load, so the counted ones
    are few beside the loads; a serialised loop waits after every one."""
    for unit in UNITS:
        waits = _waits_after_direct_loads(asm[unit])
        assert waits
        bad = {name: v for name, v in waits.items() if v[1] > max(4, v[0] // 4)}
        assert not bad, bad


def test_race_check_build_poisons_the_stages(asm):
    """The K loops fill LDS by direct loads alone: what the race-check build adds
    to a kernel's LDS writes is the poison."""
    def writes(prefix):
        return {name: sum("ds_write" in x for x in lines) for name, _, lines in streamed(asm, prefix)}
    plain, poisoned = writes(""), writes("poison:")
    assert set(plain) == set(poisoned)
    bad = {name: (plain[name], poisoned[name]) for name in plain if poisoned[name] <= plain[name]}
    assert not bad, bad
