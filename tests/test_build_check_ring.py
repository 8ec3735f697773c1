"""The build's check of waits in a loop around a ring of direct-to-LDS loads, and
of buffer loads into LDS (CPU only)."""
import pytest

from ssd_chunked_scan_amd import _build
from test_build_check import _asm


def _ring(before, inside, keep):
    """A ring's loop: `before` loads ahead of it, `inside` in each round after the wait."""
    load = "buffer_load_dwordx4 v2, s[4:7], 0 offen lds"
    return _asm(*[load] * before, ".LBB0_1:", "; ssd ring wait", f"s_waitcnt vmcnt({keep}) lgkmcnt(0)", "s_barrier", *inside,
                "s_cbranch_scc0 .LBB0_1", "s_endpgm")


def test_ring_wait_follows_the_loop_back():
    load = "buffer_load_dwordx4 v2, s[4:7], 0 offen lds"
    assert _build.check_counted_barrier_waits(_ring(6, [load] * 2, 4), "t") == 1
    # too few loads before the first round
    with pytest.raises(RuntimeError, match="short"):
        _build.check_counted_barrier_waits(_ring(3, [load] * 2, 4), "t")
    # an ordinary load among the newest, on the way around
    with pytest.raises(RuntimeError, match="ordinary"):
        _build.check_counted_barrier_waits(_ring(6, [load, "global_load_dword v3, v[4:5], off", load], 4), "t")
    with pytest.raises(RuntimeError, match="ordinary"):
        _build.check_counted_barrier_waits(_ring(6, [load, load, "buffer_store_dword v3, v4, s[4:7], 0 offen"], 4), "t")


def test_buffer_loads_to_lds_are_seen_as_such():
    load = "buffer_load_dwordx4 v2, s[4:7], 0 offen lds"
    with pytest.raises(RuntimeError, match="direct-to-LDS"):
        _build.check_counted_barrier_waits(_asm(load, "s_waitcnt vmcnt(1) lgkmcnt(0)", "s_barrier"), "t")
    assert _build.check_counted_barrier_waits(
        _asm(load, load, "; ssd lookahead wait 0", "s_waitcnt vmcnt(1) lgkmcnt(0)", "s_barrier"), "t") == 1
