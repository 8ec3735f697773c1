"""The block norm's backward workspace holds a part of the column sums for each
workgroup that gets rows, and no more (CPU only)."""
import ctypes

import pytest

import ssd_chunked_scan_amd as ssd


def workspace(rows, columns, io):
    s = ssd.BlockShape(rows, columns, 0, 0, 0, 0, 0, 1e-5, 1.0)
    return ssd.load_library().ssd_block_norm_bwd_workspace_bytes(ctypes.byref(s), io)


def parts(n, columns):
    """n parts of two sums a column, columns in whole packs of eight, in all a multiple of 256 bytes."""
    return -(-n * 2 * 4 * (-(-columns // 8) * 8) // 256) * 256


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("rows", [1, 3, 4, 5, 64, 201])
def test_four_rows_share_a_workgroup_where_a_wave_takes_one(rows, io):
    for columns in (1, 8, 96, 256):
        assert workspace(rows, columns, io) == parts(-(-rows // 4), columns), columns


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("rows", [1, 3, 64])
def test_a_row_has_a_workgroup_past_that(rows, io):
    """From 257 columns on for single columns, which the buffers' alignment may ask for."""
    for columns in (257, 512, 520, 2560, 16384):
        assert workspace(rows, columns, io) == parts(rows, columns), columns
