"""Which kernel a product runs, by its sizes (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from video_dit_block_b200 import build
    build.build()
    import video_dit_block_b200 as sba
    return sba.lib()


def plan(lib, rows, channels, codes, sms=148):
    columns, splits = ctypes.c_int(-1), ctypes.c_int(-1)
    status = lib.sba_int8_linear_plan(rows, channels, codes, sms, ctypes.byref(columns), ctypes.byref(splits))
    return status, columns.value, splits.value


def test_every_plan_can_be_launched(lib):
    for rows in (1, 2, 7, 8, 100, 128, 129, 333, 1000, 5000, 75648, 65535 * 128, 65535 * 128 + 1, 2 ** 31 - 256):
        for channels in (1, 8, 64, 65, 200, 1000, 5120, 24576, 1 << 24):
            for codes in (16, 128, 144, 512, 4096, 131056):
                status, columns, splits = plan(lib, rows, channels, codes)
                assert status == 0
                if splits == 0:
                    assert columns in (64, 128, 192, 256)
                else:
                    assert columns in (64, 128) and splits in (1, 2, 4, 8)
                    assert splits <= -(-codes // 128)          # no part without a K step
                    assert -(-rows // 128) <= 65535            # row tiles are the grid's second dimension


def test_few_rows_split_and_many_do_not(lib):
    assert plan(lib, 2, 24576, 4096)[2] > 0
    for rows, channels, codes in ((8192, 5120, 5120), (75648, 5120, 5120), (107648, 4096, 4096), (4722, 5376, 21504)):
        assert plan(lib, rows, channels, codes)[2] == 0


@pytest.mark.parametrize("args", [(0, 8, 16), (1, 0, 16), (1, 8, 0), (1, 8, 16, 0)])
def test_refuses_sizes_of_zero(lib, args):
    assert plan(lib, *args)[0] == 1
    assert lib.sba_int8_linear_plan(1, 8, 16, 148, None, None) == 1
