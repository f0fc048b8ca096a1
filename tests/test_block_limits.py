"""Sizes at the limit of a launch (less than 2^32 threads), on the CPU: the
gated scan's descriptor is refused exactly where its kernels' launch would
pass it. A workgroup has 128 bytes of channels (32 fp32, 64 bf16) of a batch
row, 8 threads a channel, whole workgroups also where there are fewer
channels; rows are rounded up to whole XCDs (64 in the check)."""

import ctypes

import pytest

gss = pytest.importorskip("gru_sequence_scan_amd")
ops = gss.block_ops

OK, E_SHAPE = 0, -2


def _status(dtype, T, B, H):
    d = gss.RnnGatedScanDesc(dtype, T, B, H, 0, 0, B * H, H, B * H, H, 0, 0)
    n = ctypes.c_size_t(0)
    got = [getattr(ops._lib(), fn)(ctypes.byref(d), ctypes.byref(n))
           for fn in ("rnn_gated_scan_workspace_bytes", "rnn_gated_scan_reserve_bytes")]
    assert got[0] == got[1]
    return got[0]


@pytest.mark.parametrize("T", [1, 9, 1000])
@pytest.mark.parametrize("dtype,lanes", [(0, 32), (1, 64)], ids=["f32", "bf16"])
@pytest.mark.parametrize("tiles", [1, 3, 100])
def test_scan_refused_where_a_launch_ends(dtype, lanes, tiles, T):
    most = (2 ** 32 - 1) // (tiles * lanes * 8) - 64     # batch rows
    for H in (tiles * lanes, (tiles - 1) * lanes + 1, (tiles - 1) * lanes + 8):
        assert _status(dtype, T, most, H) == OK
        assert _status(dtype, T, most + 1, H) == E_SHAPE


def test_scan_long_time_is_no_launch_limit():
    """Time is walked inside a workgroup, so its length does not count."""
    for dtype in (0, 1):
        assert _status(dtype, 20_000_000, 64, 4096) == OK
        assert _status(dtype, 2_000_000_000, 1, 8) == OK


@pytest.mark.parametrize("B,H", [(9_000_000, 8), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 1), (1, 2 ** 31 - 1)])
def test_scan_sizes_past_a_launch(B, H):
    assert _status(1, 9, B, H) == E_SHAPE


@pytest.mark.parametrize("dtype,lanes", [(0, 32), (1, 64)], ids=["f32", "bf16"])
def test_scan_cuts_time_only_for_few_tiles_and_long_times(dtype, lanes):
    """The workspace holds the maps of the time's segments: none where the
    tiles reach half of 256 compute units, or the time is short."""
    n = ctypes.c_size_t(0)

    def cut(T, tiles):
        d = gss.RnnGatedScanDesc(dtype, T, 1, tiles * lanes, 0, 0, 8192, 0, 8192, 0, 0, 0)
        assert ops._lib().rnn_gated_scan_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == OK
        return n.value > 0

    assert cut(1024, 1) and cut(1024, 32) and cut(4096, 96) and cut(16384, 127)
    assert not (cut(512, 1) or cut(512, 127) or cut(4096, 128) or cut(16384, 160) or cut(16384, 512))
