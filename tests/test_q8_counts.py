"""Counts near 2^31, where the kernels' loops and chunk counts would leave int32: refused on the host."""
import pytest

from test_q8_abi import _append, _map, _read, lib  # noqa: F401

TOP = 2**31 - 1


@pytest.mark.parametrize("over", [0, 1, 2000, 4095])
def test_block_map_counts(lib, over):  # noqa: F811
    assert _map(lib, n=TOP - over) == 2
    assert _map(lib, nb=TOP - over) == 2
    assert _map(lib, rows=1, mb=TOP - 1024 - over // 2, bs=1) == 2  # (a table of TOP - 4096 blocks is taken)


@pytest.mark.parametrize("over", [0, 1, 31, 4095])
def test_append_counts(lib, over):  # noqa: F811
    assert _append(lib, n=TOP - over, hk=1, d=16, kst=16, vst=16) == 2


def test_decode_chunks(lib):  # noqa: F811
    # 65535 x 32768 rows of one chunk: their count and a share's rounding up pass 2^31
    for call in ("np_paged_decode_q8_packed", "np_paged_decode_q8_check"):
        assert _read(lib, call, rows=65535, hk=32768, hq=32768, d=16, mb=1, bs=1) == 2
        assert _read(lib, call, rows=32769, hk=32768, hq=32768, d=16, mb=1, bs=1) == 2
