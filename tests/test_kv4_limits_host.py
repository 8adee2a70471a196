"""The ends of what the 4-bit cache's and the page operations' entry points accept, without a GPU."""
import pytest

import test_kv4_host as H
from test_kv4_host import BAD


@pytest.mark.parametrize("call", [H.append, H.read])
def test_scales_from_2_to_the_minus_59_to_2_to_the_58(call):
    for name in ("kg", "vg"):
        for e in (-59, 58):
            assert call(n_seq=0, **{name: 2.0 ** e}) == 0
        for e in (-61, -60, 59, 60):
            assert call(n_seq=0, **{name: 2.0 ** e}) == BAD
            assert H.attention(**{name: 2.0 ** e}) == BAD


@pytest.mark.parametrize("bad", [dict(pages_per_seq=1 << 27), dict(pages_per_seq=1 << 20, n_seq=1 << 11),
                                 dict(pages_per_seq=(1 << 31) - 1, n_seq=1), dict(pages_per_seq=1 << 16, n_seq=1 << 30)])
def test_tables_beyond_32_bits(bad):
    """2^31 entries, or rows of 2^31 tokens: the pages that a call asks for are counted in 32 bits."""
    assert H.every_call(H.desc(**bad), nbytes=1 << 50) == [BAD] * 4
    assert H._lib.load().wedlm_kv_pages_compact(H.ctypes.byref(H.desc(**bad)), None, H.P, 1 << 50, None) == BAD


@pytest.mark.parametrize("good", [dict(pages_per_seq=(1 << 27) - 1, n_seq=15), dict(pages_per_seq=(1 << 20) - 1, n_seq=1 << 11)])
def test_tables_up_to_32_bits(good):
    assert H.every_call(H.desc(**good), nbytes=1 << 50, n=0) == [0] * 4
