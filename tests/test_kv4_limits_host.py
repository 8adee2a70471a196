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
