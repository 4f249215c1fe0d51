"""Refusals of the serving decodes that need no GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def g():
    from gated_delta_rule_160_b200 import build
    build.build()
    import gated_delta_rule_160_b200 as g
    g.load_library()
    return g


@pytest.mark.parametrize("name", ["gdn2_decode_multi", "gdn2_decode_multi_prologue", "gdn2_decode_multi_q8", "gdn2_decode_multi_q8_prologue"])
@pytest.mark.parametrize("h_v", [32768, 32769])
def test_pairs_near_two_to_the_31(g, name, h_v):
    """A persistent CTA goes from one (sequence, head) pair to the next by adding the grid to a 32-bit number: within a
    grid of 2^31 the sum would turn negative and address in front of every tensor."""
    lib = g.load_library()
    X = 0x1000  # never dereferenced
    sh = g.Shape(65535, 65535, 1, h_v, 64, 64, g.GDN2_BF16, g.GDN2_F32)
    assert sh.n_seq * h_v > 2 ** 31 - 2 ** 16
    if "q8" in name:
        st = getattr(lib, name)(ctypes.byref(sh), 0, 1, X, None, X, X, X, X, X, X, X, X, 8, X, None, None, None)
    else:
        st = getattr(lib, name)(ctypes.byref(sh), 1, X, X, X, X, X, X, X, X, 8, X, None, None)
    assert st == 2 and b"pairs above 2^31 - " in lib.gdn2_last_error_string()
