"""The C++ binding of the serving operators (csrc/binding.cpp): loaded beside the library, and its own
errors. Everything here runs without a GPU."""
import sys

import pytest
import torch


@pytest.fixture(scope="module")
def g():
    from gated_delta_rule_160_b200 import build
    build.build()
    import gated_delta_rule_160_b200 as g
    g.load_library()
    return g


def test_module_is_loaded_with_the_library(g):
    assert sys.modules["gated_delta_rule_160_b200._binding"] is g._binding


def test_argument_counts(g):
    for name, n in (("store", 5), ("load", 6), ("decode", 17), ("verify", 9), ("commit", 5), ("commit_q8", 7)):
        with pytest.raises(TypeError, match=f"{n} arguments expected, 1 given"):
            getattr(g._binding, name)(None)


@pytest.mark.parametrize("bad", [None, 3, "codes", [1, 2], torch.zeros(2, 1, 64, 64, dtype=torch.int8)])
def test_anything_but_a_cuda_tensor_is_refused(g, bad):
    x = torch.zeros(2, 1, 64, 64)
    for call in (lambda: g.gdn2_state_store(x, bad, x), lambda: g.gdn2_state_load(bad, x),
                 lambda: g.gdn2_decode_multi_q8(x, x, x, x, x, x, bad, x), lambda: g.gdn2_verify_drafts(bad, x, x, x, x),
                 lambda: g.gdn2_state_commit(x, x, bad), lambda: g.gdn2_state_commit_q8(x, x, x, bad, x)):
        before = sys.getrefcount(bad)
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
        assert sys.getrefcount(bad) <= before + 1
