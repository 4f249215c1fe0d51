"""gdn2_verify_drafts at the edges of what gdn2.h says about its numbers: random numbers outside [0, 1] in
the acceptance. Every expected value follows from the header's words."""
import pytest
import torch

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_160_b200 as g
    g.load_library()
    assert torch.cuda.is_available()
    return g


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("u,p,q,accepted", [
    # below 0: as 0, so accepted exactly where the target gives the token any probability
    (-1.0, 0.0, 0.5, 0), (-INF, 0.0, 0.5, 0), (-1e-30, 0.0, 0.5, 0), (-0.0, 0.0, 0.5, 0), (0.0, 0.0, 0.5, 0),
    (-1.0, 0.25, 0.5, 1), (-INF, 0.25, 0.5, 1), (-INF, 0.25, 0.0, 1), (-INF, 0.0, 0.0, 0), (-1.0, NAN, 0.5, 0),
    # above 1: the product as it is
    (2.0, 0.1875, 0.125, 0), (2.0, 0.1875, 0.0625, 1), (1.0, 0.1875, 0.125, 1), (INF, 0.5, 0.25, 0), (INF, 0.5, 0.0, 0), (1e30, 0.5, 0.25, 0),
    # not a number: refused
    (NAN, 0.5, 0.25, 0), (NAN, 0.5, 0.0, 0),
])
def test_acceptance_outside_the_unit_interval(g, dtype, u, p, q, accepted):
    V = 8
    target = torch.zeros(1, 2, V, dtype=dtype, device="cuda")
    draft = torch.zeros(1, 1, V, dtype=dtype, device="cuda")
    target[0, :, 5] = 0.5  # what is drawn otherwise
    target[0, 0, 3], draft[0, 0, 3] = p, q
    t = torch.full((1, 1), 3, dtype=torch.int32, device="cuda")
    a, tokens = g.gdn2_verify_drafts(target, draft, t, torch.full((1, 1), u, device="cuda"), torch.full((1,), 0.999, device="cuda"))
    assert a.tolist() == [accepted]
    assert tokens.tolist() == ([[3, 5]] if accepted else [[5, -1]])


@pytest.mark.parametrize("u,p,accepted", [(-1.0, 0.0, 0), (-INF, 0.0, 0), (-1.0, 1e-30, 1), (2.0, 1.0, 0), (NAN, 1.0, 0), (0.0, 0.0, 0)])
def test_acceptance_outside_the_unit_interval_of_certain_drafts(g, u, p, accepted):
    target = torch.zeros(1, 2, 8, device="cuda")
    target[0, :, 5] = 0.5
    target[0, 0, 3] = p
    t = torch.full((1, 1), 3, dtype=torch.int32, device="cuda")
    a, _ = g.gdn2_verify_drafts(target, None, t, torch.full((1, 1), u, device="cuda"), torch.full((1,), 0.5, device="cuda"))
    assert a.tolist() == [accepted]
