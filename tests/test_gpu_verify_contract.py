"""gdn2_verify_drafts at the edges of what gdn2.h says about its numbers: random numbers outside [0, 1] in
the acceptance, and how exactly the weights of a row are summed. Every expected value is worked
out here from the header's words, in exact arithmetic."""
from fractions import Fraction

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


def _as_values(x, dtype):
    """Values of this type that add up to the fraction x exactly, largest first."""
    out = []
    while x > 0:
        v = torch.tensor(float(x), dtype=torch.float64).to(dtype).double().item()
        if Fraction(v) > x:  # rounded up: the value below it
            v = torch.nextafter(torch.tensor(v, dtype=dtype), torch.tensor(0.0, dtype=dtype)).double().item()
        out.append(v)
        x -= Fraction(v)
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("stride", [1, 4, 8])
@pytest.mark.parametrize("V,at", [(2048, 0), (2049, 0), (8192, 5), (131072, 70), (131075, 70)])
def test_sums_of_differences_keep_small_remainders(g, dtype, stride, V, at):
    """A block of 1024 weights p - q: 32 near 1, ``stride`` apart, whose rounding to 24 bits leaves 2^-24, and 992 near
    2^-24 whose rounding leaves 2^-48. If remainders were added in 24 bits, 32 times 31 of the latter could
    vanish beside one of the former: 31 2^-48 of the block. The header allows 2^-45, that is 8 2^-48, for the
    border behind the block and as much for the target. The target, 1 / 16 of the row, is put 24 2^-48
    above the block's sum: the draw is the first token behind the block."""
    big, small = (1 + 2.0 ** -7, 2.0 ** -24), (2.0 ** -24 * (1 + 2.0 ** -7), 2.0 ** -48)
    p = torch.zeros(1, 2, V, dtype=torch.float64)
    q = torch.zeros(1, 1, V, dtype=torch.float64)
    j0 = 1024 * at
    p[0, 0, j0:j0 + 1024], q[0, 0, j0:j0 + 1024] = small
    p[0, 0, j0:j0 + 32 * stride:stride], q[0, 0, j0:j0 + 32 * stride:stride] = big
    block = 32 * (Fraction(big[0]) - Fraction(big[1])) + 992 * (Fraction(small[0]) - Fraction(small[1]))
    target = block + 32 * 24 * Fraction(1, 2 ** 48)
    for i, v in enumerate(_as_values(16 * target - block, dtype)):
        p[0, 0, j0 + 1024 + i] = v
    q[0, 0, V - 1] = 0.5  # the drafted token, refused: the target gives it nothing
    p, q = p.to("cuda"), q.to("cuda")
    assert torch.equal(p.to(dtype).double(), p) and torch.equal(q.to(dtype).double(), q)
    drafts = torch.full((1, 1), V - 1, dtype=torch.int32, device="cuda")
    a, t = g.gdn2_verify_drafts(p.to(dtype), q.to(dtype), drafts, torch.full((1, 1), 0.5, device="cuda"), torch.full((1,), 1 / 16, device="cuda"))
    assert a.tolist() == [0] and t.tolist() == [[j0 + 1024, -1]]
