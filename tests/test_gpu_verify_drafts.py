"""gdn2_verify_drafts against a loop in fp64 over the same inputs (tests/serving_ref.py). The results
are whole numbers and have to be equal: the loop's sums are good to 2^-53 relative, the kernel's to 2^-48, and a border of the CDF lies
within that of a random number about once in 10^9 draws over the largest rows here."""
import numpy as np
import pytest
import torch

from tests import serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_160_b200 as g
    g.load_library()
    assert torch.cuda.is_available()
    return g


def _case(N, n, V, dtype, seed, sharp=3.0, q=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    logits = sharp * torch.randn(N, n + 1, V, generator=gen, device="cuda")
    p = torch.softmax(logits, -1).to(dtype)
    near = logits[:, :n] * 0.9 + 0.7 * torch.randn(N, n, V, generator=gen, device="cuda")
    qd = torch.softmax(near, -1).to(dtype)
    drafts = torch.distributions.Categorical(probs=qd.float().clamp(min=1e-30)).sample() if n else torch.zeros(N, 0, device="cuda")
    u = torch.rand(N, n, generator=gen, device="cuda")
    ul = torch.rand(N, generator=gen, device="cuda")
    return p.contiguous(), (qd.contiguous() if q else None), drafts.to(torch.int32), u, ul


def _ref(p, q, drafts, u, ul, lens=None):
    f = lambda x: None if x is None else x.double().cpu().numpy()  # noqa: E731
    return R.verify(f(p), f(q), drafts.cpu().numpy(), f(u), f(ul), None if lens is None else lens.cpu().numpy())


def _check(g, p, q, drafts, u, ul, lens=None):
    a, t = g.gdn2_verify_drafts(p, q, drafts, u, ul, n_drafted=lens)
    torch.cuda.synchronize()
    want_a, want_t = _ref(p, q, drafts, u, ul, lens)
    assert a.cpu().tolist() == want_a.tolist()
    assert t.cpu().tolist() == want_t.tolist()
    return a.cpu(), t.cpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 64, 1000, 1023, 1024, 1025, 4097, 8200, 33000])
@pytest.mark.parametrize("n", [0, 1, 3, 7])
@pytest.mark.parametrize("q", [True, False])
def test_matches_the_definition(g, dtype, V, n, q):
    N = 9 if V <= 8200 else 4
    p, qd, drafts, u, ul = _case(N, n, V, dtype, seed=V * 8 + n, sharp=1.5, q=q)
    gen = torch.Generator().manual_seed(V + n)
    lens = torch.randint(-1, n + 2, (N,), generator=gen).to(torch.int32).cuda()  # inactive to one too many
    _check(g, p, qd, drafts, u, ul)
    _check(g, p, qd, drafts, u, ul, lens)


def test_most_drafts(g):
    n = 31
    p, q, drafts, _, ul = _case(6, n, 500, torch.float32, seed=3, sharp=0.2)
    u = torch.zeros(6, n, device="cuda")
    u[0, 0] = u[1, 30] = u[2, 15] = 1e30
    a, t = _check(g, p, q, drafts, u, ul)
    assert a.tolist() == [0, 30, 15, 31, 31, 31]
    with pytest.raises(g.Gdn2Error, match="n_draft = 32"):
        g.gdn2_verify_drafts(*_case(1, 32, 8, torch.float32, seed=3))


@pytest.mark.parametrize("V", [130000, 262147, 1048576, 4194303, 4194304])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_vocabularies(g, V, dtype):
    """Every accepted length, the first and last tokens and both ends of the random number."""
    n, N = 2, 6
    p, q, drafts, u, ul = _case(N, n, V, dtype, seed=V)
    ul[0], ul[1], ul[2] = 0.0, 1.0, 1.0 - 2.0 ** -24
    u[0] = u[3, 0] = 1.0
    u[1] = u[4] = 0.0
    _check(g, p, q, drafts, u, ul)


def test_most_sequences(g):
    N = 65535
    p, q, drafts, u, ul = _case(N, 2, 9, torch.float32, seed=8)
    lens = (torch.arange(N, device="cuda") % 4 - 1).to(torch.int32)
    _check(g, p, q, drafts, u, ul, lens)


def test_all_the_weight_in_one_place(g):
    """The drawn token is found wherever it is: at the first and last value of the row, of a block and of
    a thread's share."""
    V = 70001
    places = [0, 1, 31, 32, 127, 128, 1023, 1024, 1025, 2047, 8191, 8192, 65535, 65536, 69999, 70000]
    p = torch.zeros(len(places), 1, V, device="cuda")
    for i, j in enumerate(places):
        p[i, 0, j] = 0.25
    none = torch.zeros(len(places), 0, device="cuda")
    for ul in (0.0, 0.5, 1.0):
        a, t = g.gdn2_verify_drafts(p, None, none.to(torch.int32), none, torch.full((len(places),), ul, device="cuda"))
        assert t[:, 0].tolist() == places and a.tolist() == [0] * len(places)


def test_borders_of_the_cdf(g):
    """Weights of exact binary fractions: a random number on a border belongs to the token behind it."""
    p = torch.tensor([0.25, 0.0, 0.5, 0.0, 0.25, 0.0], device="cuda")
    want = {0.0: 0, 0.125: 0, 0.25: 2, 0.5: 2, 0.75: 4, 0.999: 4, 1.0: 4}
    N = len(want)
    none = torch.zeros(N, 0, device="cuda")
    _, t = g.gdn2_verify_drafts(p.repeat(N, 1, 1), None, none.to(torch.int32), none, torch.tensor(list(want), device="cuda"))
    assert t[:, 0].tolist() == list(want.values())
    # acceptance is strict: u q < p
    p2 = torch.tensor([[[0.25, 0.75], [0.5, 0.5]]], device="cuda")
    q2 = torch.tensor([[[0.5, 0.5]]], device="cuda")
    for u, taken in ((0.5, 0), (0.5 - 2.0 ** -25, 1)):
        a, _ = g.gdn2_verify_drafts(p2, q2, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([[u]], device="cuda"),
                                    torch.zeros(1, device="cuda"))
        assert a.tolist() == [taken]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [50, 2048, 5001])
def test_rows_without_weight_and_bad_values(g, dtype, V):
    """Empty residuals, empty rows, NaN, infinite and negative probabilities, tokens outside the
    vocabulary, random numbers outside [0, 1]."""
    N, n = 12, 2
    p, q, drafts, u, ul = _case(N, n, V, dtype, seed=V)
    u[:] = 1.0  # every draft is refused unless p > q
    q[0] = p[0, :2]  # nothing is left of the residual
    q[1] = 2 * p[1, :2]
    p[2] = 0.0  # nothing at all
    p[3] = float("nan")
    p[4, :, ::3], q[4, :, 1::3] = float("inf"), float("nan")
    p[5, :, ::2], q[5] = -p[5, :, ::2], -1.0
    drafts[6, 0], drafts[7, 0], drafts[8, 0] = -1, V, 2 ** 31 - 1
    ul[6], ul[7], ul[8] = -3.0, 7.0, float("nan")
    u[9, 0], u[10, 0], u[11, 0] = float("nan"), -1.0, float("inf")
    a, t = _check(g, p, q, drafts, u, ul)
    assert t[2].tolist() == [-1, -1, -1] and t[3].tolist() == [-1, -1, -1]
    assert a[[6, 7, 8]].tolist() == [0, 0, 0]
    a, t = _check(g, p, None, drafts, u, ul)


def test_row_offsets_past_32_bits(g):
    """More than 2^32 bytes and 2^31 values of probabilities; only a few are not zero."""
    N, n, V = 260, 7, 1048577
    p = torch.zeros(N, n + 1, V, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(N, n, V, dtype=torch.bfloat16, device="cuda")
    assert p.numel() > 2 ** 31
    i = torch.arange(N, device="cuda")
    taken = i % 8
    drafts = (i[:, None] * 31 + torch.arange(n, device="cuda") * 7919) % V
    p.scatter_(2, torch.cat([drafts, drafts[:, :1]], 1)[..., None], 0.5)
    q.scatter_(2, drafts[..., None], 0.5)
    new = V - 1 - i
    p[i, taken, new] = 0.25
    u = torch.zeros(N, n, device="cuda")
    u[i[taken < n], taken[taken < n]] = 1.0  # refused: 1 q < p does not hold
    a, t = g.gdn2_verify_drafts(p, q, drafts.to(torch.int32), u, torch.full((N,), 0.999, device="cuda"))
    assert torch.equal(a, taken.to(torch.int32))
    assert torch.equal(t[i, taken], new.to(torch.int32))
    assert torch.equal(t[7, :7], drafts[7].to(torch.int32))


def test_unaligned_rows(g):
    """Inputs that start anywhere a value may start."""
    p, q, drafts, u, ul = _case(3, 2, 1001, torch.bfloat16, seed=5)
    want = _ref(p, q, drafts, u, ul)

    def moved(x, by):
        y = torch.empty(x.numel() + by, dtype=x.dtype, device="cuda")[by:].view(x.shape)
        y.copy_(x)
        return y

    for by in (1, 3, 4, 8):
        a, t = g.gdn2_verify_drafts(moved(p, by), moved(q, by + 1), moved(drafts, by), moved(u, by), moved(ul, 1),
                                    n_accepted=moved(torch.zeros(3, dtype=torch.int32, device="cuda"), by),
                                    tokens=moved(torch.zeros(3, 3, dtype=torch.int32, device="cuda"), by))
        assert a.tolist() == want[0].tolist() and t.tolist() == want[1].tolist()


def test_frequencies_follow_the_target(g):
    """Over 20000 sequences with drafts from q, the first token's shares are p's: within five standard
    deviations, sqrt(p (1 - p) / n) each."""
    N, V = 20000, 5
    p = torch.tensor([0.4, 0.3, 0.2, 0.1, 0.0], device="cuda")
    q = torch.tensor([0.1, 0.2, 0.3, 0.2, 0.2], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(6)
    drafts = torch.multinomial(q, N, replacement=True, generator=gen)[:, None].to(torch.int32)
    _, t = g.gdn2_verify_drafts(p.repeat(N, 2, 1), q.repeat(N, 1, 1), drafts, torch.rand(N, 1, generator=gen, device="cuda"),
                                torch.rand(N, generator=gen, device="cuda"))
    share = torch.bincount(t[:, 0].long(), minlength=V).double() / N
    assert torch.all((share.cuda() - p).abs() <= 5 * (p * (1 - p) / N).sqrt() + 1e-12)


def test_arguments_are_checked(g):
    p, q, drafts, u, ul = _case(3, 2, 100, torch.float32, seed=7)
    with pytest.raises(TypeError, match="draft_probs is"):
        g.gdn2_verify_drafts(p, q.to(torch.bfloat16), drafts, u, ul)
    with pytest.raises(TypeError, match="unsupported element type"):
        g.gdn2_verify_drafts(p.half(), q.half(), drafts, u, ul)
    with pytest.raises(ValueError, match="draft_probs has shape"):
        g.gdn2_verify_drafts(p, q[..., :99].contiguous(), drafts, u, ul)
    with pytest.raises(TypeError, match="draft_tokens is"):
        g.gdn2_verify_drafts(p, q, drafts.long(), u, ul)
    with pytest.raises(ValueError, match="contiguous"):
        g.gdn2_verify_drafts(p[..., ::2], q[..., ::2].contiguous(), drafts, u, ul)
    with pytest.raises(ValueError, match="u_sample has shape"):
        g.gdn2_verify_drafts(p, q, drafts, u, u)
    with pytest.raises(TypeError, match="n_drafted"):
        g.gdn2_verify_drafts(p, q, drafts, u, ul, n_drafted=torch.tensor([1, 1, 1], device="cuda"))
    with pytest.raises(ValueError, match="no place"):
        g.gdn2_verify_drafts(p[:, :0], None, drafts, u, ul)
