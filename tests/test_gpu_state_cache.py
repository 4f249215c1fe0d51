"""gdn2_state_store / gdn2_state_load: codes and scales to the bit against the format's definition in
fp32 (tests/serving_ref.py), the read-back, skipped and shared slots, special values, large offsets;
and gdn2_state_commit / gdn2_state_commit_q8, which move whole states."""
import numpy as np
import pytest
import torch

from tests import serving_ref as R

pytestmark = pytest.mark.gpu

FORMATS = [torch.int8, torch.float8_e4m3fn]


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_160_b200 as g
    g.load_library()
    assert torch.cuda.is_available()
    return g


def _pool(n_slots, h, dk, dv, dtype, fill=0x11):
    codes = torch.full((n_slots, h, dk, dv), fill, dtype=torch.uint8, device="cuda").view(dtype)
    return codes, torch.full((n_slots, h, dk), 7.0, device="cuda")


def _states(n, h, dk, dv, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    S = torch.randn(n, h, dk, dv, generator=gen, device="cuda")
    return S * torch.exp(10 * torch.randn(n, h, dk, 1, generator=gen, device="cuda"))  # rows from ~1e-15 to ~1e15


def _ints(slots):
    return torch.tensor(slots, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", FORMATS)
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("n,h", [(1, 1), (3, 5)])
def test_store_and_load_to_the_bit(g, dtype, dk, dv, n, h):
    S = _states(n, h, dk, dv, seed=dk + dv + n)
    S[0, 0, 0, ::2] = 0.0
    S[0, 0, 1] = torch.linspace(-448, 448, dv, device="cuda")  # ties and whole codes
    S[0, 0, 2] = torch.arange(dv, device="cuda") - dv / 2 + 0.5
    S[0, 0, 3] = 0.0
    S[0, 0, 3, 5] = 448.0
    S[0, 0, 3, 6:26] = 2.0 ** -torch.arange(3, 23, device="cuda").float()  # into e4m3's smallest steps
    n_slots = n + 2
    slots = torch.randperm(n_slots, generator=torch.Generator().manual_seed(1))[:n].tolist()
    codes, scales = _pool(n_slots, h, dk, dv, dtype)
    out = g.gdn2_state_store(S, codes, scales, slots=_ints(slots))
    assert out[0] is codes and out[1] is scales
    back = g.gdn2_state_load(codes, scales, slots=_ints(slots))
    torch.cuda.synchronize()
    want_c, want_s = R.quantise(S.cpu().numpy(), dtype)
    assert np.array_equal(R.values(codes[slots]), want_c)
    assert np.array_equal(scales[slots].cpu().numpy(), want_s)
    assert np.array_equal(back.cpu().numpy(), want_c.astype(np.float32) * want_s[..., None])
    rest = [s for s in range(n_slots) if s not in slots]
    assert torch.all(codes.view(torch.uint8)[rest] == 0x11) and torch.all(scales[rest] == 7.0)


@pytest.mark.parametrize("dtype", FORMATS)
def test_special_rows(g, dtype):
    S = _states(2, 1, 64, 64, seed=3)
    S[0, 0, 0] = 0.0
    S[0, 0, 1, 7] = float("inf")
    S[0, 0, 2, 63] = float("-inf")
    S[0, 0, 3, 0] = float("nan")
    S[0, 0, 4] = 2.0 ** -101
    S[0, 0, 5] = 2.0 ** -100
    S[0, 0, 6] = 1e-42  # subnormal
    S[0, 0, 7] = 3e38
    S[0, 0, 8] = -0.0
    S[0, 0, 9, 1] = 2.0 ** -140  # a subnormal next to ordinary values
    codes, scales = _pool(2, 1, 64, 64, dtype)
    g.gdn2_state_store(S, codes, scales)
    back = g.gdn2_state_load(codes, scales)
    torch.cuda.synchronize()
    want_c, want_s = R.quantise(S.cpu().numpy(), dtype)
    assert np.array_equal(R.values(codes), want_c)
    assert np.array_equal(scales.cpu().numpy(), want_s, equal_nan=True)
    nan = torch.isnan(back[0, 0]).all(-1).cpu()
    assert nan[1] and nan[2] and nan[3] and int(nan.sum()) == 3
    assert not torch.isnan(back[1]).any()
    assert torch.all(back[0, 0, [0, 4, 6, 8]] == 0) and torch.all(back[0, 0, 5] != 0)


@pytest.mark.parametrize("dtype", FORMATS)
def test_scale_of_every_mantissa(g, dtype):
    """The scale a / M is correctly rounded for each of the 2^23 mantissas that a can have, at three
    exponents, and the inverse M / a shows in the codes of a row's other values."""
    top = R.TOP[dtype]
    codes = torch.zeros(1024, 16, 128, 64, dtype=dtype, device="cuda")
    scales = torch.zeros(1024, 16, 128, device="cuda")
    part = 2 ** 21
    col = torch.linspace(0.001, 0.999, 64, device="cuda")
    col[5] = 1.0
    for exponent in (28, 127, 254):
        for first in range(0, 2 ** 23, part):
            a = ((exponent << 23) + first + torch.arange(part, dtype=torch.int32, device="cuda")).view(torch.float32)
            S = (a[:, None] * col).view(1024, 16, 128, 64)
            g.gdn2_state_store(S, codes, scales)
            m = torch.full_like(a, top)  # a tensor: by a number, torch multiplies with a rounded inverse
            assert torch.equal(scales.view(-1), a / m)
            want = S.view(-1, 64) * (m / a)[:, None]
            assert torch.equal(codes.view(-1, 64).float(), want.round() if dtype == torch.int8 else want.to(dtype).float())


@pytest.mark.parametrize("dtype", FORMATS)
def test_slots_skipped_shared_and_absent(g, dtype):
    n, h, d = 4, 2, 64
    S = _states(n, h, d, d, seed=4)
    codes, scales = _pool(5, h, d, d, dtype)
    g.gdn2_state_store(S, codes, scales, slots=_ints([3, -1, 5, 0]))  # -1 and 5 (>= n_slots) are not stored
    want_c, want_s = R.quantise(S.cpu().numpy(), dtype)
    for n_, slot in ((0, 3), (3, 0)):
        assert np.array_equal(R.values(codes[slot]), want_c[n_]) and np.array_equal(scales[slot].cpu().numpy(), want_s[n_])
    assert torch.all(codes.view(torch.uint8)[[1, 2, 4]] == 0x11) and torch.all(scales[[1, 2, 4]] == 7.0)
    # read back: shared slots, and zeros where nothing is cached, into a buffer that held something
    S_out = torch.full((5, h, d, d), 9.0, device="cuda")
    got = g.gdn2_state_load(codes, scales, slots=_ints([3, 3, -7, 0, 99]), S=S_out)
    assert got is S_out
    one = torch.from_numpy(R.read_back(codes, scales)).cuda()
    assert torch.equal(got, torch.stack([one[3], one[3], torch.zeros_like(one[0]), one[0], torch.zeros_like(one[0])]))
    assert torch.equal(g.gdn2_state_load(codes, scales, n_seq=2), one[:2])


@pytest.mark.parametrize("dtype", FORMATS)
def test_offsets_past_32_bits(g, dtype):
    """The last slot of a pool of more than 2^32 code bytes."""
    n_slots, d = 2 ** 18 + 3, 128
    codes = torch.zeros(n_slots, 1, d, d, dtype=torch.uint8, device="cuda").view(dtype)
    scales = torch.zeros(n_slots, 1, d, device="cuda")
    assert codes.numel() > 2 ** 32
    S = _states(2, 1, d, d, seed=5)
    slots = _ints([n_slots - 1, 1])
    g.gdn2_state_store(S, codes, scales, slots=slots)
    back = g.gdn2_state_load(codes, scales, slots=slots)
    want_c, want_s = R.quantise(S.cpu().numpy(), dtype)
    assert np.array_equal(back.cpu().numpy(), want_c.astype(np.float32) * want_s[..., None])
    assert not scales[2:n_slots - 1].any() and not scales[0].any()
    g.gdn2_state_commit_q8(codes[1:3, None], scales[1:3, None], _ints([0, 0]), codes[3:], scales[3:], slots=_ints([n_slots - 5, -1]))
    assert torch.equal(scales[n_slots - 2], scales[1])
    assert torch.equal(codes.view(torch.uint8)[n_slots - 2], codes.view(torch.uint8)[1])


# ---------------------------------------------------------------- commit
@pytest.mark.parametrize("kind", [torch.float32] + FORMATS)
@pytest.mark.parametrize("h,dk,dv", [(1, 64, 64), (3, 128, 64), (2, 128, 128), (5, 64, 128)])
@pytest.mark.parametrize("n_tok", [1, 5, 8])
def test_commit(g, kind, h, dk, dv, n_tok):
    n, n_slots = 6, 9
    gen = torch.Generator(device="cuda").manual_seed(6)
    raw = lambda *s: torch.randint(0, 255, s, generator=gen, device="cuda", dtype=torch.uint8)  # noqa: E731
    slots = [4, 8, -1, 9, 0, 7]
    index = [0, n_tok - 1, 0, 0, n_tok, -1]  # the last two: no such token
    if kind == torch.float32:
        steps, pool = raw(n, n_tok, h, dk, dv, 4), raw(n_slots, h, dk, dv, 4)
        before = pool.clone()
        as_f = lambda x: x.view(torch.float32)[..., 0]  # noqa: E731
        assert g.gdn2_state_commit(as_f(steps), _ints(index), as_f(pool), slots=_ints(slots)).data_ptr() == pool.data_ptr()
    else:
        steps, pool = raw(n, n_tok, h, dk, dv), raw(n_slots, h, dk, dv)
        ss, sc = torch.rand(n, n_tok, h, dk, generator=gen, device="cuda"), torch.rand(n_slots, h, dk, generator=gen, device="cuda")
        before, sc0 = pool.clone(), sc.clone()
        g.gdn2_state_commit_q8(steps.view(kind), ss, _ints(index), pool.view(kind), sc, slots=_ints(slots))
        for i in (0, 1):
            sc0[slots[i]] = ss[i, index[i]]
        assert torch.equal(sc, sc0)
    for i in (0, 1):
        before[slots[i]] = steps[i, index[i]]
    assert torch.equal(pool, before)


def test_commit_without_slots_and_past_32_bits(g):
    """slots None is slot n; a pool and per-token states of more than 2^32 bytes."""
    d, n_slots = 128, 2 ** 16 + 5
    pool = torch.zeros(n_slots, 1, d, d, device="cuda")
    steps = torch.randn(3, 2, 1, d, d, device="cuda")
    g.gdn2_state_commit(steps, _ints([1, 0, 1]), pool)
    assert torch.equal(pool[:3], torch.stack([steps[0, 1], steps[1, 0], steps[2, 1]])) and not pool[3:].any()
    g.gdn2_state_commit(steps, _ints([0, 5, -3]), pool, slots=_ints([n_slots - 1, 4, 5]))
    assert torch.equal(pool[-1], steps[0, 0]) and not pool[3:-1].any()


def test_arguments_are_checked(g):
    S = torch.zeros(2, 1, 64, 64, device="cuda")
    codes, scales = _pool(3, 1, 64, 64, torch.int8)
    with pytest.raises(TypeError, match="codes is torch.uint8"):
        g.gdn2_state_store(S, codes.view(torch.uint8), scales)
    with pytest.raises(ValueError, match="scales has shape"):
        g.gdn2_state_store(S, codes, scales[:2])
    with pytest.raises(ValueError, match="S has shape"):
        g.gdn2_state_store(S[:, :, :, :32].contiguous(), codes, scales)
    with pytest.raises(ValueError, match="contiguous"):
        g.gdn2_state_store(S.transpose(2, 3), codes, scales)
    with pytest.raises(TypeError, match="slots"):
        g.gdn2_state_load(codes, scales, slots=torch.tensor([0], device="cuda"))
    with pytest.raises(ValueError, match="n_seq = 3"):
        g.gdn2_state_load(codes, scales, n_seq=3, slots=_ints([0, 1]))
    with pytest.raises(g.Gdn2Error, match="n_slots = 3 too small"):
        g.gdn2_state_load(codes, scales, n_seq=4)
    with pytest.raises(ValueError, match="S_steps has shape"):
        g.gdn2_state_commit(S, _ints([0, 0]), S)
    with pytest.raises(TypeError, match="code_steps is"):
        g.gdn2_state_commit_q8(codes[:2, None].view(torch.float8_e4m3fn), scales[:2, None], _ints([0, 0]), codes, scales)
    with pytest.raises(ValueError, match="index has shape"):
        g.gdn2_state_commit(S[:, None], _ints([0]), S)
