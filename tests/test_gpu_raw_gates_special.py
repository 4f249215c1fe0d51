"""Fused pre-processing of gates that are not finite, as the formulas have it: a NaN shows in all that depends on it,
sigmoid(+-inf) is 1 or 0, and a decay exp(-softplus(a)) beyond fp32's range is 0."""
import pytest
import torch

from gated_delta_rule_160_b200 import workloads as W

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
NAMES = ("q", "k", "v", "log_alpha", "b", "w")


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_160_b200 as g
    g.load_library()
    assert torch.cuda.is_available()
    return g


def _raw(lead, dk, dv, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    shape = dict(q=dk, k=dk, v=dv, log_alpha=dk, b=dk, w=dv)
    return {n: torch.randn(*lead, 1, d, generator=gen, device="cuda").to(dtype) for n, d in shape.items()}


def _decode(g, pool, raw, S):
    """(o, state) of one call on a pool that holds S."""
    if pool == "fp32":
        S = S.clone()
        o, _ = g.gdn2_decode_multi(*(raw[n] for n in NAMES), S, prologue=True)
        return o[:, :, 0], S[:, 0]
    codes = torch.zeros(S.shape, dtype=torch.int8 if pool == "int8" else torch.float8_e4m3fn, device="cuda")
    scales = torch.zeros(S.shape[:-1], device="cuda")
    g.gdn2_state_store(S, codes, scales)
    o, _, _ = g.gdn2_decode_multi_q8(*(raw[n] for n in NAMES), codes, scales, prologue=True)
    return o[:, :, 0], g.gdn2_state_load(codes, scales)[:, 0]


@pytest.mark.parametrize("pool", ["fp32", "int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n_tok", [1, 3])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
def test_a_nan_gate_shows(g, pool, dtype, n_tok, dk, dv):
    """Sequence 0: the decay of one channel, 1: its erase gate, 2: the write gate of one column, 3: none; at the first token."""
    raw = _raw((4, n_tok), dk, dv, dtype, seed=1)
    raw["log_alpha"][0, 0, 0, 5] = NAN
    raw["b"][1, 0, 0, 5] = NAN
    raw["w"][2, 0, 0, 7] = NAN
    o, S = _decode(g, pool, raw, W.state_input(4, 1, dk, dv, 0.05, "cuda", seed=1))
    assert torch.isnan(o[:2]).all()                          # q reads the channel in every column
    assert torch.isnan(S[0]).all() and torch.isnan(S[1, 5]).all()
    others = [j for j in range(dv) if j != 7]
    assert torch.isnan(o[2, :, 7]).all() and torch.isfinite(o[2][:, others]).all()
    assert torch.isnan(S[2, :, 7]).all()
    if pool == "fp32":
        assert torch.isfinite(S[2][:, others]).all()         # (in 8 bits a row with a NaN reads back as NaN)
    assert torch.isfinite(o[3]).all() and torch.isfinite(S[3]).all()


@pytest.mark.parametrize("pool", ["fp32", "int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n_tok", [1, 3])
def test_gates_without_bound(g, pool, dtype, n_tok):
    """Decays that erase a state of 1e30 in one token (a = inf, a = 100: 4e-44): as from the zero state, to the
    bit for inf. Erase and write gates of +-inf: as those of +-40, which round to 1 and are below 2^-57."""
    raw = _raw((3, n_tok), 128, 64, dtype, seed=2)
    raw["log_alpha"][0, 0], raw["log_alpha"][1, 0] = INF, 100.0
    S = W.state_input(3, 1, 128, 64, 0.05, "cuda", seed=2)
    S[:2] *= 1e30
    raw["b"][2, 0, 0, ::3], raw["b"][2, 0, 0, 1::3] = INF, -INF
    raw["w"][2, 0, 0, ::3], raw["w"][2, 0, 0, 1::3] = INF, -INF
    raw["log_alpha"][2, 0, 0, ::5] = -INF                     # no decay
    o, St = _decode(g, pool, raw, S)
    tame = {n: t.clone() for n, t in raw.items()}
    for n in ("b", "w", "log_alpha"):
        tame[n][2] = tame[n][2].clamp(-40.0, 40.0)
    zero = S.clone()
    zero[:2] = 0.0
    tame["log_alpha"][:2, 0] = 0.0
    o2, St2 = _decode(g, pool, tame, zero)
    assert torch.equal(o[0], o2[0]) and torch.equal(St[0], St2[0])
    # a = 100: 1e30 times 4e-44 is 4e-14, beside values near 1
    assert float((o[1] - o2[1]).abs().max()) <= 1e-6 * float(o2[1].abs().max())
    # 2^-57 of the terms taken out, and their sums rounded as before: far below one fp32 rounding, which may turn one code
    assert float((o[2] - o2[2]).abs().max()) <= 2.0 ** -20 * float(o2[2].abs().max())
    assert torch.isfinite(o).all() and torch.isfinite(St).all()


@pytest.mark.parametrize("name", ["w", "b"])
def test_a_nan_gate_shows_in_the_prefill(g, name):
    T, at, ch = 130, 70, 9
    raw = _raw((T,), 128, 128, torch.bfloat16, seed=3)
    raw[name][at, 0, ch] = NAN
    o, S = g.gdn2_chunk_fwd(*(raw[n] for n in NAMES), prologue=True)
    if name == "w":  # its column, from its token on
        assert torch.isnan(o[at:, 0, ch]).all() and torch.isnan(S[0, 0, :, ch]).all()
    else:            # the channel's erase is in every column
        assert torch.isnan(o[at:]).all() and torch.isnan(S[0, 0, ch]).all()
