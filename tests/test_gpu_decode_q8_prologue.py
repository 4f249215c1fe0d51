"""gdn2_decode_multi_q8_prologue in every compiled form: each width, code format and element type, one token
without per-token states (the kernel of its own that plain serving calls), one token with them, and
several tokens. Against the fp64 oracle on the states that the codes stand for, from the oracle's
own pre-processing; the bounds are those of the decode without pre-processing."""
import numpy as np
import pytest
import torch

from tests import serving_ref as R
from tests.parity import TOL, rel_err
from tests.test_gpu_decode_q8 import FORMATS, NAMES, _check_written, _ints, _pool

pytestmark = pytest.mark.gpu
TOL32 = TOL[torch.float32]
WIDTHS = [(64, 64), (64, 128), (128, 64), (128, 128)]


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_160_b200 as g
    g.load_library()
    assert torch.cuda.is_available()
    return g


def _raw(N, n_tok, h_qk, h_v, dk, dv, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda h, d: torch.randn(N, n_tok, h, d, generator=gen, device="cuda").to(dtype)  # noqa: E731
    return dict(q=3 * rn(h_qk, dk), k=0.25 * rn(h_qk, dk), v=rn(h_v, dv), log_alpha=rn(h_v, dk), b=rn(h_v, dk), w=rn(h_v, dv))


def _oracle(oracle_mod, raw, n, upto, S0):
    f = {k: t[n, :upto].float().cpu() for k, t in raw.items()}
    q, k, la, b, w = (np.asarray(x, dtype=np.float32) for x in oracle_mod.prologue_ref(f["q"], f["k"], f["log_alpha"], f["b"], f["w"]))
    o, st = oracle_mod.fwd_ref(q, k, f["v"].numpy(), la, b, w, S0=torch.from_numpy(S0[None]), n_seq=1, bf16=False)
    return o, st[0]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", WIDTHS)
@pytest.mark.parametrize("n_tok,steps", [(1, False), (1, True), (3, False), (8, True)])
def test_matches_oracle(g, oracle_mod, fmt, dtype, dk, dv, n_tok, steps):
    """Grouped heads, sequences without a slot, a key of zeros and saturated gates."""
    slots = [4, -1, 0, 6, 2]  # -1 and 6 (>= n_slots) are skipped
    N, h_qk, h_v, n_slots = len(slots), 2, 4, 6
    raw = _raw(N, n_tok, h_qk, h_v, dk, dv, dtype, seed=dk + 2 * dv + n_tok)
    raw["k"][2, 0, 1] = 0.0
    raw["b"][0, 0, 0, ::5], raw["w"][0, 0, 0, ::7], raw["log_alpha"][0, -1, 1, ::3] = 30.0, -30.0, 30.0
    raw["log_alpha"][4, 0, 2, ::4] = -30.0
    codes, scales = _pool(n_slots, h_v, dk, dv, fmt, seed=dv + 1)
    S0, c0, s0 = R.read_back(codes, scales), codes.clone(), scales.clone()
    o = torch.full((N, n_tok, h_v, dv), 123.0, device="cuda")
    _, cs, ss = g.gdn2_decode_multi_q8(*(raw[k] for k in NAMES), codes, scales, slots=_ints(slots), o=o, want_steps=steps, prologue=True)
    torch.cuda.synchronize()
    got, want = [], []
    for n, s in enumerate(slots):
        if not 0 <= s < n_slots:
            assert torch.all(o[n] == 123.0)
            continue
        for t in range(n_tok if steps else 0):
            _check_written(cs[n, t], ss[n, t], _oracle(oracle_mod, raw, n, t + 1, S0[s])[1], fmt)
        ref_o, ref_s = _oracle(oracle_mod, raw, n, n_tok, S0[s])
        _check_written(codes[s], scales[s], ref_s, fmt)
        got.append(o[n])
        want.append(ref_o)
    assert rel_err(torch.stack(got), np.stack(want)) <= TOL32
    rest = [s for s in range(n_slots) if s not in slots]
    assert torch.equal(codes.view(torch.uint8)[rest], c0.view(torch.uint8)[rest]) and torch.equal(scales[rest], s0[rest])
    assert g.gdn2_device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", WIDTHS)
def test_one_token_with_and_without_per_token_states(g, fmt, dtype, dk, dv):
    """Two kernels, the same bits; more (sequence, head) pairs than the GPU holds CTAs, some sequences without a slot."""
    N, H = 70, 32
    raw = _raw(N, 1, 16, H, dk, dv, dtype, seed=21)
    codes, scales = _pool(N, H, dk, dv, fmt, seed=21)
    slots = torch.randperm(N, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    slots[::9] = -1
    o = torch.full((N, 1, H, dv), 123.0, device="cuda")
    c1, s1, o1 = codes.clone(), scales.clone(), o.clone()
    g.gdn2_decode_multi_q8(*(raw[k] for k in NAMES), codes, scales, slots=slots.cuda(), o=o, prologue=True)
    _, cs, ss = g.gdn2_decode_multi_q8(*(raw[k] for k in NAMES), c1, s1, slots=slots.cuda(), o=o1, want_steps=True, prologue=True)
    assert torch.equal(o, o1) and torch.equal(codes.view(torch.uint8), c1.view(torch.uint8)) and torch.equal(scales, s1)
    live = [n for n in range(N) if slots[n] >= 0]
    home = slots[live].long().cuda()
    assert torch.equal(cs.view(torch.uint8)[live, 0], codes.view(torch.uint8)[home]) and torch.equal(ss[live, 0], scales[home])
    assert torch.all(o[::9] == 123.0) and not torch.any(o[live] == 123.0)
