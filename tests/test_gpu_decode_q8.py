"""gdn2_decode_multi_q8: decode on an 8-bit pool, against the fp64 oracle run from the states that
the codes stand for. The output bound is the repository's for fp32 arithmetic (the state is exact
when it is read). What is written may be off the oracle's state by half a step of its code plus
that bound."""
import numpy as np
import pytest
import torch

from gated_delta_rule_160_b200 import workloads as W
from tests import serving_ref as R
from tests.parity import TOL, rel_err

pytestmark = pytest.mark.gpu

FORMATS = [torch.int8, torch.float8_e4m3fn]
NAMES = ("q", "k", "v", "log_alpha", "b", "w")
TOL32 = TOL[torch.float32]


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_160_b200 as g
    g.load_library()
    assert torch.cuda.is_available()
    return g


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tokens(N, n_tok, h_qk, h_v, dk, dv, dtype, seed):
    d = W.token_inputs(N * n_tok, h_qk, h_v, dk, dv, dtype, "cuda", seed=seed)
    return {k_: t.view(N, n_tok, *t.shape[1:]) for k_, t in d.items()}


def _pool(n_slots, h, dk, dv, dtype, seed):
    S = W.state_input(n_slots, h, dk, dv, 0.05, "cuda", seed=seed)
    c, s = R.quantise(S.cpu().numpy(), dtype)
    codes = torch.from_numpy(c.astype(np.float32)).cuda().to(dtype).contiguous()
    return codes, torch.from_numpy(s).cuda()


def _check_written(codes, scales, want, dtype):
    """codes, scales of states whose unrounded values should be ``want`` (fp64, [..., dk, dv])."""
    back = R.read_back(codes, scales).astype(np.float64)
    rms = np.sqrt(np.mean(want ** 2))
    assert np.all(np.abs(back - want) <= R.half_step(want, dtype) + 2 * TOL32 * rms)
    top = R.TOP[dtype]
    amax = np.abs(want).max(-1)
    assert np.all(np.abs(scales.cpu().numpy() * top - amax) <= 2 * TOL32 * rms)


def _oracle(oracle_mod, d, n, upto, S0):
    sl = {k_: d[k_][n, :upto].float().cpu() for k_ in NAMES}
    o, st = oracle_mod.fwd_ref(*(sl[k_] for k_ in NAMES), S0=S0[None], n_seq=1)
    return o, st[0]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("n_tok", [1, 2, 3, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_matches_oracle(g, oracle_mod, fmt, dk, dv, n_tok, dtype):
    """Grouped heads, skipped slots, the state after each token, every width, type and format."""
    slots = [4, -1, 8, 0, 9, 2]  # -1 and 9 (>= n_slots) are skipped
    N, h_qk, h_v, n_slots = len(slots), 2, 4, 9
    d = _tokens(N, n_tok, h_qk, h_v, dk, dv, dtype, seed=n_tok + dk)
    codes, scales = _pool(n_slots, h_v, dk, dv, fmt, seed=dv)
    S0, c0, s0 = R.read_back(codes, scales), codes.clone(), scales.clone()
    o = torch.full((N, n_tok, h_v, dv), 123.0, device="cuda")
    cs = torch.full((N, n_tok, h_v, dk, dv), 0x11, dtype=torch.uint8, device="cuda").view(fmt)
    ss = torch.full((N, n_tok, h_v, dk), 7.0, device="cuda")
    ret = g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), codes, scales, slots=_ints(slots), o=o, code_steps=cs, scale_steps=ss)
    assert ret[0] is o and ret[1] is cs and ret[2] is ss
    torch.cuda.synchronize()
    o_got, o_ref = [], []
    for n, s in enumerate(slots):
        if not 0 <= s < n_slots:
            assert torch.all(o[n] == 123.0) and torch.all(cs.view(torch.uint8)[n] == 0x11) and torch.all(ss[n] == 7.0)
            continue
        for t in range(n_tok):
            ref_o, ref_s = _oracle(oracle_mod, d, n, t + 1, torch.from_numpy(S0[s]))
            _check_written(cs[n, t], ss[n, t], ref_s, fmt)
        o_got.append(o[n])
        o_ref.append(ref_o)
        assert torch.equal(codes[s].view(torch.uint8), cs[n, -1].view(torch.uint8)) and torch.equal(scales[s], ss[n, -1])
    assert rel_err(torch.stack(o_got), np.stack(o_ref)) <= TOL32
    rest = [s for s in range(n_slots) if s not in slots]
    assert torch.equal(codes.view(torch.uint8)[rest], c0.view(torch.uint8)[rest]) and torch.equal(scales[rest], s0[rest])
    # without the per-token states: the same pool and output to the bit
    c1, s1 = c0.clone(), s0.clone()
    o1 = torch.full_like(o, 123.0)
    _, none_c, none_s = g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), c1, s1, slots=_ints(slots), o=o1)
    assert none_c is None and none_s is None
    assert torch.equal(o1, o) and torch.equal(c1.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s1, scales)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n_tok", [1, 4])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
def test_fused_preprocessing(g, oracle_mod, fmt, dtype, n_tok, dk, dv):
    N, h_qk, h_v = 3, 1, 2
    gen = torch.Generator(device="cuda").manual_seed(8)
    rn = lambda h, d: torch.randn(N, n_tok, h, d, generator=gen, device="cuda").to(dtype)  # noqa: E731
    raw = dict(q=rn(h_qk, dk), k=rn(h_qk, dk), v=rn(h_v, dv), log_alpha=rn(h_v, dk), b=rn(h_v, dk), w=rn(h_v, dv))
    raw["k"][1, 0] = 0.0  # a zero key stays zero
    codes, scales = _pool(N, h_v, dk, dv, fmt, seed=9)
    S0 = R.read_back(codes, scales)
    o, cs, ss = g.gdn2_decode_multi_q8(*(raw[k_] for k_ in NAMES), codes, scales, want_steps=True, prologue=True)
    torch.cuda.synchronize()
    flat = {k_: t.reshape(N * n_tok, *t.shape[2:]).float().cpu() for k_, t in raw.items()}
    q_, k_, la_, b_, w_ = oracle_mod.prologue_ref(flat["q"], flat["k"], flat["log_alpha"], flat["b"], flat["w"])
    f32 = lambda x: np.asarray(x, dtype=np.float32)  # noqa: E731
    o_ref, s_ref = oracle_mod.fwd_ref(f32(q_), f32(k_), flat["v"].numpy(), f32(la_), f32(b_), f32(w_), S0=torch.from_numpy(S0), n_seq=N, bf16=False)
    assert rel_err(o.reshape(N * n_tok, h_v, dv), o_ref) <= TOL32
    _check_written(codes, scales, s_ref, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("n_tok", [1, 2])
def test_bf16_output_is_the_fp32_one_rounded(g, fmt, dv, n_tok):
    d = _tokens(3, n_tok, 2, 2, 64, dv, torch.bfloat16, seed=10)
    codes, scales = _pool(3, 2, 64, dv, fmt, seed=10)
    c2, s2 = codes.clone(), scales.clone()
    o32, _, _ = g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), codes, scales)
    o16, _, _ = g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), c2, s2, out_dtype=torch.bfloat16)
    assert o16.dtype == torch.bfloat16 and torch.equal(o16, o32.to(torch.bfloat16))
    assert torch.equal(codes.view(torch.uint8), c2.view(torch.uint8))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_tok", [1, 2])
def test_states_written_elsewhere(g, fmt, n_tok):
    """Two sequences go on from one prefix's slot, each in a slot of its own; one writes nowhere."""
    d = _tokens(4, n_tok, 2, 2, 128, 128, torch.bfloat16, seed=11)
    codes, scales = _pool(8, 2, 128, 128, fmt, seed=11)
    c0, s0 = codes.clone(), scales.clone()
    slots, out = [5, 5, 6, 7], [0, 1, -1, 7]
    o, _, _ = g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), codes, scales, slots=_ints(slots), slots_out=_ints(out))
    # the same, each sequence by itself and in place
    for n, s in enumerate(slots):
        c, sc = c0[s:s + 1].clone(), s0[s:s + 1].clone()
        o1, _, _ = g.gdn2_decode_multi_q8(*(d[k_][n:n + 1] for k_ in NAMES), c, sc)
        assert torch.equal(o[n], o1[0])
        if out[n] >= 0:
            assert torch.equal(codes.view(torch.uint8)[out[n]], c.view(torch.uint8)[0]) and torch.equal(scales[out[n]], sc[0])
    rest = [2, 3, 4, 5, 6]
    assert torch.equal(codes.view(torch.uint8)[rest], c0.view(torch.uint8)[rest]) and torch.equal(scales[rest], s0[rest])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_tok", [1, 2])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 64), (128, 128)])
def test_more_items_than_the_gpu_holds(g, fmt, n_tok, dk, dv):
    """Enough (sequence, head) pairs that a resident CTA takes several: bit for bit what one sequence
    at a time gives, with skipped sequences among them."""
    N, H = 160, 32
    d = _tokens(N, n_tok, H, H, dk, dv, torch.bfloat16, seed=12)
    codes, scales = _pool(N, H, dk, dv, fmt, seed=12)
    c0, s0 = codes.clone(), scales.clone()
    slots = torch.randperm(N, generator=torch.Generator().manual_seed(2)).to(torch.int32)
    slots[::7] = -1
    o = torch.full((N, n_tok, H, dv), 123.0, device="cuda")
    g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), codes, scales, slots=slots.cuda(), o=o)
    for n in (1, 2, 50, 97, 158, 159):
        s = int(slots[n])
        c, sc = c0[s:s + 1].clone(), s0[s:s + 1].clone()
        o1, _, _ = g.gdn2_decode_multi_q8(*(d[k_][n:n + 1] for k_ in NAMES), c, sc)
        assert torch.equal(o[n], o1[0]) and torch.equal(codes[s].view(torch.uint8), c[0].view(torch.uint8)) and torch.equal(scales[s], sc[0])
    idle = [int(s) for s in range(N) if s not in set(slots.tolist())]
    assert torch.all(o[::7] == 123.0)
    assert torch.equal(codes.view(torch.uint8)[idle], c0.view(torch.uint8)[idle])
    assert g.gdn2_device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("steps", [False, True])
def test_special_states_and_decays(g, fmt, steps):
    """A zero state, a row read back as NaN, a decay that erases everything (log_alpha = -inf) and
    infinite tokens: what is finite stays exact, what is not shows in the output and in the pool."""
    d = _tokens(5, 1, 1, 1, 64, 64, torch.float32, seed=13)
    codes, scales = _pool(5, 1, 64, 64, fmt, seed=13)
    codes.view(torch.uint8)[0] = 0
    scales[0] = 0.0
    scales[1, 0, 9] = float("nan")
    d["log_alpha"][2] = float("-inf")
    d["b"][2], d["w"][3] = 0.0, 0.0
    d["b"][3] = 0.0
    d["log_alpha"][3] = 0.0  # no decay, no edit: the state stays
    d["v"][4, 0, 0, 5] = float("inf")
    before = R.read_back(codes, scales)
    o, _, _ = g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), codes, scales, want_steps=steps)
    torch.cuda.synchronize()
    f = {k_: t[:, 0, 0].double().cpu().numpy() for k_, t in d.items()}
    x = f["w"] * f["v"]
    for n in (0, 2):  # nothing was there: the state is k x^T
        S = f["k"][n][:, None] * x[n][None]
        _check_written(codes[n], scales[n], S[None], fmt)
        assert np.abs(o[n, 0, 0].cpu().numpy() - f["q"][n] @ S).max() <= TOL32 * np.abs(f["q"][n] @ S).max()
    assert torch.isnan(o[1]).all()  # every column reads the NaN row
    assert torch.isnan(scales[1]).all() and not codes[1].float().any()
    assert np.all(np.abs(R.read_back(codes[3:4], scales[3:4]) - before[3:4]) <= np.abs(before[3:4]).max() * 2.0 ** -21)
    assert torch.isnan(scales[4]).all() and not torch.isfinite(o[4, 0, 0, 5]) and torch.isfinite(o[4, 0, 0, :5]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_offsets_past_32_bits(g, fmt):
    n_slots = 2 ** 18 + 3
    codes = torch.zeros(n_slots, 1, 128, 128, dtype=torch.uint8, device="cuda").view(fmt)
    scales = torch.zeros(n_slots, 1, 128, device="cuda")
    small = _pool(2, 1, 128, 128, fmt, seed=14)
    codes.view(torch.uint8)[-2:], scales[-2:] = small[0].view(torch.uint8), small[1]
    d = _tokens(2, 1, 1, 1, 128, 128, torch.bfloat16, seed=14)
    o, _, _ = g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), codes, scales, slots=_ints([n_slots - 2, n_slots - 1]))
    o1, _, _ = g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), *small)
    assert torch.equal(o, o1) and torch.equal(codes.view(torch.uint8)[-2:], small[0].view(torch.uint8)) and torch.equal(scales[-2:], small[1])
    assert not scales[:-2].any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_run_stays_near_the_fp32_pool(g, fmt):
    """64 one-token steps. Each rounding adds at most half a step of noise to the state, and the decay of
    the recipe (mean log_alpha -0.8) forgets it: alpha's mean square is below 0.3, so independent
    roundings sum to less than sqrt(1 / 0.7) = 1.2 of one. A code's rms error is 1 / sqrt(3) of half a
    step: 1 / 440 of the row's largest magnitude (int8) or 2^-4 / sqrt(3) = 3.7e-2 of the value (e4m3); a
    row's largest magnitude is under 4.5 of its rms. Allowed: twice that."""
    N, H = 2, 2
    S = W.state_input(N, H, 128, 128, 0.05, "cuda", seed=15)
    codes, scales = _pool(N, H, 128, 128, fmt, seed=15)
    allow = 2 * 1.2 * (4.5 / 440 if fmt == torch.int8 else 3.7e-2)
    for i in range(64):
        d = _tokens(N, 1, H, H, 128, 128, torch.bfloat16, seed=100 + i)
        o8, _, _ = g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), codes, scales)
        o, _ = g.gdn2_decode_multi(*(d[k_] for k_ in NAMES), S)
    back = g.gdn2_state_load(codes, scales)
    assert float((back - S).norm() / S.norm()) <= allow
    assert float((o8 - o).norm() / o.norm()) <= allow


def test_arguments_are_checked(g):
    d = _tokens(3, 2, 2, 2, 64, 64, torch.bfloat16, seed=16)
    codes, scales = _pool(4, 2, 64, 64, torch.int8, seed=16)
    run = lambda **kw: g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), kw.pop("codes", codes), kw.pop("scales", scales), **kw)  # noqa: E731
    with pytest.raises(TypeError, match="codes is torch.bfloat16"):
        run(codes=codes.to(torch.bfloat16))
    with pytest.raises(ValueError, match="codes has shape"):
        run(codes=torch.zeros(4, 2, 64, 128, dtype=torch.int8, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        run(codes=codes.transpose(2, 3))
    with pytest.raises(ValueError, match="scales has shape"):
        run(scales=scales[:, :1].contiguous())
    with pytest.raises(TypeError, match="slots_out"):
        run(slots_out=torch.tensor([0, 1, 2], device="cuda"))
    with pytest.raises(ValueError, match="together"):
        run(code_steps=torch.zeros(3, 2, 2, 64, 64, dtype=torch.int8, device="cuda"))
    with pytest.raises(TypeError, match="unsupported element type"):
        run(out_dtype=torch.float16)
    with pytest.raises(g.Gdn2Error, match="n_slots = 2 too small"):
        run(codes=codes[:2], scales=scales[:2])
    with pytest.raises(g.Gdn2Error, match="n_tok"):
        e = _tokens(1, 9, 2, 2, 64, 64, torch.bfloat16, seed=16)
        g.gdn2_decode_multi_q8(*(e[k_] for k_ in NAMES), codes, scales)


@pytest.mark.parametrize("n_tok", [1, 3])
def test_loads_that_never_land_are_reported(g, n_tok):
    """The loads withheld, the waits for them run out: nothing is written and the status word says so; the
    next call works."""
    d = _tokens(2, n_tok, 2, 2, 64, 64, torch.bfloat16, seed=17)
    codes, scales = _pool(2, 2, 64, 64, torch.int8, seed=17)
    c0, s0 = codes.clone(), scales.clone()
    o = torch.full((2, n_tok, 2, 64), 123.0, device="cuda")
    assert g.gdn2_device_status() == 0
    lib = g.load_library()
    lib.gdn2_testing_set_wait_limit(2_000_000, 1)
    try:
        g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), codes, scales, o=o)
        assert g.gdn2_device_status() == g.GDN2_DEVICE_WAIT_TIMEOUT
    finally:
        lib.gdn2_testing_set_wait_limit(0, 0)
    assert torch.all(o == 123.0) and torch.equal(codes, c0) and torch.equal(scales, s0)
    g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), codes, scales, o=o)
    assert g.gdn2_device_status() == 0 and not torch.any(o == 123.0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("steps", [False, True])
@pytest.mark.parametrize("size", [1e-25, 1e-3, 1e20])
def test_states_and_keys_of_any_size(g, oracle_mod, fmt, steps, size):
    """States, keys and queries far from 1, rows of very different size next to each other, and a head whose
    keys are zero."""
    d = _tokens(3, 1, 1, 1, 128, 64, torch.float32, seed=18)
    gen = torch.Generator().manual_seed(18)
    S = torch.randn(3, 1, 128, 64, generator=gen) * size * torch.exp(4 * torch.randn(3, 1, 128, 1, generator=gen))
    d["k"][1] *= 1e-12
    d["q"][1] *= 1e9
    d["k"][2] = 0.0
    d["v"] *= size
    c, sc = R.quantise(S.numpy(), fmt)
    codes, scales = torch.from_numpy(c.astype(np.float32)).cuda().to(fmt), torch.from_numpy(sc).cuda()
    S0 = R.read_back(codes, scales)
    o, _, _ = g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), codes, scales, want_steps=steps)
    for n in range(3):
        ref_o, ref_s = _oracle(oracle_mod, d, n, 1, torch.from_numpy(S0[n]))
        assert rel_err(o[n], ref_o) <= TOL32
        _check_written(codes[n], scales[n], ref_s, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_tok,steps", [(1, False), (1, True), (8, False), (8, True)])
@pytest.mark.parametrize("what", ["decay", "write", "key", "erase", "scale"])
def test_factors_that_leave_the_ordinary_range(g, oracle_mod, fmt, n_tok, steps, what):
    """Decays that erase in one token or over several, values of 1e12 and 1e30, keys of 1e8, erase gates of 4096,
    scales from 1e-30 to 1e30, next to ordinary rows, tokens and columns."""
    N = 2
    d = _tokens(N, n_tok, 1, 2, 128, 64, torch.float32, seed=19)
    gen = torch.Generator(device="cuda").manual_seed(19)
    S = 0.05 * torch.randn(N, 2, 128, 64, generator=gen, device="cuda")
    if what == "decay":
        d["log_alpha"][:, :, 0, ::3] = -30.0
        d["log_alpha"][:, n_tok // 2, 1, 1::5] = float("-inf")
        d["log_alpha"][:, :, 1, 2::7] = -9.0
    elif what == "write":
        d["v"][:, n_tok // 2, 0, 3] = 1e12
        d["v"][:, -1, 1] *= 1e30
    elif what == "key":
        d["k"][:, n_tok // 2, 0, ::4] *= 1e8
        d["b"][:] *= 1e-9  # (an erase along such a key would blow the state up)
    elif what == "erase":
        d["b"][:, 0, :, ::9] = 4096.0
        d["k"][:] *= 1e-2
    else:
        S *= torch.logspace(-30, 30, 128, device="cuda")[torch.randperm(128, generator=gen, device="cuda")][:, None]
        d["k"][:] *= 1e-3
    c, sc = R.quantise(S.cpu().numpy(), fmt)
    codes, scales = torch.from_numpy(c.astype(np.float32)).cuda().to(fmt), torch.from_numpy(sc).cuda()
    S0 = R.read_back(codes, scales)
    o, cs, ss = g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), codes, scales, want_steps=steps)
    torch.cuda.synchronize()
    heads = lambda x, h: x[:, h:h + 1] if x.shape[1] == 2 else x  # noqa: E731
    for n in range(N):
        for h in range(2):  # a head by itself: the bounds go by its own sizes
            sl = {k_: heads(d[k_][n], h).cpu().contiguous() for k_ in NAMES}
            for t in range(n_tok if steps else 0):
                _, ref = oracle_mod.fwd_ref(*(sl[k_][:t + 1].contiguous() for k_ in NAMES), S0=torch.from_numpy(S0[n:n + 1, h:h + 1]), n_seq=1)
                _check_written(cs[n, t, h], ss[n, t, h], ref[0, 0], fmt)
            ref_o, ref = oracle_mod.fwd_ref(*(sl[k_] for k_ in NAMES), S0=torch.from_numpy(S0[n:n + 1, h:h + 1]), n_seq=1)
            for t in range(n_tok):
                assert rel_err(o[n, t, h], ref_o[t, 0]) <= TOL32
            _check_written(codes[n, h], scales[n, h], ref[0, 0], fmt)
    assert g.gdn2_device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_tok", [1, 2])
def test_most_sequences(g, fmt, n_tok):
    """65535 sequences, nearly all idle: the active ones at both ends and in between as by themselves."""
    N = 65535
    live = [0, 1, 591, 592, 40000, 65533, 65534]
    d = _tokens(N, n_tok, 1, 1, 64, 64, torch.bfloat16, seed=20)
    codes, scales = _pool(len(live), 1, 64, 64, fmt, seed=20)
    c0, s0 = codes.clone(), scales.clone()
    slots = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    slots[live] = torch.arange(len(live), dtype=torch.int32, device="cuda")
    o = torch.full((N, n_tok, 1, 64), 123.0, device="cuda")
    g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), codes, scales, slots=slots, o=o)
    o1, _, _ = g.gdn2_decode_multi_q8(*(d[k_][live].contiguous() for k_ in NAMES), c0, s0)
    assert torch.equal(o[live], o1) and torch.equal(codes.view(torch.uint8), c0.view(torch.uint8)) and torch.equal(scales, s0)
    o[live] = 123.0
    assert torch.all(o == 123.0) and g.gdn2_device_status() == 0
