"""The references of the serving operators' tests, checked against what they have to satisfy, and
the refusals that need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from tests import serving_ref as R

FORMATS = [torch.int8, torch.float8_e4m3fn]


def test_e4m3_rounding_gives_representable_values():
    """Every finite e4m3 value rounds to itself; halfway points go to the even neighbour; what lies
    past the largest value stays there."""
    all_codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    finite = np.unique(all_codes[np.isfinite(all_codes)])
    assert finite[-1] == 448.0 and len(finite) == 253
    assert np.array_equal(R.e4m3_round(finite), finite)
    mid = (finite[1:] + finite[:-1]) / 2
    got = R.e4m3_round(mid)
    assert np.all((got == finite[1:]) | (got == finite[:-1]))
    code = {float(v): i for i, v in enumerate(finite[finite >= 0])}  # position = code, 0 upwards
    assert all(code[float(abs(g))] % 2 == 0 for g in got)
    assert R.e4m3_round(1e9) == 448.0 and R.e4m3_round(-449.0) == -448.0


@pytest.mark.parametrize("dtype", FORMATS)
def test_format_error_is_within_half_a_step(dtype):
    rng = np.random.default_rng(1)
    S = (rng.standard_normal((64, 128)) * np.exp(rng.uniform(-40, 40, (64, 1)))).astype(np.float32)
    code, scale = R.quantise(S, dtype)
    back = (code.astype(np.float32) * scale[:, None]).astype(np.float64)
    assert np.all(np.abs(back - S) <= R.half_step(S.astype(np.float64), dtype))


@pytest.mark.parametrize("dtype", FORMATS)
def test_format_of_special_rows(dtype):
    S = np.zeros((4, 64), np.float32)
    S[1, 3], S[2, 5], S[3] = np.inf, np.nan, 2.0 ** -101
    code, scale = R.quantise(S, dtype)
    assert not code.any()
    assert scale[0] == 0 and np.isnan(scale[1]) and np.isnan(scale[2]) and scale[3] == 0


def test_verification_keeps_the_target_distribution():
    """Accept-or-replace leaves the first token distributed as p, whatever q: on a grid of both random
    numbers, the shares of the tokens are p's to the grid's resolution."""
    p = np.array([0.5, 0.25, 0.125, 0.125])
    q = np.array([0.125, 0.5, 0.25, 0.125])
    G = 64
    grid = (np.arange(G) + 0.5) / G
    share = np.zeros(4)
    for t in range(4):
        for u in grid:
            for ul in grid:
                a, tok = R.verify(np.stack([p, p])[None], q[None, None], np.array([[t]]), np.array([[u]]), np.array([ul]))
                share[tok[0, 0]] += q[t] / (G * G)
    assert np.abs(share - p).max() <= 4 / G


def test_verification_by_hand():
    p = np.array([[[0.1, 0.9, 0.0], [0.2, 0.3, 0.5], [0.0, 0.0, 1.0]]])
    q = np.array([[[0.5, 0.5, 0.0], [0.6, 0.2, 0.2]]])
    run = lambda d, u, ul, **kw: [x.tolist() for x in R.verify(p, q, np.array([d]), np.array([u]), np.array([ul]), **kw)]  # noqa: E731
    assert run([1, 2], [0.9, 0.9], 0.5) == [[2], [[1, 2, 2]]]  # both accepted: one more from the last place
    assert run([0, 2], [0.3, 0.0], 0.0) == [[0], [[1, -1, -1]]]  # 0.3 0.5 >= 0.1: only token 1 has more than its draft
    assert run([1, 0], [0.0, 0.99], 0.0) == [[1], [[1, 1, -1]]]  # residual (0, 0.1, 0.3)
    assert run([1, 0], [0.0, 0.99], 0.5) == [[1], [[1, 2, -1]]]
    assert run([1, 2], [0.0, 0.0], 0.5, lens=[0])[0] == [0] and run([1, 2], [0.0, 0.0], 0.5, lens=[-1]) == [[-1], [[-1, -1, -1]]]


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def g():
    from gated_delta_rule_160_b200 import build
    build.build()
    import gated_delta_rule_160_b200 as g
    g.load_library()
    return g


def _err(g):
    return g.load_library().gdn2_last_error_string()


def test_state_calls_reject_before_device_work(g):
    lib = g.load_library()
    X = 0x1000  # never dereferenced: every call below is refused first

    def store(n=2, h=2, dk=64, dv=64, fmt=0, S=X, slots=X, codes=X, scales=X, n_slots=4):
        return lib.gdn2_state_store(n, h, dk, dv, fmt, S, slots, codes, scales, n_slots, None)

    assert store(n=0) == 1 and b"n_seq = 0" in _err(g)
    assert store(n=65536) == 1
    assert store(h=0) == 1
    assert store(dk=96) == 2 and b"dk = 96" in _err(g)
    assert store(dv=256) == 2
    assert store(fmt=2) == 1 and b"8-bit format 2" in _err(g)
    assert store(n=65535, h=32768, n_slots=65535) == 2 and b"above 2^30 - 1" in _err(g)
    assert store(n_slots=0) == 1
    assert store(slots=None, n_slots=1) == 1 and b"n_slots = 1 too small" in _err(g)
    assert store(S=None) == 1 and b"S is NULL" in _err(g)
    assert store(S=0x1008) == 1 and b"S = 0x1008 is not 16-byte aligned" in _err(g)
    assert store(S=X, slots=0x1002) == 1

    def load(**kw):
        d = dict(n=2, h=2, dk=64, dv=64, fmt=1, codes=X, scales=X, n_slots=4, slots=X, S=X) | kw
        return lib.gdn2_state_load(d["n"], d["h"], d["dk"], d["dv"], d["fmt"], d["codes"], d["scales"], d["n_slots"], d["slots"], d["S"], None)

    assert load(n=0) == 1 and load(dk=32) == 2 and load(fmt=-1) == 1 and load(S=None) == 1 and load(slots=None, n_slots=1) == 1

    def commit(n=2, n_tok=4, steps=X, index=X, slots=X, pool=X, n_slots=4):
        return lib.gdn2_state_commit(n, 2, 64, 64, n_tok, steps, index, slots, pool, n_slots, None)

    assert commit(n_tok=0) == 1 and b"n_tok = 0" in _err(g)
    assert commit(n_tok=9) == 1
    assert commit(steps=None) == 1 and b"S_steps is NULL" in _err(g)
    assert commit(index=None) == 1
    assert commit(slots=None, n_slots=1) == 1
    assert lib.gdn2_state_commit_q8(2, 2, 64, 64, 4, X, None, X, X, X, X, 4, None) == 1


def test_decode_q8_rejects_before_device_work(g):
    lib = g.load_library()
    X = 0x1000

    def call(n_tok=2, n_slots=4, slots=None, fmt=0, code_steps=None, scale_steps=None, q=X, prologue=False, **shape):
        sh = g.Shape(**(dict(n_seq=2, T_total=4, h_qk=1, h_v=2, dk=64, dv=64, dtype=g.GDN2_BF16, o_dtype=g.GDN2_F32) | shape))
        fn = lib.gdn2_decode_multi_q8_prologue if prologue else lib.gdn2_decode_multi_q8
        return fn(ctypes.byref(sh), fmt, n_tok, slots, None, q, X, X, X, X, X, X, X, n_slots, X, code_steps, scale_steps, None)

    for prologue in (False, True):
        assert call(n_tok=0, prologue=prologue) == 1
        assert call(n_tok=9, T_total=18, prologue=prologue) == 1
        assert call(n_tok=3, prologue=prologue) == 1 and b"not n_seq * n_tok" in _err(g)
        assert call(n_slots=1, prologue=prologue) == 1
        assert call(fmt=5, prologue=prologue) == 1
        assert call(dk=96, prologue=prologue) == 2
        assert call(h_qk=2, h_v=3, prologue=prologue) == 1
        assert call(code_steps=X, prologue=prologue) == 1 and b"together" in _err(g)
        assert call(scale_steps=X, prologue=prologue) == 1
        assert call(q=None, prologue=prologue) == 1 and b"q is NULL" in _err(g)


def test_verify_rejects_before_device_work(g):
    lib = g.load_library()
    X = 0x1000

    def call(n=2, m=3, V=100, dt=0, p=X, q=X, d=X, lens=None, u=X, ul=X, acc=X, tok=X):
        return lib.gdn2_verify_drafts(n, m, V, dt, p, q, d, lens, u, ul, acc, tok, None)

    assert call(n=0) == 1 and call(n=65536) == 1
    assert call(m=-1) == 1 and call(m=g.GDN2_VERIFY_MAX_DRAFTS + 1) == 2
    assert call(V=0) == 1 and call(V=g.GDN2_VERIFY_MAX_VOCAB + 1) == 2 and b"vocab" in _err(g)
    assert call(dt=2) == 1
    assert call(p=None) == 1 and b"target_probs is NULL" in _err(g)
    assert call(d=None) == 1 and call(u=None) == 1 and call(ul=None) == 1 and call(acc=None) == 1 and call(tok=None) == 1
    assert call(p=0x1002) == 1 and b"4-byte aligned" in _err(g)


def test_binding_rejects_host_tensors(g):
    S = torch.zeros(2, 1, 64, 64)
    c, sc = torch.zeros(2, 1, 64, 64, dtype=torch.int8), torch.zeros(2, 1, 64)
    x = torch.zeros(2, 1, 1, 64)
    i = torch.zeros(2, dtype=torch.int32)
    p = torch.zeros(2, 2, 10)
    for call in (lambda: g.gdn2_state_store(S, c, sc), lambda: g.gdn2_state_load(c, sc),
                 lambda: g.gdn2_decode_multi_q8(x, x, x, x, x, x, c, sc),
                 lambda: g.gdn2_state_commit(S[:, None], i, S), lambda: g.gdn2_state_commit_q8(c[:, None], sc[:, None], i, c, sc),
                 lambda: g.gdn2_verify_drafts(p, p[:, :1], i[:, None], p[:, :1, 0], p[:, 0, 0])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_limits_match_the_header(g):
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gdn2.h")).read()
    for name in ("GDN2_VERIFY_MAX_DRAFTS", "GDN2_VERIFY_MAX_VOCAB", "GDN2_DECODE_MAX_TOKENS"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(g, name)
