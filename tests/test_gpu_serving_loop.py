"""The serving operators as they are used together: prefill, states put into the pool, decode steps over
drafted tokens, verification, roll-back, states taken out again; captured into a graph, on a side
stream, and two at once."""
import numpy as np
import pytest
import torch

from gated_delta_rule_160_b200 import workloads as W
from tests import serving_ref as R

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "log_alpha", "b", "w")
N, H, D, V, DRAFTS = 5, 4, 128, 4099, 3
TOK = DRAFTS + 1


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_160_b200 as g
    g.load_library()
    assert torch.cuda.is_available()
    return g


def _step_inputs(seed):
    d = W.token_inputs(N * TOK, H, H, D, D, torch.bfloat16, "cuda", seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    p = torch.softmax(3 * torch.randn(N, TOK, V, generator=gen, device="cuda"), -1)
    q = torch.softmax(torch.log(p[:, :DRAFTS]) + 0.5 * torch.randn(N, DRAFTS, V, generator=gen, device="cuda"), -1)
    drafts = torch.multinomial(q.reshape(-1, V), 1, generator=gen).view(N, DRAFTS).to(torch.int32)
    return {k_: t.view(N, TOK, *t.shape[1:]) for k_, t in d.items()} | dict(
        p=p, draft=q.contiguous(), drafts=drafts, u=rand(N, DRAFTS), ul=rand(N))


def _slots():
    return torch.tensor([6, 1, -1, 3, 0], dtype=torch.int32, device="cuda")


def _step_fp32(g, x, pool, steps, slots, o, acc, tok):
    g.gdn2_decode_multi(*(x[k_] for k_ in NAMES), pool, slots=slots, o=o, S_steps=steps)
    g.gdn2_verify_drafts(x["p"], x["draft"], x["drafts"], x["u"], x["ul"], n_accepted=acc, tokens=tok)
    g.gdn2_state_commit(steps, acc, pool, slots=slots)


def _step_q8(g, x, pool, steps, slots, o, acc, tok, stream=None):
    g.gdn2_decode_multi_q8(*(x[k_] for k_ in NAMES), *pool, slots=slots, o=o, code_steps=steps[0], scale_steps=steps[1], stream=stream)
    g.gdn2_verify_drafts(x["p"], x["draft"], x["drafts"], x["u"], x["ul"], n_accepted=acc, tokens=tok, stream=stream)
    g.gdn2_state_commit_q8(*steps, acc, *pool, slots=slots, stream=stream)


def _buffers():
    return (torch.zeros(N, TOK, H, D, device="cuda"), torch.zeros(N, dtype=torch.int32, device="cuda"),
            torch.zeros(N, TOK, dtype=torch.int32, device="cuda"))


def _q8_buffers(fmt):
    return (torch.zeros(8, H, D, D, dtype=fmt, device="cuda"), torch.zeros(8, H, D, device="cuda")), \
        (torch.zeros(N, TOK, H, D, D, dtype=fmt, device="cuda"), torch.zeros(N, TOK, H, D, device="cuda"))


def test_fp32_pool_keeps_the_accepted_tokens(g, oracle_mod):
    """After three steps each pool state is the oracle's over the accepted tokens alone."""
    S0 = W.state_input(8, H, D, D, 0.05, "cuda", seed=20)
    pool, slots = S0.clone(), _slots()
    steps = torch.zeros(N, TOK, H, D, D, device="cuda")
    o, acc, tok = _buffers()
    kept = [[] for _ in range(N)]
    for i in range(3):
        x = _step_inputs(200 + i)
        _step_fp32(g, x, pool, steps, slots, o, acc, tok)
        want_a, want_t = R.verify(*(x[k_].double().cpu().numpy() for k_ in ("p", "draft")), x["drafts"].cpu().numpy(), *(x[k_].double().cpu().numpy() for k_ in ("u", "ul")))
        assert acc.tolist() == want_a.tolist() and tok.tolist() == want_t.tolist()
        for n in range(N):
            kept[n].append({k_: x[k_][n, :want_a[n] + 1] for k_ in NAMES})
    for n, s in enumerate(slots.tolist()):
        if s < 0:
            continue
        sl = {k_: torch.cat([c[k_] for c in kept[n]]).cpu() for k_ in NAMES}
        _, want = oracle_mod.fwd_ref(*(sl[k_] for k_ in NAMES), S0=S0[s:s + 1].cpu(), n_seq=1)
        got = pool[s].double().cpu().numpy()
        assert np.abs(got - want[0]).max() <= 1e-4 * np.sqrt(np.mean(want[0] ** 2))
    rest = [2, 4, 5, 7]
    assert torch.equal(pool[rest], S0[rest])


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
def test_prefill_store_decode_verify_commit_load(g, fmt):
    """The 8-bit pool through a whole round, against the same calls one sequence at a time."""
    lens = [65, 3, 130, 64, 200]
    T = sum(lens)
    d = W.token_inputs(T, H, H, D, D, torch.bfloat16, "cuda", seed=30)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    _, S = g.gdn2_chunk_fwd(*(d[k_] for k_ in NAMES), cu_seqlens=cu)
    pool, steps = _q8_buffers(fmt)
    slots = _slots()
    g.gdn2_state_store(S, *pool, slots=slots)
    o, acc, tok = _buffers()
    x = _step_inputs(31)
    _step_q8(g, x, pool, steps, slots, o, acc, tok)
    back = g.gdn2_state_load(*pool, slots=slots)
    # the next prefill goes on from the cached states
    o2, S2 = g.gdn2_chunk_fwd(*(d[k_] for k_ in NAMES), S0=back, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert torch.isfinite(o2).all() and torch.isfinite(S2).all()
    c, s = R.quantise(S.cpu().numpy(), fmt)
    for n, slot in enumerate(slots.tolist()):
        if slot < 0:
            assert not back[n].any()
            continue
        one = torch.from_numpy(c[n:n + 1].astype(np.float32)).cuda().to(fmt), torch.from_numpy(s[n:n + 1]).cuda()
        keep = int(acc[n]) + 1
        g.gdn2_decode_multi_q8(*(x[k_][n:n + 1, :keep].contiguous() for k_ in NAMES), *one)
        assert torch.equal(one[0][0].view(torch.uint8), pool[0][slot].view(torch.uint8)) and torch.equal(one[1][0], pool[1][slot])
        assert torch.equal(back[n], one[0][0].float() * one[1][0][..., None])


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
def test_captured_round_replays(g, fmt):
    """decode, verification, commit and the read-back captured in one graph; replayed on new inputs in the same
    buffers it gives what the eager calls give."""
    slots = _slots()
    S = W.state_input(N, H, D, D, 0.05, "cuda", seed=40)
    x = _step_inputs(41)
    pool, steps = _q8_buffers(fmt)
    g.gdn2_state_store(S, *pool, slots=slots)
    o, acc, tok = _buffers()
    back = torch.zeros(N, H, D, D, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        _step_q8(g, x, pool, steps, slots, o, acc, tok)
        g.gdn2_state_load(*pool, slots=slots, S=back)
    e_pool, e_steps = _q8_buffers(fmt)
    g.gdn2_state_store(S, *e_pool, slots=slots)
    e_o, e_acc, e_tok = _buffers()
    for seed in (41, 42, 43):
        new = _step_inputs(seed)
        for k_ in x:
            x[k_].copy_(new[k_])
        graph.replay()
        _step_q8(g, new, e_pool, e_steps, slots, e_o, e_acc, e_tok)
        e_back = g.gdn2_state_load(*e_pool, slots=slots)
        torch.cuda.synchronize()
        for a, b in ((o, e_o), (acc, e_acc), (tok, e_tok), (pool[0].view(torch.uint8), e_pool[0].view(torch.uint8)), (pool[1], e_pool[1]),
                     (back, e_back)):
            assert torch.equal(a, b)
    del graph


def test_two_streams_at_once(g):
    """Rounds on two pools, queued on two streams, give what they give one after the other."""
    def run(s1, s2):
        out = []
        for fmt, stream, seed in ((torch.int8, s1, 50), (torch.float8_e4m3fn, s2, 51)):
            stream.wait_stream(torch.cuda.current_stream())
            x = _step_inputs(seed)
            pool, steps = _q8_buffers(fmt)
            bufs = _buffers()
            S = W.state_input(N, H, D, D, 0.05, "cuda", seed=seed)
            torch.cuda.synchronize()
            out.append((fmt, stream, x, pool, steps, bufs, S))
        for fmt, stream, x, pool, steps, bufs, S in out:
            g.gdn2_state_store(S, *pool, slots=_slots(), stream=stream)
        torch.cuda.synchronize()
        for _ in range(4):
            for fmt, stream, x, pool, steps, bufs, S in out:
                _step_q8(g, x, pool, steps, x.setdefault("slots", _slots()), *bufs, stream=stream)
        torch.cuda.synchronize()
        return [t for _, _, _, pool, _, bufs, _ in out for t in (pool[0].view(torch.uint8), pool[1], *bufs)]

    one = torch.cuda.Stream()
    serial = run(one, one)
    both = run(torch.cuda.Stream(), torch.cuda.Stream())
    assert all(torch.equal(a, b) for a, b in zip(serial, both))


def test_fused_preprocessing_in_the_loop(g):
    """Raw projections through the prologue decode: the pool ends where the plain decode on the activated
    inputs ends, to fp32 arithmetic plus one code's step."""
    gen = torch.Generator(device="cuda").manual_seed(60)
    raw = {k_: torch.randn(N, TOK, H, D, generator=gen, device="cuda") for k_ in NAMES}
    act = dict(q=raw["q"] / raw["q"].norm(dim=-1, keepdim=True), k=raw["k"] / raw["k"].norm(dim=-1, keepdim=True), v=raw["v"],
               log_alpha=-torch.nn.functional.softplus(raw["log_alpha"]), b=torch.sigmoid(raw["b"]), w=torch.sigmoid(raw["w"]))
    S = W.state_input(N, H, D, D, 0.05, "cuda", seed=61)
    pools = []
    for inputs, pro in ((raw, True), (act, False)):
        pool, _ = _q8_buffers(torch.int8)
        g.gdn2_state_store(S, pool[0][:N], pool[1][:N])
        o, _, _ = g.gdn2_decode_multi_q8(*(inputs[k_].contiguous() for k_ in NAMES), *pool, prologue=pro)
        pools.append((o, g.gdn2_state_load(*pool, n_seq=N)))
    (o1, s1), (o2, s2) = pools
    assert float((o1 - o2).abs().max()) <= 1e-4 * float(o2.square().mean().sqrt())
    step = s2.abs().amax(-1, keepdim=True) / 127
    assert torch.all((s1 - s2).abs() <= 1.01 * step)


def test_streams_of_another_device_are_refused(g):
    class Elsewhere:
        device = torch.device("cuda", 7)
        cuda_stream = 0
    S = W.state_input(1, 1, 64, 64, 0.05, "cuda", seed=1)
    with pytest.raises(ValueError, match="stream is on cuda:7"):
        g.gdn2_state_store(S, torch.zeros(1, 1, 64, 64, dtype=torch.int8, device="cuda"), torch.zeros(1, 1, 64, device="cuda"), stream=Elsewhere())


def test_calls_keep_no_references(g):
    import sys
    S = W.state_input(2, 1, 64, 64, 0.05, "cuda", seed=2)
    codes, scales = torch.zeros(2, 1, 64, 64, dtype=torch.int8, device="cuda"), torch.zeros(2, 1, 64, device="cuda")
    d = {k_: t.view(2, 1, *t.shape[1:]) for k_, t in W.token_inputs(2, 1, 1, 64, 64, torch.float32, "cuda", seed=2).items()}
    p = torch.full((2, 1, 8), 0.125, device="cuda")
    none = torch.zeros(2, 0, device="cuda")
    index = torch.zeros(2, dtype=torch.int32, device="cuda")
    u = torch.rand(2, device="cuda")
    held = [S, codes, scales, p, none, index, u, *d.values()]

    def once():
        g.gdn2_state_store(S, codes, scales)
        g.gdn2_state_load(codes, scales, S=S)
        g.gdn2_state_load(codes, scales)
        _, cs, ss = g.gdn2_decode_multi_q8(*(d[k_] for k_ in NAMES), codes, scales, want_steps=True)
        g.gdn2_state_commit_q8(cs, ss, index, codes, scales)
        g.gdn2_state_commit(S[:, None], index, S)
        g.gdn2_verify_drafts(p, None, none.to(torch.int32), none, u)
        with pytest.raises(ValueError):
            g.gdn2_state_store(S[:, :, :32].contiguous(), codes, scales)

    once()
    before = [sys.getrefcount(x) for x in held]
    torch.cuda.synchronize()
    memory = torch.cuda.memory_allocated()
    for _ in range(50):
        once()
    torch.cuda.synchronize()
    assert [sys.getrefcount(x) for x in held] == before and torch.cuda.memory_allocated() == memory


def test_calls_from_several_threads(g):
    """Each thread on its own stream, some of their calls refused: results and messages stay with their thread."""
    import threading
    results = {}

    def work(i):
        stream = torch.cuda.Stream()
        x = _step_inputs(300 + i)
        pool, steps = _q8_buffers(torch.int8 if i % 2 else torch.float8_e4m3fn)
        bufs = _buffers()
        S = W.state_input(N, H, D, D, 0.05, "cuda", seed=300 + i)
        slots = _slots()
        torch.cuda.synchronize()
        g.gdn2_state_store(S, *pool, slots=slots, stream=stream)
        errors = []
        for k in range(20):
            _step_q8(g, x, pool, steps, slots, *bufs, stream=stream)
            try:
                g.gdn2_state_load(pool[0][:1 + i], pool[1][:1 + i], n_seq=2 + i, stream=stream)
            except g.Gdn2Error as e:
                errors.append(str(e))
        stream.synchronize()
        results[i] = (pool, bufs, errors)

    def alone(i):
        work(i)
        return results.pop(i)

    want = [alone(i) for i in range(4)]
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(4):
        (pool, bufs, errors), (w_pool, w_bufs, w_errors) = results[i], want[i]
        assert errors == w_errors and len(errors) == 20 and f"n_slots = {1 + i} too small" in errors[0]
        assert torch.equal(pool[0].view(torch.uint8), w_pool[0].view(torch.uint8)) and torch.equal(pool[1], w_pool[1])
        assert all(torch.equal(a, b) for a, b in zip(bufs, w_bufs))
