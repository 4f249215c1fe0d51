"""The serving operators around the state pool, as measured cases.

Four operators, each reached through the package's public functions:

  cache    gdn2_state_store then gdn2_state_load: states written to an 8-bit pool (int8 or e4m3
           codes, one fp32 scale a key row) and read back
  decode   gdn2_decode_multi_q8: 1-8 tokens a sequence, straight on the 8-bit pool
  verify   gdn2_verify_drafts: drafted tokens against the target's probabilities
  commit   gdn2_state_commit / gdn2_state_commit_q8: the state after the last accepted token
           goes back to its slot

Where ``own`` is false the same results come from elementary torch operations.
"""
import math

import torch

own = False

DEV = "cuda"
TINY = 2.0 ** -100  # a row whose largest magnitude is below this is stored as zeros
TOP = {"int8": 127.0, "e4m3": 448.0}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TYPE = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def _cache(name, n, h, dk, dv, fmt, idle=0):
    return dict(name=name, op="cache", n=n, h=h, dk=dk, dv=dv, fmt=fmt, idle=idle)


def _decode(name, n, hq, h, dk, dv, tok, fmt, dtype="bf16", out="fp32", steps=False, raw=False, idle=0):
    return dict(name=name, op="decode", n=n, hq=hq, h=h, dk=dk, dv=dv, tok=tok, fmt=fmt, dtype=dtype, out=out,
                steps=steps, raw=raw, idle=idle)


def _verify(name, n, drafts, vocab, dtype, ragged=False, sure=False):
    return dict(name=name, op="verify", n=n, drafts=drafts, vocab=vocab, dtype=dtype, ragged=ragged, sure=sure)


def _commit(name, n, h, dk, dv, tok, fmt, idle=0):
    return dict(name=name, op="commit", n=n, h=h, dk=dk, dv=dv, tok=tok, fmt=fmt, idle=idle)


def listed():
    return [
        # one conversation's prefix state put away and taken up again, on a small layer
        _cache("cache_one_small", 1, 2, 64, 64, "int8"),
        # a batch of finished prefills put away, some sequences without a slot
        _cache("cache_batch", 61, 16, 128, 128, "int8", idle=3),
        # every state of the full decode batch (256 sequences x 32 heads)
        _cache("cache_full", 256, 32, 128, 128, "e4m3"),
        # one user, one token: latency
        _decode("decode_one", 1, 16, 16, 128, 128, 1, "e4m3"),
        # the full decode batch, one token a sequence
        _decode("decode_full", 256, 32, 32, 128, 128, 1, "e4m3"),
        # drafted tokens: four tokens a sequence and the state after each, for the roll-back
        _decode("decode_drafts", 64, 32, 32, 128, 128, 4, "e4m3", steps=True),
        # fp32 inputs, shared query/key heads, narrow keys, int8 codes, an odd batch with idle rows
        _decode("decode_odd", 37, 4, 8, 64, 128, 3, "int8", dtype="fp32", idle=2),
        # one user's three drafted tokens
        _verify("verify_one", 1, 3, 32768, "fp32"),
        # a decode batch's four drafted tokens a sequence over a large vocabulary
        _verify("verify_full", 256, 4, 131072, "fp32"),
        # an odd vocabulary in bf16, draft lengths that differ from sequence to sequence
        _verify("verify_odd", 48, 7, 50257, "bf16", ragged=True),
        # a few sequences roll back in the 8-bit pool
        _commit("commit_few", 5, 16, 128, 128, 4, "e4m3"),
        # the full batch rolls back in the fp32 pool
        _commit("commit_full", 192, 32, 128, 128, 4, "fp32", idle=7),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(("cache", "decode", "decode", "verify", "verify", "commit"))
    dk, dv = rng.choice((64, 128, 128)), rng.choice((64, 128, 128))
    n = log(1, 256)
    idle = rng.randint(0, n // 4)
    if op == "cache":
        return {k: v for k, v in _cache("", n, log(1, 32), dk, dv, rng.choice(("int8", "e4m3")), idle).items() if k != "name"}
    if op == "decode":
        tok, group = rng.randint(1, 8) if rng.random() < 0.6 else 1, rng.choice((1, 1, 2, 4))
        h = log(1, 32 // group) * group
        steps = tok > 1 and rng.random() < 0.6
        n = min(n, 256 // tok)
        c = _decode("", n, h // group, h, dk, dv, tok, rng.choice(("int8", "e4m3", "e4m3")), rng.choice(("bf16", "bf16", "fp32")),
                    rng.choice(("fp32", "fp32", "bf16")), steps, rng.random() < 0.25, min(idle, n - 1))
        return {k: v for k, v in c.items() if k != "name"}
    if op == "verify":
        c = _verify("", n, rng.randint(0, 7), log(1000, 131072), rng.choice(("fp32", "bf16")), rng.random() < 0.5, rng.random() < 0.25)
        c["drafts"] = min(c["drafts"], 1 + 256 * 4 * 131072 // (c["n"] * c["vocab"]))
        return {k: v for k, v in c.items() if k != "name"}
    tok = rng.randint(2, 8)
    n = min(n, 192 * 4 // tok)
    return {k: v for k, v in _commit("", n, log(1, 32), dk, dv, tok, rng.choice(("fp32", "int8", "e4m3")), min(idle, n)).items() if k != "name"}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _slots(n, n_slots, idle, g):
    """A slot of the pool for each sequence, -1 for the idle ones; and which sequences are active."""
    s = torch.randperm(n_slots, generator=g, device=DEV)[:n].to(torch.int32)
    who = torch.randperm(n, generator=g, device=DEV)
    s[who[:idle]] = -1
    return s, who[idle:].sort().values


def _states(shape, g):
    """States as the recurrence leaves them: key rows of different magnitude, by their decays."""
    return 0.05 * torch.randn(shape, generator=g, device=DEV) * torch.exp(0.7 * torch.randn(shape[:-1] + (1,), generator=g, device=DEV))


def _tokens(c, g):
    lead = (c["n"], c["tok"])
    dt = TYPE[c["dtype"]]
    rn = lambda h, d: torch.randn(lead + (h, d), generator=g, device=DEV)  # noqa: E731
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
    t = dict(q=rn(c["hq"], c["dk"]), k=rn(c["hq"], c["dk"]), v=rn(c["h"], c["dv"]), a=rn(c["h"], c["dk"]), b=rn(c["h"], c["dk"]), w=rn(c["h"], c["dv"]))
    if not c["raw"]:  # normalised keys, activated gates; else the raw projections go in
        t = dict(q=unit(t["q"]), k=unit(t["k"]), v=t["v"], a=-torch.log1p(torch.exp(t["a"])), b=torch.sigmoid(t["b"]), w=torch.sigmoid(t["w"]))
    return {k: x.to(torch.float32 if k == "a" and not c["raw"] else dt).contiguous() for k, x in t.items()}


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(case=c)
    if c["op"] == "verify":
        n, m, v, dt = c["n"], c["drafts"], c["vocab"], TYPE[c["dtype"]]
        logits = 3.0 * torch.randn(n, m + 1, v, generator=g, device=DEV)
        st["p"] = torch.softmax(logits, -1).to(dt).contiguous()
        # a smaller model's guess at the same distribution, and tokens drawn from it
        near = logits[:, :m].mul_(0.9).add_(torch.randn(n, m, v, generator=g, device=DEV))
        q = torch.softmax(near, -1).to(dt).contiguous()
        if c["sure"]:  # drafts without probabilities: each was certain
            st["tokens"] = near.argmax(-1).to(torch.int32)
            st["q"] = None
        else:
            u = torch.rand(n, m, 1, generator=g, device=DEV, dtype=torch.float64)
            st["tokens"] = torch.cat([(q[i].double().cumsum(-1) < u[i] * 0.999).sum(-1).clamp_(max=v - 1)[None] for i in range(n)]).to(torch.int32)
            st["q"] = q
        st["u"] = torch.rand(n, m, generator=g, device=DEV)
        st["last"] = torch.rand(n, generator=g, device=DEV)
        st["lens"] = torch.randint(0, m + 1, (n,), generator=g, device=DEV, dtype=torch.int32) if c["ragged"] else None
        return st
    n, h, dk, dv = c["n"], c["h"], c["dk"], c["dv"]
    n_slots = 2 * n + 3
    st["slots"], st["active"] = _slots(n, n_slots, c["idle"], g)
    if c["op"] == "cache":
        st["S"] = _states((n, h, dk, dv), g)
        st["codes"] = torch.zeros(n_slots, h, dk, dv, dtype=CODE[c["fmt"]], device=DEV)
        st["scales"] = torch.zeros(n_slots, h, dk, device=DEV)
        st["back"] = torch.zeros(n, h, dk, dv, device=DEV)
    elif c["op"] == "decode":
        st["codes"], st["scales"] = _quantise(_states((n_slots, h, dk, dv), g), c["fmt"])
        # each sequence goes on in another slot than the one that it was forked from
        taken = torch.zeros(n_slots, dtype=torch.bool, device=DEV)
        taken[st["slots"][st["active"]].long()] = True
        st["slots_out"] = torch.argsort(taken.to(torch.int32), stable=True)[:n].to(torch.int32)
        st |= _tokens(c, g)
        st["o"] = torch.zeros(n, c["tok"], h, dv, dtype=TYPE[c["out"]], device=DEV)
        if c["steps"]:
            st["code_steps"] = torch.zeros(n, c["tok"], h, dk, dv, dtype=CODE[c["fmt"]], device=DEV)
            st["scale_steps"] = torch.zeros(n, c["tok"], h, dk, device=DEV)
    else:
        steps = _states((n, c["tok"], h, dk, dv), g)
        pool = _states((n_slots, h, dk, dv), g)
        st["index"] = torch.randint(0, c["tok"], (n,), generator=g, device=DEV, dtype=torch.int32)
        if c["fmt"] == "fp32":
            st["steps"], st["pool"] = steps, pool
        else:
            st["steps"], st["step_scales"] = _quantise(steps, c["fmt"])
            st["pool"], st["scales"] = _quantise(pool, c["fmt"])
    return st


# ---------------------------------------------------------------- plain forms

def _quantise(S, fmt):
    """Codes and the scale of each key row (the last axis)."""
    amax = S.abs().amax(-1)
    fine = amax >= TINY
    top = torch.full_like(amax, TOP[fmt])  # a tensor: by a number, torch multiplies with a rounded inverse
    scale = torch.where(fine, amax / top, torch.zeros_like(amax))
    inv = torch.where(fine, top / amax, torch.zeros_like(amax))
    x = S * inv[..., None]
    x = torch.round(x) if fmt == "int8" else x.clamp(-TOP[fmt], TOP[fmt])
    return x.to(CODE[fmt]), scale


def _plain_cache(st):
    at, to = st["active"], st["slots"][st["active"]].long()
    codes, scales = _quantise(st["S"][at], st["case"]["fmt"])
    _bytes(st["codes"])[to] = _bytes(codes)
    st["scales"][to] = scales
    st["back"].zero_()
    st["back"][at] = st["codes"][to].float() * st["scales"][to][..., None]
    return dict(S=st["back"], scales=st["scales"])


def _bytes(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _token_vectors(st):
    """q, k, decay, erase and write vectors of the active sequences, [n, tok, h, d] in 32 bits."""
    c, at = st["case"], st["active"]
    f = {k: st[k][at].float() for k in ("q", "k", "v", "a", "b", "w")}
    if c["raw"]:
        norm = lambda x: x / x.square().sum(-1, keepdim=True).sqrt().clamp(min=1e-12)  # noqa: E731
        f["q"], f["k"] = norm(f["q"]), norm(f["k"])
        decay, f["b"], f["w"] = 1 / (1 + torch.exp(f["a"])), 1 / (1 + torch.exp(-f["b"])), 1 / (1 + torch.exp(-f["w"]))
    else:
        decay = torch.exp(f["a"])
    share = c["h"] // c["hq"]
    q, k = f["q"].repeat_interleave(share, 2), f["k"].repeat_interleave(share, 2)
    return q, k, decay, f["b"] * k, f["w"] * f["v"]


def _plain_decode(st):
    c, at = st["case"], st["active"]
    src, dst = st["slots"][at].long(), st["slots_out"][at].long()
    q, k, decay, e, x = _token_vectors(st)
    S = st["codes"][src].float() * st["scales"][src][..., None]
    for t in range(c["tok"]):
        S = S * decay[:, t, :, :, None]
        r = (S * k[:, t, :, :, None]).sum(-2, keepdim=True)
        S = S - e[:, t, :, :, None] * r + k[:, t, :, :, None] * x[:, t, :, None, :]
        st["o"][at, t] = (S * q[:, t, :, :, None]).sum(-2).to(st["o"].dtype)
        codes, scales = _quantise(S, c["fmt"]) if c["steps"] or t == c["tok"] - 1 else (None, None)
        if c["steps"]:
            _bytes(st["code_steps"])[at, t] = _bytes(codes)
            st["scale_steps"][at, t] = scales
    _bytes(st["codes"])[dst] = _bytes(codes)
    st["scales"][dst] = scales
    return _decode_out(st)


def _decode_out(st):
    """Outputs, and the pool. Codes are compared as values: e4m3 as they are, int8 in a type that holds
    their whole numbers, since a last bit of the state can turn a rounding."""
    value = lambda x: x.to(torch.bfloat16) if x.dtype == torch.int8 else x  # noqa: E731
    out = dict(o=st["o"], codes=value(st["codes"]), scales=st["scales"])
    if st["case"]["steps"]:
        out |= dict(code_steps=value(st["code_steps"]), scale_steps=st["scale_steps"])
    return out


def _plain_verify(st):
    c, p, q, m = st["case"], st["p"], st["q"], st["case"]["drafts"]
    n, v = c["n"], c["vocab"]
    rows = torch.arange(n, device=DEV)
    t = st["tokens"].long()
    lens = torch.full((n,), m, device=DEV) if st["lens"] is None else st["lens"].long()
    # in 64 bits: values next to a border
    pt = p[:, :m].gather(-1, t[..., None])[..., 0].double()
    qt = torch.ones_like(pt) if q is None else q.gather(-1, t[..., None])[..., 0].double()
    yes = (st["u"].double() * qt < pt) & (torch.arange(m, device=DEV) < lens[:, None])
    taken = yes.long().cumprod(-1).sum(-1)
    row = p[rows, taken].double()
    refused = taken < lens
    if m:
        at = taken.clamp(max=m - 1)
        if q is None:
            less = torch.zeros_like(row).scatter_(1, t[rows, at][:, None], float("inf"))
        else:
            less = q[rows, at].double()
        left = torch.where(refused[:, None], row - less, row).clamp(min=0)
        row = torch.where(left.sum(-1, keepdim=True) > 0, left, row)
    cum = row.cumsum(-1)
    over = (cum > st["last"].double()[:, None] * cum[:, -1:]) & (row > 0)
    # the first place past the border; past the last one, the last place that has any probability
    place = torch.arange(v, device=DEV)
    first = torch.where(over, place, v).amin(-1)
    last = torch.where(row > 0, place, -1).amax(-1)
    new = torch.where(first < v, first, last)
    tokens = torch.cat([t, t.new_zeros(n, 1)], 1)
    i = torch.arange(m + 1, device=DEV)
    tokens = torch.where(i < taken[:, None], tokens, torch.where(i == taken[:, None], new[:, None], -1))
    return dict(n_accepted=taken.to(torch.int32), tokens=tokens.to(torch.int32))


def _plain_commit(st):
    at = st["active"]
    to, i = st["slots"][at].long(), st["index"][at].long()
    _bytes(st["pool"])[to] = _bytes(st["steps"])[at, i]
    if st["case"]["fmt"] == "fp32":
        return dict(pool=st["pool"])
    st["scales"][to] = st["step_scales"][at, i]
    return dict(codes=st["pool"], scales=st["scales"])


# ---------------------------------------------------------------- one pass

def run(state):
    st, c = state, state["case"]
    if not own:
        return {"cache": _plain_cache, "decode": _plain_decode, "verify": _plain_verify, "commit": _plain_commit}[c["op"]](st)
    import gated_delta_rule_160_b200 as g
    if c["op"] == "cache":
        g.gdn2_state_store(st["S"], st["codes"], st["scales"], slots=st["slots"])
        g.gdn2_state_load(st["codes"], st["scales"], slots=st["slots"], S=st["back"])
        return dict(S=st["back"], scales=st["scales"])
    if c["op"] == "decode":
        g.gdn2_decode_multi_q8(st["q"], st["k"], st["v"], st["a"], st["b"], st["w"], st["codes"], st["scales"], slots=st["slots"],
                               slots_out=st["slots_out"], o=st["o"], code_steps=st.get("code_steps"), scale_steps=st.get("scale_steps"),
                               prologue=c["raw"])
        return _decode_out(st)
    if c["op"] == "verify":
        n_accepted, tokens = g.gdn2_verify_drafts(st["p"], st["q"], st["tokens"], st["u"], st["last"], n_drafted=st["lens"])
        return dict(n_accepted=n_accepted, tokens=tokens)
    if c["fmt"] == "fp32":
        g.gdn2_state_commit(st["steps"], st["index"], st["pool"], slots=st["slots"])
        return dict(pool=st["pool"])
    g.gdn2_state_commit_q8(st["steps"], st["step_scales"], st["index"], st["pool"], st["scales"], slots=st["slots"])
    return dict(codes=st["pool"], scales=st["scales"])


def work(case):
    c = case
    if c["op"] == "verify":
        es = 4 if c["dtype"] == "fp32" else 2
        rows = 1 if c["sure"] or not c["drafts"] else 2
        return dict(bytes=c["n"] * (rows * es * c["vocab"] + c["drafts"] * (2 * es + 12) + 16), flops=c["n"] * c["vocab"] * 3)
    n = c["n"] - c["idle"]
    elts = n * c["h"] * c["dk"] * c["dv"]
    packed = elts + 4 * n * c["h"] * c["dk"]  # codes and scales
    if c["op"] == "cache":  # states in, codes and scales out, states out (idle ones as zeros)
        return dict(bytes=4 * elts + packed + 4 * c["n"] * c["h"] * c["dk"] * c["dv"], flops=3 * elts)
    if c["op"] == "commit":
        return dict(bytes=2 * (4 * elts if c["fmt"] == "fp32" else packed), flops=0)
    es, tok = (4 if c["dtype"] == "fp32" else 2), n * c["tok"]
    token = tok * (2 * c["hq"] * c["dk"] * es + c["h"] * (2 * c["dv"] * es + c["dk"] * (es + (es if c["raw"] else 4)) + c["dv"] * (4 if c["out"] == "fp32" else 2)))
    return dict(bytes=(2 + (c["tok"] if c["steps"] else 0)) * packed + token, flops=9 * elts * c["tok"])


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _format64(S, fmt):
    """The 8-bit format's definition: scale and its inverse are fp32 numbers, and a code is the nearest to
    the fp32 product; everything before them in 64 bits. Returns the codes' values and the scales."""
    amax = S.abs().max(-1, keepdim=True).values.float().double()
    keep = amax >= TINY
    scale = (amax / TOP[fmt]).float().double()
    x = (S * (TOP[fmt] / amax).float().double()).float().double()
    if fmt == "int8":
        code = torch.round(x)
    else:  # 3 bits behind the leading one, exponents from -6: the step at |x| in [2^e, 2^(e+1)) is 2^(e-3)
        e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
        code = (torch.round(x / torch.exp2(e - 3)) * torch.exp2(e - 3)).clamp(-448, 448)
    return torch.where(keep, code, 0.0), torch.where(keep, scale, 0.0)[..., 0]


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "verify":
        return _exact_verify(c, st)
    live = [(i, s) for i, s in enumerate(st["slots"].tolist()) if s >= 0]
    if c["op"] == "commit":
        pool = st["pool"].to(torch.float64)
        scales = None if c["fmt"] == "fp32" else st["scales"].double()
        for i, s in live:
            j = int(st["index"][i])
            pool[s] = st["steps"][i, j].to(torch.float64)
            if scales is not None:
                scales[s] = st["step_scales"][i, j].double()
        return dict(pool=pool) if scales is None else dict(codes=pool, scales=scales)
    if c["op"] == "cache":
        S, scales = torch.zeros_like(st["S"], dtype=torch.float64), st["scales"].double()
        for i, s in live:
            code, scales[s] = _format64(st["S"][i].double(), c["fmt"])
            S[i] = code * scales[s][..., None]
        return dict(S=S, scales=scales)
    if c["n"] * c["h"] * c["tok"] > 20000:  # a state and token after the other: too long
        return None
    codes, scales, o = st["codes"].to(torch.float64), st["scales"].double(), st["o"].double()
    code_steps = st["code_steps"].to(torch.float64) if c["steps"] else None
    scale_steps = st["scale_steps"].double() if c["steps"] else None
    for i, s in live:
        S = st["codes"][s].double() * st["scales"][s].double()[..., None]
        head = torch.arange(c["h"], device=DEV) // (c["h"] // c["hq"])
        for t in range(c["tok"]):
            q, k, v, a, b, w = (st[x][i, t].double() for x in ("q", "k", "v", "a", "b", "w"))
            if c["raw"]:
                q, k = q / torch.linalg.vector_norm(q, dim=-1, keepdim=True), k / torch.linalg.vector_norm(k, dim=-1, keepdim=True)
                a, b, w = -torch.nn.functional.softplus(a), torch.sigmoid(b), torch.sigmoid(w)
            q, k = q[head], k[head]
            S = torch.exp(a)[..., None] * S
            S = S - torch.einsum("hi,hl,hlj->hij", b * k, k, S) + torch.einsum("hi,hj->hij", k, w * v)
            o[i, t] = torch.einsum("hij,hi->hj", S, q)
            if c["steps"]:
                code_steps[i, t], scale_steps[i, t] = _format64(S, c["fmt"])
        to = int(st["slots_out"][i])
        codes[to], scales[to] = _format64(S, c["fmt"])
    out = dict(o=o, codes=codes, scales=scales)
    return out | (dict(code_steps=code_steps, scale_steps=scale_steps) if c["steps"] else {})


def _exact_verify(c, st):
    taken, tokens = [], []
    for n in range(c["n"]):
        m = c["drafts"] if st["lens"] is None else int(st["lens"][n])
        got, i = [], 0
        while i < m:
            t = int(st["tokens"][n, i])
            ratio = 1.0 if st["q"] is None else float(st["q"][n, i, t])
            if float(st["u"][n, i]) * ratio >= float(st["p"][n, i, t]):
                break
            got.append(t)
            i += 1
        row = st["p"][n, i].double()
        if i < m:
            left = row.clone()
            if st["q"] is None:
                left[int(st["tokens"][n, i])] = 0
            else:
                left = torch.relu(row - st["q"][n, i].double())
            row = left if bool(left.any()) else row
        sums = torch.cumsum(row, 0)
        new = int(torch.searchsorted(sums, float(st["last"][n]) * sums[-1], right=True).clamp(max=c["vocab"] - 1))
        taken.append(i)
        tokens.append(got + [new] + [-1] * (c["drafts"] - i))
    return dict(n_accepted=torch.tensor(taken, dtype=torch.int32), tokens=torch.tensor(tokens, dtype=torch.int32))
