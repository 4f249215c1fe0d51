"""Plain references for the operators around the state pool (test infrastructure, numpy).

The 8-bit format is stated in fp32 arithmetic (gdn2.h), so its codes and scales are reproduced
here to the bit; draft verification is a loop in fp64 over Python floats.
"""
import numpy as np
import torch

TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
TINY = np.float32(2.0 ** -100)


def e4m3_round(x):
    """Nearest e4m3 value (3 mantissa bits, exponents from -6, largest 448), ties to even, fp64 in and out."""
    x = np.asarray(x, dtype=np.float64)
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    step = np.exp2(e - 3)
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def quantise(S, dtype):
    """Codes' values (fp64) and scales (fp32) of states S [..., dk, dv] fp32."""
    S = np.asarray(S, dtype=np.float32)
    top = np.float32(TOP[dtype])
    with np.errstate(all="ignore"):
        mag = np.where(np.isnan(S), np.float32(np.inf), np.abs(S))
        a = mag.max(-1)
        bad, tiny = ~np.isfinite(a), a < TINY
        scale = np.where(bad, np.float32(np.nan), np.where(tiny, np.float32(0), a / top)).astype(np.float32)
        inv = np.where(bad | tiny, np.float32(0), top / a).astype(np.float32)
        x = np.where((bad | tiny)[..., None], np.float32(0), S * inv[..., None]).astype(np.float64)
    return (np.rint(x) if dtype == torch.int8 else e4m3_round(x)), scale


def values(codes):
    """Codes as fp64 numbers."""
    return codes.detach().float().cpu().numpy().astype(np.float64)


def read_back(codes, scales):
    """fp32 states of a pool's codes and scales."""
    c = codes.detach().float().cpu().numpy()
    return c * scales.detach().cpu().numpy()[..., None]


def half_step(S, dtype):
    """Largest rounding error of each element of fp64 states S [..., dk, dv] in the 8-bit format:
    half a step of the code, and 2^-22 of the row's largest magnitude for the roundings of the scale,
    its inverse and the two products (four of 2^-24 each)."""
    a = np.abs(S).max(-1, keepdims=True)
    half = a / 254 if dtype == torch.int8 else np.maximum(np.abs(S) * 2.0 ** -4, a / 458752)
    return half + a * 2.0 ** -22


def clean(x):
    """A probability, or a row of them, as it counts: 0 unless it is positive and finite."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        return np.where((x > 0) & np.isfinite(x), x, 0.0)


def verify(p, q, drafts, u, u_last, lens=None):
    """p [N, n + 1, V], q [N, n, V] or None, drafts [N, n], u [N, n], u_last [N], lens [N] or None,
    all numpy (probabilities as fp64). Returns (n_accepted, tokens)."""
    N, n1, V = p.shape
    n = n1 - 1
    taken, tokens = [], []
    for s in range(N):
        m = n if lens is None else min(int(lens[s]), n)
        if m < 0:
            taken.append(-1)
            tokens.append([-1] * n1)
            continue
        a = 0
        while a < m:
            t = int(drafts[s, a])
            if not 0 <= t < V:
                break
            qt = 1.0 if q is None else clean(q[s, a, t])
            if not float(u[s, a]) * float(qt) < float(clean(p[s, a, t])):
                break
            a += 1
        row = clean(p[s, a])
        if a < m:
            rest = row.copy()
            if q is None:
                if 0 <= drafts[s, a] < V:
                    rest[drafts[s, a]] = 0.0
            else:
                rest = np.maximum(row - clean(q[s, a]), 0.0)
            row = rest if rest.sum() > 0 else row
        cum = np.cumsum(row)
        ul = float(u_last[s])
        ul = 0.0 if np.isnan(ul) else min(max(ul, 0.0), 1.0)
        some = np.nonzero(row > 0)[0]
        over = np.nonzero((cum > ul * cum[-1]) & (row > 0))[0]
        new = -1 if not len(some) else int(over[0] if len(over) else some[-1])
        taken.append(a)
        tokens.append([int(t) for t in drafts[s, :a]] + [new] + [-1] * (n - a))
    return np.array(taken), np.array(tokens)
