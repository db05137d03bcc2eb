"""Plain 64-bit implementation of the 4-bit KV cache (test infrastructure, numpy on the host).

A cache is a list of slots; a slot holds, per KV head, rows as arrays of the values they stand
for, with their positions and accumulated weights."""
import numpy as np

GROUP = 32


def bf16_round(x):
    """float64 -> nearest bf16 (ties to even), kept as float64; subnormals and the range included."""
    x = np.asarray(x, np.float64)
    e = np.maximum(np.frexp(x)[1], -125)       # 2**-126 is the smallest normal: 0.5 * 2**-125
    return np.ldexp(np.rint(np.ldexp(x, 8 - e)), e - 8)


SCALE_MAX = 145 * 2.0 ** 118     # the largest scale whose 7-fold is a finite bf16
F32_MAX = float(np.finfo(np.float32).max)


def code_rows(x):
    """(codes, scales) of rows x [..., D] (float64 holding the given values)."""
    x = np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=F32_MAX, neginf=-F32_MAX)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    # the format takes a seventh by an fp32 product
    seventh = np.abs(g).max(-1, keepdims=True).astype(np.float32) * (np.float32(1) / np.float32(7))
    s = np.minimum(bf16_round(seventh), SCALE_MAX)
    # quotients of 64 bits: exact at the borders, whose 12 significant bits they hold
    c = np.clip(np.rint(np.divide(g, s, out=np.zeros_like(g), where=s > 0)), -7, 7)
    return c.reshape(x.shape), s[..., 0]


def values(x):
    """The values rows x stand for once coded."""
    c, s = code_rows(x)
    return bf16_round(c * np.repeat(s, GROUP, -1))


def attend(q, k, v, group, scale, window=0):
    """q [m, H, D] newest tokens over k, v [T, KVH, D]; returns out [m, H, D], gained [KVH, T]."""
    m, heads, d = q.shape
    t, kvh = k.shape[0], k.shape[1]
    out = np.zeros((m, heads, d))
    gained = np.zeros((kvh, t))
    for h in range(heads):
        for i in range(m):
            last = t - m + i
            lo = max(0, last - window + 1) if window else 0
            if last < lo:
                continue
            s = (k[lo:last + 1, h // group] @ q[i, h]) * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h] = p @ v[lo:last + 1, h // group]
            gained[h // group, lo:last + 1] += p
    return out, gained


def evict_source(pos, weight, budget, recent):
    """Row that each of the min(len, budget) kept places takes (one KV head)."""
    n = len(pos)
    if n <= budget:
        return np.arange(n)
    w = np.where(np.isnan(weight), -np.inf, weight.astype(np.float64))
    nan_last = np.isnan(weight)
    safe = pos.astype(np.int64) > int(pos.max()) - recent
    order = sorted(range(n), key=lambda r: (not safe[r], bool(nan_last[r]), -w[r], r))
    keep = set(order[:budget])
    movers = iter(sorted(r for r in keep if r >= budget))
    return np.array([r if r in keep else next(movers) for r in range(budget)])
