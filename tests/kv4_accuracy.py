"""Relative errors that tell a right attention over the 4-bit cache from a wrong one (test
infrastructure; torch on any device).

Inputs are drawn so that scores have a standard deviation of one to two and values are not ordered:
an output row of d numbers is then a sum of many small terms, and independent errors of the terms
add up as their squares do.  Errors are taken per output row (token, head), as |error| / |row|:

* rounding the result: each number is off by at most u = eps / 2 of itself, by u / sqrt(3) in the
  root mean square; 0.65 u leaves room for rows of 64 numbers.  However few numbers make up a row, it
  is off by at most u: sum (u x_i)^2 = u^2 |x|^2 (`few`);
* scores: a score is the sum of d products in d / 16 steps per query part (bf16 one, fp16 two, fp32
  three), each step off by at most 2^-23 of numbers that stay below 4 after the softmax scale.  An
  error ds of the scores changes the weights by the factor 1 + ds, and a row by about ds (twice
  that is allowed: the row's own weighted mean moves with it);
* weights: 2^-17 of each (two bf16 parts) or 2^-24 (three, for fp32), the exponential's 2^-22;
* sums over the keys: one step per 16 keys and part in a warp, each off by at most 2^-23 of the sum.

An account is a sum of weights, each off by the factor 1 + ds and by 2^-22 of the exponential and
2^-24 of a logarithm below 32."""
import math

import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
PARTS = {"f32": 3, "bf16": 1, "f16": 2}


def score_error(dtype, d):
    return PARTS[dtype] * d / 16 * 4 * 2.0 ** -23


def row_limit(dtype, d, keys, few=False):
    u = torch.finfo(TYPES[dtype]).eps / 2
    weight = 2.0 ** -22 + (2.0 ** -24 if dtype == "f32" else 2.0 ** -17)
    steps = (keys / 64 + 16) * 3 * 2.0 ** -23
    return (1.0 if few else 0.65) * u + 2 * score_error(dtype, d) + weight + steps


def gain_limit(dtype, d):
    return 2 * score_error(dtype, d) + 2.0 ** -20


def inputs(n, keys, kvh, group, q_len, d, dtype, seed):
    """q, k, v on the host: normed keys with some strong channels, values of uneven size."""
    g = torch.Generator().manual_seed(seed)
    gain = 1 + 3 * (torch.rand(kvh, d, generator=g) < 0.05)
    k = torch.randn(n, keys, kvh, d, generator=g) * gain
    v = torch.randn(n, keys, kvh, d, generator=g) * (0.25 + torch.rand(n, keys, kvh, 1, generator=g))
    q = torch.randn(n, q_len, kvh * group, d, generator=g)
    return [x.to(TYPES[dtype]) for x in (q, k, v)]


def attend(q, k, v, scale=None, window=0):
    """64-bit attention of q [m, H, d], the newest tokens, over k, v [T, KVH, d] (the values the rows
    stand for): output [m, H, d] and gains [KVH, T]."""
    m, heads, d = q.shape
    t, kvh = k.shape[0], k.shape[1]
    qq = q.double().reshape(m, kvh, heads // kvh, d)
    s = torch.einsum("mkgd,tkd->kgmt", qq, k.double()) * (1 / math.sqrt(d) if scale is None else scale)
    j = torch.arange(t, device=q.device)
    last = t - m + torch.arange(m, device=q.device)[:, None]
    hidden = j > last
    if window:
        hidden = hidden | (j <= last - window)
    p = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
    p = torch.where(hidden.all(-1)[:, None], 0.0, p)               # a token that sees nothing
    out = torch.einsum("kgmt,tkd->mkgd", p, v.double()).reshape(m, heads, d)
    return out, p.sum((1, 2))


def row_errors(out, want):
    """|error| / |row| of every output row; rows that should be zero have to be."""
    err, size = (out.double() - want).norm(dim=-1), want.norm(dim=-1)
    return torch.where(size > 0, err / torch.where(size > 0, size, 1.0), torch.where(err > 0, math.inf, 0.0))


def right(out, want, dtype, keys, few=False):
    return bool((row_errors(out, want) <= row_limit(dtype, want.shape[-1], keys, few)).all())


def gains_right(gained, want, dtype, d):
    """Per KV head, in the root mean square over the keys."""
    err = (gained.double() - want).norm(dim=-1)
    return bool((err <= gain_limit(dtype, d) * want.norm(dim=-1)).all())
