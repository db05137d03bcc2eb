"""The 4-bit KV cache's operators, as they are measured: append, read, attend and evict.

A cache row of one KV head is a key and a value of head_dim numbers, each held as signed 4-bit
codes with one bf16 scale per 32 numbers: s = bf16(max|v| / 7), c = round-half-even(v / s)
clipped to +-7, and the row stands for the values bf16(c * s).  Rows live in slots (one per
sequence), either at fixed places or in pages that a page table names.

  append  codes new key/value rows into the cache (here: and reads them back);
  read    gives rows back as the values they stand for;
  attend  softmax attention of 1 to 64 query tokens per sequence over its rows, the query tokens
          being the newest rows (causal), optionally within a sliding window, optionally adding
          each row's attention weights (over query tokens and heads) to the row's account;
  evict   keeps, per sequence and KV head, `budget` rows: the newest `recent` positions and, of
          the others, those with the most accumulated weight; ties stay at the lowest row.  Kept
          rows from beyond the budget move into the places of evicted ones, both in row order.

Without `own` every operator is computed in elementary torch operations on a packed cache of
the same content; with it the calls are those of runtime.KV4Cache.
"""
import math
import random

import torch

own = False

GROUP = 32
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step's K/V rows of eight agents, in the decoder's fp32 activations
        dict(name="append step b8 d256 f32", op="append", n_seq=8, rows=1, at=639, heads=8, kv_heads=1, head_dim=256,
             dtype="f32", page=0),
        # prompts of 16 sequences coded after their prefill, four KV heads, paged, ragged
        dict(name="append prompts b16 d128 bf16", op="append", n_seq=16, rows=2100, at=37, heads=32, kv_heads=4,
             head_dim=128, dtype="bf16", page=128),
        # a short session taken out of its slot
        dict(name="read one session d256", op="read", n_seq=1, rows=639, at=0, heads=8, kv_heads=1, head_dim=256,
             dtype="bf16", page=0),
        # eight agents' contexts handed over in fp16, wide heads, paged
        dict(name="read contexts b8 d512", op="read", n_seq=8, rows=8639, at=0, heads=8, kv_heads=1, head_dim=512,
             dtype="f16", page=128),
        # one sequence early in its answer: latency
        dict(name="decode b1 t200 d256 f32", op="attend", n_seq=1, q_len=1, keys=200, heads=8, kv_heads=1,
             head_dim=256, dtype="f32", page=0, window=0, accumulate=False),
        # the benchmark's largest batch on a sliding layer
        dict(name="decode b64 w512 d256 f32", op="attend", n_seq=64, q_len=1, keys=640, heads=8, kv_heads=1,
             head_dim=256, dtype="f32", page=0, window=512, accumulate=False),
        # agent replay at its last context on a full layer, ragged, paged, weights accounted
        dict(name="decode b8 t8639 d512 bf16", op="attend", n_seq=8, q_len=1, keys=8639, heads=8, kv_heads=1,
             head_dim=512, dtype="bf16", page=128, window=0, accumulate=True),
        # a grouped-query model's batch at long contexts: the largest decode
        dict(name="decode b64 t8192 gqa d128", op="attend", n_seq=64, q_len=1, keys=8192, heads=32, kv_heads=8,
             head_dim=128, dtype="bf16", page=128, window=0, accumulate=False),
        # a block of 64 prompt tokens appended to long contexts, weights accounted
        dict(name="block b8 q64 t8000 d256", op="attend", n_seq=8, q_len=64, keys=8000, heads=8, kv_heads=1,
             head_dim=256, dtype="bf16", page=128, window=0, accumulate=True),
        # a verification of a few drafted tokens, odd sizes, fp16
        dict(name="draft b5 q7 t1531 d64", op="attend", n_seq=5, q_len=7, keys=1531, heads=12, kv_heads=4,
             head_dim=64, dtype="f16", page=16, window=0, accumulate=True),
        # a bounded cache in steady decoding: one row in, one row out
        dict(name="evict step b8 keep 1024", op="evict", n_seq=8, rows=1, budget=1024, recent=128, heads=8,
             kv_heads=1, head_dim=256, dtype="f32", page=0),
        # a turn's appended prompt cut back to the budget
        dict(name="evict turn b8 2500 to 512", op="evict", n_seq=8, rows=1988, budget=512, recent=100, heads=16,
             kv_heads=2, head_dim=128, dtype="bf16", page=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["append", "read", "attend", "attend", "attend", "evict"])
    kv_heads = rng.choice([1, 1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8, 3, 5]) if kv_heads > 1 else rng.choice([4, 8, 8, 7])
    c = dict(op=op, n_seq=_log_int(rng, 1, 64), heads=kv_heads * group, kv_heads=kv_heads,
             head_dim=rng.choice([64, 128, 256, 512]), dtype=rng.choice(["f32", "bf16", "f16"]),
             page=rng.choice([0, 16, 32, 64, 128]))
    wide = kv_heads * c["head_dim"]  # numbers of a row's keys
    if op in ("append", "read"):
        most = max(1, min(9000, (36 << 20) // (wide * c["n_seq"])))
        c.update(rows=_log_int(rng, 1, most), at=rng.choice([0, rng.randrange(0, 300)]))
    elif op == "attend":
        many = rng.random() < 0.4
        q_len = _log_int(rng, 2, 64) if many else 1
        if many:
            c["n_seq"] = min(c["n_seq"], 8)
        most = min(12000, (512 << 20) // (wide * c["n_seq"]))
        if many:
            most = min(most, (1 << 25) // (c["n_seq"] * c["heads"] * q_len))
        c.update(q_len=q_len, keys=max(q_len, _log_int(rng, 1, max(2, most))))
        c["window"] = rng.choice([0, 0, _log_int(rng, 1, 2000)])
        c["accumulate"] = c["window"] == 0 and rng.random() < 0.5
    else:
        c["n_seq"] = min(c["n_seq"], 16)
        budget = _log_int(rng, 16, max(17, min(4000, (16 << 20) // (wide * c["n_seq"]))))
        c.update(budget=budget, recent=rng.randrange(0, budget // 2 + 1), rows=_log_int(rng, 1, 2 * budget))
    return c


def _counts(case):
    """Rows (append, read) or keys (attend) of every sequence: a ragged batch, the first the longest."""
    n, most = case["n_seq"], case["keys"] if case["op"] == "attend" else case["rows"]
    least = case.get("q_len", 1)
    return [max(least, most - (most * ((7 * i) % n)) // (2 * n)) for i in range(n)]


def work(case):
    d, kvh, h, n = case["head_dim"], case["kv_heads"], case["heads"], case["n_seq"]
    coded = 2 * (d // 2 + d // 16) * kvh          # bytes of one cache row, K and V
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("append", "read"):
        rows = sum(_counts(case))
        dense_in = 2 * d * kvh * es if case["op"] == "append" else 0
        dense_out = 2 * d * kvh * (2 if case["op"] == "append" else es)
        return {"bytes": rows * (dense_in + coded + dense_out), "flops": rows * 2 * d * kvh * 4}
    if case["op"] == "attend":
        read, pairs = 0, 0
        for t in _counts(case):
            lo = max(0, t - case["q_len"] + 1 - case["window"]) if case["window"] else 0
            read += t - lo
            for i in range(case["q_len"]):
                last = t - case["q_len"] + i
                pairs += min(last + 1, case["window"] or last + 1)
        dense = 2 * n * case["q_len"] * h * d * es
        kept = 8 * read * kvh if case["accumulate"] else 0
        return {"bytes": read * coded + dense + kept, "flops": 4 * pairs * h * d}
    new, rows = n * case["rows"], n * (case["budget"] + case["rows"])
    out = n * case["budget"]
    return {"bytes": new * (2 * d * kvh * es + coded) + rows * kvh * 8 + out * (coded + 4 * d * kvh + 8 * kvh),
            "flops": new * 2 * d * kvh * 4}


# ------------------------------------------------------------------------------- the inputs
def _inputs(case, seed):
    """Everything that the case's numbers are made of, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, kvh, n = case["head_dim"], case["kv_heads"], case["n_seq"]
    typ = TYPES[case["dtype"]]

    def rows(m):
        """Keys and values of m rows per sequence: normed keys with some strong channels, values of uneven size."""
        gain = 1 + 3 * (torch.rand(kvh, d, device="cuda", generator=g) < 0.05)
        k = torch.empty(n, m, kvh, d, dtype=typ, device="cuda")
        v = torch.empty(n, m, kvh, d, dtype=typ, device="cuda")
        for i in range(n):
            k[i] = torch.randn(m, kvh, d, device="cuda", generator=g) * gain
            v[i] = torch.randn(m, kvh, d, device="cuda", generator=g) * torch.rand(m, kvh, 1, device="cuda", generator=g)
        return k, v

    x = {}
    if case["op"] == "append" or case["op"] == "read":
        x["first"], x["held"] = [case["at"]] * n, case["at"] + case["rows"]
        x["k"], x["v"] = rows(case["rows"])
    elif case["op"] == "attend":
        x["held"] = case["keys"]
        x["k"], x["v"] = rows(case["keys"])
        q = torch.randn(n, case["q_len"], case["heads"], d, device="cuda", generator=g)
        x["q"] = q.to(typ)
        if case["accumulate"]:
            x["weights"] = 4 * torch.rand(n, kvh, case["keys"], device="cuda", generator=g)
    else:
        x["held"] = case["budget"] + case["rows"]
        x["k"], x["v"] = rows(case["budget"])
        x["new_k"], x["new_v"] = rows(case["rows"])
        # accumulated weights: a few rows take most, as attention does
        heavy = lambda m: torch.exp(2 * torch.randn(n, kvh, m, device="cuda", generator=g))
        x["weights"] = heavy(case["budget"])
        x["new_weights"] = heavy(case["rows"]) if case["rows"] > 1 else None
        # positions that an earlier eviction left: rising within a row of holes, another per head
        gaps = torch.randint(1, 4, (n, kvh, case["budget"]), device="cuda", generator=g)
        x["positions"] = torch.cumsum(gaps, 2).to(torch.int32)
        start = x["positions"].amax(2, keepdim=True).amax(1, keepdim=True) + 1
        x["new_positions"] = (start + torch.arange(case["rows"], device="cuda", dtype=torch.int32)).to(
            torch.int32).expand(n, kvh, case["rows"]).contiguous()
    x["slots"] = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    page = case["page"]
    if page:
        per = -(-x["held"] // page)
        x["table"] = torch.randperm(n * per, generator=g, device="cuda").to(torch.int32).view(n, per)
    return x


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    x = _inputs(case, seed)
    n, kvh, page = case["n_seq"], case["kv_heads"], case["page"]
    s = {"case": case, "slots": x["slots"], "q": x.get("q"), "table": x.get("table")}
    counts = _counts(case) if case["op"] != "evict" else [case["budget"] + case["rows"]] * n
    s["counts"] = _i32(counts)
    s["start"] = _i32([case["at"]] * n if "at" in case else [case["budget"]] * n if case["op"] == "evict" else [0] * n)
    s["zeros"] = _i32([0] * n)
    if case["op"] == "append":
        s["new_k"], s["new_v"] = x["k"], x["v"]
    if case["op"] == "evict":
        s["new_k"], s["new_v"], s["new_weights"] = x["new_k"], x["new_v"], x["new_weights"]
        s["new_positions"] = x["new_positions"].clone()
    tracked = case["op"] == "evict" or bool(case.get("accumulate"))
    if own:
        from accelerator_decode_gb300 import runtime
        s["cache"] = runtime.KV4Cache(n_slots=n, capacity=x["held"], num_q_heads=case["heads"], num_kv_heads=kvh,
                                      head_dim=case["head_dim"], max_q_len=case.get("q_len", 1), track=tracked,
                                      page_size=page, page_table=x.get("table"))
        if case["op"] != "append":
            s["cache"].append(x["k"], x["v"], s["slots"], s["start"] if case["op"] == "read" else s["zeros"],
                              positions=x.get("positions"), weights=x.get("weights"))
    else:
        d = case["head_dim"]
        total = n * (-(-x["held"] // page) * page if page else x["held"])
        s["kc"] = torch.zeros(total, kvh, d // 2, dtype=torch.uint8, device="cuda")
        s["vc"] = torch.zeros(total, kvh, d // 2, dtype=torch.uint8, device="cuda")
        s["ks"] = torch.zeros(total, kvh, d // GROUP, dtype=torch.bfloat16, device="cuda")
        s["vs"] = torch.zeros(total, kvh, d // GROUP, dtype=torch.bfloat16, device="cuda")
        s["held"] = x["held"]
        if tracked:
            s["positions"] = torch.zeros(total, kvh, dtype=torch.int32, device="cuda")
            s["weights"] = torch.zeros(total, kvh, device="cuda")
        if case["op"] != "append":
            m = x["k"].shape[1]
            at = _places(s, s["start"] if case["op"] == "read" else s["zeros"], m)
            for i in range(n):
                s["kc"][at[i]], s["ks"][at[i]] = _code(x["k"][i])
                s["vc"][at[i]], s["vs"][at[i]] = _code(x["v"][i])
            if tracked:
                s["weights"][at] = x["weights"].transpose(1, 2)
                if "positions" in x:
                    s["positions"][at] = x["positions"].transpose(1, 2)
    return s


# ------------------------------------------------------------------------- the plain forms
def _code(x):
    """Packed codes (two to a byte) and scales of rows x [..., head_dim]; 64 bits next to the rounding borders."""
    g = x.double().unflatten(-1, (-1, GROUP))
    s = (g.abs().amax(-1, keepdim=True).float() / 7).bfloat16()
    c = torch.where(s == 0, 0.0, torch.round(g / torch.where(s == 0, 1.0, s.double()))).clamp(-7, 7)
    u = (c + 8).to(torch.uint8).flatten(-2)
    return u[..., 0::2] | (u[..., 1::2] << 4), s.squeeze(-1)


def _values(codes, scales):
    """The values, bf16(code * scale), in 32 bits."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8
    return (c.unflatten(-1, (-1, GROUP)) * scales.float().unsqueeze(-1)).flatten(-2).bfloat16().float()


def _places(s, start, m):
    """Pool places of rows start .. start + m of the sequences' slots [n, m] (within the capacity)."""
    r = (start.long()[:, None] + torch.arange(m, device="cuda")).clamp(max=s["held"] - 1)
    slot = s["slots"].long()[:, None]
    if s["table"] is None:
        return slot * s["held"] + r
    page = s["case"]["page"]
    return s["table"].long()[slot, r // page] * page + r % page


def _plain_append(s, k, v, counts):
    m = k.shape[1]
    at = _places(s, s["start"], m)
    live = torch.arange(m, device="cuda")[None] < counts[:, None]
    for name, x in (("k", k), ("v", v)):
        codes, scales = _code(x)
        s[name + "c"][at[live]] = codes[live]
        s[name + "s"][at[live]] = scales[live]
    return at, live


def _plain_read(s, start, m, counts, typ):
    at = _places(s, start, m)
    live = (torch.arange(m, device="cuda")[None] < counts[:, None])[..., None, None]
    return tuple(torch.where(live, _values(s[n + "c"][at], s[n + "s"][at]), 0.0).to(typ) for n in "kv")


def _plain_attend(s):
    c, q = s["case"], s["q"]
    n, m, h, d = q.shape
    t = c["keys"]
    at = _places(s, s["zeros"], t)
    qf = q.float().view(n, m, c["kv_heads"], h // c["kv_heads"], d)
    keys = _values(s["kc"][at], s["ks"][at])                                   # [n, t, kv, d]
    scores = torch.einsum("nmkgd,ntkd->nkgmt", qf, keys) * (1 / math.sqrt(d))
    del keys
    j = torch.arange(t, device="cuda")
    last = s["counts"][:, None] - m + torch.arange(m, device="cuda")[None]      # row of each query token
    seen = j <= last[..., None]
    if c["window"]:
        seen &= j > last[..., None] - c["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    p /= p.sum(-1, keepdim=True)
    out = torch.einsum("nkgmt,ntkd->nmkgd", p, _values(s["vc"][at], s["vs"][at])).reshape(n, m, h, d).to(q.dtype)
    if not c["accumulate"]:
        return out
    gained = p.sum((2, 3))                                                     # [n, kv, t]
    w = s["weights"][at].transpose(1, 2) + gained
    live = (j[None] < s["counts"][:, None])
    s["weights"][at[live]] = w.transpose(1, 2)[live]
    return out, torch.where(live[:, None], w, 0.0)


def _plain_evict(s):
    c = s["case"]
    n, b, t = c["n_seq"], c["budget"], c["budget"] + c["rows"]
    at, _ = _plain_append(s, s["new_k"], s["new_v"], torch.full_like(s["counts"], c["rows"]))
    s["positions"][at] = s["new_positions"].transpose(1, 2)
    s["weights"][at] = 0.0 if s["new_weights"] is None else s["new_weights"].transpose(1, 2)
    s["new_positions"].add_(c["rows"])
    at = _places(s, s["zeros"], t)
    pos, w = s["positions"][at].transpose(1, 2), s["weights"][at].transpose(1, 2)      # [n, kv, t]
    safe = pos > pos.amax(-1, keepdim=True) - c["recent"]
    order = torch.sort(torch.where(safe, math.inf, w), dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(safe).scatter_(-1, order[..., :b], True)
    movers = torch.sort((~kept[..., b:]).int(), dim=-1, stable=True).indices + b
    hole = (torch.cumsum((~kept[..., :b]).int(), -1) - 1).clamp(0, t - b - 1)
    src = torch.where(kept[..., :b], torch.arange(b, device="cuda"), movers.gather(-1, hole))  # [n, kv, b]
    from_ = at.gather(1, src.flatten(1)).view_as(src).transpose(1, 2)                  # [n, b, kv]
    head = torch.arange(c["kv_heads"], device="cuda")
    to = at[:, :b, None]
    for name in ("kc", "vc", "ks", "vs", "positions", "weights"):
        s[name][to, head] = s[name][from_, head]
    k, v = _plain_read(s, s["zeros"], b, torch.full_like(s["counts"], b), torch.bfloat16)
    return (torch.clamp(s["counts"], max=b), s["positions"][at[:, :b]].transpose(1, 2),
            s["weights"][at[:, :b]].transpose(1, 2), k, v)


# -------------------------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    if c["op"] == "append":
        if own:
            s["cache"].append(s["new_k"], s["new_v"], s["slots"], s["start"], counts=s["counts"])
            return s["cache"].read(s["slots"], s["start"], c["rows"], counts=s["counts"])
        _plain_append(s, s["new_k"], s["new_v"], s["counts"])
        return _plain_read(s, s["start"], c["rows"], s["counts"], torch.bfloat16)
    if c["op"] == "read":
        if own:
            return s["cache"].read(s["slots"], s["start"], c["rows"], counts=s["counts"], dtype=TYPES[c["dtype"]])
        return _plain_read(s, s["start"], c["rows"], s["counts"], TYPES[c["dtype"]])
    if c["op"] == "attend":
        if not own:
            return _plain_attend(s)
        out = s["cache"].attend(s["q"], s["slots"], s["counts"], window=c["window"], accumulate=c["accumulate"])
        if not c["accumulate"]:
            return out
        return out, s["cache"].account(s["slots"], s["zeros"], c["keys"], counts=s["counts"])[1]
    if not own:
        return _plain_evict(s)
    s["cache"].append(s["new_k"], s["new_v"], s["slots"], s["start"], positions=s["new_positions"],
                      weights=s["new_weights"])
    s["new_positions"].add_(c["rows"])
    lens = s["cache"].evict(s["slots"], s["counts"], c["budget"], c["recent"])
    positions, weights = s["cache"].account(s["slots"], s["zeros"], c["budget"])
    k, v = s["cache"].read(s["slots"], s["zeros"], c["budget"])
    return lens, positions, weights, k, v


# ------------------------------------------------------------------- the definition, 64 bits
def _bf16_of(x):
    """x (64 bits) rounded to eight significant bits, ties to even: 45 of the 52 stored ones go."""
    u = x.contiguous().view(torch.int64)
    return ((u + ((1 << 44) - 1) + ((u >> 45) & 1)) >> 45 << 45).view(torch.float64)


def _stands_for(x):
    """The values that coded rows x [..., head_dim] stand for: each number by the borders it lies between."""
    g = x.to(torch.float64).reshape(*x.shape[:-1], -1, GROUP)
    s = _bf16_of(g.abs().max(-1, keepdim=True).values / 7)
    a, code = g.abs(), torch.zeros_like(g)
    for c in range(7):
        border = (c + 0.5) * s
        code += (a > border) | ((a == border) & (c % 2 == 1))
    return _bf16_of(torch.sign(g) * code * s).reshape(x.shape)


def exact(case, seed):
    x = _inputs(case, seed)
    n, kvh, d = case["n_seq"], case["kv_heads"], case["head_dim"]
    if case["op"] in ("append", "read"):
        outs = []
        for t in (x["k"], x["v"]):
            o = torch.zeros(t.shape, dtype=torch.float64, device="cuda")
            for i, m in enumerate(_counts(case)):
                o[i, :m] = _stands_for(t[i, :m])
            outs.append(o)
        return tuple(outs)
    if case["op"] == "attend":
        m, h, t = case["q_len"], case["heads"], case["keys"]
        g = h // kvh
        out = torch.zeros(n, m, h, d, dtype=torch.float64, device="cuda")
        account = torch.zeros(n, kvh, t, dtype=torch.float64, device="cuda")
        for i, held in enumerate(_counts(case)):
            row = torch.arange(held - m, held, device="cuda").repeat_interleave(g)
            key = torch.arange(held, device="cuda")
            hidden = key[None] > row[:, None]
            if case["window"]:
                hidden |= key[None] <= row[:, None] - case["window"]
            for k in range(kvh):
                keys, vals = _stands_for(x["k"][i, :held, k]), _stands_for(x["v"][i, :held, k])
                q = x["q"][i, :, k * g:(k + 1) * g].reshape(m * g, d).double()
                p = torch.softmax(((q @ keys.T) / math.sqrt(d)).masked_fill(hidden, -math.inf), -1)
                out[i, :, k * g:(k + 1) * g] = (p @ vals).reshape(m, g, d)
                if case["accumulate"]:
                    account[i, k, :held] = x["weights"][i, k, :held].double() + p.sum(0)
        return (out, account) if case["accumulate"] else out
    b, m = case["budget"], case["rows"]
    w = torch.cat([x["weights"], torch.zeros(n, kvh, m, device="cuda") if x["new_weights"] is None else x["new_weights"]], 2)
    pos = torch.cat([x["positions"], x["new_positions"]], 2)
    k, v = (torch.cat([_stands_for(x[a]), _stands_for(x["new_" + a])], 1) for a in "kv")
    src = torch.zeros(n, kvh, b, dtype=torch.long)
    ws, ps = w.cpu().tolist(), pos.cpu().tolist()
    for i in range(n):
        for j in range(kvh):
            oldest_safe = max(ps[i][j]) - case["recent"] + 1
            rank = sorted(range(b + m), key=lambda r: (0, 0) if ps[i][j][r] >= oldest_safe else (1, -ws[i][j][r]))
            keep = set(rank[:b])
            movers = iter(sorted(r for r in keep if r >= b))
            src[i, j] = torch.tensor([r if r in keep else next(movers) for r in range(b)])
    src = src.cuda()
    rows = src.transpose(1, 2)[..., None].expand(n, b, kvh, d)
    return (None, None, w.double().gather(2, src), k.gather(1, rows), v.gather(1, rows))
