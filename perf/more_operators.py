"""The operators of a paged serving batch, as they are measured: the plan of its pages, the store of
its rows, the attention of whole prompts and the attention of tokens behind a shared prefix.

Keys and values are held in pools [pages, kv_heads, page_size, head_dim] of 16-bit numbers.  A page
table names each slot's pages; pages not in use lie on a stack, and what is taken last in is given
first out.

  plan    cuts slots back to the rows that stay (pages behind them return to the stack) and extends
          them by new rows: pages for those, the pool row of every new row (packed, in the order
          of the sequences), each sequence's offset among them, and the new lengths;
  store   puts packed keys and values into the pools at given pool rows (-1: left out);
  prompt  causal softmax attention of packed sequences, optionally within a sliding window;
  shared  softmax attention of one token per sequence over the slot's rows, whose first pages are the
          same for every slot of the batch.

Without `own` every operator is computed in elementary torch operations; with it the calls are those
of runtime.PageTable and runtime.Attention.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a verification step's four drafts and a token of 64 sequences: what was rejected goes, the next rows come
        dict(name="plan drafts b64", op="plan", n_seq=64, base=1200, rows=5, shared=0, page=16),
        # a wave of requests behind one long instruction that all of them share
        dict(name="plan prompts b250", op="plan", n_seq=250, base=0, rows=1790, shared=1024, page=16),
        # one decode step's rows of eight sequences, one wide KV head
        dict(name="store step b8 d256", op="store", rows=8, spare=300, kv_heads=1, head_dim=256, dtype="bf16", page=128),
        # the prompts of a batch put away after their attention, a padded end
        dict(name="store prompts d128 gqa", op="store", rows=33111, spare=2000, kv_heads=8, head_dim=128, dtype="bf16", page=64),
        # one short request on a sliding layer: latency
        dict(name="prompt b1 t128 d256", op="prompt", n_seq=1, tokens=128, heads=8, kv_heads=1, head_dim=256, dtype="bf16", window=512),
        # eight prompts on a sliding layer, ragged
        dict(name="prompt b8 t4000 d256 w512", op="prompt", n_seq=8, tokens=4000, heads=8, kv_heads=1, head_dim=256, dtype="bf16", window=512),
        # the same on a full layer of wide heads
        dict(name="prompt b8 t4000 d512", op="prompt", n_seq=8, tokens=4000, heads=8, kv_heads=1, head_dim=512, dtype="bf16", window=0),
        # many short questions of narrow heads, odd group, fp16
        dict(name="prompt b61 t333 d64 f16", op="prompt", n_seq=61, tokens=333, heads=12, kv_heads=4, head_dim=64, dtype="f16", window=0),
        # one long document of a grouped-query model
        dict(name="prompt b1 t16384 d128 gqa", op="prompt", n_seq=1, tokens=16384, heads=32, kv_heads=8, head_dim=128, dtype="bf16", window=0),
        # eight agents early in their answers behind the same instructions
        dict(name="shared b8 p2048 d256", op="shared", n_seq=8, prefix=2048, rows=333, heads=8, kv_heads=1, head_dim=256, dtype="bf16", page=128),
        # samples of one problem, odd sizes, fp16
        dict(name="shared b29 p1504 d64 f16", op="shared", n_seq=29, prefix=1504, rows=777, heads=12, kv_heads=4, head_dim=64, dtype="f16", page=16),
        # a full batch behind a long document
        dict(name="shared b64 p16384 d128 gqa", op="shared", n_seq=64, prefix=16384, rows=1100, heads=32, kv_heads=8, head_dim=128, dtype="bf16", page=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng: random.Random):
    op = rng.choice(["plan", "store", "prompt", "prompt", "shared", "shared"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "plan":
        n = _log_int(rng, 1, 256)
        return dict(op=op, n_seq=n, base=rng.choice([0, _log_int(rng, 1, 4000)]), rows=_log_int(rng, 1, (1 << 19) // n),
                    shared=rng.choice([0, page * _log_int(rng, 1, 32)]), page=page)
    kv_heads = rng.choice([1, 1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8, 3, 5]) if kv_heads > 1 else rng.choice([4, 8, 8, 7, 16])
    c = dict(op=op, kv_heads=kv_heads, head_dim=rng.choice([64, 128, 256, 512]), dtype=rng.choice(["bf16", "bf16", "f16"]))
    wide = kv_heads * c["head_dim"]
    if op == "store":
        c.update(rows=_log_int(rng, 1, (32 << 20) // wide), spare=rng.randrange(0, 500), page=page)
        return c
    c["heads"] = kv_heads * group
    if op == "prompt":
        c["n_seq"] = _log_int(rng, 1, 64)
        # at most a quarter of the largest listed case's products, and no more tokens' numbers than it has
        most = math.sqrt(16384 * 16384 * 32 * 128 / 4 / (c["n_seq"] * c["heads"] * c["head_dim"]))
        most = min(most, 16384 * 40 * 128 / (c["n_seq"] * (c["heads"] + kv_heads) * c["head_dim"]))
        c.update(tokens=_log_int(rng, 1, int(most)), window=rng.choice([0, 0, _log_int(rng, 1, 2000)]))
        return c
    c["n_seq"] = _log_int(rng, 1, 96)
    most = (1 << 26) // wide
    prefix = min(_log_int(rng, page, max(page, min(20000, most // 2))), (1 << 25) // (c["n_seq"] * c["heads"]))
    c.update(prefix=prefix // page * page, rows=_log_int(rng, 1, max(1, min(4000, most // c["n_seq"]))), page=page)
    return c


def _ragged(n, most):
    """Rows of every sequence: a ragged batch, the first the longest."""
    return [max(1, most - (most * ((7 * i) % n)) // (2 * n)) for i in range(n)]


def _pairs(t, window):
    w = window if 0 < window < t else t
    return w * (w + 1) // 2 + (t - w) * w


def work(case):
    if case["op"] == "plan":
        n, rows = case["n_seq"], sum(_ragged(case["n_seq"], case["rows"]))
        pages = rows // case["page"] + n
        # counts, lengths and slots in; rows, offsets, lengths and the pages' names out; pages off and on the stack
        return {"bytes": 4 * (3 * n + rows + 2 * n + 4 * pages), "flops": 2 * rows}
    wide = case["kv_heads"] * case["head_dim"]
    if case["op"] == "store":
        return {"bytes": case["rows"] * (4 + 8 * wide), "flops": 0}
    h, d, n = case["heads"], case["head_dim"], case["n_seq"]
    if case["op"] == "prompt":
        lens = _ragged(n, case["tokens"])
        return {"bytes": sum(lens) * (4 * h * d + 4 * wide), "flops": 4 * h * d * sum(_pairs(t, case["window"]) for t in lens)}
    rows = _ragged(n, case["rows"])
    return {"bytes": 4 * wide * (case["prefix"] + sum(rows)) + 4 * n * h * d,
            "flops": 4 * h * d * (n * case["prefix"] + sum(rows))}


# ------------------------------------------------------------------------------- the inputs
def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _inputs(case, seed):
    """Everything that the case's numbers are made of, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = {}
    if case["op"] == "plan":
        n = case["n_seq"]
        x["slots"] = torch.randperm(n + 1, generator=g, device="cuda")[:n].to(torch.int32)
        r = torch.rand(n, generator=g, device="cuda").cpu().tolist()
        x["base"] = [int(case["base"] * (0.5 + 0.5 * u)) for u in r]
        x["rows"] = _ragged(n, case["rows"])
        return x
    typ, kvh, d = TYPES[case["dtype"]], case["kv_heads"], case["head_dim"]
    gain = 1 + 3 * (torch.rand(kvh, d, device="cuda", generator=g) < 0.05)

    def kv(m):
        """Keys and values of m rows: normed keys with some strong channels, values of uneven size."""
        k = (torch.randn(m, kvh, d, device="cuda", generator=g) * gain).to(typ)
        v = (torch.randn(m, kvh, d, device="cuda", generator=g) * torch.rand(m, kvh, 1, device="cuda", generator=g)).to(typ)
        return k, v

    if case["op"] == "store":
        m, page = case["rows"], case["page"]
        x["pages"] = -(-(m + case["spare"]) // page)
        x["k"], x["v"] = kv(m)
        # sequences of consecutive rows in scattered pages; some rows are left out
        at = torch.randperm(x["pages"], generator=g, device="cuda")[:, None] * page + torch.arange(page, device="cuda")
        keep = torch.rand(m, generator=g, device="cuda") < 0.98
        x["rows"] = torch.where(keep, at.flatten()[:m], -1).to(torch.int32)
        return x
    lens = _ragged(case["n_seq"], case["tokens"]) if case["op"] == "prompt" else [1] * case["n_seq"]
    x["q"] = torch.randn(sum(lens), case["heads"], d, device="cuda", generator=g).to(typ)
    if case["op"] == "prompt":
        x["k"], x["v"] = kv(sum(lens))
        x["offsets"] = [sum(lens[:i]) for i in range(len(lens) + 1)]
        return x
    x["rows"] = _ragged(case["n_seq"], case["rows"])
    x["prefix_k"], x["prefix_v"] = kv(case["prefix"])
    x["k"], x["v"] = kv(sum(x["rows"]))
    x["slots"] = torch.randperm(case["n_seq"], generator=g, device="cuda").to(torch.int32)
    return x


def prepare(case, seed):
    x = _inputs(case, seed)
    s = {"case": case}
    if case["op"] == "plan":
        page, n, pre = case["page"], case["n_seq"], case["shared"]
        most = -(-(pre + case["base"] + case["rows"]) // page)
        # (a slot's shared pages, those of its base rows and those of its new ones)
        total = pre // page + sum(-(-b // page) + -(-r // page) + 1 for b, r in zip(x["base"], x["rows"])) + 5
        s.update(slots=x["slots"], counts=_i32(x["rows"]), base=_i32([pre + b for b in x["base"]]), total=sum(x["rows"]))
        first, held = _i32([n + 1]), sum(x["base"])
        if own:
            from accelerator_decode_gb300 import runtime
            s["table"] = runtime.PageTable(n_slots=n + 2, n_pages=total, page_size=page, max_pages=most)
            plan = s["table"]
        else:
            s.update(page=page, table=torch.full((n + 2, most), -1, dtype=torch.int32, device="cuda"),
                     lens=torch.zeros(n + 2, dtype=torch.int32, device="cuda"),
                     refs=torch.zeros(total + 1, dtype=torch.int32, device="cuda"),
                     free=torch.arange(total, -1, -1, dtype=torch.int32, device="cuda") - 1,
                     top=torch.full((1,), total, dtype=torch.int64, device="cuda"))
            plan = _Plain(s)
        if pre:
            plan.extend(first, _i32([pre]), pre)
            plan.share(x["slots"], n + 1, pre // page)
        if held:
            plan.extend(x["slots"], _i32(x["base"]), held)
        return s
    if case["op"] == "store":
        s.update(k=x["k"], v=x["v"], rows=x["rows"])
        shape = (x["pages"], case["kv_heads"], case["page"], case["head_dim"])
        s["k_pool"], s["v_pool"] = (torch.zeros(shape, dtype=TYPES[case["dtype"]], device="cuda") for _ in "kv")
        if own:
            from accelerator_decode_gb300 import runtime
            s["table"] = runtime.PageTable(n_slots=1, n_pages=x["pages"], page_size=case["page"], max_pages=x["pages"])
        return s
    if own:
        from accelerator_decode_gb300 import runtime
        s["attn"] = runtime.Attention(case["heads"], case["kv_heads"], case["head_dim"], dtype=TYPES[case["dtype"]],
                                      max_seqs=case["n_seq"])
    s["q"] = x["q"]
    if case["op"] == "prompt":
        s.update(k=x["k"], v=x["v"], offsets=_i32(x["offsets"]), lens=[b - a for a, b in zip(x["offsets"], x["offsets"][1:])])
        return s
    # the pools with the prefix in the pages of a slot of its own and the sequences' rows behind it,
    # grown in turns as a batch grows, so that their pages are scattered
    page, n, pre = case["page"], case["n_seq"], case["prefix"]
    most = -(-(pre + case["rows"]) // page)
    total = pre // page + sum(-(-r // page) for r in x["rows"])
    shape = (total, case["kv_heads"], page, case["head_dim"])
    s["k_pool"], s["v_pool"] = (torch.zeros(shape, dtype=TYPES[case["dtype"]], device="cuda") for _ in "kv")
    s["slots"], s["longest"] = x["slots"], case["rows"]
    if own:
        s["table"] = runtime.PageTable(n_slots=n + 1, n_pages=total, page_size=page, max_pages=most)
        rows = s["table"].extend(_i32([n]), _i32([pre]), pre)[0]
        s["table"].store(x["prefix_k"], x["prefix_v"], rows, s["k_pool"], s["v_pool"])
        s["table"].share(s["slots"], n, pre // page)
        first = torch.tensor([sum(x["rows"][:i]) for i in range(n)], device="cuda")
        for a, b in zip([0, 40, 200], [40, 200, 1 << 30]):
            counts = [max(0, min(r, b) - a) for r in x["rows"]]
            if sum(counts) == 0:
                break
            rows, offsets, _ = s["table"].extend(s["slots"], _i32(counts), sum(counts))
            seq = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(counts, device="cuda"))
            at = first[seq] + a + torch.arange(sum(counts), device="cuda") - offsets[seq]
            s["table"].store(x["k"][at], x["v"][at], rows, s["k_pool"], s["v_pool"])
        return s
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    ids = torch.randperm(total, generator=g, device="cuda")
    s["table"] = torch.zeros(n, most, dtype=torch.int64, device="cuda")
    s["table"][:, :pre // page] = ids[:pre // page]
    s["lens"] = torch.zeros(n, dtype=torch.int64, device="cuda")
    used, done = pre // page, 0
    for i, r in enumerate(x["rows"]):
        slot, mine = int(x["slots"][i]), -(-r // page)
        s["table"][slot, pre // page:pre // page + mine] = ids[used:used + mine]
        s["lens"][slot] = pre + r
        at = _places(ids[used:used + mine], page)[:r]
        _plain_store(s, x["k"][done:done + r], x["v"][done:done + r], at)
        used, done = used + mine, done + r
    _plain_store(s, x["prefix_k"], x["prefix_v"], _places(ids[:pre // page], page))
    return s


# ------------------------------------------------------------------------- the plain forms
def _places(pages, page):
    return (pages.long()[:, None] * page + torch.arange(page, device="cuda")).flatten()


class _Plain:
    """The page table in elementary torch operations on the state's tensors."""

    def __init__(self, s):
        self.s = s

    def _pages(self, rows):
        return (rows + self.s["page"] - 1) // self.s["page"]

    def extend(self, slots, counts, n_rows):
        s, slots, page = self.s, slots.long(), self.s["page"]
        held = s["lens"][slots]
        old, need = self._pages(held), self._pages(held + counts) - self._pages(held)
        base = torch.cumsum(need, 0) - need
        col = torch.arange(s["table"].shape[1], device="cuda")
        fresh = (col >= old[:, None]) & (col < (old + need)[:, None])
        page_id = s["free"][(s["top"] - 1 - (base - old)[:, None] - col).clamp(0, s["free"].numel() - 1)]
        s["table"][slots] = torch.where(fresh, page_id, s["table"][slots])
        s["refs"].index_add_(0, torch.where(fresh, page_id, s["refs"].numel() - 1).flatten().long(), fresh.flatten().to(torch.int32))
        s["top"].sub_(need.sum())
        s["lens"][slots] = held + counts
        offsets = torch.zeros(slots.numel() + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = torch.cumsum(counts, 0)
        t = torch.arange(n_rows, device="cuda")
        seq = torch.searchsorted(offsets[1:].long(), t, right=True)
        at = held[seq] + t - offsets[seq]
        rows = s["table"][slots[seq], at // page] * page + at % page
        return rows.to(torch.int32), offsets, held + counts

    def share(self, slots, source, n_pages):
        s, slots = self.s, slots.long()
        s["table"][slots, :n_pages] = s["table"][source, :n_pages]
        s["refs"][s["table"][source, :n_pages].long()] += slots.numel()
        s["lens"][slots] = n_pages * s["page"]

    def truncate(self, slots, lens):
        s, slots = self.s, slots.long()
        held = s["lens"][slots]
        keep, old = self._pages(torch.minimum(lens, held)), self._pages(held)
        col = torch.arange(s["table"].shape[1], device="cuda")
        gone = (col >= keep[:, None]) & (col < old[:, None])
        ids = torch.where(gone, s["table"][slots], s["refs"].numel() - 1).long()
        s["refs"].index_add_(0, ids.flatten(), -gone.flatten().to(torch.int32))
        freed = (gone & (s["refs"][ids] == 0)).flatten()   # (no page is let go by two slots in one of these calls)
        rank = torch.cumsum(freed, 0)
        where = torch.where(freed, s["top"] + rank[-1] - rank, s["free"].numel() - 1)
        s["free"][where] = torch.where(freed, ids.flatten(), 0).to(torch.int32)
        s["top"].add_(rank[-1])
        s["table"][slots] = torch.where(gone, -1, s["table"][slots])
        s["lens"][slots] = torch.minimum(lens, held)


def _plain_store(s, k, v, rows):
    live = rows >= 0
    page = s["case"]["page"]
    at, row = (rows // page)[live].long(), (rows % page)[live].long()
    s["k_pool"][at, :, row] = k[live]
    s["v_pool"][at, :, row] = v[live]


def _plain_prompt(s):
    c, q = s["case"], s["q"]
    h, d, kvh = c["heads"], c["head_dim"], c["kv_heads"]
    out = torch.empty_like(q)
    done = 0
    for t in s["lens"]:
        part = max(1, min(t, (1 << 28) // (t * h // kvh)))          # query tokens at a time
        for k in range(kvh):
            heads = slice(k * (h // kvh), (k + 1) * (h // kvh))
            keys, vals = (s[n][done:done + t, k].float() for n in "kv")
            for a in range(0, t, part):
                b = min(t, a + part)
                lo = max(0, a - c["window"] + 1) if c["window"] else 0
                qf = q[done + a:done + b, heads].float().transpose(0, 1)            # [g, b - a, d]
                scores = torch.matmul(qf, keys[lo:b].T) * (1 / math.sqrt(d))
                i, j = torch.arange(a, b, device="cuda")[:, None], torch.arange(lo, b, device="cuda")
                seen = j <= i
                if c["window"]:
                    seen &= j > i - c["window"]
                scores.masked_fill_(~seen, -math.inf)
                p = torch.exp(scores - scores.amax(-1, keepdim=True))
                o = torch.matmul(p, vals[lo:b]) / p.sum(-1, keepdim=True)
                out[done + a:done + b, heads] = o.transpose(0, 1).to(q.dtype)
        done += t
    return out


def _plain_shared(s):
    c, q = s["case"], s["q"]
    n, h, d = q.shape
    kvh, page, pre = c["kv_heads"], c["page"], c["prefix"]
    slots = s["slots"].long()
    table, lens = s["table"][slots], s["lens"][slots]
    qf = q.float().view(n, kvh, h // kvh, d) * (1 / math.sqrt(d))
    out = torch.empty(n, kvh, h // kvh, d, dtype=q.dtype, device="cuda")
    pages = table[:, pre // page:]
    j = torch.arange(pages.shape[1] * page, device="cuda")
    hidden = (j >= (lens - pre)[:, None])[:, None]
    for k in range(kvh):
        # the prefix once for all, each sequence's own rows, and both under one softmax
        keys, vals = (s[p][table[0, :pre // page], k].float().view(pre, d) for p in ("k_pool", "v_pool"))
        own_keys, own_vals = (s[p][pages, k].float().view(n, -1, d) for p in ("k_pool", "v_pool"))
        before = torch.matmul(qf[:, k], keys.T)                                     # [n, g, pre]
        scores = torch.matmul(qf[:, k], own_keys.transpose(1, 2)).masked_fill_(hidden, -math.inf)
        top = torch.maximum(before.amax(-1, keepdim=True), scores.amax(-1, keepdim=True))
        before, scores = torch.exp(before - top), torch.exp(scores - top)
        total = before.sum(-1, keepdim=True) + scores.sum(-1, keepdim=True)
        out[:, k] = ((torch.matmul(before, vals) + torch.matmul(scores, own_vals)) / total).to(q.dtype)
    return out.view(n, h, d)


# -------------------------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    if c["op"] == "plan":
        plan = s["table"] if own else _Plain(s)
        plan.truncate(s["slots"], s["base"])
        rows, offsets, lens = plan.extend(s["slots"], s["counts"], s["total"])
        return rows, offsets, lens, s["table"].table if own else s["table"]
    if c["op"] == "store":
        if own:
            s["table"].store(s["k"], s["v"], s["rows"], s["k_pool"], s["v_pool"])
        else:
            _plain_store(s, s["k"], s["v"], s["rows"])
        return s["k_pool"], s["v_pool"]
    if c["op"] == "prompt":
        return s["attn"].prompt(s["q"], s["k"], s["v"], s["offsets"], window=c["window"]) if own else _plain_prompt(s)
    if not own:
        return _plain_shared(s)
    return s["attn"].shared(s["q"], s["k_pool"], s["v_pool"], s["table"], s["slots"], c["prefix"] // c["page"])


# ------------------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    x = _inputs(case, seed)
    if case["op"] == "plan":
        return _exact_plan(case, x)
    kvh, d = case["kv_heads"], case["head_dim"]
    if case["op"] == "store":
        pools = [torch.zeros(x["pages"], kvh, case["page"], d, dtype=torch.float64, device="cuda") for _ in "kv"]
        where = [(i, r) for i, r in enumerate(x["rows"].cpu().tolist()) if r >= 0]
        src = torch.tensor([i for i, _ in where], dtype=torch.long, device="cuda")
        to = torch.tensor([r for _, r in where], dtype=torch.long, device="cuda")
        for pool, t in zip(pools, (x["k"], x["v"])):
            flat = torch.zeros(x["pages"] * case["page"], kvh, d, dtype=torch.float64, device="cuda")
            flat[to] = t.to(torch.float64)[src]
            pool.copy_(flat.view(x["pages"], case["page"], kvh, d).transpose(1, 2))
        return tuple(pools)
    h = case["heads"]
    out = torch.zeros(x["q"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "prompt":
        for a, b in zip(x["offsets"], x["offsets"][1:]):
            for head in range(h):
                k, v = x["k"][a:b, head * kvh // h].double(), x["v"][a:b, head * kvh // h].double()
                for i in range(a, b, 2048):
                    e = min(b, i + 2048)
                    back = torch.arange(i - a, e - a, device="cuda")[:, None] - torch.arange(e - a, device="cuda")
                    far = back < 0 if not case["window"] else (back < 0) | (back >= case["window"])
                    score = (x["q"][i:e, head].double() @ k[:e - a].T / math.sqrt(d)).masked_fill(far, -math.inf)
                    out[i:e, head] = torch.softmax(score, -1) @ v[:e - a]
        return out
    done = 0
    for i, r in enumerate(x["rows"]):
        for head in range(kvh):
            q = x["q"][i, head * (h // kvh):(head + 1) * (h // kvh)].double()
            k = torch.cat([x["prefix_k"][:, head], x["k"][done:done + r, head]]).double()
            v = torch.cat([x["prefix_v"][:, head], x["v"][done:done + r, head]]).double()
            out[i, head * (h // kvh):(head + 1) * (h // kvh)] = torch.softmax(q @ k.T / math.sqrt(d), -1) @ v
        done += r
    return out


def _exact_plan(case, x):
    """The plan written out page by page: a list of free pages whose end is the top of the stack."""
    n, page, pre = case["n_seq"], case["page"], case["shared"]
    total = pre // page + sum(-(-b // page) + -(-r // page) + 1 for b, r in zip(x["base"], x["rows"])) + 5
    most = -(-(pre + case["base"] + case["rows"]) // page)
    free, slots = list(range(total))[::-1], x["slots"].cpu().tolist()
    prefix = [free.pop() for _ in range(pre // page)]
    pages = {slot: list(prefix) for slot in slots}
    held = {slot: pre for slot in slots}
    rows, offsets, lens = [], [0], []
    for counts, last in ((x["base"], False), (x["rows"], True)):
        for slot, m in zip(slots, counts):
            for r in range(held[slot], held[slot] + m):
                if r % page == 0:
                    pages[slot].append(free.pop())
                if last:
                    rows.append(pages[slot][r // page] * page + r % page)
            held[slot] += m
            if last:
                offsets.append(len(rows))
                lens.append(held[slot])
    table = [[-1] * most for _ in range(n + 2)]
    for slot, ids in list(pages.items()) + [(n + 1, prefix)]:
        table[slot][:len(ids)] = ids
    return _i32(rows), _i32(offsets), _i32(lens), _i32(table)
