"""What is timed of the operators around the verify-and-commit step, and their plain forms.

Four families of calls, all in the packed ragged layout of the step (request b
has K_b draft tokens, so a window of K_b + 1 rows):

  logprobs   log probability, rank, entropy and top alternatives of tokens
  attention  attention of whole windows over a paged key-value cache
  append     the window's key and value rows written to their pages
  pages      one round of the page operations: free, fork, reserve (with the
             copy of shared partial pages), append, commit (the kept
             candidate's rows moved to the front, the rest released)

A case is a dict of plain values. `run` takes the plain form (elementary torch
operations, in 32 bits) unless the module's name `own` is true; then it makes
the library's calls.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    lp = dict(op="logprobs", ragged=False, masked=False, committed=True)
    at = dict(op="attention", ragged=False, cand=1)
    ap = dict(op="append", ragged=False, cand=1)
    pg = dict(op="pages", ragged=False)
    return [
        # One request's window, five logprobs a token: a chat reply at batch size one.
        dict(lp, name="lp-one-request", B=1, K=4, V=32000, dtype="fp32", T=1.0, n_top=5),
        # The benchmark batch: the committed rows' logprobs with the usual largest number of alternatives.
        dict(lp, name="lp-batch", B=256, K=7, V=151936, dtype="bf16", T=0.7, n_top=20),
        # Scoring of every row, ragged windows, a vocabulary that is no multiple of a vector, some rows under a grammar's mask.
        dict(lp, name="lp-score-odd", B=211, K=8, V=128255, dtype="fp32", T=1.0, n_top=8, ragged=True, masked=True, committed=False),
        # One new token of one sequence over a long history: a draft model's step.
        dict(at, name="at-one-token", B=1, K=0, Hq=32, Hkv=8, D=128, page=16, ctx_min=8192, ctx_max=8192, dtype="bf16"),
        # The benchmark batch's windows over a middling history: the target's step.
        dict(at, name="at-batch", B=256, K=7, Hq=32, Hkv=8, D=128, page=16, ctx_min=1024, ctx_max=4096, dtype="bf16"),
        # Four candidates a request in one window, sixty-four requests of very unlike lengths.
        dict(at, name="at-candidates", B=64, K=5, cand=4, Hq=64, Hkv=8, D=64, page=32, ctx_min=17, ctx_max=8192, dtype="bf16", ragged=True),
        # An fp32 model of odd sizes: three query heads to a kv head, pages of seven tokens.
        dict(at, name="at-fp32-odd", B=37, K=3, Hq=12, Hkv=4, D=64, page=7, ctx_min=0, ctx_max=1000, dtype="fp32", ragged=True),
        # A decode step's rows of one layer.
        dict(ap, name="ap-batch", B=128, K=5, Hkv=8, D=128, page=16, ctx_min=1, ctx_max=2048, layers=1, dtype="bf16"),
        # Prompts of 64 sequences, ragged: the rows of one layer.
        dict(ap, name="ap-prompts", B=64, K=1023, Hkv=8, D=128, page=16, ctx_min=0, ctx_max=100, layers=1, dtype="bf16", ragged=True),
        # One request that is forked four times.
        dict(pg, name="pg-one-request", S=1, forks=4, K=4, cand=1, Hkv=4, D=64, page=16, ctx_min=500, ctx_max=600, layers=4, dtype="bf16"),
        # Sixty-four requests with four candidates each, of which one is kept.
        dict(pg, name="pg-candidates", S=64, forks=1, K=4, cand=4, Hkv=8, D=128, page=16, ctx_min=100, ctx_max=2000, layers=4, dtype="bf16", ragged=True),
        # A large pool: many forks of long shared prefixes, pages of 64 tokens.
        dict(pg, name="pg-many-forks", S=32, forks=8, K=7, cand=2, Hkv=8, D=128, page=64, ctx_min=64, ctx_max=4096, layers=4, dtype="bf16", ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "attention", "attention", "append", "pages"])
    if op == "logprobs":
        V = _log_int(rng, 1000, 256000)
        if rng.random() < 0.5:
            V = -(-V // 8) * 8
        K = rng.randint(0, 8)
        B = _log_int(rng, 1, max(1, min(256, int(2.5e8 / (V * (K + 1))))))
        return dict(op=op, B=B, K=K, V=V, dtype=rng.choice(["bf16", "fp32"]), T=rng.choice([0.5, 0.7, 1.0, 1.3]),
                    n_top=rng.choice([0, 1, 5, 8, 20, 32]), ragged=rng.random() < 0.6, masked=rng.random() < 0.3,
                    committed=rng.random() < 0.6)
    if op == "attention":
        Hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 3, 4, 5, 8])
        D = rng.choice([64, 128])
        cand = rng.choice([1, 1, 1, 2, 4])
        K = rng.randint(0, 8)
        page = rng.choice([1, 7, 16, 32, 64, 128])
        ctx = _log_int(rng, 1, 32000)
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        most = (2e9 if dtype == "bf16" else 1e8) / (ctx * Hkv * D * 4)
        B = _log_int(rng, 1, max(1, min(256, int(most))))
        return dict(op=op, B=B, K=K, cand=cand, Hq=Hkv * g, Hkv=Hkv, D=D, page=page, ctx_min=rng.choice([0, ctx // 2, ctx]),
                    ctx_max=ctx, dtype=dtype, ragged=rng.random() < 0.5)
    if op == "append":
        K = _log_int(rng, 1, 1024) - 1
        B = _log_int(rng, 1, max(1, min(256, 60000 // (K + 1))))
        return dict(op=op, B=B, K=K, cand=rng.choice([1, 1, 2]), Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]),
                    page=rng.choice([1, 7, 16, 32, 64]), ctx_min=0, ctx_max=rng.randint(0, 300), layers=rng.choice([1, 1, 2]),
                    dtype=rng.choice(["bf16", "fp32"]), ragged=rng.random() < 0.6)
    S = _log_int(rng, 1, 48)
    return dict(op=op, S=S, forks=rng.randint(1, max(1, min(8, 128 // S))), K=rng.randint(0, 7), cand=rng.choice([1, 2, 3, 4]),
                Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), page=rng.choice([1, 7, 16, 32, 64]), ctx_min=0,
                ctx_max=_log_int(rng, 1, 2000), layers=rng.choice([1, 2, 4]), dtype=rng.choice(["bf16", "fp32"]),
                ragged=rng.random() < 0.6)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _windows(c, n, gen):
    """Draft lengths of n requests and their offsets (int64 on the GPU): the same lengths for every seed, in another order."""
    if c["ragged"]:
        k = (c["K"] - torch.arange(n, device="cuda") % (c["K"] + 1))[torch.randperm(n, generator=gen, device="cuda")]
    else:
        k = torch.full((n,), c["K"], device="cuda", dtype=torch.int64)
    cu = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    cu[1:] = k.cumsum(0)
    return k, cu


def _randn(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _lengths(c, n, gen):
    """Lengths spread evenly from ctx_min to ctx_max, in an order of the seed's."""
    at = torch.arange(n, device="cuda")
    ctx = c["ctx_max"] - (c["ctx_max"] - c["ctx_min"]) * at // max(1, n - 1)
    return ctx[torch.randperm(n, generator=gen, device="cuda")]


def _tables(held, width, pool, gen):
    """Page tables of sequences that hold `held` pages each, from a shuffled pool of that many pages."""
    total = int(held.sum())
    perm = torch.randperm(pool, generator=gen, device="cuda")
    at = torch.arange(width, device="cuda")[None]
    first = (held.cumsum(0) - held)[:, None]
    table = torch.where(at < held[:, None], perm[(first + at).clamp_(max=pool - 1)], -1)
    ref = torch.zeros(pool, dtype=torch.int64, device="cuda")
    ref[perm[:total]] = 1
    return table.to(torch.int32), ref.to(torch.int32)


def _pack_bits(ref):
    """Bit p % 32 of word p / 32 is set where page p is free."""
    free = torch.zeros(-(-ref.shape[0] // 32) * 32, dtype=torch.int64, device=ref.device)
    free[: ref.shape[0]] = (ref == 0).to(torch.int64)
    words = (free.view(-1, 32) << torch.arange(32, device=ref.device)).sum(1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "logprobs":
        k, cu = _windows(c, c["B"], gen)
        R = int(cu[-1]) + c["B"]
        z = _randn((R, c["V"]), torch.float32, gen)
        z *= 2.0
        # A peaked head of sixteen tokens a row, as a trained model's rows have.
        at = torch.randint(0, c["V"], (R, 16), generator=gen, device="cuda")
        z.scatter_(1, at, 4.0 + 12.0 * torch.rand((R, 16), generator=gen, device="cuda"))
        if c["masked"]:  # one row in four allows a dozen tokens, the others of its vocabulary are -inf
            some = torch.randperm(R, generator=gen, device="cuda")[: max(1, R // 4)]
            kept = z[some].gather(1, at[some, :12])
            z[some] = -math.inf
            z[some[:, None], at[some, :12]] = kept
        tok = torch.where(torch.rand(R, generator=gen, device="cuda") < 0.5, z.argmax(1), at[:, 3])
        if not c["masked"]:
            rare = torch.rand(R, generator=gen, device="cuda") < 0.1
            tok = torch.where(rare, torch.randint(0, c["V"], (R,), generator=gen, device="cuda"), tok)
        s["logits"] = z.to(_DT[c["dtype"]])
        s["tokens"] = tok.to(torch.int32)
        s["cu_draft"] = cu.to(torch.int32) if c["committed"] else None
        n = torch.minimum((torch.rand(c["B"], generator=gen, device="cuda") * (k + 1)).to(torch.int64), k) + 1
        s["out_len"] = n.to(torch.int32) if c["committed"] else None
        f = dict(device="cuda", dtype=torch.float32)
        i = dict(device="cuda", dtype=torch.int32)
        s["out"] = {"logprob": torch.zeros(R, **f), "rank": torch.zeros(R, **i), "entropy": torch.zeros(R, **f),
                    "top_ids": torch.zeros((R, c["n_top"]), **i), "top_logprobs": torch.zeros((R, c["n_top"]), **f)}
        return s

    if c["op"] == "pages":
        S, B = c["S"], c["S"] * c["forks"]
        _, cu = _windows(c, B * c["cand"], gen)
        rows = (cu[1:] - cu[:-1] + 1).view(B, c["cand"])
        ctx = _lengths(c, S, gen)
        held = (ctx + c["page"] - 1) // c["page"]
        window = (c["K"] + 1) * c["cand"]
        most = (c["ctx_max"] + window + c["page"] - 1) // c["page"]
        src = torch.arange(S, device="cuda").repeat_interleave(c["forks"])
        table, ref = _tables(held, most, int(held.sum()) + B * ((window + c["page"] - 1) // c["page"] + 1), gen)
        s["page_table"] = torch.cat([table, torch.full((B, most), -1, dtype=torch.int32, device="cuda")])
        s["ctx_len"] = torch.cat([ctx, torch.zeros(B, dtype=torch.int64, device="cuda")]).to(torch.int32)
        s["src"], s["dst"] = src.to(torch.int32), torch.arange(S, S + B, device="cuda", dtype=torch.int32)
        s["cu_cand"] = torch.arange(B + 1, device="cuda", dtype=torch.int32) * c["cand"]
        best = torch.randint(0, c["cand"], (B,), generator=gen, device="cuda")
        s["best"] = (best + torch.arange(B, device="cuda") * c["cand"]).to(torch.int32)
        u = torch.rand(B * c["cand"], generator=gen, device="cuda")
        s["out_len"] = (torch.minimum((u * rows.view(-1)).to(torch.int64), rows.view(-1) - 1) + 1).to(torch.int32)
        s["granted"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    else:
        n = c["B"] * c["cand"]
        _, cu = _windows(c, n, gen)
        rows = (cu[1:] - cu[:-1] + 1).view(c["B"], c["cand"]).sum(1)
        ctx = _lengths(c, c["B"], gen)
        held = (ctx + rows + c["page"] - 1) // c["page"]
        most = (ctx + (c["K"] + 1) * c["cand"] + c["page"] - 1) // c["page"]
        s["page_table"], ref = _tables(held, int(most.max()), int(most.sum()) + 3, gen)
        s["ctx_len"] = ctx.to(torch.int32)
        s["cu_cand"] = torch.arange(c["B"] + 1, device="cuda", dtype=torch.int32) * c["cand"] if c["cand"] > 1 else None
    s["cu_draft"] = cu.to(torch.int32)
    R = int(cu[-1]) + cu.shape[0] - 1
    dt = _DT[c["dtype"]]
    layers = c.get("layers", 1)
    shape = (layers, ref.shape[0], c["page"], c["Hkv"], c["D"])
    s["k"], s["v"] = _randn(shape, dt, gen), _randn(shape, dt, gen)
    s["page_ref"], s["free_bits"] = ref, _pack_bits(ref)
    if c["op"] == "attention":
        s["q"] = _randn((R, c["Hq"], c["D"]), dt, gen) * 2.0
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((R, c["Hq"]), device="cuda")
    else:
        s["k_new"] = _randn((layers, R, c["Hkv"], c["D"]), dt, gen)
        s["v_new"] = _randn((layers, R, c["Hkv"], c["D"]), dt, gen)
    if own:  # the handle that a serving program keeps of its cache
        from speculative_decoding_verification_27_gb300 import api
        s["cache"] = api.KVCache(s["k"], s["v"], s["page_ref"], s["free_bits"])
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _owners(cu_draft, cu_cand):
    """Per window row: its request, its place in the request's window, and where its candidate begins there."""
    cu = cu_draft.long()
    C = cu.shape[0] - 1
    first = cu + torch.arange(C + 1, device=cu.device)  # first row of each candidate, and R at the end
    cand = torch.repeat_interleave(torch.arange(C, device=cu.device), first[1:] - first[:-1])
    edge = cu_cand.long() if cu_cand is not None else torch.arange(C + 1, device=cu.device)
    req = torch.searchsorted(edge, cand, right=True) - 1
    base = first[edge]  # first row of each request
    row = torch.arange(cand.shape[0], device=cu.device)
    return req, row - base[req], first[cand] - base[req], base


def _logprobs(s):
    c, o = s["case"], s["out"]
    R = s["logits"].shape[0]
    rows = torch.arange(R, device="cuda")
    if s["cu_draft"] is not None:
        req, place, _, _ = _owners(s["cu_draft"], None)
        rows = rows[place < s["out_len"].long()[req]]
    z = s["logits"][rows].float() + 0.0  # -0 counts as 0
    tok = s["tokens"][rows].long()[:, None]
    m = z.amax(1, keepdim=True)
    t = (z - m) / c["T"]
    e = t.exp()
    S = e.sum(1, dtype=torch.float64)
    log_S = S.log()[:, None]
    o["logprob"][rows] = (t.gather(1, tok) - log_S).float()[:, 0]
    o["entropy"][rows] = (log_S[:, 0] - torch.where(e > 0, e * t, 0.0).sum(1, dtype=torch.float64) / S).float()
    zt = z.gather(1, tok)
    at = torch.arange(c["V"], device="cuda")[None]
    o["rank"][rows] = (1 + (z > zt).sum(1) + ((z == zt) & (at < tok)).sum(1)).to(torch.int32)
    if c["n_top"]:
        # Order by value and then by the lowest index, as one whole number.
        bits = z.view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32) + (0x7FFFFFFF - at)
        n = min(c["n_top"], c["V"])
        ids = 0x7FFFFFFF - (key.topk(n, dim=1).values & 0xFFFFFFFF)
        lp = (t.gather(1, ids) - log_S).float()
        o["top_ids"][rows, :n] = torch.where(lp > -math.inf, ids, -1).to(torch.int32)
        o["top_logprobs"][rows, :n] = lp
    return o


def _attention(s):
    c = s["case"]
    req, place, begin, base = _owners(s["cu_draft"], s["cu_cand"])
    B, Hkv, D, g = c["B"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    ctx = s["ctx_len"].long()
    width = base[1:] - base[:-1]
    W, L = int(width.max()), int((ctx + width).max())
    at = torch.arange(L, device="cuda")
    page = s["page_table"].long()[:, at // c["page"]].clamp_(min=0)
    k = s["k"][0][page, at % c["page"]].float()  # [B, L, Hkv, D]
    v = s["v"][0][page, at % c["page"]].float()
    q = torch.zeros((B, W, c["Hq"], D), device="cuda")
    q[req, place] = s["q"].float()
    lo = torch.zeros((B, W), dtype=torch.int64, device="cuda")
    lo[req, place] = begin
    q = q.view(B, W, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, W * g, D)
    scores = (q @ k.permute(0, 2, 3, 1)) / math.sqrt(D)
    rel = at[None] - ctx[:, None]  # place in the window, below zero in the history
    seen = (rel[:, None] < 0) | ((rel[:, None] >= lo[:, :, None]) & (rel[:, None] <= torch.arange(W, device="cuda")[None, :, None]))
    seen = seen[:, None, :, None].expand(B, 1, W, g, L).reshape(B, 1, W * g, L)
    scores = torch.where(seen, scores, -math.inf)
    m = scores.amax(3, keepdim=True)
    p = (scores - m).exp()
    S = p.sum(3, keepdim=True)
    out = (p @ v.transpose(1, 2)) / S
    out = out.view(B, Hkv, W, g, D).permute(0, 2, 1, 3, 4).reshape(B, W, c["Hq"], D)
    lse = (m + S.log()).view(B, Hkv, W, g).permute(0, 2, 1, 3).reshape(B, W, c["Hq"])
    s["out"][:] = out[req, place].to(s["out"].dtype)
    s["lse"][:] = lse[req, place]
    return [s["out"], s["lse"]]


def _append(s, table, ctx):
    req, place, _, _ = _owners(s["cu_draft"], s["cu_cand"])
    at = ctx.long()[req] + place
    n = s["case"]["page"]
    page = table.long()[req, at // n]
    s["k"][:, page, at % n] = s["k_new"]
    s["v"][:, page, at % n] = s["v_new"]


def _pages(s):
    c = s["case"]
    n, S = c["page"], c["S"]
    table, ctx, ref = s["page_table"], s["ctx_len"], s["page_ref"]
    src, dst = s["src"].long(), s["dst"].long()
    col = torch.arange(table.shape[1], device="cuda")[None]
    # free: the forks of the last round
    held = (ctx[dst].long()[:, None] + n - 1) // n
    gone = table[dst][col < held].long()
    ref.index_add_(0, gone, torch.full_like(gone, -1).to(torch.int32))
    table[dst] = torch.where(col < held, -1, table[dst])
    ctx[dst] = 0
    # fork
    held = (ctx[src].long()[:, None] + n - 1) // n
    table[dst] = torch.where(col < held, table[src], table[dst])
    kept = table[dst][col < held].long()
    ref.index_add_(0, kept, torch.ones_like(kept).to(torch.int32))
    ctx[dst] = ctx[src]
    # reserve: a shared partial page is copied (by all but its last holder), then the window's pages, from the lowest free ones
    mine, length = table[S:], ctx[S:].long()
    _, _, _, base = _owners(s["cu_draft"], s["cu_cand"])
    rows = base[1:] - base[:-1]
    part = torch.where(length % n > 0, mine.long().gather(1, (length // n).clamp(max=table.shape[1] - 1)[:, None])[:, 0], -1)
    same = (part[:, None] == part[None]) & (part >= 0)[:, None]
    before = torch.tril(same, -1).sum(1)
    copy = (part >= 0) & (ref.long()[part.clamp(min=0)] - before > 1)
    held = (length + n - 1) // n
    new = (length + rows + n - 1) // n - held
    need = new + copy.long()
    free = torch.nonzero(ref == 0)[:, 0][: int(need.sum())]
    ref[free] = 1
    first = need.cumsum(0) - need
    target = torch.where(copy, free[first.clamp(max=free.shape[0] - 1)] if free.shape[0] else first, 0)
    who = torch.nonzero(copy)[:, 0]
    s["k"][:, target[who]] = _upto(s["k"], part[who], target[who], (length % n)[who], n)
    s["v"][:, target[who]] = _upto(s["v"], part[who], target[who], (length % n)[who], n)
    ref.index_add_(0, part[who], torch.full_like(part[who], -1).to(torch.int32))
    mine[who, (length // n)[who]] = target[who].to(torch.int32)
    req = torch.repeat_interleave(torch.arange(rows.shape[0], device="cuda"), new)
    place = torch.arange(req.shape[0], device="cuda") - (new.cumsum(0) - new)[req]
    mine[req, held[req] + place] = free[first[req] + copy.long()[req] + place].to(torch.int32)
    s["granted"][:] = rows.to(torch.int32)
    _append(s, mine, ctx[S:])
    # commit: the kept candidate's rows to the front of the window, the pages behind them released
    cu = s["cu_draft"].long()
    best = s["best"].long()
    count = s["out_len"].long()[best]
    begin = cu[best] + best - base[:-1]
    req = torch.repeat_interleave(torch.arange(rows.shape[0], device="cuda"), count)
    place = torch.arange(req.shape[0], device="cuda") - (count.cumsum(0) - count)[req]
    a, b = length[req] + begin[req] + place, length[req] + place
    pa, pb = mine.long()[req, a // n], mine.long()[req, b // n]
    s["k"][:, pb, b % n] = s["k"][:, pa, a % n]
    s["v"][:, pb, b % n] = s["v"][:, pa, a % n]
    keep, have = (length + count + n - 1) // n, (length + rows + n - 1) // n
    out = (col >= keep[:, None]) & (col < have[:, None])
    gone = mine[out].long()
    ref.index_add_(0, gone, torch.full_like(gone, -1).to(torch.int32))
    mine[out] = -1
    ctx[S:] += count.to(torch.int32)
    s["free_bits"][:] = _pack_bits(ref)
    return _page_outputs(s)


def _upto(pool, old, new, count, n):
    """Pages `new` with the first `count` tokens of pages `old` in them."""
    take = (torch.arange(n, device=pool.device)[None] < count[:, None])[None, :, :, None, None]
    return torch.where(take, pool[:, old], pool[:, new])


def _page_outputs(s):
    return {x: s[x] for x in ("k", "v", "page_table", "ctx_len", "page_ref", "free_bits", "granted")}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _own(s, op)
    if op == "logprobs":
        return _logprobs(s)
    if op == "attention":
        return _attention(s)
    if op == "append":
        _append(s, s["page_table"], s["ctx_len"])
        return [s["k"], s["v"]]
    return _pages(s)


def _own(s, op):
    from speculative_decoding_verification_27_gb300 import api
    if op == "logprobs":
        o, c = s["out"], s["case"]
        api.sv_token_logprobs(s["logits"], s["tokens"], cu_draft=s["cu_draft"], out_len=s["out_len"], temperature=c["T"],
                              n_top=c["n_top"], out_logprob=o["logprob"], out_rank=o["rank"], out_entropy=o["entropy"],
                              out_top_ids=o["top_ids"], out_top_logprobs=o["top_logprobs"])
        return o
    if op == "attention":
        api.sv_window_attention(s["q"], s["cache"], 0, s["page_table"], s["ctx_len"], s["cu_draft"], s["cu_cand"], out=s["out"],
                                out_lse=s["lse"])
        return [s["out"], s["lse"]]
    if op == "append":
        api.sv_cache_append(s["cache"], 0, s["k_new"], s["v_new"], s["page_table"], s["ctx_len"], s["cu_draft"], s["cu_cand"])
        return [s["k"], s["v"]]
    S, cache = s["case"]["S"], s["cache"]
    table, ctx = s["page_table"], s["ctx_len"]
    api.sv_cache_free(cache, table, ctx, s["dst"])
    api.sv_cache_fork(cache, table, ctx, s["src"], s["dst"])
    table, ctx = table[S:], ctx[S:]
    api.sv_cache_reserve(cache, table, ctx, s["cu_draft"], s["cu_cand"], granted=s["granted"])
    api.sv_cache_append(cache, 0, s["k_new"], s["v_new"], table, ctx, s["cu_draft"], s["cu_cand"])
    api.sv_cache_commit(cache, table, ctx, s["cu_draft"], s["out_len"], s["cu_cand"], s["best"])
    return _page_outputs(s)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    """Bytes and operations at the mean of the case's random lengths."""
    c = case
    size = 2 if c["dtype"] == "bf16" else 4
    K = c["K"] / 2 if c["ragged"] else c["K"]
    if c["op"] == "logprobs":
        rows = c["B"] * ((K + 2) / 2 if c["committed"] else K + 1)
        return {"bytes": rows * (c["V"] * size + 16 + 8 * c["n_top"]), "flops": rows * c["V"] * 6}
    ctx = (c["ctx_min"] + c["ctx_max"]) / 2
    token = 2 * c["Hkv"] * c["D"] * size  # one token's key and value rows of one layer
    window = (K + 1) * c["cand"]
    if c["op"] == "attention":
        io = c["B"] * window * c["Hq"] * (2 * c["D"] * size + 4)
        return {"bytes": c["B"] * (ctx + window) * token + io,
                "flops": 4 * c["B"] * window * c["Hq"] * c["D"] * (ctx + (K + 2) / 2)}
    if c["op"] == "append":
        return {"bytes": 2 * c["B"] * window * token * c["layers"] + 8, "flops": 0}
    B = c["S"] * c["forks"]
    copied = (c["page"] - 1) / 2  # tokens of a partial page
    moved = (K + 2) / 2 * (c["cand"] - 1) / c["cand"]
    table = 4 * (ctx / c["page"] + 1)
    return {"bytes": B * (2 * token * c["layers"] * (copied + window + moved) + 4 * table), "flops": 0}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "attention": _exact_attention, "append": _exact_append, "pages": _exact_pages}[case["op"]](s)


def _spans(s):
    """Per request the list of its candidates' row ranges, as whole numbers."""
    cu = s["cu_draft"].tolist()
    first = [a + i for i, a in enumerate(cu)]
    if s.get("cu_cand") is None:
        return [[(first[i], first[i + 1])] for i in range(len(cu) - 1)]
    e = s["cu_cand"].tolist()
    return [[(first[i], first[i + 1]) for i in range(a, b)] for a, b in zip(e[:-1], e[1:])]


def _exact_logprobs(s):
    c, o = s["case"], {k: (v.double() if v.is_floating_point() else v.long()) for k, v in s["out"].items()}
    rows = list(range(s["logits"].shape[0]))
    if s["cu_draft"] is not None:
        rows = [r for [(a, b)], n in zip(_spans(s), s["out_len"].tolist()) for r in range(a, a + n)]
    for i in range(0, len(rows), 64):
        r = torch.tensor(rows[i:i + 64], device="cuda")
        z = s["logits"][r].double()
        lp = torch.log_softmax(z / c["T"], 1)
        tok = s["tokens"][r].long()[:, None]
        o["logprob"][r] = lp.gather(1, tok)[:, 0]
        p = lp.exp()
        o["entropy"][r] = -torch.special.xlogy(p, p).sum(1)
        value, ids = torch.sort(z, dim=1, descending=True, stable=True)
        o["rank"][r] = 1 + (ids == tok).long().argmax(1)
        n = min(c["n_top"], c["V"])
        if n:
            value, ids = value[:, :n], ids[:, :n]
            o["top_ids"][r, :n] = torch.where(value == -math.inf, -1, ids)
            o["top_logprobs"][r, :n] = lp.gather(1, ids)
    return o


def _exact_attention(s):
    c = s["case"]
    out, lse = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64), s["lse"].double()
    g, n = c["Hq"] // c["Hkv"], c["page"]
    for b, spans in enumerate(_spans(s)):
        ctx, r0, r1 = int(s["ctx_len"][b]), spans[0][0], spans[-1][1]
        at = torch.arange(ctx + r1 - r0, device="cuda")
        page = s["page_table"][b].long()[at // n]
        k, v = s["k"][0][page, at % n].double(), s["v"][0][page, at % n].double()
        mask = torch.full((r1 - r0, at.shape[0]), -math.inf, device="cuda", dtype=torch.float64)
        mask[:, :ctx] = 0
        for a, e in spans:
            for r in range(a, e):
                mask[r - r0, ctx + a - r0: ctx + r - r0 + 1] = 0
        q = s["q"][r0:r1].double().view(r1 - r0, c["Hkv"], g, c["D"])
        x = torch.einsum("whgd,lhd->whgl", q, k) / math.sqrt(c["D"]) + mask[:, None, None]
        lse[r0:r1] = torch.logsumexp(x, 3).view(r1 - r0, c["Hq"])
        out[r0:r1] = torch.einsum("whgl,lhd->whgd", torch.softmax(x, 3), v).reshape(r1 - r0, c["Hq"], c["D"])
    return [out, lse]


def _put(s, table, ctx):
    n = s["case"]["page"]
    for b, spans in enumerate(_spans(s)):
        r0, r1 = spans[0][0], spans[-1][1]
        for p in range(ctx[b] // n, (ctx[b] + r1 - r0 + n - 1) // n):
            lo, hi = max(p * n, ctx[b]), min((p + 1) * n, ctx[b] + r1 - r0)
            for pool, new in ((s["k"], s["k_new"]), (s["v"], s["v_new"])):
                pool[:, table[b][p], lo - p * n: hi - p * n] = new[:, r0 + lo - ctx[b]: r0 + hi - ctx[b]]


def _exact_append(s):
    _put(s, s["page_table"].tolist(), s["ctx_len"].tolist())
    return [s["k"], s["v"]]


def _exact_pages(s):
    c = s["case"]
    n, S = c["page"], c["S"]
    table, ctx, ref = s["page_table"].tolist(), s["ctx_len"].tolist(), s["page_ref"].tolist()
    spans = _spans(s)

    def lowest():
        p = ref.index(0)
        ref[p] = 1
        return p

    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        ctx[b] = ctx[a]
        for i in range(-(-ctx[a] // n)):
            table[b][i] = table[a][i]
            ref[table[a][i]] += 1
    for b, sp in enumerate(spans):
        row, length, held = table[S + b], ctx[S + b], -(-ctx[S + b] // n)
        if length % n and ref[row[held - 1]] > 1:
            old, row[held - 1] = row[held - 1], lowest()
            ref[old] -= 1
            for pool in (s["k"], s["v"]):
                pool[:, row[held - 1], : length % n] = pool[:, old, : length % n]
        for i in range(held, -(-(length + sp[-1][1] - sp[0][0]) // n)):
            row[i] = lowest()
    _put(s, table[S:], ctx[S:])
    for b, (sp, best) in enumerate(zip(spans, s["best"].tolist())):
        row, length, count = table[S + b], ctx[S + b], int(s["out_len"][best])
        begin = sp[best - b * c["cand"]][0] - sp[0][0]
        for j in range(count if begin else 0):
            a, d = length + begin + j, length + j
            for pool in (s["k"], s["v"]):
                pool[:, row[d // n], d % n] = pool[:, row[a // n], a % n]
        for i in range(-(-(length + count) // n), -(-(length + sp[-1][1] - sp[0][0]) // n)):
            ref[row[i]] -= 1
            row[i] = -1
        ctx[S + b] = length + count
    back = lambda x: torch.tensor(x, device="cuda")  # noqa: E731
    words = [sum(1 << i for i in range(32) if w * 32 + i < len(ref) and not ref[w * 32 + i]) for w in range(-(-len(ref) // 32))]
    return {"k": s["k"], "v": s["v"], "page_table": back(table), "ctx_len": back(ctx), "page_ref": back(ref),
            "free_bits": back([w - (1 << 32) if w >> 31 else w for w in words]),
            "granted": back([sp[-1][1] - sp[0][0] for sp in spans])}
