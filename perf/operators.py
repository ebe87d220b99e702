"""The operators of a paged key-value cache, as calls that can be timed and checked: the sampling step over
a paged cache, the append to it, the accumulated attention weight of its rows, and the eviction of its
lightest rows.

``run`` computes each of them in its plain form (elementary torch operations in 32 bits), or, with ``own``
true, through the calls that a user makes of this package.  Notation: B entries, Hq query heads on Hkv
key-value heads (G = Hq / Hkv), head size d, S rows of a block (1: a single token), P[b] cached rows of entry
b, pools of pages [pages][Hkv][page][d] with a page table [B][max_pages] (page 0 in a case: contiguous caches
[B][Hkv][capacity][d] without a table).

  sample:  out = softmax(scale q [k_cache[:P]; k_blk]^T) [v_cache[:P]; v_blk], lse = its log-sum-exp
  append:  cache rows P..P+S-1 = the new rows; their weight = 0, their position = tokens..tokens+S-1
  weigh:   weight_out[j] = weight[j] + sum over the G S query rows i of exp(scale q_i.k_j - lse_i),  j < P
  evict:   of the P rows, `keep` stay: those at positions >= tokens - recent, then the heaviest (ties: lowest
           row).  Kept rows below `keep` stay where they are; the i-th kept row at or past `keep` moves to the
           i-th row below `keep` that is not kept, with its weight and position.
"""
import torch

own = False

NEG = float("-inf")


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one sequence, one token: the latency of a single decoding call (one attention layer)
        {"name": "sample token B1 P500", "op": "sample", "B": 1, "Hq": 16, "Hkv": 8, "d": 128, "S": 1, "page": 64,
         "shortest": 500, "longest": 500, "block": True},
        # a serving batch of single tokens with prompts of every length, some of them empty
        {"name": "sample tokens B32 ragged", "op": "sample", "B": 32, "Hq": 32, "Hkv": 8, "d": 128, "S": 1,
         "page": 16, "shortest": 0, "longest": 8192, "block": True},
        # the denoising step of a block, the sampling workload of the benchmark over pages
        {"name": "sample blocks B32 P2048", "op": "sample", "B": 32, "Hq": 16, "Hkv": 8, "d": 128, "S": 16,
         "page": 64, "shortest": 2048, "longest": 2048, "block": True},
        # the long-context loop's heads (G S = 64), four times its longest prefix
        {"name": "sample blocks B4 P32768", "op": "sample", "B": 4, "Hq": 32, "Hkv": 8, "d": 128, "S": 16,
         "page": 128, "shortest": 31000, "longest": 32768, "block": True},
        # odd sizes: head size 64, seven rows, pages of 48, the block already in the cache
        {"name": "sample odd d64", "op": "sample", "B": 5, "Hq": 12, "Hkv": 4, "d": 64, "S": 7, "page": 48,
         "shortest": 1, "longest": 3001, "block": False},
        # every layer's append of a finished block to the cache, a serving batch
        {"name": "append blocks B32", "op": "append", "B": 32, "Hkv": 8, "d": 128, "S": 16, "page": 64,
         "shortest": 100, "longest": 2000},
        # a prompt of 4095 tokens written into pages after its encoding
        {"name": "append prompts B4", "op": "append", "B": 4, "Hkv": 8, "d": 128, "S": 4095, "page": 16,
         "shortest": 0, "longest": 33},
        # weights after a finished block, the sampling workload's sizes
        {"name": "weigh blocks B32 P2064", "op": "weigh", "B": 32, "Hq": 16, "Hkv": 8, "d": 128, "S": 16, "page": 64,
         "shortest": 2064, "longest": 2064},
        # weights after one token, contiguous caches, head size 64, odd lengths
        {"name": "weigh token d64", "op": "weigh", "B": 6, "Hq": 16, "Hkv": 16, "d": 64, "S": 1, "page": 0,
         "shortest": 130, "longest": 1999},
        # a full cache gives up as many rows as the next block brings
        {"name": "evict block B32 2064", "op": "evict", "B": 32, "Hkv": 8, "d": 128, "page": 64,
         "shortest": 2064, "longest": 2064, "keep": 2048, "recent": 64},
        # a long prompt is cut to a budget once
        {"name": "evict prompt B4 32768", "op": "evict", "B": 4, "Hkv": 8, "d": 128, "page": 128,
         "shortest": 30011, "longest": 32768, "keep": 8192, "recent": 512},
        # one short sequence, contiguous caches
        {"name": "evict odd B1 777", "op": "evict", "B": 1, "Hkv": 5, "d": 64, "page": 0,
         "shortest": 777, "longest": 777, "keep": 500, "recent": 33},
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    """One more case: an operator, heads, a page size and lengths over the listed ones' range.  At most 2^20 cached rows
    of all heads (fewer where more than 64 query rows read each), so no drawn case costs more than the largest listed."""
    op = rng.choice(("sample", "sample", "append", "weigh", "evict"))
    case = {"op": op, "B": _log(rng, 1, 32), "Hkv": rng.choice((1, 2, 3, 4, 8)), "d": rng.choice((32, 64, 128, 128)),
            "page": rng.choice((0, 16, 32, 48, 64, 128))}
    heads, most = case["B"] * case["Hkv"], 1 << 20
    if op in ("sample", "weigh"):
        G = rng.choice((1, 2, 4, 8))
        case["Hq"] = case["Hkv"] * G
        case["S"] = rng.choice((1, 1, _log(rng, 1, 16)))
        most = min(most, (1 << 26) // (G * case["S"]))
    if op == "append":
        case["S"] = _log(rng, 1, min(4095, (1 << 18) // heads))
    case["longest"] = _log(rng, 2, min(16384, most // heads))
    case["shortest"] = rng.randint(0, case["longest"])
    if op == "sample":
        case["block"] = rng.random() < 0.75
    if op == "weigh":
        case["shortest"] = max(1, case["shortest"])
    if op == "evict":
        case["keep"] = rng.randint(1, case["longest"])
        case["recent"] = rng.randint(0, min(case["keep"], 512))
    return case


def lengths(case):
    """P[b]: entry b's share of the range, the first entry the longest and the second the shortest."""
    lo, hi, n = case["shortest"], case["longest"], case["B"]
    mid = [lo + int((hi - lo) * ((0.6180339887 * b) % 1.0)) for b in range(2, n)]
    return ([hi, lo] + mid)[:n]


def capacity(case):
    """Rows that an entry's cache can hold: the longest length, the block after it, and up to one page more."""
    rows = case["longest"] + (case["S"] if case["op"] == "append" else 16)
    if case["page"] == 0:
        return rows
    return -(-rows // case["page"]) * case["page"]


# ---------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    B, Hkv, d, op = case["B"], case["Hkv"], case["d"], case["op"]
    cap, P = capacity(case), lengths(case)
    st = {"op": op, "P": torch.tensor(P, dtype=torch.int32, device="cuda"), "table": None, "cap": cap}
    if case["page"]:
        # a pool with a few pages more than the entries use, in an order that has nothing to do with them
        each = cap // case["page"]
        pages, rows = B * each + 3, case["page"]
        order = torch.randperm(pages, generator=g, device="cuda")[:B * each].view(B, each).to(torch.int32)
        if op != "append":
            # an entry of the table past an entry's length names no page
            used = (st["P"][:, None] + rows - 1) // rows
            order = torch.where(torch.arange(each, device="cuda")[None, :] < used, order, -1)
        st["table"] = order.contiguous()
    else:
        pages, rows = B, cap
    st["k"] = normal(pages, Hkv, rows, d)
    if op != "weigh":
        st["v"] = normal(pages, Hkv, rows, d)
    if op in ("sample", "weigh"):
        Hq, S = case["Hq"], case["S"]
        st["q"] = normal(B, Hq, S, d)
        if op == "sample" and case["block"]:
            st["k_blk"], st["v_blk"] = normal(B, Hkv, S, d), normal(B, Hkv, S, d)
    if op == "append":
        st["k_new"], st["v_new"] = normal(B, Hkv, case["S"], d), normal(B, Hkv, case["S"], d)
    if op != "sample":
        # weights as attention leaves them: a few rows carry much, many carry little, the newest none yet
        st["weight"] = torch.exp(2.0 * torch.randn((B, Hkv, cap), generator=g, device="cuda") - 3.0)
        st["weight"].masked_fill_(torch.arange(cap, device="cuda") >= st["P"][:, None, None] - 4, 0.0)
        st["pos"] = torch.arange(cap, dtype=torch.int32, device="cuda").expand(B, Hkv, cap).contiguous()
        st["tokens"] = st["P"].clone()
    if op == "weigh":
        # the log-sum-exp that the attention over the same rows returned
        s = _scores(st)
        st["lse"] = torch.logsumexp(s, dim=-1).view(B, case["Hq"], case["S"]).contiguous()
        st["weight_out"] = torch.zeros_like(st["weight"])
    if op == "evict":
        # positions as earlier evictions leave them: not in the order of the rows, other ones in each head
        for b, n in enumerate(P):
            st["pos"][b, :, :n] = torch.rand((Hkv, n), generator=g, device="cuda").argsort(dim=-1).to(torch.int32)
        st["weight_out"], st["pos_out"] = torch.zeros_like(st["weight"]), torch.zeros_like(st["pos"])
        st["P_out"] = torch.zeros_like(st["P"])
        st["keep"], st["recent"] = case["keep"], case["recent"]
    return st


# ---------------------------------------------------------------------------------------------- plain forms
def _rows(st, pool):
    """[B][Hkv][capacity][d] of a pool, in 32 bits."""
    if st["table"] is None:
        return pool.float()
    B, Hkv = st["P"].shape[0], pool.shape[1]
    x = pool[st["table"].long().clamp(min=0)]  # [B][each][Hkv][page][d]
    return x.transpose(1, 2).reshape(B, Hkv, st["cap"], pool.shape[3]).float()


def _place(st, row):
    """(page, row in page) of row `row` [B][...] of each entry."""
    if st["table"] is None:
        return torch.arange(row.shape[0], device=row.device).view(-1, *[1] * (row.dim() - 1)).expand_as(row), row
    page = st["k"].shape[2]
    each = torch.gather(st["table"].long(), 1, (row // page).reshape(row.shape[0], -1)).view(row.shape)
    return each, row % page


def _scores(st):
    """scale q.k of every query row and cached row, [B][Hkv][G S][capacity]; rows past the length: -inf."""
    q, k = st["q"].float(), _rows(st, st["k"])
    B, Hq, S, d = q.shape
    Hkv = k.shape[1]
    s = torch.matmul(q.view(B, Hkv, Hq // Hkv * S, d), k.transpose(2, 3)) * d ** -0.5
    return s.masked_fill(torch.arange(st["cap"], device=q.device) >= st["P"][:, None, None, None], NEG)


def _sample(st):
    q = st["q"]
    B, Hq, S, d = q.shape
    Hkv = st["k"].shape[1]
    s, v = _scores(st), _rows(st, st["v"])
    if "k_blk" in st:
        rows = q.float().view(B, Hkv, Hq // Hkv * S, d)
        s = torch.cat([s, torch.matmul(rows, st["k_blk"].float().transpose(2, 3)) * d ** -0.5], dim=-1)
        v = torch.cat([v, st["v_blk"].float()], dim=2)
    m = s.amax(dim=-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(s - m)
    total = e.sum(dim=-1, keepdim=True)
    out = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)  # a row that sees nothing: zeros
    lse = (m + torch.log(total)).masked_fill(total == 0, NEG)
    return out.view(B, Hq, S, d).to(q.dtype), lse.view(B, Hq, S)


def _append(st):
    k_new = st["k_new"]
    B, Hkv, S, d = k_new.shape
    at = torch.arange(S, device=k_new.device)
    row = (st["P"].long()[:, None] + at)  # [B][S]
    page, r = _place(st, row)
    st["k"][page, :, r] = k_new.transpose(1, 2)
    st["v"][page, :, r] = st["v_new"].transpose(1, 2)
    where = row[:, None, :].expand(B, Hkv, S)
    st["weight"].scatter_(2, where, 0.0)
    st["pos"].scatter_(2, where, (st["tokens"][:, None] + at)[:, None, :].expand(B, Hkv, S).to(torch.int32))
    return st["k"], st["v"], st["weight"], st["pos"]


def _weigh(st):
    B, Hq, S, d = st["q"].shape
    Hkv = st["k"].shape[1]
    p = torch.exp(_scores(st) - st["lse"].view(B, Hkv, Hq // Hkv * S, 1))
    seen = torch.arange(st["cap"], device=p.device) < st["P"][:, None, None]
    st["weight_out"].copy_(torch.where(seen, st["weight"] + p.sum(dim=2), st["weight_out"]))
    return st["weight_out"]


def _evict(st):
    keep, P = st["keep"], st["P"].long()
    w, pos = st["weight"], st["pos"]
    B, Hkv, cap = w.shape
    row = torch.arange(cap, device=w.device).expand(B, Hkv, cap)
    key = torch.where(pos >= (st["tokens"] - st["recent"])[:, None, None], float("inf"), w)
    key = key.masked_fill(row >= P[:, None, None], NEG)
    rank = torch.argsort(torch.argsort(key, dim=-1, descending=True, stable=True), dim=-1)
    kept = (rank < keep) & (row < P[:, None, None])
    hole = (row < torch.clamp(P, max=keep)[:, None, None]) & ~kept
    mover = (row >= keep) & kept
    # the i-th mover's place is the i-th hole
    b, h, src = torch.nonzero(mover, as_tuple=True)
    _, _, dst = torch.nonzero(hole, as_tuple=True)  # as many in each head, in the same order
    out = row < torch.clamp(P, max=keep)[:, None, None]
    w_new, pos_new = torch.where(out, w, st["weight_out"]), torch.where(out, pos, st["pos_out"])
    w_new[b, h, dst], pos_new[b, h, dst] = w[b, h, src], pos[b, h, src]
    st["weight_out"].copy_(w_new)
    st["pos_out"].copy_(pos_new)
    if st["table"] is None:
        sp, sr, dp, dr = b, src, b, dst
    else:
        page, table = st["k"].shape[2], st["table"].long()
        sp, sr, dp, dr = table[b, src // page], src % page, table[b, dst // page], dst % page
    st["k"][dp, h, dr] = st["k"][sp, h, sr]
    st["v"][dp, h, dr] = st["v"][sp, h, sr]
    st["P_out"].copy_(torch.clamp(st["P"], max=keep))
    return st["k"], st["v"], st["weight_out"], st["pos_out"], st["P_out"]


# ---------------------------------------------------------------------------------------------- one pass
def run(state):
    st = state
    if not own:
        return {"sample": _sample, "append": _append, "weigh": _weigh, "evict": _evict}[st["op"]](st)
    from block_discrete_diffusion_tcgen05_b200 import attn

    if st["op"] == "sample":
        if "workspace" not in st:  # allocated once, as a serving loop does
            st["workspace"] = attn.sample_paged_workspace(st["q"], st["k"])
        return attn.decoder_sample_paged(st["q"], st["k"], st["v"], st["table"], st["P"], st.get("k_blk"),
                                         st.get("v_blk"), workspace=st["workspace"])
    if st["op"] == "append":
        attn.kv_cache_append_paged(st["k"], st["v"], st["table"], st["P"], st["k_new"], st["v_new"],
                                   weight=st["weight"], pos=st["pos"], tokens=st["tokens"])
        return st["k"], st["v"], st["weight"], st["pos"]
    if st["op"] == "weigh":
        return attn.kv_cache_weigh(st["q"], st["k"], st["table"], st["P"], st["lse"], st["weight"],
                                   out=st["weight_out"])
    if "workspace" not in st:
        st["workspace"] = attn.evict_workspace(st["weight"])
    attn.kv_cache_evict(st["k"], st["v"], st["table"], st["P"], st["weight"], st["pos"], st["tokens"], st["keep"],
                        recent=st["recent"], weight_out=st["weight_out"], pos_out=st["pos_out"], P_out=st["P_out"],
                        workspace=st["workspace"])
    return st["k"], st["v"], st["weight_out"], st["pos_out"], st["P_out"]


# ---------------------------------------------------------------------------------------------- its work
def work(case):
    B, Hkv, d, op, P = case["B"], case["Hkv"], case["d"], case["op"], lengths(case)
    table = 4 * sum(-(-p // case["page"]) for p in P) if case["page"] else 0
    if op in ("sample", "weigh"):
        GS = case["Hq"] // Hkv * case["S"]
        q = B * Hkv * GS
    if op == "sample":
        own_rows = case["S"] if case["block"] else 0
        rows = Hkv * sum(p + own_rows for p in P)
        return {"bytes": rows * d * 4 + q * (d * 4 + 4) + table + 4 * B, "flops": 4 * rows * GS * d}
    if op == "append":
        rows = B * Hkv * case["S"]
        return {"bytes": rows * (d * 8 + 8) + 8 * B, "flops": 0}
    if op == "weigh":
        rows = Hkv * sum(P)
        return {"bytes": rows * (d * 2 + 8) + q * (d * 2 + 4) + table + 4 * B, "flops": 2 * rows * GS * d}
    # evict: every weight and position read once, those of the kept rows written.  A kept row past `keep`
    # moves, K and V read and written: with weights that have nothing to do with the row, the share of the
    # rows past `keep` that is kept is keep / P.
    keep = case["keep"]
    moves = sum(round((p - keep) * keep / p) for p in P if p > keep) * Hkv
    return {"bytes": Hkv * sum(8 * p + 8 * min(p, keep) for p in P) + moves * d * 8 + 12 * B + table, "flops": 0}


# ---------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The attention and the weights by their definition, entry by entry and head by head.  The append and the
    eviction copy values: they compute none."""
    if case["op"] not in ("sample", "weigh"):
        return None
    st = prepare(case, seed)
    B, Hq, S, d = st["q"].shape
    Hkv, G, page = case["Hkv"], case["Hq"] // case["Hkv"], case["page"]
    if case["op"] == "sample":
        out = torch.zeros((B, Hq, S, d), dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq, S), NEG, dtype=torch.float64, device="cuda")
    else:
        wout = st["weight_out"].double()

    def cached(name, b, h, n):
        pool = st[name]
        if not page:
            return pool[b, h, :n].double()
        ids = st["table"][b, :-(-n // page)].tolist()
        return torch.cat([pool[i, h] for i in ids] + [pool[0, h, :0]])[:n].double()

    for b, n in enumerate(lengths(case)):
        for h in range(Hkv):
            q = st["q"][b, h * G:(h + 1) * G].double()  # [G][S][d]
            k = cached("k", b, h, n)
            if case["op"] == "weigh":
                p = torch.einsum("gsd,nd->gsn", q, k).div(d ** 0.5).sub(st["lse"][b, h * G:(h + 1) * G, :, None].double()).exp()
                wout[b, h, :n] = st["weight"][b, h, :n].double() + p.sum(dim=(0, 1))
                continue
            v = cached("v", b, h, n)
            if case["block"]:
                k, v = torch.cat([k, st["k_blk"][b, h].double()]), torch.cat([v, st["v_blk"][b, h].double()])
            if not k.shape[0]:
                continue
            a = torch.einsum("gsd,nd->gsn", q, k).div(d ** 0.5)
            out[b, h * G:(h + 1) * G] = torch.einsum("gsn,nd->gsd", a.softmax(dim=-1), v)
            lse[b, h * G:(h + 1) * G] = a.logsumexp(dim=-1)
    return (out, lse) if case["op"] == "sample" else wout
