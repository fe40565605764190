"""Timed cases of the decode-step operators: beam selection, reordering of
beam states, and the block tables, slot maps and moves of a paged cache.

Each case names an operator ("op") and its sizes:
  select   the M best continuations over beams and vocabulary
           c(w, v) = score_w + z_w(v)/T - ln sum_u exp(z_w(u)/T)
  reorder  beam j of every cache takes over the state of beam parent_j, in
           place, on dense caches [B*W, G, S, D] or through block tables
  extend   pages for the new tokens of every request from a free list, the
           block tables, and the slot, position and request of every token
  commit   lengths after a verify step, unused pages back to the free list
  compact  cache entries along the accepted path of a token tree moved to
           consecutive positions
`run` computes a case in plain torch operations, or with the package's
kernels where `own` is true.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _select(name, B, W, V, M, dtype, T=1.0, finished=0, masked=0.0, pad=0):
    return {"name": name, "op": "select", "B": B, "W": W, "V": V, "M": M, "dtype": dtype, "T": T,
            "finished": finished, "masked": masked, "pad": pad}


def _reorder(name, B, W, pools, G, S, D, dtype, page=0):
    return {"name": name, "op": "reorder", "B": B, "W": W, "pools": pools, "G": G, "S": S, "D": D,
            "dtype": dtype, "page": page}


def _extend(name, B, page, blocks, most_new):
    return {"name": name, "op": "extend", "B": B, "page": page, "blocks": blocks, "most_new": most_new}


def _commit(name, B, page, blocks, most_new, finished):
    return {"name": name, "op": "commit", "B": B, "page": page, "blocks": blocks, "most_new": most_new,
            "finished": finished}


def _compact(name, B, N, depth, pools, G, page, D, blocks, dtype):
    return {"name": name, "op": "compact", "B": B, "N": N, "depth": depth, "pools": pools, "G": G,
            "page": page, "D": D, "blocks": blocks, "dtype": dtype}


def listed():
    return [
        # one request with four beams: the step's latency
        _select("select 1x4x32000 fp32", 1, 4, 32000, 8, "fp32"),
        # an odd vocabulary (rows at any alignment), one beam of each request
        # finished, a grammar that leaves a tenth of the tokens
        _select("select 8x5x50021 bf16 odd", 8, 5, 50021, 10, "bf16", T=0.7, finished=1, masked=0.9),
        # a serving batch, twice as many candidates as beams
        _select("select 64x8x152064 bf16", 64, 8, 152064, 16, "bf16"),
        # fp32 logits of a large batch
        _select("select 128x4x128256 fp32", 128, 4, 128256, 8, "fp32", T=0.8),
        # the dense caches of a small batch, heads before positions
        _reorder("reorder 8x4 dense", 8, 4, 16, 8, 1024, 128, "bf16"),
        # one request's beams in a paged cache: few bytes, many small rows
        _reorder("reorder 1x4 paged", 1, 4, 32, 1, 600, 1024, "bf16", page=16),
        # a decode step: K + 1 = 6 tokens a request
        _extend("extend 64 decode", 64, 16, 512, 6),
        # requests in prefill: long ragged runs of new tokens
        _extend("extend 256 prefill", 256, 16, 1024, 4096),
        # the end of a decode step
        _commit("commit 64 decode", 64, 16, 512, 6, 0.0),
        # a large batch, one request in twenty finished and all its pages free
        _commit("commit 2000 finished", 2000, 16, 512, 8, 0.05),
        # a tree of 20 nodes (4, 2, 1), up to three accepted
        _compact("compact 4 tree 20", 4, 20, 3, 32, 1, 16, 1024, 16, "bf16"),
        # deep trees in a batch, heads before positions in a page
        _compact("compact 64 tree 60", 64, 60, 8, 32, 8, 16, 128, 16, "bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("select", "select", "reorder", "extend", "commit", "compact"))
    if op == "select":
        dtype = rng.choice(("fp32", "bf16"))
        W, V = _log_uniform(rng, 1, 16), _log_uniform(rng, 1000, 160000)
        most = (240 << 20) // (W * V * (4 if dtype == "fp32" else 2))
        return _select("", _log_uniform(rng, 1, max(1, min(256, most))), W, V, rng.randint(W, 2 * W), dtype,
                       T=rng.choice((1.0, 0.6, 1.3)), finished=rng.choice((0, W // 4)),
                       masked=rng.choice((0.0, 0.5)), pad=rng.choice((0, 0, 8, 27)))
    if op == "reorder":
        page = rng.choice((0, 8, 16, 64))
        W, G, D = rng.randint(2, 16), rng.choice((1, 2, 8)), rng.choice((64, 80, 128, 576))
        S = _log_uniform(rng, 40, 1500)
        pools = rng.choice((2, 9, 16))
        most = (1 << 30) // (W * G * S * D * pools * 4)
        return _reorder("", _log_uniform(rng, 1, max(1, min(16, most))), W, pools, G, S, D,
                        rng.choice(("bf16", "fp32")), page=page)
    if op == "extend":
        most = _log_uniform(rng, 1, 4096)
        return _extend("", _log_uniform(rng, 1, max(1, min(3000, (1 << 20) // most))), rng.choice((1, 8, 16, 64)),
                       rng.randint(4200, 6000) if most > 64 else rng.randint(100, 900), most)
    if op == "commit":
        return _commit("", _log_uniform(rng, 1, 3000), rng.choice((1, 8, 16, 64)), rng.randint(40, 700),
                       rng.randint(1, 30), rng.choice((0.0, 0.1)))
    N = rng.randint(2, 100)
    return _compact("", _log_uniform(rng, 1, 64), N, rng.randint(1, min(N, 12)), rng.choice((2, 16, 32)),
                    rng.choice((1, 4)), rng.choice((8, 16, 64)), rng.choice((64, 80, 256)), rng.randint(14, 20),
                    rng.choice(("bf16", "fp32")))


# ---------------------------------------------------------------------------
# Inputs.


def _tables(rng, lengths, blocks, page, pages):
    """Block tables [rows, blocks] that give every row the pages its length
    needs, in a random order from pages 1..pages-1 (page 0 belongs to nobody),
    -1 behind them; the free list and how many pages it holds."""
    dev = lengths.device
    order = torch.randperm(pages - 1, generator=rng, device=dev) + 1
    need = (lengths + page - 1) // page
    start = torch.cumsum(need, 0) - need
    j = torch.arange(blocks, device=dev)
    at = (start[:, None] + j[None, :]).clamp(max=pages - 2)
    table = torch.where(j[None, :] < need[:, None], order[at], -1).to(torch.int32).contiguous()
    used = need.sum()
    free = torch.roll(order, 0).to(torch.int32)
    # the free list's first entries are the pages nobody holds
    free = free[(torch.arange(pages - 1, device=dev) + used) % (pages - 1)]
    return table, torch.cat([free, free.new_zeros(1)]), (pages - 1 - used).to(torch.int32).reshape(1)


def _rand(rng, lo, hi, size):
    return torch.randint(lo, hi + 1, size, generator=rng, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    rng = torch.Generator(device="cuda").manual_seed(int(seed))
    c, B = case, case["B"]
    s = {"case": dict(case)}
    if c["op"] == "select":
        W, V, dt = c["W"], c["V"], DTYPES[c["dtype"]]
        # a heavy-tailed row: 3 N(0, 1) - 1.1 ln(rank), ranks drawn at random
        z = torch.rand((B, W, V + c["pad"]), generator=rng, device="cuda").mul_(V).floor_().add_(1).log_().mul_(-1.1)
        z += 3.0 * torch.randn(z.shape, generator=rng, device="cuda")
        if c["masked"]:
            z.masked_fill_(torch.rand(z.shape, generator=rng, device="cuda") < c["masked"], -math.inf)
        s["logits"] = z.to(dt)[:, :, :V]
        # cumulative log-probabilities of beams in competition
        s["scores"] = -20.0 - 2.0 * torch.rand((B, W), generator=rng, device="cuda")
        s["temperature"] = torch.full((B,), c["T"], device="cuda")
        s["finished"], s["eos"] = None, -1
        if c["finished"]:
            order = torch.rand((B, W), generator=rng, device="cuda").argsort(1)
            s["finished"], s["eos"] = (order < c["finished"]).to(torch.int32), 2
    elif c["op"] == "reorder":
        W, S, page = c["W"], c["S"], c["page"]
        s["parent"] = _rand(rng, 0, W - 1, (B, W))
        s["length"] = _rand(rng, 1, S, (B,))
        shape = (B * W, c["G"], S, c["D"])
        s["table"] = s["start"] = None
        if page:
            blocks = -(-S // page)
            # the prompt's part stays where it is
            s["start"] = (s["length"] * torch.rand((B,), generator=rng, device="cuda") * 0.5).to(torch.int32)
            s["table"] = _tables(rng, s["length"].repeat_interleave(W).long(), blocks, page, B * W * blocks + 1)[0]
            shape = (B * W * blocks + 1, c["G"], page, c["D"])
        s["pools"] = torch.randn((c["pools"], *shape), generator=rng, device="cuda", dtype=DTYPES[c["dtype"]])
    elif c["op"] in ("extend", "commit"):
        page, blocks, most = c["page"], c["blocks"], c["most_new"]
        new = _rand(rng, 0, most, (B,))
        s["seq_len"] = _rand(rng, 0, blocks * page - most, (B,))
        held = s["seq_len"] + (new if c["op"] == "commit" else 0)
        s["table"], s["free_list"], s["free_count"] = _tables(rng, held.long(), blocks, page, B * blocks + 2)
        s["free_out"] = torch.empty_like(s["free_count"])
        if c["op"] == "extend":
            s["new_len"] = new
        else:
            s["reserved"] = new
            s["accepted"] = (torch.rand((B,), generator=rng, device="cuda") * (new + 1)).to(torch.int32).minimum(new) - 1
            s["finished"] = (torch.rand((B,), generator=rng, device="cuda") < c["finished"]).to(torch.int32)
            s["len_out"] = torch.empty_like(s["seq_len"])
    else:
        page, blocks, N = c["page"], c["blocks"], c["N"]
        most = blocks * page - N - 1
        assert most >= 0
        s["seq_len"] = _rand(rng, 0, most, (B,))
        s["table"] = _tables(rng, (s["seq_len"] + N + 1).long(), blocks, page, B * blocks + 1)[0]
        s["accepted"] = _rand(rng, 0, c["depth"], (B,))
        order = torch.rand((B, N), generator=rng, device="cuda").argsort(1).to(torch.int32)
        i = torch.arange(N, device="cuda")[None, :]
        order = torch.where(i < s["accepted"][:, None], order, N).sort(1).values  # an ascending path
        s["path"] = torch.where(i < s["accepted"][:, None], order, -1).to(torch.int32).contiguous()
        s["pools"] = torch.randn((c["pools"], B * blocks + 1, c["G"], page, c["D"]), generator=rng, device="cuda",
                                 dtype=DTYPES[c["dtype"]])
    if own:
        s["call"] = _bind(s)
    return s


def _bind(s):
    """The operator with its buffers bound once, as a decode loop keeps it."""
    import draft_token_verification_03_amd as sv

    c = s["case"]
    if c["op"] == "select":
        return sv.BeamSelector(s["logits"], s["scores"], c["M"], temperature=s["temperature"],
                               finished=s["finished"], eos=s["eos"])
    if c["op"] == "reorder":
        return sv.BeamReorder(s["pools"], s["parent"], length=s["length"], block_table=s["table"], start=s["start"])
    if c["op"] == "extend":
        return sv.CacheExtend(s["seq_len"], s["table"], s["free_list"], s["free_count"], c["page"],
                              c["B"] * c["most_new"], new_len=s["new_len"], free_count_out=s["free_out"])
    if c["op"] == "commit":
        return sv.CacheCommit(s["seq_len"], s["reserved"], s["accepted"], s["table"], s["free_list"],
                              s["free_count"], c["page"], extra=1, finished=s["finished"],
                              seq_len_out=s["len_out"], free_count_out=s["free_out"])
    return sv.CacheCompact(s["pools"], s["table"], s["seq_len"], s["path"], s["accepted"])


# ---------------------------------------------------------------------------
# One pass.


def run(s):
    op = s["case"]["op"]
    if own:
        out = s["call"]()
        if op == "select":
            return list(out[:3])
        if op == "extend":
            return [*out[:5], s["table"], s["free_out"]]
        if op == "commit":
            return [s["len_out"], s["free_out"], s["free_list"]]
        return [s["pools"]]
    return {"select": _plain_select, "reorder": _plain_reorder, "extend": _plain_extend,
            "commit": _plain_commit, "compact": _plain_compact}[op](s)


def _plain_select(s):
    c = s["case"]
    B, W, V, M = c["B"], c["W"], c["V"], c["M"]
    z = s["logits"].float() + 0.0
    t = s["temperature"].double().view(B, 1, 1)
    top = z.amax(2, keepdim=True).double()
    top = torch.where(top == -math.inf, 0.0, top)
    # candidates of different beams lie close together: 64 bits for their order
    lse = top / t + ((z.double() - top) / t).exp().sum(2, keepdim=True).log()
    # the best of each beam, by (logit, lower token): distinct whole numbers
    bits = z.contiguous().view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7fffffff)).long() * 2**32 + (V - 1 - torch.arange(V, device=z.device))
    k = min(M, V)
    token = V - 1 - (key.topk(k, dim=2).values & 0xffffffff)
    best = z.gather(2, token).double()
    value = torch.where(best == -math.inf, -math.inf, s["scores"].double()[:, :, None] + best / t - lse)
    if s["finished"] is not None:
        done = s["finished"][:, :, None] != 0
        only = torch.where(torch.arange(k, device=z.device) == 0, s["scores"].double()[:, :, None], -math.inf)
        value = torch.where(done, only, value)
        token = torch.where(done, s["eos"], token)
    value, order = value.view(B, W * k).sort(dim=1, descending=True, stable=True)
    value, order = value[:, :M], order[:, :M]
    token = token.reshape(B, W * k).gather(1, order)
    some = value > -math.inf
    out = [value.float(), torch.where(some, order // k, -1).int(), torch.where(some, token, -1).int()]
    lack = M - W * k
    if lack > 0:
        out = [torch.nn.functional.pad(x, (0, lack), value=v) for x, v in zip(out, (-math.inf, -1, -1))]
    return out


def _plain_reorder(s):
    c = s["case"]
    B, W, S = c["B"], c["W"], c["S"]
    pools, dev = s["pools"], s["pools"].device
    parent = s["parent"].long()
    source = (torch.arange(B, device=dev)[:, None] * W + parent).view(-1)
    at = torch.arange(S, device=dev)
    if not c["page"]:
        keep = (at[None, :] < s["length"].repeat_interleave(W)[:, None]).view(1, B * W, 1, S, 1)
        pools.copy_(torch.where(keep, pools.index_select(1, source), pools))
        return [pools]
    page = c["page"]
    inside = (at[None, :] >= s["start"][:, None]) & (at[None, :] < s["length"][:, None])
    inside = inside.repeat_interleave(W, 0)
    table = s["table"].long()
    mine = torch.where(inside, table[:, at // page], 0)
    theirs = torch.where(inside, table[source][:, at // page], 0)
    off = (at % page).expand(B * W, S)
    pools[:, mine, :, off] = pools[:, theirs, :, off]
    return [pools]


def _plain_extend(s):
    c = s["case"]
    B, page, most = c["B"], c["page"], c["B"] * c["most_new"]
    dev = s["table"].device
    length, new = s["seq_len"].long(), s["new_len"].long()
    end = torch.cumsum(new, 0)
    query = torch.cat([end.new_zeros(1), end])
    first = (length + page - 1) // page
    need = (length + new + page - 1) // page - first
    before = torch.cumsum(need, 0) - need
    free = s["free_count"].long()
    fits = (need == 0) | (before + need <= free)
    j = torch.arange(s["table"].shape[1], device=dev)[None, :] - first[:, None]
    take = (j >= 0) & (j < need[:, None]) & fits[:, None]
    pick = (free - 1 - before[:, None] - j).clamp(0, s["free_list"].numel() - 1)
    s["table"].copy_(torch.where(take, s["free_list"][pick], s["table"]))
    s["free_out"].copy_(free - torch.where(fits, need, 0).sum())
    t = torch.arange(most, device=dev)
    b = torch.searchsorted(end, t, right=True)
    some = b < B
    b = b.clamp(max=B - 1)
    at = torch.where(some, length[b] + t - query[b], 0)
    slot = s["table"][b, at // page].long() * page + at % page
    return [torch.where(some & fits[b], slot, -1), at.int(), torch.where(some, b, -1).int(), query.int(),
            torch.where(fits, new, 0).int(), s["table"], s["free_out"]]


def _plain_commit(s):
    page = s["case"]["page"]
    table, free = s["table"], s["free_count"].long()
    length, held = s["seq_len"].long(), s["reserved"].long()
    keep = (s["accepted"].long() + 1).clamp(min=0).minimum(held)
    now = torch.where(s["finished"] != 0, 0, length + keep)
    first = (now + page - 1) // page
    count = (length + held + page - 1) // page - first
    before = torch.cumsum(count, 0) - count
    total = count.sum()
    j = torch.arange(table.shape[1], device=table.device)[None, :] - first[:, None]
    back = (j >= 0) & (j < count[:, None])
    # the page taken last comes back first; what is not given back goes behind the list
    end = s["free_list"].numel()
    to = torch.where(back, free + total - 1 - before[:, None] - j, end)
    longer = torch.cat([s["free_list"], s["free_list"].new_zeros(1)])
    longer.scatter_(0, to.view(-1), torch.where(back, table, 0).view(-1))
    s["free_list"].copy_(longer[:end])
    s["free_out"].copy_(free + total)
    s["len_out"].copy_(now)
    return [s["len_out"], s["free_out"], s["free_list"]]


def _plain_compact(s):
    c = s["case"]
    pools, page, N = s["pools"], c["page"], c["N"]
    i = torch.arange(N, device=pools.device)[None, :]
    moved = i < s["accepted"][:, None]
    base = s["seq_len"].long()[:, None] + 1
    to = torch.where(moved, base + i, 0)
    of = torch.where(moved, base + s["path"].long(), 0)
    table = s["table"].long()
    to_page = torch.where(moved, table.gather(1, to // page), 0)
    of_page = torch.where(moved, table.gather(1, of // page), 0)
    pools[:, to_page, :, to % page] = pools[:, of_page, :, of % page]
    return [pools]


# ---------------------------------------------------------------------------
# What a pass cannot do without.


def work(case):
    c, B = case, case["B"]
    elt = 4 if c.get("dtype") == "fp32" else 2
    if c["op"] == "select":
        read = B * (c["W"] - c["finished"]) * c["V"]
        # an exponent, an exponential and a sum for each logit
        return {"bytes": read * elt + B * c["W"] * 4 + B * c["M"] * 12, "flops": 3 * read}
    if c["op"] == "reorder":
        W = c["W"]
        # beams with another parent, and parents that some other beam has
        rows = W * (1 - 1 / W) + W * (1 - (1 - 1 / W) ** (W - 1))
        positions = (c["S"] + 1) / 2 * (0.75 if c["page"] else 1.0)
        return {"bytes": B * rows * positions * c["pools"] * c["G"] * c["D"] * elt + B * W * 4, "flops": 0}
    if c["op"] == "extend":
        pages = B * c["most_new"] / 2 / c["page"]
        return {"bytes": B * c["most_new"] * 16 + B * 16 + pages * 8, "flops": 0}
    if c["op"] == "commit":
        pages = B * (c["most_new"] / 2 / c["page"] + c["finished"] * c["blocks"] / 2)
        return {"bytes": B * 20 + pages * 8, "flops": 0}
    return {"bytes": B * c["depth"] / 2 * c["pools"] * c["G"] * c["D"] * elt * 2 + B * c["N"] * 4, "flops": 0}


# ---------------------------------------------------------------------------
# The same from the definitions, request by request.


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    c = case
    if c["op"] == "select":
        B, W, V, M = c["B"], c["W"], c["V"], c["M"]
        out = torch.full((B, M), -math.inf, dtype=torch.float64, device="cuda")
        parent = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
        token = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
        for b in range(B):
            z = s["logits"][b].double() / float(s["temperature"][b])
            lp = z - torch.logsumexp(z, dim=1, keepdim=True) + s["scores"][b].double()[:, None]
            if s["finished"] is not None:
                for w in torch.nonzero(s["finished"][b]).view(-1).tolist():
                    lp[w] = -math.inf
                    lp[w, s["eos"]] = s["scores"][b, w].double()
            v, i = lp.view(-1).sort(dim=0, descending=True, stable=True)
            n = min(M, int((v[:M] > -math.inf).sum()))
            out[b, :n], parent[b, :n], token[b, :n] = v[:n], (i[:n] // V).int(), (i[:n] % V).int()
        return [out, parent, token]
    if c["op"] == "reorder":
        W, old = c["W"], s["pools"].double()
        new = old.clone()
        length, parent = s["length"].tolist(), s["parent"].tolist()
        table = s["table"].tolist() if c["page"] else None
        for b in range(c["B"]):
            for j, p in enumerate(parent[b]):
                if not c["page"]:
                    new[:, b * W + j, :, :length[b]] = old[:, b * W + p, :, :length[b]]
                    continue
                at = int(s["start"][b])
                while at < length[b]:
                    k, lo = at // c["page"], at % c["page"]
                    hi = min(c["page"], lo + length[b] - at)
                    new[:, table[b * W + j][k], :, lo:hi] = old[:, table[b * W + p][k], :, lo:hi]
                    at += hi - lo
        return [new]
    if c["op"] == "compact":
        old = s["pools"].double()
        new = old.clone()
        table, path, lens, page = s["table"].tolist(), s["path"].tolist(), s["seq_len"].tolist(), c["page"]
        for b, d in enumerate(s["accepted"].tolist()):
            for i in range(d):
                to, of = lens[b] + 1 + i, lens[b] + 1 + path[b][i]
                new[:, table[b][to // page], :, to % page] = old[:, table[b][of // page], :, of % page]
        return [new]
    return None  # lengths, pages and slots are whole numbers
