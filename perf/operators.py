"""The operators over a paged latent cache, as they are measured.

Three operators of a server that keeps a multi-head latent attention cache (rows of 576 bf16
values: 512 latent + 64 rotary) in pages or slots on the GPU:

  attend  attention of a chunk of new tokens over the cache: each request's new rows sit at the
          end of its context and see, causally, every token, a sliding window with the first
          tokens kept visible, or the row's own selection (the sparse prefill's top-k);
  weigh   the attention weight every cached token receives from such a chunk, accumulated with a
          decay over the steps;
  evict   the victims of a cache that has to shrink: the lightest tokens of each request, the
          first and the most recent ones spared.

Where ``own`` is false the operators run in plain torch operations, else through
``sparse_attention_kv_echo_gb300``.
"""
import math

import torch

own = False

DQK, DV = 576, 512
SCALE = 1.0 / math.sqrt(192.0)
DECAY = 0.9375


def _attend(name, requests, length, rows, heads=128, page=64, window=0, sinks=0, k=0, absent=0, op="attend"):
    # length, rows: (first, last) over the requests, geometrically spaced; absent: percent of the
    # cached tokens that hold no row (page 1 only)
    return {"name": name, "op": op, "requests": requests, "len_a": length[0], "len_b": length[1], "rows_a": rows[0],
            "rows_b": rows[1], "heads": heads, "page": page, "window": window, "sinks": sinks, "k": k,
            "absent": absent}


def _evict(name, requests, slots, length, keep, sinks, recent):
    return {"name": name, "op": "evict", "requests": requests, "slots": slots, "length": length, "keep": keep,
            "sinks": sinks, "recent": recent}


def listed():
    return [
        # one user's single token: the latency of a call
        _attend("decode 1x1000", 1, (1000, 1000), (1, 1)),
        # a decode batch whose contexts differ by a factor of sixteen
        _attend("decode 32 ragged", 32, (1024, 16384), (1, 1)),
        # a prompt's chunk in the middle of its prefill
        _attend("chunk 2048 of 8192", 1, (8192, 8192), (2048, 2048)),
        # several prompts' chunks and draft tokens together, on a shard of the heads
        _attend("chunks 6 ragged, 16 heads", 6, (700, 9001), (3, 515), heads=16, page=16),
        # the sparse prefill: 1024 rows of a prompt, each over its own 2048 selected tokens in the cache's slots
        _attend("selected 1024 rows", 1, (32768, 32768), (1024, 1024), page=1, k=2048),
        # long conversations served with a window and the first tokens kept
        _attend("window decode 32", 32, (20000, 131072), (1, 1), window=4096, sinks=4),
        # a long prompt's chunk through the same window
        _attend("window chunk 2048", 1, (32768, 32768), (2048, 2048), window=1024, sinks=16),
        # the weights of a decode step over caches that have been evicted from
        _attend("weights decode 32", 32, (2048, 8192), (1, 1), page=1, absent=25, op="weigh"),
        # the weights of a prompt's chunk: what its eviction starts from
        _attend("weights chunk 1024", 1, (8192, 8192), (1024, 1024), op="weigh"),
        # a few requests make room for the next tokens
        _evict("evict 8x4096", 8, 4096, 32768, 3900, 4, 256),
        # a batch shrinks to half its slots
        _evict("evict 32x8192", 32, 8192, 131072, 4096, 4, 512),
        # one long prompt's cache of 260000 slots
        _evict("evict 1x260000", 1, 260000, 300001, 200000, 16, 2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "window", "selected", "weigh", "evict"))
    if op == "evict":
        requests = _log(rng, 1, 48)
        slots = 32 * _log(rng, 4, 8192 if requests == 1 else max(8, 8192 // requests))
        length = _log(rng, slots, 4 * slots)
        return {"op": "evict", "requests": requests, "slots": slots, "length": length,
                "keep": rng.randint(0, slots * 9 // 10), "sinks": rng.choice((0, 1, 4, 33)), "recent": rng.choice((0, 1, 100))}
    heads = rng.choice((128, 128, 64, 40, 16, 1))
    page = rng.choice((1, 16, 48, 64, 256))
    c = {"op": "weigh" if op == "weigh" else "attend", "requests": _log(rng, 1, 40), "rows_a": 1, "rows_b": 1,
         "heads": heads, "page": page, "window": 0, "sinks": 0, "k": 0, "absent": 0}
    c["len_a"], c["len_b"] = _log(rng, 1, 20000), _log(rng, 64, 20000)
    if rng.random() < 0.5:
        c["requests"] = rng.randint(1, 4)
        c["rows_a"], c["rows_b"] = _log(rng, 1, 600), _log(rng, 1, 600)
    if op == "window":
        c["window"], c["sinks"] = _log(rng, 1, 8192), rng.choice((0, 1, 4, 17, 128))
    if op == "selected":
        c["requests"], c["page"], c["k"], c["rows_a"], c["rows_b"] = 1, 1, _log(rng, 16, 2048), 1, _log(rng, 1, 600)
        c["rows_a"] = c["rows_b"]
    if page == 1 and rng.random() < 0.5:
        c["absent"] = rng.randint(1, 60)
    return c


def _spaced(a, b, n):
    return [int(round(a * (b / a) ** (i / max(n - 1, 1)))) for i in range(n)]


def _lengths(case):
    lens = _spaced(case["len_a"], case["len_b"], case["requests"])
    rows = [min(r, n) for r, n in zip(_spaced(case["rows_b"], case["rows_a"], case["requests"]), lens)]
    return lens, rows


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "evict":
        return _prepare_evict(case, g, dev)
    lens, rows = _lengths(case)
    H, page, B = case["heads"], case["page"], case["requests"]
    room = [n + 7 for n in lens]                       # contexts grow inside their regions
    tok_off = torch.tensor([0] + room, dtype=torch.int64).cumsum(0)
    n_tokens = int(tok_off[-1])
    row_off = torch.tensor([0] + rows, dtype=torch.int64).cumsum(0)
    n_rows, n_pages = int(row_off[-1]), -(-n_tokens // page)
    kv = torch.randn(((n_pages + 3) * page, DQK), generator=g, device=dev).to(torch.bfloat16)
    tab = torch.randperm(n_pages + 3, generator=g, device=dev)[:n_pages].to(torch.int32)
    if case["absent"]:
        tab[torch.rand(n_pages, generator=g, device=dev) < case["absent"] / 100.0] = -1
    st = {"case": case, "lens": lens, "rows": rows, "n_tokens": n_tokens, "n_rows": n_rows,
          "row_off": row_off.to(dev), "tok_off": tok_off.to(dev), "page_tab": tab, "kv": kv,
          "tok_end": (tok_off[:-1] + torch.tensor(lens)).to(dev),
          "q": torch.randn((n_rows, H, DQK), generator=g, device=dev).to(torch.bfloat16),
          "sel": None, "status": torch.zeros(1, dtype=torch.int32, device=dev)}
    if case["k"]:
        st["sel"] = _selection(case, st, g, dev)
    if case["op"] == "weigh":
        st["lse"] = _plain_attend(st)[1]
        st["mass"] = torch.rand(n_tokens, generator=g, device=dev)
        st["mass_out"] = st["mass"].clone()
    else:
        st["out"] = torch.empty((n_rows, H, DV), dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.empty((n_rows, H), dtype=torch.float32, device=dev)
    return st


def _selection(case, st, g, dev):
    # k different tokens of each row's causal prefix, ascending, -1 behind them (all of a shorter prefix)
    R, n, k = st["n_rows"], st["lens"][0], case["k"]
    pos = n - R + torch.arange(R, device=dev)
    step = (pos + 1).double() / k
    at = (torch.arange(k, device=dev) + torch.rand((R, k), generator=g, device=dev)).double() * step[:, None]
    sel = torch.minimum(at.long(), pos[:, None])
    short = pos[:, None] < k                          # the whole prefix, then padding
    every = torch.arange(k, device=dev)[None, :].expand(R, k)
    sel = torch.where(short, torch.where(every <= pos[:, None], every, -1), sel)
    return sel.to(torch.int32).contiguous()


def _prepare_evict(case, g, dev):
    B, C, n = case["requests"], case["slots"], case["length"]
    tok_off = torch.arange(B + 1, dtype=torch.int64, device=dev) * (n + 5)
    # every request holds a random set of its tokens, in slots of no particular order; some slots are free
    order = torch.rand((B, n), generator=g, device=dev).argsort(1)[:, :C].to(torch.int32)
    if C > 64:
        order[:, ::37] = -1
    u = torch.rand(B * (n + 5), generator=g, device=dev)
    mass = (-torch.log(u.clamp_min(1e-7))) ** 3
    mass = torch.where(u > 0.9, torch.zeros_like(u), mass)         # never attended: ties at zero
    mass = torch.where(u < 0.2, (mass * 4).round() / 4, mass)      # more ties
    return {"case": case, "n_tokens": B * (n + 5), "tok_off": tok_off, "tok_end": tok_off[:-1] + n,
            "slot2tok": order.contiguous(), "mass": mass,
            "evict_tok": torch.empty((B, C), dtype=torch.int32, device=dev),
            "evict_slot": torch.empty((B, C), dtype=torch.int32, device=dev),
            "evict_cnt": torch.empty(B, dtype=torch.int32, device=dev),
            "status": torch.zeros(1, dtype=torch.int32, device=dev)}


# ---------------------------------------------------------------- the plain forms
def _keys(st):
    """The tokens any row of a request may see: token ids [B, V], their cache rows, which exist."""
    case, dev = st["case"], st["q"].device
    lens, n = torch.tensor(st["lens"], device=dev), torch.tensor(st["rows"], device=dev)
    first = lens - n
    lo = (first - case["window"] + 1).clamp_min(0) if case["window"] else torch.zeros_like(first)
    kept = lo.clamp_max(case["sinks"])
    host = [(min(case["sinks"], max(l - r - case["window"] + 1, 0)) if case["window"] else 0)
            + l - (max(l - r - case["window"] + 1, 0) if case["window"] else 0) for l, r in zip(st["lens"], st["rows"])]
    v = torch.arange(max(host), device=dev)[None, :]
    tok = torch.where(v < kept[:, None], v, v - kept[:, None] + lo[:, None])
    ok = tok < lens[:, None]
    at = (st["tok_off"][:-1, None] + tok).clamp_max(st["n_tokens"] - 1)
    pg = st["page_tab"].long()[at // case["page"]]
    ok = ok & (pg >= 0)
    return tok, at, pg.clamp_min(0) * case["page"] + at % case["page"], ok, first


def _visible(st, tok, ok, first, N):
    case = st["case"]
    pos = first[:, None] + torch.arange(N, device=tok.device)[None, :]
    t, p = tok[:, None, :], pos[:, :, None]
    vis = ok[:, None, :] & (t <= p)
    if case["window"]:
        vis = vis & ((t > p - case["window"]) | (t < case["sinks"]))
    return vis                                         # [B, N, V]


def _rows_of(st):
    """(request, row within it) of every row, and the rows padded to [B, N]."""
    dev = st["q"].device
    n = torch.tensor(st["rows"], device=dev)
    req = torch.repeat_interleave(torch.arange(len(st["rows"]), device=dev), n, output_size=st["n_rows"])
    i = torch.arange(st["n_rows"], device=dev) - st["row_off"][:-1][req]
    N = max(st["rows"])
    pad = (st["row_off"][:-1, None] + torch.arange(N, device=dev)[None, :]).clamp_max(st["n_rows"] - 1)
    return req, i, N, pad


def _plain_attend(st):
    H = st["case"]["heads"]
    if st["sel"] is not None:
        return _plain_selected(st)
    tok, _, row, ok, first = _keys(st)
    req, i, N, pad = _rows_of(st)
    B, V = tok.shape
    kf = st["kv"][row].float()
    s = torch.bmm(st["q"][pad].float().view(B, N * H, DQK), kf.transpose(1, 2)).mul_(SCALE).view(B, N, H, V)
    s.masked_fill_(~_visible(st, tok, ok, first, N)[:, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m.clamp_min(-3e38)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(B, N * H, V), kf[:, :, :DV]).view(B, N, H, DV) / l.clamp_min(1e-38)
    lse = (m + l.log()).squeeze(-1)
    return o[req, i].to(torch.bfloat16), lse[req, i]


def _plain_selected(st):
    sel, case = st["sel"].long(), st["case"]
    at = st["tok_off"][0] + sel.clamp_min(0)
    pg = st["page_tab"].long()[at // case["page"]]
    ok = (sel >= 0) & (pg >= 0)
    kf = st["kv"][pg.clamp_min(0) * case["page"] + at % case["page"]].float()
    s = torch.bmm(st["q"].float(), kf.transpose(1, 2)).mul_(SCALE)
    s.masked_fill_(~ok[:, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m.clamp_min(-3e38)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.bmm(p, kf[:, :, :DV]) / l.clamp_min(1e-38)
    return o.to(torch.bfloat16), (m + l.log()).squeeze(-1)


def _plain_weigh(st):
    H = st["case"]["heads"]
    tok, at, row, ok, first = _keys(st)
    req, i, N, pad = _rows_of(st)
    B, V = tok.shape
    s = torch.bmm(st["q"][pad].float().view(B, N * H, DQK), st["kv"][row].float().transpose(1, 2)).mul_(SCALE)
    inside = torch.arange(N, device=tok.device)[None, :] < torch.tensor(st["rows"], device=tok.device)[:, None]
    vis = _visible(st, tok, ok, first, N) & inside[:, :, None]
    w = s.view(B, N, H, V).sub_(st["lse"][pad].clamp_min(-3e38)[..., None]).exp_()
    w.masked_fill_(~vis[:, :, None, :], 0.0)
    got = w.sum((1, 2))                                # [B, V]
    t = torch.arange(st["n_tokens"], device=tok.device)
    owner = torch.searchsorted(st["tok_off"][1:], t, right=True)
    new = torch.where(t < st["tok_end"][owner], st["mass"] * DECAY, st["mass_out"])
    return new.index_add(0, at[ok], got[ok])


def _plain_evict(st):
    case = st["case"]
    s2t = st["slot2tok"].long()
    held = s2t >= 0
    mass = st["mass"][st["tok_off"][:-1, None] + s2t.clamp_min(0)] + 0.0
    bits = mass.view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    n = case["length"]
    may = held & (s2t >= case["sinks"]) & (s2t < n - case["recent"])
    want = torch.minimum(held.sum(1) - case["keep"], may.sum(1)).clamp_min(0)
    key = torch.where(may, (key << 31) + s2t, torch.full_like(key, 2 ** 63 - 1))
    rank = key.argsort(dim=1, stable=True).argsort(dim=1, stable=True)
    out = rank < want[:, None]
    place = torch.where(out, out.long().cumsum(1) - 1, s2t.shape[1])
    slot = torch.arange(s2t.shape[1], device=s2t.device)[None, :].expand_as(s2t)
    pad = torch.full((s2t.shape[0], s2t.shape[1] + 1), -1, dtype=torch.long, device=s2t.device)
    tok = pad.scatter(1, place, s2t)[:, :-1]
    slot = pad.scatter(1, place, slot)[:, :-1]
    return tok.to(torch.int32), slot.to(torch.int32), want.to(torch.int32)


# ---------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    if not own:
        return {"attend": _plain_attend, "weigh": _plain_weigh, "evict": _plain_evict}[case["op"]](st)
    from sparse_attention_kv_echo_gb300 import lib as L
    if case["op"] == "evict":
        L.evict_select(st["tok_off"], st["n_tokens"], st["slot2tok"], st["mass"], case["keep"], st["evict_tok"],
                       st["evict_slot"], st["evict_cnt"], st["status"], sinks=case["sinks"], recent=case["recent"],
                       tok_end=st["tok_end"])
        return st["evict_tok"], st["evict_slot"], st["evict_cnt"]
    if "pages" not in st:                              # what a server keeps for its cache and its stream
        st["pages"] = L.KVPages(st["page_tab"], st["kv"], case["page"])
        st["ws"] = torch.empty(L.mla_chunk_workspace_size(st["n_rows"], case["heads"], case["requests"]),
                               dtype=torch.uint8, device=st["q"].device)
    if case["op"] == "attend":
        L.mla_chunk(st["row_off"], st["q"], st["tok_off"], st["n_tokens"], st["pages"], SCALE, st["out"], st["lse"],
                    st["ws"], st["status"], tok_end=st["tok_end"], window=case["window"], sinks=case["sinks"],
                    sel=st["sel"])
        return st["out"], st["lse"]
    L.mla_mass(st["row_off"], st["q"], st["lse"], st["tok_off"], st["n_tokens"], st["pages"], SCALE, st["mass"],
               st["mass_out"], st["status"], decay=DECAY, tok_end=st["tok_end"], window=case["window"],
               sinks=case["sinks"])
    return st["mass_out"]


# ---------------------------------------------------------------- what a pass cannot do without
def _pairs(case):
    """(row, token) pairs that are seen, and the tokens any row sees."""
    lens, rows = _lengths(case)
    pairs = seen = 0
    for n, r in zip(lens, rows):
        w = case["window"]
        for p in range(n - r, n):
            if case["k"]:
                pairs += min(p + 1, case["k"])
            elif w:
                lo = max(p - w + 1, 0)
                pairs += p + 1 - lo + min(case["sinks"], lo)
            else:
                pairs += p + 1
        lo = max(n - r - w + 1, 0) if w else 0
        seen += n - lo + min(case["sinks"], lo)
        if case["k"]:
            seen = min(n, r * case["k"])
    there = 1.0 - case["absent"] / 100.0
    return pairs * there, seen * there, sum(rows), sum(lens)


def work(case):
    if case["op"] == "evict":
        n = case["requests"] * case["slots"]
        return {"bytes": n * (4 + 4 + 8), "flops": n}
    pairs, seen, rows, total = _pairs(case)
    H = case["heads"]
    if case["op"] == "attend":
        extra = rows * case["k"] * 4
        return {"bytes": seen * DQK * 2 + rows * H * (DQK * 2 + DV * 2 + 4) + extra,
                "flops": 2.0 * pairs * H * (DQK + DV)}
    return {"bytes": seen * DQK * 2 + rows * H * (DQK * 2 + 4) + 8 * total, "flops": 2.0 * pairs * H * DQK}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "evict":
        return None                                    # whole numbers: the plain form's are exact
    st = prepare(case, seed)
    H, page, dev = case["heads"], case["page"], st["q"].device
    n_rows = st["n_rows"]
    out = torch.zeros((n_rows, H, DV), dtype=torch.float64, device=dev)
    lse = torch.full((n_rows, H), -math.inf, dtype=torch.float64, device=dev)
    mass = None
    if case["op"] == "weigh":
        mass = st["mass_out"].double()
    r0 = 0
    for b, (n, r) in enumerate(zip(st["lens"], st["rows"])):
        off = int(st["tok_off"][b])
        g = off + torch.arange(n, device=dev)
        phys = st["page_tab"][torch.div(g, page, rounding_mode="floor")].long()
        there = phys >= 0
        cache_row = torch.where(there, phys, 0) * page + torch.remainder(g, page)
        if mass is not None:
            mass[off:off + n] = st["mass"][off:off + n].double() * DECAY
        block = max(1, min(r, int(2e9 / (8.0 * H * n)))) if not case["k"] else 8
        for i0 in range(0, r, block):
            i1 = min(r, i0 + block)
            p = torch.arange(n - r + i0, n - r + i1, device=dev)
            qd = st["q"][r0 + i0:r0 + i1].double()
            if case["k"]:
                pick = st["sel"][i0:i1].long()
                use = (pick >= 0) & there[pick.clamp_min(0)]
                kd = st["kv"][cache_row[pick.clamp_min(0)]].double()
                s = SCALE * torch.matmul(qd, kd.mT)
                s = torch.where(use[:, None, :], s, -math.inf)
                lse[r0 + i0:r0 + i1] = torch.logsumexp(s, -1)
                out[r0 + i0:r0 + i1] = torch.matmul(torch.exp(s - lse[r0 + i0:r0 + i1, :, None]).nan_to_num(0.0),
                                                    kd[..., :DV])
                continue
            a, z = 0, int(p[-1]) + 1
            if case["window"] and case["sinks"] == 0:
                a = max(0, int(p[0]) - case["window"] + 1)
            t = torch.arange(a, z, device=dev)
            if case["window"] and case["sinks"]:
                t = t[(t < case["sinks"]) | (t > int(p[0]) - case["window"])]
            see = (t[None, :] <= p[:, None]) & there[t][None, :]
            if case["window"]:
                see &= (t[None, :] < case["sinks"]) | (p[:, None] - t[None, :] < case["window"])
            kd = st["kv"][cache_row[t]].double()
            s = SCALE * (qd.reshape(-1, DQK) @ kd.T).reshape(i1 - i0, H, -1)
            s = torch.where(see[:, None, :], s, -math.inf)
            if mass is not None:
                w = torch.exp(s - st["lse"][r0 + i0:r0 + i1].double()[:, :, None]).nan_to_num(0.0)
                mass[off + t] += w.sum((0, 1))
            else:
                lse[r0 + i0:r0 + i1] = torch.logsumexp(s, -1)
                w = torch.exp(s - lse[r0 + i0:r0 + i1, :, None]).nan_to_num(0.0)
                out[r0 + i0:r0 + i1] = (w.reshape(-1, t.numel()) @ kd[:, :DV]).reshape(i1 - i0, H, DV)
        r0 += r
    return mass if mass is not None else (out, lse)
