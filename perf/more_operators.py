"""The operators of speculative decoding over a paged latent cache, as they are measured.

A server drafts a tree of tokens per request (node 0: the last token it committed, the others: drafts,
each under its parent), runs the model over the trees, keeps the path that the target accepts and goes on:

  tree    attention of the trees' nodes over the cache: each node sees the whole context before its
          tree, itself and its ancestors (rows of 576 bf16 values: 512 latent + 64 rotary);
  verify  the walk down each tree: a draft is accepted with min(1, p / q) against the target's
          probabilities, siblings against what the rejections left of them, and the token behind the
          path is drawn from that residual, all from given uniform numbers; or greedily;
  pages   the cache's pages meanwhile: the accepted path's rows moved together ("keep"), a prompt's
          pages shared by its samples ("fork"), and a pool closed up while requests leave and come ("turn").

Where ``own`` is false the operators run in plain torch operations, else through
``sparse_attention_kv_echo_gb300``.
"""
import math
import random

import torch

own = False

DQK, DV = 576, 512
SCALE = 1.0 / math.sqrt(192.0)


def _tree(name, requests, length, nodes, heads=128, page=64, reach=4):
    # length, nodes: (first, last) over the requests, geometrically spaced; a node's parent is one of
    # the `reach` nodes before it (1: a chain)
    return {"name": name, "op": "tree", "requests": requests, "len_a": length[0], "len_b": length[1],
            "nodes_a": nodes[0], "nodes_b": nodes[1], "heads": heads, "page": page, "reach": reach}


def _verify(name, requests, nodes, vocab, half=False, mode="sample", reach=1):
    # mode "sample": drafts drawn from the draft model's probabilities; "certain": drafts without
    # probabilities (looked up, or the draft's best); "greedy": the target's best token only
    return {"name": name, "op": "verify", "requests": requests, "nodes_a": nodes[0], "nodes_b": nodes[1],
            "vocab": vocab, "half": half, "mode": mode, "reach": reach}


def _pages(name, kind, requests, length, nodes=0, page=64, layers=4, copies=0):
    return {"name": name, "op": "pages", "kind": kind, "requests": requests, "len_a": length[0], "len_b": length[1],
            "nodes": nodes, "page": page, "layers": layers, "copies": copies}


def listed():
    return [
        # one user's small tree: the latency of a call
        _tree("tree 1x8 of 1000", 1, (1000, 1000), (8, 8)),
        # a batch whose contexts differ by a factor of sixteen
        _tree("trees 16 ragged", 16, (2048, 32768), (12, 48)),
        # one user's long context under a large tree
        _tree("tree 1x64 of 131072", 1, (131072, 131072), (64, 64)),
        # many short chats on a shard of the heads, chains of three drafts
        _tree("chains 48, 16 heads", 48, (100, 4001), (4, 4), heads=16, page=16, reach=1),
        # one user's chain of four drafts: the latency of a call
        _verify("verify chain 1x5", 1, (5, 5), 32000),
        # a batch of chains over a large vocabulary
        _verify("verify chains 64x6", 64, (6, 6), 131072),
        # trees with many siblings, probabilities in 16 bits
        _verify("verify trees 32x48", 32, (32, 48), 131072, half=True, reach=8),
        # greedy decoding of trees, a vocabulary of odd size
        _verify("verify greedy 16x24", 16, (8, 24), 50001, half=True, mode="greedy", reach=4),
        # one user's accepted path, one layer: the latency of the three calls behind a verification
        _pages("keep 1x8", "keep", 1, (1000, 1000), nodes=8, layers=1),
        # a batch's accepted paths through several layers' caches
        _pages("keep 64x16", "keep", 64, (512, 6000), nodes=16, layers=8),
        # four prompts, sixteen samples of each
        _pages("fork 4 to 64", "fork", 4, (3001, 8000), copies=16),
        # half of a pool's requests leave, the others move together, as many come
        _pages("turn 48", "turn", 48, (4096, 4096), page=64, layers=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tree", "verify", "pages"))
    if op == "tree":
        while True:
            c = _tree(None, _log(rng, 1, 48), (_log(rng, 64, 32768), _log(rng, 64, 131072)),
                      (_log(rng, 1, 64), _log(rng, 1, 64)), rng.choice((128, 128, 64, 40, 16)), rng.choice((1, 16, 48, 64, 256)),
                      rng.choice((1, 2, 4, 16)))
            lens, nodes = _spread(c["len_a"], c["len_b"], c["requests"]), _spread(c["nodes_a"], c["nodes_b"], c["requests"])
            # the plain form pads to the longest request and the largest tree
            if c["heads"] * max(nodes) * max(n + m for n, m in zip(lens, nodes)) * c["requests"] <= 128 * 64 * 131072:
                break
    elif op == "verify":
        while True:
            c = _verify(None, _log(rng, 1, 64), (_log(rng, 1, 48), _log(rng, 1, 48)), _log(rng, 1000, 131072),
                        rng.random() < 0.5, rng.choice(("sample", "sample", "certain", "greedy")), rng.choice((1, 2, 8)))
            if max(c["nodes_a"], c["nodes_b"]) * c["requests"] * c["vocab"] <= 48 * 32 * 131072:
                break
    else:
        kind = rng.choice(("keep", "fork", "turn"))
        page = rng.choice((16, 48, 64, 128))
        while True:
            if kind == "keep":
                n = _log(rng, 1, 64)
                c = _pages(None, kind, _log(rng, 1, 64), (_log(rng, n + 1, 6000), _log(rng, n + 1, 6000)), n, page, rng.randint(1, 8))
            elif kind == "fork":
                c = _pages(None, kind, _log(rng, 1, 8), (_log(rng, 1, 8000), _log(rng, 1, 8000)), 0, page, rng.randint(1, 6),
                           _log(rng, 1, 16))
            else:
                n = _log(rng, 100, 8192)
                c = _pages(None, kind, 2 * _log(rng, 1, 32), (n, n), 0, page, rng.randint(1, 6))
            if _pool_rows(c) * c["layers"] <= 48 * 4200 * 4:
                break
    del c["name"]
    return c


def _spread(a, b, n):
    return [int(round(a * (b / a) ** (i / max(n - 1, 1)))) for i in range(n)]


def _offsets(counts, dev):
    return torch.tensor([0] + list(counts), dtype=torch.int64).cumsum(0).to(dev)


def _parents(sizes, reach, rng):
    # the root of each tree is its node 0
    return [-1 if i == 0 else rng.randrange(max(0, i - reach), i) for n in sizes for i in range(n)]


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rng = random.Random(seed)
    return {"tree": _prepare_tree, "verify": _prepare_verify, "pages": _prepare_pages}[case["op"]](case, g, rng, dev)


def _prepare_tree(case, g, rng, dev):
    B, H, page = case["requests"], case["heads"], case["page"]
    nodes = _spread(case["nodes_a"], case["nodes_b"], B)
    lens = [n + m for n, m in zip(_spread(case["len_a"], case["len_b"], B), nodes)]  # the trees' rows are cached too
    region = [-(-(n + 7) // page) * page for n in lens]
    tok_off = _offsets(region, dev)
    n_tokens = sum(region)
    pages = n_tokens // page
    tab = torch.randperm(pages + 3, generator=g, device=dev)[:pages].to(torch.int32)
    kv = torch.randn(((pages + 3) * page, DQK), generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)
    n_rows, words = sum(nodes), -(-max(nodes) // 32)
    i32 = dict(dtype=torch.int32, device=dev)
    return {"case": case, "lens": lens, "nodes": nodes, "n_rows": n_rows, "n_tokens": n_tokens, "words": words,
            "tok_off": tok_off, "tok_end": tok_off[:-1] + torch.tensor(lens, device=dev), "row_off": _offsets(nodes, dev),
            "parent": torch.tensor(_parents(nodes, case["reach"], rng), **i32), "page_tab": tab, "kv": kv,
            "q": (1.5 * torch.randn((n_rows, H, DQK), generator=g, device=dev)).to(torch.bfloat16),
            "mask": torch.zeros((n_rows, words), **i32), "depth": torch.zeros(n_rows, **i32),
            "out": torch.empty((n_rows, H, DV), dtype=torch.bfloat16, device=dev),
            "lse": torch.empty((n_rows, H), dtype=torch.float32, device=dev), "status": torch.zeros(1, **i32)}


def _prepare_verify(case, g, rng, dev):
    B, V = case["requests"], case["vocab"]
    nodes = _spread(case["nodes_a"], case["nodes_b"], B)
    n = sum(nodes)
    dtype = torch.bfloat16 if case["half"] else torch.float32
    parents = _parents(nodes, case["reach"], rng)
    i32 = dict(dtype=torch.int32, device=dev)
    row_off = _offsets(nodes, dev)
    parent = torch.tensor(parents, **i32)
    owner = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(nodes, device=dev), output_size=n)
    above = (row_off[owner] + parent.clamp_min(0)).long()
    target = torch.empty((n, V), dtype=dtype, device=dev)
    draft = torch.empty((n, V), dtype=dtype, device=dev) if case["mode"] == "sample" else None
    token = torch.empty(n, dtype=torch.int64, device=dev)
    # the draft model's logits are the target's, disturbed; a child is drawn from its parent's row
    rows = torch.empty((n, V), dtype=dtype, device=dev)
    step = max(1, (1 << 28) // V)
    for i in range(0, n, step):
        t = 3.0 * torch.randn((min(step, n - i), V), generator=g, device=dev)
        d = t + 0.8 * torch.randn(t.shape, generator=g, device=dev)
        target[i:i + step] = t if case["mode"] == "greedy" else torch.softmax(t, -1)
        rows[i:i + step] = torch.softmax(d, -1)
    for i in range(0, n, step):
        if case["mode"] == "sample":
            u = torch.rand((min(step, n - i), V), generator=g, device=dev).clamp_min_(1e-20)
            token[i:i + step] = (rows[above[i:i + step]].float() / -u.log()).argmax(-1)
        else:  # the draft's best, or one of its next
            token[i:i + step] = rows[above[i:i + step]].float().topk(min(4, V), -1)[1].gather(
                1, torch.randint(0, min(4, V), (min(step, n - i), 1), generator=g, device=dev) *
                (torch.rand((min(step, n - i), 1), generator=g, device=dev) < 0.4))[:, 0]
    if draft is not None:
        draft = rows
    some = case["mode"] != "greedy"
    return {"case": case, "n_rows": n, "N": max(nodes), "row_off": row_off, "parent": parent, "token": token.to(torch.int32),
            "target": target, "draft": draft,
            "u_node": torch.rand(n, generator=g, device=dev) if some else None,
            "u_pick": torch.rand(B, generator=g, device=dev) if some else None,
            "path": torch.empty(n, **i32), "count": torch.empty(B, **i32), "next": torch.empty(B, **i32),
            "status": torch.zeros(1, **i32)}


def _region(case):
    """Tokens of a request's region: whole pages, room for what it grows to."""
    page, most = case["page"], max(case["len_a"], case["len_b"])
    return -(-(most + 2 * case["nodes"]) // page) * page


def _pool_rows(case):
    B = case["requests"]
    per = case["copies"] + 1 if case["kind"] == "fork" else 1
    return B * per * _region(case)


def _prepare_pages(case, g, rng, dev):
    B, page, layers, kind = case["requests"], case["page"], case["layers"], case["kind"]
    region = _region(case)
    E = region // page                                              # table entries per request
    lens = _spread(case["len_a"], case["len_b"], B)
    i32 = dict(dtype=torch.int32, device=dev)
    all_ = B * (1 + case["copies"]) if kind == "fork" else B       # the prompts, then their samples
    tok_off = torch.arange(all_ + 1, dtype=torch.int64, device=dev) * region
    held = torch.tensor([-(-n // page) for n in lens], device=dev)  # pages in use
    e = torch.arange(E, device=dev)[None, :]
    used = e < held[:, None]
    n_pages = all_ * E + 5
    if kind == "turn":  # the even requests hold the lower half of what is used
        order = torch.arange(n_pages, device=dev)
        rank = torch.cat((torch.arange(0, B, 2), torch.arange(1, B, 2))).argsort().to(dev)
        tab = torch.where(used, rank[:, None] * int(held[0]) + e, -1)
    else:
        order = torch.randperm(n_pages, generator=g, device=dev)
        tab = torch.where(used, order[:B * E].view(B, E), -1)
    if kind == "fork":
        tab = torch.cat((tab, torch.full(((all_ - B), E), -1, device=dev)))
    tab = tab.to(torch.int32).reshape(-1).contiguous()
    refs = torch.zeros(n_pages, **i32)
    refs[tab[tab >= 0].long()] = 1
    kv = torch.empty((layers, n_pages * page, DQK), dtype=torch.bfloat16, device=dev)
    for l in range(layers):
        kv[l] = torch.randn(kv.shape[1:], generator=g, device=dev)
    n = torch.tensor(lens, device=dev)
    st = {"case": case, "B": all_, "E": E, "n_tokens": all_ * region, "n_pages": n_pages, "tok_off": tok_off,
          "page_tab": tab, "refs": refs, "kv": kv, "status": torch.zeros(1, **i32)}
    if kind == "keep":  # the trees are the last rows of their requests; about half of their nodes' depth is accepted
        N = case["nodes"]
        path, count = [], []
        for b in range(B):
            c = rng.randint(1, max(1, N // 2))
            at = [0] + sorted(rng.sample(range(1, N), c - 1)) if N > 1 else [0]
            count.append(len(at))
            path += at + [-1] * (N - len(at))
        st |= {"tok_end": tok_off[:-1] + n, "row_off": torch.arange(B + 1, device=dev) * N, "path": torch.tensor(path, **i32),
               "count": torch.tensor(count, **i32), "new_end": torch.empty(B, dtype=torch.int64, device=dev),
               "nodes": torch.full((B,), N, dtype=torch.int64, device=dev), "room": torch.empty(B, dtype=torch.int64, device=dev)}
    elif kind == "fork":
        k = case["copies"]
        st |= {"tok_end": tok_off[:-1] + torch.cat((n, torch.zeros(all_ - B, dtype=torch.int64, device=dev))),
               "src": torch.arange(B, device=dev).repeat_interleave(k).to(torch.int32),
               "dst": torch.arange(B, all_, device=dev).to(torch.int32)}
    else:
        full = tok_off[:-1] + n
        odd = torch.arange(B, device=dev) % 2 == 1
        st |= {"left": (torch.where(odd, full, tok_off[:-1]), torch.where(odd, tok_off[:-1], full)), "want": full, "turn": 0,
               "room": torch.empty(B, dtype=torch.int64, device=dev), "used": torch.empty(1, **i32)}
    return st


# ---------------------------------------------------------------- the plain forms
def _padded(row_off, N, n_rows):
    """Rows of every request padded to [B, N], and which of them there are."""
    i = torch.arange(N, device=row_off.device)[None, :]
    ok = i < (row_off[1:] - row_off[:-1])[:, None]
    return (row_off[:-1, None] + i).clamp_max(n_rows - 1), ok


def _ancestors(parent, pad, ok):
    """[B, N, N]: node j is i or an ancestor of i."""
    B, N = pad.shape
    up = parent[pad].long()
    j = torch.arange(N, device=pad.device)
    a = ((up[:, :, None] == j) | (j[:, None] == j[None, :])).float()
    for _ in range(max(N - 1, 1).bit_length()):
        a = (torch.bmm(a, a) > 0).float()
    return (a > 0) & ok[:, :, None] & ok[:, None, :]


def _plain_tree(st):
    case, dev = st["case"], st["q"].device
    H, page, N, words = case["heads"], case["page"], max(st["nodes"]), st["words"]
    pad, ok = _padded(st["row_off"], N, st["n_rows"])
    up = _ancestors(st["parent"], pad, ok)
    bit = torch.arange(words * 32, device=dev)
    bits = torch.zeros(up.shape[:2] + (words * 32,), dtype=torch.int64, device=dev)
    bits[..., :N] = up
    mask = (bits << (bit % 32)).view(up.shape[0], N, words, 32).sum(-1)
    mask = torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).to(torch.int32)
    req = torch.repeat_interleave(torch.arange(pad.shape[0], device=dev), st["row_off"][1:] - st["row_off"][:-1],
                                  output_size=st["n_rows"])
    i = torch.arange(st["n_rows"], device=dev) - st["row_off"][:-1][req]
    L = max(st["lens"])
    t = torch.arange(L, device=dev)[None, :]
    n = (st["tok_end"] - st["tok_off"][:-1])[:, None]
    first = n - (st["row_off"][1:] - st["row_off"][:-1])[:, None]   # where the tree starts
    at = (st["tok_off"][:-1, None] + t).clamp_max(st["n_tokens"] - 1)
    kf = st["kv"][st["page_tab"].long()[at // page] * page + at % page].float()
    s = torch.bmm(st["q"][pad].float().view(-1, N * H, DQK), kf.transpose(1, 2)).mul_(SCALE).view(-1, N, H, L)
    node = (t - first).clamp(0, N - 1)
    see = (t < first)[:, None, :] | ((t < n)[:, None, :] & up.gather(2, node[:, None, :].expand(-1, N, -1)))
    s.masked_fill_(~see[:, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-3e38)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(-1, N * H, L), kf[:, :, :DV]).view(-1, N, H, DV) / l.clamp_min(1e-38)
    lse = (m + l.log()).squeeze(-1)
    return {"out": o[req, i].to(torch.bfloat16), "lse": lse[req, i], "mask": mask[req, i], "depth": up.sum(-1)[req, i].to(torch.int32) - 1}


def _links(parent, pad, ok):
    """First child and next sibling of every node, N where there is none: [B, N]."""
    B, N = pad.shape
    up = torch.where(ok, parent[pad].long(), -2)
    j = torch.arange(N, device=pad.device)
    child = torch.where(up[:, None, :] == j[None, :, None], j, N).amin(-1)
    next_ = torch.where((up[:, None, :] == up[:, :, None]) & (j[None, :] > j[:, None]), j, N).amin(-1)
    return child, next_


def _plain_verify(st):
    case, dev = st["case"], st["target"].device
    B, V, N = case["requests"], case["vocab"], st["N"]
    pad, ok = _padded(st["row_off"], N, st["n_rows"])
    tok = st["token"][pad].long()
    child, next_ = _links(st["parent"], pad, ok)
    b = torch.arange(B, device=dev)
    wide = torch.full((B, N + 1), -1, dtype=torch.int64, device=dev)
    v = torch.zeros(B, dtype=torch.int64, device=dev)
    count = torch.ones_like(v)
    wide[:, 0] = 0
    if case["mode"] == "greedy":
        x = st["target"].float()
        best = torch.where(x == x.amax(-1, keepdim=True), torch.arange(V, device=dev), V).amin(-1)[pad]
        c = child[b, v]
        for _ in range(N - 1):
            here = c.clamp_max(N - 1)
            yes = (c < N) & (tok[b, here] == best[b, v])
            wide[b, torch.where(yes, count, N)] = torch.where(yes, here, -1)
            count, v = count + yes, torch.where(yes, here, v)
            c = torch.where(yes, child[b, here], torch.where(c < N, next_[b, here], N))
        token = best[b, v]
    else:
        # what is left of p after the rejections at a node is max(0, p - S q): the first rejection leaves
        # max(0, p - q) with the sum R, the next max(0, max(0, p - q) - R q), and so on.  In 64 bits: the
        # path and the token hang on which side of a border a sum falls
        S, R = torch.zeros(B, dtype=torch.float64, device=dev), torch.ones(B, dtype=torch.float64, device=dev)
        c = child[b, v]
        certain = st["draft"] is None
        chain = case["reach"] == 1
        gone = torch.zeros((B, V), dtype=torch.bool, device=dev) if certain else None
        if chain:  # every test on its own, then up to the first that fails
            x = tok[:, 1:]
            px = st["target"][pad[:, :-1], x].double()
            qx = 1.0 if certain else st["draft"][pad[:, :-1], x].double()
            yes = (st["u_node"][pad[:, 1:]].double() * qx < px) & ok[:, 1:]
            v = yes.long().cumprod(1).sum(1)
            count = v + 1
            wide[:, :N] = torch.where(torch.arange(N, device=dev)[None, :] <= v[:, None], torch.arange(N, device=dev)[None, :], -1)
            failed = child[b, v] < N
            if certain:
                gone[b, tok[b, child[b, v].clamp_max(N - 1)]] = failed
            else:
                S = failed.double()
                left = (st["target"][pad[b, v]].double() - st["draft"][pad[b, v]].double()).clamp_min_(0).sum(-1)
                S = torch.where(left > 0, S, 0.0)
        for _ in range(0 if chain else N - 1):
            here = c.clamp_max(N - 1)
            x = tok[b, here]
            px = st["target"][pad[b, v], x].double()
            if certain:
                rx, qx = torch.where(gone[b, x], 0.0, px), 1.0
            else:
                qx = st["draft"][pad[b, v], x].double()
                rx = (px - S * qx).clamp_min(0)
            on = c < N
            yes = on & (st["u_node"][pad[b, here]].double() * qx * R < rx)
            no = on & ~yes
            # a rejection
            p = st["target"][pad[b, v]].double()
            if certain:
                was = gone[b, x]
                gone[b, x] = was | no
                left = p.masked_fill_(gone, 0.0).sum(-1)
                keep = no & (left > 0)
                gone[b, x] = torch.where(no & ~keep, was, gone[b, x])
                R = torch.where(keep, left, R)
            else:
                left = p.sub_((S + R)[:, None] * st["draft"][pad[b, v]].double()).clamp_min_(0).sum(-1)
                keep = no & (left > 0)
                S, R = torch.where(keep, S + R, S), torch.where(keep, left, R)
            # an acceptance
            wide[b, torch.where(yes, count, N)] = torch.where(yes, here, -1)
            count, v = count + yes, torch.where(yes, here, v)
            S, R = torch.where(yes, 0.0, S), torch.where(yes, 1.0, R)
            if certain:
                gone &= ~yes[:, None]
            c = torch.where(yes, child[b, here], torch.where(on, next_[b, here], N))
        p = st["target"][pad[b, v]].double()
        if certain:
            p = torch.where(gone & (p.masked_fill(gone, 0.0).sum(-1) > 0)[:, None], 0.0, p)
        else:
            p = p.sub_(S[:, None] * st["draft"][pad[b, v]].double()).clamp_min_(0)
        up = p.cumsum(-1)
        token = (up <= st["u_pick"].double()[:, None] * up[:, -1:]).sum(-1).clamp_max(V - 1)
    req = torch.repeat_interleave(b, st["row_off"][1:] - st["row_off"][:-1], output_size=st["n_rows"])
    path = wide[req, torch.arange(st["n_rows"], device=dev) - st["row_off"][:-1][req]]
    return {"path": path.to(torch.int32), "count": count.to(torch.int32), "next": token.to(torch.int32)}


def _place(st, at):
    """Cache row of token row `at`."""
    page = st["case"]["page"]
    return st["page_tab"].long()[at // page] * page + at % page


def _plain_free(st, end):
    E = st["E"]
    start = torch.arange(st["page_tab"].numel(), device=end.device) * st["case"]["page"]
    drop = (st["page_tab"] >= 0) & (start >= end.repeat_interleave(E, output_size=start.numel()))
    st["refs"].index_add_(0, st["page_tab"].clamp_min(0).long(), -drop.to(torch.int32))
    st["page_tab"].masked_fill_(drop, -1)


def _plain_reserve(st, end, want):
    """No page of these requests is shared, and the pool has room."""
    E, tab, refs = st["E"], st["page_tab"], st["refs"]
    start = torch.arange(tab.numel(), device=end.device) * st["case"]["page"]
    need = (tab < 0) & (start < want.repeat_interleave(E, output_size=start.numel()))
    free = (refs > 0).to(torch.int32).argsort(stable=True)
    new = free[(need.long().cumsum(0) - 1).clamp_min(0)].to(torch.int32)
    tab.copy_(torch.where(need, new, tab))
    refs.index_add_(0, tab.clamp_min(0).long(), need.to(torch.int32))
    st["room"].copy_(want)


def _plain_keep(st):
    B, N, kv = st["B"], st["case"]["nodes"], st["kv"]
    path = st["path"].view(B, N).long()
    i = torch.arange(N, device=kv.device)[None, :]
    base = (st["tok_end"] - N)[:, None]
    to = _place(st, base + i)
    fro = torch.where(i < st["count"][:, None], _place(st, base + path.clamp_min(0)), to)
    kv[:, to.reshape(-1)] = kv[:, fro.reshape(-1)]
    st["new_end"].copy_(base[:, 0] + st["count"])
    _plain_free(st, st["new_end"])
    _plain_reserve(st, st["new_end"], st["new_end"] + N)
    return {"kv": kv, "page_tab": st["page_tab"], "refs": st["refs"], "new_end": st["new_end"], "room": st["room"]}


def _plain_fork(st):
    page, E, tab, refs, kv = st["case"]["page"], st["E"], st["page_tab"].view(-1, st["E"]), st["refs"], st["kv"]
    src, dst = st["src"].long(), st["dst"].long()
    n = (st["tok_end"] - st["tok_off"][:-1])[src]
    e = torch.arange(E, device=kv.device)[None, :]
    old = tab[dst]
    refs.index_add_(0, old.clamp_min(0).reshape(-1).long(), -(old >= 0).to(torch.int32).reshape(-1))
    new = torch.where(e < (n // page)[:, None], tab[src], -1)
    refs.index_add_(0, new.clamp_min(0).reshape(-1).long(), (new >= 0).to(torch.int32).reshape(-1))
    rest = n % page                                                 # rows of the last page, which is copied
    some = rest > 0
    free = (refs > 0).to(torch.int32).argsort(stable=True)
    tail = free[(some.long().cumsum(0) - 1).clamp_min(0)]
    last = (n // page).clamp_max(E - 1)
    new[torch.arange(dst.numel(), device=kv.device), last] = torch.where(some, tail.to(torch.int32), new.gather(1, last[:, None])[:, 0])
    refs.index_add_(0, tail, some.to(torch.int32))
    r = torch.arange(page, device=kv.device)[None, :]
    fro = tab[src].gather(1, last[:, None]).long() * page + r
    to = torch.where(r < rest[:, None], tail[:, None] * page + r, fro)
    kv[:, to.reshape(-1)] = kv[:, fro.reshape(-1)]
    tab[dst] = new
    st["tok_end"][dst] = st["tok_off"][:-1][dst] + n
    return {"kv": kv, "page_tab": st["page_tab"], "refs": refs, "tok_end": st["tok_end"]}


def _plain_turn(st):
    case, tab, refs, kv = st["case"], st["page_tab"], st["refs"], st["kv"]
    left = st["left"][st["turn"]]
    st["turn"] ^= 1
    _plain_free(st, left)
    # the pages in use behind the first `used` places move down into the free ones among those
    P = st["n_pages"]
    p = torch.arange(P, device=kv.device)
    live = refs > 0
    used = live.sum()
    hole, far = ~live & (p < used), live & (p >= used)
    most = P // 2
    to = torch.where(hole, p, P).sort()[0][:most]
    fro = torch.where(far, p, P).sort()[0][:most]
    some = to < P
    to, fro = torch.where(some, to, P - 1), torch.where(some, fro, P - 1)  # the last page has no request's rows
    place = p.scatter(0, fro, torch.where(some, to, fro))
    tab.copy_(torch.where(tab >= 0, place[tab.clamp_min(0).long()], -1))
    rows = kv.view(kv.shape[0], P, -1)
    rows[:, to] = rows[:, fro]
    moved = refs[fro]
    refs[fro] = torch.where(some, 0, moved)
    refs[to] = torch.where(some, moved, refs[to])
    st["used"].copy_(used[None])
    _plain_reserve(st, left, st["want"])
    return {"kv": kv, "page_tab": tab, "refs": refs, "used": st["used"], "room": st["room"]}


# ---------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    if not own:
        if case["op"] == "pages":
            return {"keep": _plain_keep, "fork": _plain_fork, "turn": _plain_turn}[case["kind"]](st)
        return {"tree": _plain_tree, "verify": _plain_verify}[case["op"]](st)
    from sparse_attention_kv_echo_gb300 import lib as L
    if case["op"] == "tree":
        if "pages" not in st:                          # what a server keeps for its cache and its stream
            st["pages"] = L.KVPages(st["page_tab"], st["kv"], case["page"])
            st["ws"] = torch.empty(L.mla_chunk_workspace_size(st["n_rows"], case["heads"], case["requests"]),
                                   dtype=torch.uint8, device=st["q"].device)
        L.tree_masks(st["row_off"], st["parent"], st["mask"], st["status"], depth=st["depth"])
        L.mla_tree(st["row_off"], st["q"], st["mask"], st["tok_off"], st["n_tokens"], st["pages"], SCALE, st["out"], st["lse"],
                   st["ws"], st["status"], tok_end=st["tok_end"])
        return {"out": st["out"], "lse": st["lse"], "mask": st["mask"], "depth": st["depth"]}
    if case["op"] == "verify":
        L.draft_verify(st["row_off"], st["parent"], st["token"], st["target"], st["path"], st["count"], st["next"], st["status"],
                       draft=st["draft"], u_node=st["u_node"], u_pick=st["u_pick"])
        return {"path": st["path"], "count": st["count"], "next": st["next"]}
    if "pool" not in st:
        st["pool"] = L.PagePool(st["page_tab"], st["refs"], st["kv"], case["page"])
        st["ws"] = torch.empty(L.pages_workspace_size(st["B"], st["n_pages"]), dtype=torch.uint8, device=st["kv"].device)
    pool, ws, off, n, status = st["pool"], st["ws"], st["tok_off"], st["n_tokens"], st["status"]
    if case["kind"] == "keep":
        L.rows_keep(st["row_off"], st["path"], st["count"], off, st["tok_end"], n, pool, st["new_end"], status)
        L.pages_free(off, st["new_end"], n, pool, status)
        L.pages_reserve(off, st["new_end"], st["new_end"] + st["nodes"], n, pool, st["room"], ws, status)
        return {"kv": st["kv"], "page_tab": st["page_tab"], "refs": st["refs"], "new_end": st["new_end"], "room": st["room"]}
    if case["kind"] == "fork":
        L.pages_fork(st["src"], st["dst"], off, st["tok_end"], n, pool, ws, status)
        return {"kv": st["kv"], "page_tab": st["page_tab"], "refs": st["refs"], "tok_end": st["tok_end"]}
    left = st["left"][st["turn"]]
    st["turn"] ^= 1
    L.pages_free(off, left, n, pool, status)
    L.pages_compact(n, pool, st["used"], ws, status)
    L.pages_reserve(off, left, st["want"], n, pool, st["room"], ws, status)
    return {"kv": st["kv"], "page_tab": st["page_tab"], "refs": st["refs"], "used": st["used"], "room": st["room"]}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    B = case["requests"]
    if case["op"] == "tree":
        nodes, lens = _spread(case["nodes_a"], case["nodes_b"], B), _spread(case["len_a"], case["len_b"], B)
        # a node sees at least the context and itself; every cached row, the trees' among them, is read once
        pairs = sum(m * (n + 1) for n, m in zip(lens, nodes))
        rows = sum(nodes)
        return {"bytes": 2 * DQK * sum(n + m for n, m in zip(lens, nodes)) + rows * case["heads"] * (2 * DQK + 2 * DV + 4)
                + 4 * rows * (2 + -(-max(nodes) // 32)) + 4 * sum(lens) // case["page"],
                "flops": 2.0 * (DQK + DV) * case["heads"] * pairs}
    if case["op"] == "verify":
        # the row of the token behind the path, and of the draft under it; which and how many more the
        # walk needs is up to the data
        rows = 2 if case["mode"] == "sample" else 1
        n = sum(_spread(case["nodes_a"], case["nodes_b"], B))
        return {"bytes": B * case["vocab"] * rows * (2 if case["half"] else 4) + 16 * n, "flops": 3.0 * B * case["vocab"]}
    row, page, layers = 2 * DQK, case["page"], case["layers"]
    lens = _spread(case["len_a"], case["len_b"], B)
    entries = _pool_rows(case) // page
    if case["kind"] == "keep":  # a quarter of the nodes on average, read and written
        return {"bytes": 2 * row * layers * B * max(1, case["nodes"] // 4) + 4 * 2 * entries, "flops": 0}
    if case["kind"] == "fork":
        return {"bytes": 2 * row * layers * case["copies"] * sum(n % page for n in lens) + 4 * 4 * entries, "flops": 0}
    return {"bytes": 2 * row * layers * (B // 2) * -(-lens[0] // page) * page + 4 * 6 * entries, "flops": 0}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(st)
    if case["op"] == "verify":
        return _exact_verify(st)
    return _exact_pages(st)


def _exact_tree(st):
    case = st["case"]
    H, page, dev = case["heads"], case["page"], st["q"].device
    out = torch.empty((st["n_rows"], H, DV), dtype=torch.float64, device=dev)
    lse = torch.empty((st["n_rows"], H), dtype=torch.float64, device=dev)
    parent = st["parent"].tolist()
    r0 = 0
    for b, (n, m) in enumerate(zip(st["lens"], st["nodes"])):
        at = int(st["tok_off"][b]) + torch.arange(n, device=dev)
        kd = st["kv"][st["page_tab"][torch.div(at, page, rounding_mode="floor")].long() * page + torch.remainder(at, page)].double()
        see = torch.zeros((m, n), dtype=torch.bool)
        see[:, :n - m] = True
        for i in range(m):
            j = i
            while j >= 0:
                see[i, n - m + j] = True
                j = parent[r0 + j]
        see = see.to(dev)
        block = max(1, min(m, int(2e9 / (8.0 * H * n))))
        for i0 in range(0, m, block):
            i1 = min(m, i0 + block)
            s = SCALE * (st["q"][r0 + i0:r0 + i1].double().reshape(-1, DQK) @ kd.T).reshape(i1 - i0, H, n)
            s = torch.where(see[i0:i1, None, :], s, -math.inf)
            lse[r0 + i0:r0 + i1] = torch.logsumexp(s, -1)
            w = torch.exp(s - lse[r0 + i0:r0 + i1, :, None])
            out[r0 + i0:r0 + i1] = (w.reshape(-1, n) @ kd[:, :DV]).reshape(i1 - i0, H, DV)
        r0 += m
    return {"out": out, "lse": lse, "mask": None, "depth": None}


def _exact_verify(st):
    """One request, one child, one rejection after the other, the residual carried along as it is defined."""
    case = st["case"]
    off, parent, token = st["row_off"].tolist(), st["parent"].tolist(), st["token"].tolist()
    paths, counts, picks = [], [], []
    for b in range(case["requests"]):
        r0, n = off[b], off[b + 1] - off[b]
        v, path = 0, [0]
        while True:
            row = st["target"][r0 + v].double()
            kids = [i for i in range(v + 1, n) if parent[r0 + i] == v]
            went = None
            if case["mode"] == "greedy":
                pick = int((row == row.max()).nonzero()[0])
                went = next((i for i in kids if token[r0 + i] == pick), None)
            else:
                left, total = row, 1.0
                for i in kids:
                    x = token[r0 + i]
                    if st["draft"] is None:
                        q = torch.zeros_like(row)
                        q[x] = 1.0
                    else:
                        q = st["draft"][r0 + v].double()
                    if float(st["u_node"][r0 + i]) * float(q[x]) * total < float(left[x]):
                        went = i
                        break
                    then = (left - total * q).clamp_min(0)
                    if float(then.sum()) > 0:
                        left, total = then, float(then.sum())
                if went is None:
                    c = left.cumsum(0)
                    pick = int((c > float(st["u_pick"][b]) * float(c[-1])).nonzero()[0])
            if went is None:
                break
            v = went
            path.append(v)
        paths += path + [-1] * (n - len(path))
        counts.append(len(path))
        picks.append(pick)
    i32 = dict(dtype=torch.int32, device=st["target"].device)
    return {"path": torch.tensor(paths, **i32), "count": torch.tensor(counts, **i32), "next": torch.tensor(picks, **i32)}


def _exact_pages(st):
    """The calls on lists, then the rows moved by them; they are copies, and as exact in 64 bits as in 16."""
    case, kv = st["case"], st["kv"]
    page, E, B = case["page"], st["E"], st["B"]
    tab, refs, off = st["page_tab"].tolist(), st["refs"].tolist(), st["tok_off"].tolist()
    moves = []                                                       # (from row, to row)

    def free(end):
        for b in range(B):
            for e in range(b * E, (b + 1) * E):
                if e * page >= end[b] and tab[e] >= 0:
                    refs[tab[e]] -= 1
                    tab[e] = -1

    def reserve(want):
        spare = [p for p, r in enumerate(refs) if r == 0]
        for e in range(B * E):
            if tab[e] < 0 and e * page < want[e // E]:
                tab[e] = spare.pop(0)
                refs[tab[e]] = 1

    more = {}
    if case["kind"] == "keep":
        end, N, path, count = st["tok_end"].tolist(), case["nodes"], st["path"].tolist(), st["count"].tolist()
        row = lambda t: tab[t // page] * page + t % page  # noqa: E731
        for b in range(B):
            moves += [(row(end[b] - N + path[b * N + i]), row(end[b] - N + i)) for i in range(count[b])]
            end[b] += count[b] - N
        free(end)
        want = [x + N for x in end]
        reserve(want)
        more = {"new_end": end, "room": want}
    elif case["kind"] == "fork":
        end = st["tok_end"].tolist()
        tails = []
        for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
            n = end[s] - off[s]
            for e in range(n // page):
                tab[d * E + e] = tab[s * E + e]
                refs[tab[s * E + e]] += 1
            end[d] = off[d] + n
            if n % page:
                tails.append((s, d, n // page, n % page))
        spare = [p for p, r in enumerate(refs) if r == 0]
        for s, d, e, rest in tails:
            tab[d * E + e] = spare.pop(0)
            refs[tab[d * E + e]] = 1
            moves += [(tab[s * E + e] * page + r, tab[d * E + e] * page + r) for r in range(rest)]
        more = {"tok_end": end}
    else:
        free(st["left"][0].tolist())
        live = [p for p, r in enumerate(refs) if r > 0]
        holes = [p for p in range(len(live)) if refs[p] == 0]
        place = dict(zip([p for p in live if p >= len(live)], holes))
        tab[:] = [place.get(p, p) for p in tab]
        for a, z in place.items():
            refs[z], refs[a] = refs[a], 0
            moves += [(a * page + r, z * page + r) for r in range(page)]
        reserve(st["want"].tolist())
        more = {"used": [len(live)], "room": st["want"].tolist()}
    rows = torch.tensor(moves, dtype=torch.int64).view(-1, 2).to(kv.device)
    wide = kv.double()
    for l in range(case["layers"]):
        wide[l, rows[:, 1]] = wide[l, rows[:, 0]]
    kinds = {"used": torch.int32}
    got = {"kv": wide, "page_tab": torch.tensor(tab, dtype=torch.int32), "refs": torch.tensor(refs, dtype=torch.int32)}
    return got | {k: torch.tensor(x, dtype=kinds.get(k, torch.int64)) for k, x in more.items()}
