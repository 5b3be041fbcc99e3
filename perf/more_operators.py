"""Drafted tokens over the paged resident cache, as they are measured: the operators' cases, plain forms and definition in 64 bits.

A step brings each sequence a tree of drafted rows: row 0 is the last token that is certain, the others are drafts, and
parent [T] names for each row the one it follows, counted within its sequence (-1: it follows the cached tokens). Row i's
position is its depth behind the cached ones. Pages, row0 and seq_len are those of the resident paged cache.

  tree    softmax attention of every head of the rows over the cached tokens and the row's own branch
  verify  which drafts the target's probabilities accept, from given random numbers, and the token that follows them
  accept  the accepted rows of each tree move together behind the cached tokens; the lengths without the others
  copy    pages of a pool are copied to others, whole or their first rows (forked sequences, a pool that is packed)
"""
import math
import random

import torch

own = False

ROW, VAL = 576, 512
SCALE = 1.0 / math.sqrt(192.0)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one conversation, eight drafts, a shard of 16 heads: latency
        dict(name="tree-1x8-h16-1k", op="tree", B=1, rows=8, H=16, ctx=999, page=64, window=0, sink=0, ragged=False, mix=1),
        # a decode batch of the benchmark's 32 sequences, small trees of different sizes, all 128 heads
        dict(name="tree-32x12-h128-8k", op="tree", B=32, rows=12, H=128, ctx=8192, page=64, window=0, sink=0, ragged=True, mix=2),
        # few sequences, wide trees, a long cache
        dict(name="tree-4x64-h128-16k", op="tree", B=4, rows=64, H=128, ctx=16384, page=64, window=0, sink=0, ragged=False, mix=3),
        # windowed layer, odd page size: only the first tokens and the window are read of long caches
        dict(name="tree-window-16x27-h32-50k", op="tree", B=16, rows=27, H=32, ctx=50000, page=24, window=1024, sink=4, ragged=True, mix=4),
        # one conversation, four drafts in a row, proposed without randomness
        dict(name="verify-1x5-32000", op="verify", B=1, rows=5, V=32000, bf16=False, chain=True, drawn=False, mix=5),
        # a batch whose chains were drawn from a drafting model's probabilities
        dict(name="verify-32x6-drawn-128000", op="verify", B=32, rows=6, V=128000, bf16=True, chain=True, drawn=True, mix=6),
        # small trees, a vocabulary of odd size: rows that begin at every alignment
        dict(name="verify-8x26-50021", op="verify", B=8, rows=26, V=50021, bf16=True, chain=False, drawn=False, mix=7),
        # a large batch of wide trees: a few rows of each decide
        dict(name="verify-64x60-128000", op="verify", B=64, rows=60, V=128000, bf16=True, chain=False, drawn=False, mix=8),
        # one conversation's accepted drafts
        dict(name="accept-1x8", op="accept", B=1, rows=8, ctx=999, page=64, mix=9),
        # a large batch of wide trees, page ends inside the trees
        dict(name="accept-256x60", op="accept", B=256, rows=60, ctx=700, page=24, mix=10),
        # twelve samples fork off their prompts: the last, partly filled page of each
        dict(name="copy-12-partial", op="copy", pages=12, page=64, partial=True, spare=100, mix=11),
        # a pool is packed: 131072 rows change their place
        dict(name="copy-2048", op="copy", pages=2048, page=64, partial=False, spare=3000, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "verify", "verify", "accept", "copy"])
    page, mix = rng.choice([1, 16, 24, 32, 48, 64, 100, 128]), rng.randrange(1 << 20)
    if op == "copy":
        page = max(page, 16)
        return dict(op=op, pages=_log(rng, 1, 131072 // page), page=page, partial=rng.random() < 0.5, spare=rng.randint(1, 500), mix=mix)
    if op == "accept":
        return dict(op=op, B=_log(rng, 1, 256), rows=_log(rng, 2, 64), ctx=_log(rng, 1, 700), page=page, mix=mix)
    if op == "verify":
        V, B = _log(rng, 1000, 160000), _log(rng, 1, 128)
        rows = _log(rng, 2, 64)
        rows = max(2, min(rows, int(4.9e8 / (V * B))))
        chain = rng.random() < 0.5
        return dict(op=op, B=B, rows=rows, V=V, bf16=rng.random() < 0.6, chain=chain, drawn=chain and rng.random() < 0.6, mix=mix)
    H = rng.choice([1, 8, 16, 24, 32, 64, 128])
    B, rows = _log(rng, 1, 64), _log(rng, 2, 128)
    most = 5.0e8                                  # padded (row, head, token) triples: under the largest listed case's
    rows = max(2, min(rows, int(most / (B * H * 1000))))
    ctx = _log(rng, 1, max(2, min(60000, 800000 // B, int(most / (B * H * rows)) - rows)))
    window = _log(rng, 1, 4096) if rng.random() < 0.4 else 0
    return dict(op=op, B=B, rows=rows, H=H, ctx=ctx, page=page, window=window, sink=rng.choice([0, 1, 4, 64]) if window else 0,
                ragged=rng.random() < 0.6, mix=mix)


def _tree(r, n, chain=False):
    """Parents of a tree of n rows, row 0 its root; a draft follows any earlier row, so depths stay near 2 ln n."""
    return [-1] + [i - 1 if chain else r.randrange(i) for i in range(1, n)]


def _depths(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _sizes(case):
    """(parents of each sequence's rows, lengths with them), from the case alone."""
    r = random.Random(case["mix"])
    R, trees, lens = case["rows"], [], []
    for b in range(case["B"]):
        n = R if not case.get("ragged") or b == 0 else r.choice([0, 1, r.randint(2, R), r.randint(2, R), R])
        trees.append(_tree(r, n, case.get("chain", False)) if n else [])
        ctx = case.get("ctx", 0)
        lens.append(n + (ctx if not case.get("ragged") or b == 0 else r.randint(ctx // 2, ctx)))
    return trees, lens


# ---------------------------------------------------------------- what a program has in hand
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev = dict(device="cuda")

    def rows_of(n):   # cached rows: unit latents with a spread of magnitudes between tokens
        x = torch.randn((n, ROW), generator=g, **dev)
        return (x * torch.exp(0.3 * torch.randn((n, 1), generator=g, **dev))).to(torch.bfloat16)

    if case["op"] == "copy":
        n, ps = case["pages"], case["page"]
        total = 2 * n + case["spare"]
        perm = torch.randperm(total, generator=g, **dev).to(torch.int32)
        st = dict(case=case, ps=ps, n=n, pool=rows_of(total * ps), src=perm[:n].contiguous(), dst=perm[n:2 * n].contiguous(), count=None)
        if case["partial"]:
            st["count"] = torch.randint(0, ps + 1, (n,), generator=g, dtype=torch.int32, **dev)
        return st
    trees, lens = _sizes(case)
    B, off = case["B"], [0]
    for t in trees:
        off.append(off[-1] + len(t))
    T = off[-1]
    st = dict(case=case, B=B, T=T, max_rows=max(len(t) for t in trees), row0=torch.tensor(off, dtype=torch.int32, **dev),
              parent=torch.tensor([p for t in trees for p in t], dtype=torch.int32, **dev),
              depth=max(max(_depths(t)) for t in trees if t))
    if case["op"] == "verify":
        return _prepare_verify(st, g)
    ps, max_len = case["page"], max(lens)
    npg = -(-max_len // ps)
    perm = torch.randperm(B * npg + 1, generator=g, **dev).to(torch.int32)
    st.update(ps=ps, max_len=max_len, table=perm[: B * npg].view(B, npg).contiguous(), seq_len=torch.tensor(lens, dtype=torch.int32, **dev),
              pool=rows_of((B * npg + 1) * ps))
    if case["op"] == "tree":
        st["q"] = torch.randn((T, case["H"], ROW), generator=g, **dev).to(torch.bfloat16)
        return st
    # accept: a branch of each tree, its rows in order
    r = random.Random(int(seed))
    kept = []
    for t in trees:
        d = _depths(t)
        at, path = r.choice([i for i in range(len(t)) if d[i] >= min(2, max(d))]), []
        while at >= 0:
            path.insert(0, at)
            at = t[at]
        kept.append(path + [-1] * (st["depth"] + 1 - len(path)))
    st["kept"] = torch.tensor(kept, dtype=torch.int32, **dev)
    st["n_kept"] = (st["kept"] >= 0).sum(1, dtype=torch.int32)
    return st


def _prepare_verify(st, g):
    """Target logits with a few likely tokens a row; drafts that are mostly among them; temperatures of single requests, some greedy."""
    case, T, B, V = st["case"], st["T"], st["B"], st["case"]["V"]
    dev = dict(device="cuda")
    x = torch.randn((T, V), generator=g, **dev).mul_(1.5)
    x += 9.0 * (torch.rand((T, V), generator=g, **dev) < 12.0 / V)
    st["temperature"] = torch.where(torch.arange(B, **dev) % 5 == 3, 0.0, 0.6 + 0.4 * torch.rand(B, generator=g, **dev))
    n = st["row0"][1:] - st["row0"][:-1]
    first = torch.repeat_interleave(st["row0"][:-1], n)
    at = (first + st["parent"].clamp(min=0)).long()
    if case["drawn"]:
        temp = torch.repeat_interleave(st["temperature"], n).clamp(min=0.3).view(T, 1)
        st["draft"] = torch.softmax((x + 0.7 * torch.randn((T, V), generator=g, **dev)) / temp, -1)
        tok = torch.multinomial(st["draft"], 1, generator=g)[:, 0][at]
    else:
        top = torch.topk(x, 8, dim=1).indices
        turn = torch.arange(T, **dev) % 3           # the best, second or third token of the row before
        tok = top[at, turn]
        tok = torch.where(torch.rand(T, generator=g, **dev) < 0.15, torch.randint(0, V, (T,), generator=g, **dev), tok)
    st["tokens"] = tok.to(torch.int32)
    st["logits"] = x.to(torch.bfloat16) if case["bf16"] else x
    st["u"] = torch.rand(T, generator=g, **dev)
    return st


# ---------------------------------------------------------------- plain forms
def _slots(st, table, n):
    t = torch.arange(n, device="cuda")
    return table[:, t // st["ps"]].long() * st["ps"] + t % st["ps"]


def _padded(st):
    """(rows of each sequence [B, R], which of them exist, ancestors-or-self [B, R, R])."""
    B, R = st["B"], st["max_rows"]
    n = (st["row0"][1:] - st["row0"][:-1]).view(B, 1)
    i = torch.arange(R, device="cuda").view(1, R)
    at = (st["row0"][:-1].view(B, 1) + i).clamp(max=st["T"] - 1).long()
    parent = torch.where(i < n, st["parent"][at], -1)
    step = (parent.unsqueeze(-1) == torch.arange(R, device="cuda")).double()
    line = torch.linalg.matrix_power(step + torch.eye(R, dtype=torch.float64, device="cuda"), max(1, st["depth"])) > 0
    return at, i < n, parent, line


def _flat(st, x):
    """[B, rows, ...] -> the batch's rows one after another [T, ...]."""
    t = torch.arange(st["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(st["row0"][1:], t, right=True)
    return x[b, (t - st["row0"][b]).long()]


def _plain_tree(st):
    case, B, L, R, H = st["case"], st["B"], st["max_len"], st["max_rows"], st["case"]["H"]
    at, live, _, line = _padded(st)
    k = st["pool"][_slots(st, st["table"], L)].float()
    s = torch.matmul(st["q"][at].float().view(B, R * H, ROW), k.transpose(1, 2)).view(B, R, H, L).mul_(SCALE)
    ctx = st["seq_len"] - (st["row0"][1:] - st["row0"][:-1])
    depth = line.sum(-1) - 1
    t = torch.arange(L, device="cuda").view(1, L)
    node = (t - ctx.view(B, 1)).long()                              # of token t; below 0: cached
    of = node.clamp(0, R - 1)
    pos = torch.where(node < 0, t, ctx.view(B, 1) + depth.gather(1, of)).unsqueeze(1)
    mine = (ctx.view(B, 1) + depth).unsqueeze(-1)
    vis = torch.where((node < 0).unsqueeze(1), True, line.gather(2, of.unsqueeze(1).expand(B, R, L)))
    vis = vis & (t < st["seq_len"].view(B, 1)).unsqueeze(1) & live.unsqueeze(-1)
    if case["window"]:
        vis = vis & ((pos > mine - case["window"]) | (pos < case["sink"]))
    s = s.masked_fill_(~vis.unsqueeze(2), -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, R * H, L), k[..., :VAL]).view(B, R, H, VAL) / torch.where(l == 0, torch.ones_like(l), l)
    return _flat(st, o.to(torch.bfloat16)), _flat(st, (m + l.log()).squeeze(-1))


def _plain_verify(st):
    """In 64 bits: each decision compares a random number with a sum over the vocabulary."""
    case, B, R, V = st["case"], st["B"], st["max_rows"], st["case"]["V"]
    at, live, parent, line = _padded(st)
    temp = torch.repeat_interleave(st["temperature"], st["row0"][1:] - st["row0"][:-1]).double().view(-1, 1)
    x = st["logits"].double()
    top, first = x.max(-1, keepdim=True)
    best = torch.where(x == top, torch.arange(V, device="cuda"), V).amin(-1)
    w = x.sub_(top).div_(torch.where(temp > 0, temp, torch.ones_like(temp))).exp_()
    total = w.sum(-1)
    greedy = (st["temperature"] <= 0).view(B, 1)
    u = st["u"].double()[at]
    tok, before = st["tokens"].long()[at], torch.gather(at, 1, parent.clamp(min=0).long())
    is_child = live & (parent >= 0)
    mass = torch.where(is_child, w[before, tok], 0.0)
    if case["drawn"]:
        ok = (mass > 0) & (u * st["draft"].double()[before, tok] < mass / total[before])
        older = torch.zeros((B, R, R), dtype=torch.bool, device="cuda")
    else:
        i = torch.arange(R, device="cuda")
        older = (parent.unsqueeze(2) == parent.unsqueeze(1)) & (i.view(1, 1, R) < i.view(1, R, 1)) & is_child.unsqueeze(1)
        again = (older & (tok.unsqueeze(2) == tok.unsqueeze(1))).any(-1)
        mass = torch.where(again, 0.0, mass)
        left = total[before] - torch.matmul(older.double(), mass.unsqueeze(-1)).squeeze(-1)
        ok = (mass > 0) & (u * left < mass)
    ok = torch.where(greedy, tok == best[before], ok) & is_child
    taken = ok & ~(older & ok.unsqueeze(1)).any(-1)
    taken[:, 0] = True
    depth = line.sum(-1) - 1
    on = live & line[..., 0] & (depth <= st["depth"]) & ~(line & ~taken.unsqueeze(1)).any(-1)
    n_kept = on.sum(1, dtype=torch.int32)
    kept = torch.where(on, torch.arange(R, device="cuda"), R).sort(1).values
    kept = torch.nn.functional.pad(kept, (0, max(0, st["depth"] + 1 - R)), value=R)[:, : st["depth"] + 1]
    kept = torch.where(kept < R, kept, -1).to(torch.int32)
    end = (n_kept - 1).clamp(min=0).long().view(B, 1)
    last = kept.gather(1, end).clamp(min=0).long()                  # the node where the branch ends
    row = at.gather(1, last)[:, 0]
    tried = is_child & (parent == last) & (end < st["depth"])       # its children, all rejected
    p = w[row]
    if case["drawn"]:
        p = p / total[row].view(B, 1)
        rest = (p - st["draft"][row].double()).clamp(min=0)
        p = torch.where(tried.any(1, keepdim=True) & (rest.sum(1, keepdim=True) > 0), rest, p)
    else:
        p = p.scatter_reduce(1, tok, torch.where(tried, 0.0, 1.0).double(), "prod")
    cum = p.cumsum(1)
    aim = st["u"].double()[st["row0"][:-1].long()].view(B, 1) * cum[:, -1:]
    nxt = torch.minimum((cum <= aim).sum(1), (cum < cum[:, -1:]).sum(1))
    return kept, n_kept, torch.where(greedy[:, 0], best[row], nxt).to(torch.int32)


def _plain_accept(st):
    B = st["B"]
    ctx = (st["seq_len"] - (st["row0"][1:] - st["row0"][:-1])).view(B, 1).long()
    kept = st["kept"].long()
    j = torch.arange(kept.shape[1], device="cuda").view(1, -1)
    valid = j < st["n_kept"].view(B, 1)                             # the others move the first row onto itself
    a, d = ctx + torch.where(valid, kept, 0), ctx + torch.where(valid, j, 0)
    b = torch.arange(B, device="cuda").view(B, 1)
    src, dst = (st["table"][b, t // st["ps"]].long() * st["ps"] + t % st["ps"] for t in (a, d))
    st["pool"][dst.view(-1)] = st["pool"][src.view(-1)]
    return st["pool"], (ctx[:, 0] + st["n_kept"]).to(torch.int32)


def _plain_copy(st):
    j = torch.arange(st["ps"], device="cuda").view(1, -1)
    src, dst = (st[k].long().view(-1, 1) * st["ps"] + j for k in ("src", "dst"))
    if st["count"] is not None:
        dst = torch.where(j < st["count"].view(-1, 1), dst, src)    # what is not copied moves onto itself
    st["pool"][dst.view(-1)] = st["pool"][src.view(-1)]
    return st["pool"]


def run(st):
    case, op = st["case"], st["case"]["op"]
    if not own:
        return {"tree": _plain_tree, "verify": _plain_verify, "accept": _plain_accept, "copy": _plain_copy}[op](st)
    import indexer_top_kv_amd as ech
    dev = dict(device="cuda")
    if op == "copy":
        ech.ech_paged_copy(st["pool"], st["ps"], st["src"], st["dst"], rows=st["count"])
        return st["pool"]
    B, T, R = st["B"], st["T"], st["max_rows"]
    if op == "accept":
        if "len_out" not in st:
            st["len_out"] = torch.empty_like(st["seq_len"])
        ech.ech_paged_accept(st["pool"], st["table"], st["ps"], st["row0"], st["seq_len"], st["kept"], st["n_kept"], R, st["max_len"],
                             st["len_out"])
        return st["pool"], st["len_out"]
    if op == "verify":
        if "ws" not in st:   # kept by the program for as long as its shapes stay
            st["ws"] = torch.empty(ech.ech_draft_verify_ws_bytes(B, T, case["V"], R, st["depth"] + 1), dtype=torch.uint8, **dev)
            st["kept"] = torch.empty((B, st["depth"] + 1), dtype=torch.int32, **dev)
            st["n_kept"], st["next"] = torch.empty(B, dtype=torch.int32, **dev), torch.empty(B, dtype=torch.int32, **dev)
        ech.ech_draft_verify(st["logits"], st["tokens"], st["row0"], R, st["u"], st["kept"], st["n_kept"], st["next"],
                             parent=None if case["chain"] else st["parent"], draft=st.get("draft"), temperature=st["temperature"],
                             ws=st["ws"])
        return st["kept"], st["n_kept"], st["next"]
    H = case["H"]
    if "ws" not in st:
        st["ws"] = torch.empty(ech.ech_paged_tree_attn_ws_bytes(B, T, H, R, st["max_len"], case["window"], case["sink"]),
                               dtype=torch.uint8, **dev)
        st["out"] = torch.empty((T, H, VAL), dtype=torch.bfloat16, **dev)
        st["lse"] = torch.empty((T, H), dtype=torch.float32, **dev)
    ech.ech_paged_tree_attn(st["q"], st["pool"], st["table"], st["ps"], st["row0"], st["seq_len"], st["parent"], R, st["max_len"],
                            SCALE, st["out"], st["lse"], window=case["window"], n_sink=case["sink"], ws=st["ws"])
    return st["out"], st["lse"]


# ---------------------------------------------------------------- what a pass cannot do without
def _line(parent, i):
    a = []
    while i >= 0:
        a.append(i)
        i = parent[i]
    return a


def work(case):
    if case["op"] == "copy":
        rows = case["pages"] * case["page"] * (0.5 if case["partial"] else 1)
        return {"bytes": rows * 2 * ROW * 2 + 8 * case["pages"], "flops": 0}
    trees, lens = _sizes(case)
    if case["op"] == "accept":   # about half of a branch's rows are not in their place
        moved = sum(max(_depths(t)) for t in trees)
        return {"bytes": moved * ROW * 2 + 16 * case["B"], "flops": 0}
    if case["op"] == "verify":   # the rows of one branch, half of its length on average, and a drafting row
        rows = sum(1 + max(_depths(t)) // 2 for t in trees)
        V = case["V"]
        return {"bytes": rows * V * (2 if case["bf16"] else 4) + (case["B"] * V * 4 if case["drawn"] else 0), "flops": 4 * rows * V}
    H, w, s = case["H"], case["window"], case["sink"]
    T = pairs = tokens = 0
    for t, length in zip(trees, lens):
        n, d = len(t), _depths(t)
        c = length - n
        T += n
        for i in range(n):
            line = _line(t, i)
            if not w:
                pairs += c + len(line)
                continue
            lo = max(0, c + d[i] - w + 1)
            pairs += max(0, c - lo) + min(s, lo, c) + sum(1 for a in line if d[i] - d[a] < w or c + d[a] < s)
        if n:
            lo = max(0, c - w + 1) if w else 0
            tokens += max(0, c - lo) + min(s, lo, c) + n
    return {"bytes": T * H * (ROW * 2 + VAL * 2 + 4) + tokens * ROW * 2, "flops": 2 * pairs * H * (ROW + VAL)}


# ---------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    if case["op"] != "tree":
        return None          # values that move as they are, and whole numbers
    st = prepare(case, seed)
    trees, lens = _sizes(case)
    ps, table, H, first = st["ps"], st["table"].cpu(), case["H"], 0
    out = torch.zeros((st["T"], H, VAL), dtype=torch.float64, device="cuda")
    lse = torch.full((st["T"], H), -math.inf, dtype=torch.float64, device="cuda")
    for b, (parent, length) in enumerate(zip(trees, lens)):
        n, d = len(parent), _depths(parent)
        c = length - n
        at = [int(table[b, t // ps]) * ps + t % ps for t in range(length)] if n else []
        kv = st["pool"][torch.tensor(at, dtype=torch.int64, device="cuda")].to(torch.float64)
        for i in range(n):
            w, lo = case["window"], 0
            see = _line(parent, i)[::-1]
            if w:
                lo = max(0, c + d[i] - w + 1)
                see = [a for a in see if d[i] - d[a] < w or c + d[a] < case["sink"]]
            head = kv[: min(case["sink"], lo, c)]
            k = torch.cat([head, kv[min(lo, c):c], kv[torch.tensor([c + a for a in see], dtype=torch.int64, device="cuda")]])
            sc = (st["q"][first + i].to(torch.float64) @ k.t()) * float(torch.tensor(SCALE, dtype=torch.float32))
            lse[first + i] = torch.logsumexp(sc, -1)
            out[first + i] = torch.softmax(sc, -1) @ k[:, :VAL]
        first += n
    return out, lse
