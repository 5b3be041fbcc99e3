"""The paged resident cache's operators, as they are measured: their cases, their plain forms and their definition in 64 bits.

A layer that keeps its rows on the device holds them in pages of a pool [slots, 576] of bf16 rows (absorbed-MLA rows: all
576 values are the key, the first 512 the value). `row0` [B + 1] says which of a step's new rows belong to which
sequence, `seq_len` [B] how long each sequence is with its new rows. A new row at position p sees the tokens t <= p, and
with a window only those with t > p - window or t < sink.

  append   the new rows go into their sequences' pages
  attn     softmax attention of every head of the new rows over the pages (a chunk, a single token, a ragged mix)
  weight   the attention weight that each cached token received, summed over rows and heads, joins a decayed running sum
  evict    the `keep` tokens of each sequence that stay (first ones, latest ones, then by accumulated weight), moved to
           the pages given for them
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
        # one short conversation, one token, a shard of 16 heads: latency
        dict(name="attn-1x1-h16-1k", op="attn", B=1, rows=1, H=16, ctx=999, page=64, window=0, sink=0, ragged=False, mix=1),
        # a decode batch of the benchmark's 32 sequences, all 128 heads on one GPU, ragged lengths
        dict(name="attn-32x1-h128-16k", op="attn", B=32, rows=1, H=128, ctx=16384, page=64, window=0, sink=0, ragged=True, mix=2),
        # a prompt's chunk over a long cache
        dict(name="attn-1x1024-h128-16k", op="attn", B=1, rows=1024, H=128, ctx=15360, page=64, window=0, sink=0, ragged=False, mix=3),
        # a step of a continuous batch: a few tokens each (drafts, ends of prompts), some sequences none, odd page size
        dict(name="attn-12x77-h16-5k", op="attn", B=12, rows=77, H=16, ctx=5003, page=24, window=0, sink=0, ragged=True, mix=4),
        # windowed layer, decode: only the first tokens and the window are read of long caches
        dict(name="window-64x1-h32-100k", op="attn", B=64, rows=1, H=32, ctx=100000, page=128, window=1024, sink=4, ragged=True, mix=5),
        # windowed layer, a prompt's chunk
        dict(name="window-2x2048-h16-8k", op="attn", B=2, rows=2048, H=16, ctx=8191, page=32, window=512, sink=64, ragged=False, mix=6),
        # weights of a decode step of the batch above
        dict(name="weight-32x1-h128-16k", op="weight", B=32, rows=1, H=128, ctx=16384, page=64, window=0, sink=0, ragged=True, mix=7),
        # weights of a prompt's last rows (the observation window that ranks a prompt's tokens)
        dict(name="weight-4x64-h64-10k", op="weight", B=4, rows=64, H=64, ctx=10007, page=16, window=0, sink=0, ragged=False, mix=8),
        # one token of each of 64 sequences joins its pages
        dict(name="append-64x1", op="append", B=64, rows=1, ctx=4096, page=64, ragged=False, mix=9),
        # prompts' chunks join their pages
        dict(name="append-4x4096", op="append", B=4, rows=4096, ctx=110000, page=48, ragged=True, mix=10),
        # budgeted caches, trimmed to their budget
        dict(name="evict-32-16k-to-8k", op="evict", B=32, ctx=16384, keep=8192, sink=4, recent=1024, page=64, ragged=True, mix=11),
        # one long prompt cut down to what decoding keeps
        dict(name="evict-1-131072-to-4096", op="evict", B=1, ctx=131072, keep=4096, sink=16, recent=512, page=64, ragged=False, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "weight", "append", "evict", "evict"])
    page = rng.choice([1, 16, 24, 32, 48, 64, 100, 128])
    ragged, mix = rng.random() < 0.6, rng.randrange(1 << 20)
    if op == "append":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, rows=_log(rng, 1, 16384 // B), ctx=_log(rng, 1, 20000), page=page, ragged=ragged, mix=mix)
    if op == "evict":
        B = _log(rng, 1, 64)
        ctx = _log(rng, 64, min(131072, 524288 // B))
        keep = max(1, int(ctx * rng.uniform(0.03, 0.9)))
        sink = rng.randint(0, min(16, keep // 4))
        return dict(op=op, B=B, ctx=ctx, keep=keep, sink=sink, recent=rng.randint(0, keep // 2), page=page, ragged=ragged, mix=mix)
    H = rng.choice([1, 8, 16, 24, 32, 64, 128])
    B = _log(rng, 1, 64)
    rows = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
    most = 2.0e9 if op == "attn" else 1.0e9       # padded (row, head, token) triples: under the largest listed case's
    rows = max(1, min(rows, int(most / (B * H * 1000))))
    ctx = _log(rng, 1, max(2, min(100000, 1200000 // B, int(most / (B * H * rows)) - rows)))
    window = _log(rng, 1, 4096) if rng.random() < 0.45 else 0
    return dict(op=op, B=B, rows=rows, H=H, ctx=ctx, page=page, window=window, sink=rng.choice([0, 1, 4, 64, 130]) if window else 0,
                ragged=ragged, mix=mix)


def _sizes(case):
    """(new rows, lengths with them) of the sequences, from the case alone."""
    r = random.Random(case["mix"])
    B, R, ctx = case["B"], case.get("rows", 0), case["ctx"]
    rows, lens = [], []
    for b in range(B):
        n = R if not case["ragged"] or b == 0 or R < 2 else r.choice([0, 1, r.randint(1, R), r.randint(1, R)])
        c = ctx if not case["ragged"] or b == 0 else r.randint(ctx // 2, ctx)
        rows.append(n)
        lens.append(n + c)
    return rows, lens


# ---------------------------------------------------------------- what a program has in hand
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev = dict(device="cuda")
    rows, lens = _sizes(case)
    B, ps, T = case["B"], case["page"], sum(rows)
    max_len = max(lens)
    npg = -(-max_len // ps)
    n_pages = B * npg + 1
    perm = torch.randperm(n_pages, generator=g, **dev).to(torch.int32)
    st = dict(case=case, B=B, T=T, ps=ps, max_len=max_len, max_rows=max(rows), table=perm[: B * npg].view(B, npg).contiguous(),
              seq_len=torch.tensor(lens, dtype=torch.int32, **dev))
    off = [0]
    for n in rows:
        off.append(off[-1] + n)
    st["row0"] = torch.tensor(off, dtype=torch.int32, **dev)

    def rows_of(n):   # cached rows: unit latents with a spread of magnitudes between tokens
        x = torch.randn((n, ROW), generator=g, **dev)
        return (x * torch.exp(0.3 * torch.randn((n, 1), generator=g, **dev))).to(torch.bfloat16)

    if case["op"] == "append":
        st["rows"] = rows_of(T)
        st["pool"] = torch.zeros((n_pages * ps, ROW), dtype=torch.bfloat16, **dev)
        return st
    if case["op"] == "evict":
        # accumulated weights: heavy-tailed, many tokens that never received any (ties)
        acc = torch.exp(2.0 * torch.randn((B, max_len), generator=g, **dev))
        st["acc"] = torch.where(torch.rand((B, max_len), generator=g, **dev) < 0.3, torch.zeros_like(acc), acc)
        nk = -(-case["keep"] // ps)
        st["pool"] = torch.cat([rows_of(n_pages * ps), torch.zeros(((B * nk + 1) * ps, ROW), dtype=torch.bfloat16, **dev)])
        dst = n_pages + torch.randperm(B * nk, generator=g, **dev).to(torch.int32)
        st["dst"] = torch.full((B, npg), -1, dtype=torch.int32, **dev)
        st["dst"][:, : min(nk, npg)] = dst.view(B, nk)[:, : min(nk, npg)]
        return st
    st["pool"] = rows_of(n_pages * ps)
    st["q"] = torch.randn((T, case["H"], ROW), generator=g, **dev).to(torch.bfloat16)
    if case["op"] == "weight":
        st["acc"] = torch.rand((B, max_len), generator=g, **dev)
        s, vis, _ = _scores(st)
        m = s.masked_fill(~vis, -math.inf).amax(-1, keepdim=True)
        l = (m + (s - m).exp().mul(vis).sum(-1, keepdim=True).log()).squeeze(-1)
        st["lse"] = _flat(st, l).contiguous()
    return st


# ---------------------------------------------------------------- plain forms
def _slots(st, table, n):
    t = torch.arange(n, device="cuda")
    return table[:, t // st["ps"]].long() * st["ps"] + t % st["ps"]


def _scores(st):
    """Scaled scores [B, rows, H, tokens] in 32 bits, which of them count [B, rows, 1, tokens], the keys [B, tokens, 576]."""
    case, B, L, R, H = st["case"], st["B"], st["max_len"], st["max_rows"], st["case"]["H"]
    k = st["pool"][_slots(st, st["table"], L)].float()
    n = (st["row0"][1:] - st["row0"][:-1]).view(B, 1)
    i = torch.arange(R, device="cuda").view(1, R)
    q = st["q"][(st["row0"][:-1].view(B, 1) + i).clamp(max=st["T"] - 1).long()].float()
    s = torch.matmul(q.view(B, R * H, ROW), k.transpose(1, 2)).view(B, R, H, L).mul_(SCALE)
    p = (st["seq_len"].view(B, 1) - n + i).view(B, R, 1, 1)
    t = torch.arange(L, device="cuda")
    vis = (t <= p) & (i < n).view(B, R, 1, 1)
    if case["window"]:
        vis &= (t > p - case["window"]) | (t < case["sink"])
    return s, vis, k


def _flat(st, x):
    """[B, rows, ...] -> the batch's rows one after another [T, ...]."""
    t = torch.arange(st["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(st["row0"][1:], t, right=True)
    return x[b, (t - st["row0"][b]).long()]


def _plain_attn(st):
    s, vis, k = _scores(st)
    B, R, H, L = s.shape
    s = s.masked_fill_(~vis, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, R * H, L), k[..., :VAL]).view(B, R, H, VAL) / torch.where(l == 0, torch.ones_like(l), l)
    return _flat(st, o.to(torch.bfloat16)), _flat(st, (m + l.log()).squeeze(-1))


def _plain_weight(st):
    s, vis, _ = _scores(st)
    B, R, H, L = s.shape
    i = (st["row0"][:-1].view(B, 1) + torch.arange(R, device="cuda").view(1, R)).clamp(max=st["T"] - 1).long()
    w = s.sub_(st["lse"][i].unsqueeze(-1)).exp_().masked_fill_(~vis, 0.0).view(B, R * H, L).sum(1)
    t = torch.arange(L, device="cuda")
    return torch.where(t < st["seq_len"].view(B, 1), st["acc"] * 0.9 + w, torch.zeros_like(w))


def _plain_append(st):
    t = torch.arange(st["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(st["row0"][1:], t, right=True)
    p = (st["seq_len"][b] - st["row0"][b + 1] + t).long()
    st["pool"][st["table"][b, p // st["ps"]].long() * st["ps"] + p % st["ps"]] = st["rows"]
    return st["pool"]


def _plain_evict(st):
    case, B, L = st["case"], st["B"], st["max_len"]
    keep, n = case["keep"], st["seq_len"].view(B, 1)
    t = torch.arange(L, device="cuda").view(1, L)
    a = st["acc"].masked_fill((t < case["sink"]) | (t >= n - case["recent"]), math.inf).masked_fill(t >= n, -math.inf)
    order = torch.sort(a, dim=1, descending=True, stable=True).indices[:, :keep]
    new_len = st["seq_len"].clamp(max=keep)
    W = order.shape[1]
    j = torch.arange(W, device="cuda").view(1, W)
    order = torch.where(j < new_len.view(B, 1), order, L).sort(dim=1).values
    live = order < L
    at = order.clamp(max=L - 1)
    kept = torch.full((B, keep), -1, dtype=torch.int32, device="cuda")
    kept[:, :W] = torch.where(live, order, -1)
    acc = torch.zeros_like(st["acc"])
    acc[:, :W] = torch.where(live, st["acc"].gather(1, at), 0.0)
    spare = st["pool"].shape[0] - 1   # a slot of no sequence: places that stay free move it onto itself
    src = torch.where(live, _slots(st, st["table"], L).gather(1, at), spare)
    dst = torch.where(live, _slots(st, st["dst"], W), spare)
    st["pool"][dst.view(-1)] = st["pool"][src.view(-1)]
    return st["pool"], kept, new_len, acc


def run(st):
    case, op = st["case"], st["case"]["op"]
    if not own:
        return {"attn": _plain_attn, "weight": _plain_weight, "append": _plain_append, "evict": _plain_evict}[op](st)
    import indexer_top_kv_amd as ech
    dev = dict(device="cuda")
    if op == "append":
        ech.ech_paged_append(st["pool"], st["table"], st["ps"], st["row0"], st["seq_len"], st["rows"])
        return st["pool"]
    if op == "evict":
        if "ws" not in st:   # kept by the program for as long as its shapes stay
            st["ws"] = torch.empty(ech.ech_paged_evict_ws_bytes(st["B"], st["max_len"], case["keep"]), dtype=torch.uint8, **dev)
            st["kept"] = torch.empty((st["B"], case["keep"]), dtype=torch.int32, **dev)
            st["len_out"] = torch.empty_like(st["seq_len"])
            st["acc_out"] = torch.empty_like(st["acc"])
        ech.ech_paged_evict(st["acc"], st["seq_len"], st["max_len"], case["keep"], case["sink"], case["recent"], st["kept"],
                            st["len_out"], acc_out=st["acc_out"], pool=st["pool"], src_table=st["table"], dst_table=st["dst"],
                            page_size=st["ps"], ws=st["ws"])
        return st["pool"], st["kept"], st["len_out"], st["acc_out"]
    H, T, B = case["H"], st["T"], st["B"]
    if op == "attn":
        if "ws" not in st:
            st["ws"] = torch.empty(ech.ech_paged_attn_ws_bytes(B, T, H, st["max_rows"], st["max_len"], case["window"], case["sink"]),
                                   dtype=torch.uint8, **dev)
            st["out"] = torch.empty((T, H, VAL), dtype=torch.bfloat16, **dev)
            st["lse"] = torch.empty((T, H), dtype=torch.float32, **dev)
        ech.ech_paged_attn(st["q"], st["pool"], st["table"], st["ps"], st["row0"], st["seq_len"], st["max_rows"], st["max_len"],
                           SCALE, st["out"], st["lse"], window=case["window"], n_sink=case["sink"], ws=st["ws"])
        return st["out"], st["lse"]
    if "ws" not in st:
        st["ws"] = torch.empty(ech.ech_paged_weight_ws_bytes(B, T, H, st["max_rows"], st["max_len"]), dtype=torch.uint8, **dev)
        st["acc_out"] = torch.zeros_like(st["acc"])
    ech.ech_paged_weight(st["q"], st["lse"], st["pool"], st["table"], st["ps"], st["row0"], st["seq_len"], st["max_rows"],
                         st["max_len"], SCALE, st["acc"], st["acc_out"], decay=0.9, window=case["window"], n_sink=case["sink"],
                         ws=st["ws"])
    return st["acc_out"]


# ---------------------------------------------------------------- what a pass cannot do without
def _seen(case, n, length):
    """(pairs of a new row and a token it sees, tokens that some new row sees) of one sequence."""
    w, s = case["window"], case["sink"]
    if not n:
        return 0, 0
    p0, p1 = length - n, length - 1
    if not w:
        return sum_to(p1 + 1) - sum_to(p0), length
    pairs = sum(min(p + 1, w) + min(s, max(0, p + 1 - w)) for p in range(p0, p1 + 1))
    lo = max(0, p0 - w + 1)
    return pairs, length - lo + min(s, lo)


def sum_to(n):
    return n * (n + 1) // 2


def work(case):
    rows, lens = _sizes(case)
    T = sum(rows)
    if case["op"] == "append":
        return {"bytes": 2 * T * ROW * 2 + 4 * T // case["page"] + 8 * case["B"], "flops": 0}
    if case["op"] == "evict":
        kept = sum(min(case["keep"], n) for n in lens)
        return {"bytes": 4 * sum(lens) + kept * (2 * ROW * 2 + 4) + 4 * case["B"] * max(lens), "flops": 0}
    H = case["H"]
    pairs = tokens = 0
    for n, length in zip(rows, lens):
        p, t = _seen(case, n, length)
        pairs, tokens = pairs + p, tokens + t
    if case["op"] == "weight":
        return {"bytes": T * H * (ROW * 2 + 4) + tokens * ROW * 2 + 8 * sum(lens), "flops": 2 * pairs * H * ROW}
    return {"bytes": T * H * (ROW * 2 + VAL * 2 + 4) + tokens * ROW * 2, "flops": 2 * pairs * H * (ROW + VAL)}


# ---------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    rows, lens = _sizes(case)
    ps, table, pool = st["ps"], st["table"].cpu(), st["pool"]
    if case["op"] in ("append", "evict"):
        return None          # values that move as they are: nothing is computed
    H, first = case["H"], 0
    q = st["q"].to(torch.float64)
    out = torch.zeros((st["T"], H, VAL), dtype=torch.float64, device="cuda")
    lse = torch.full((st["T"], H), -math.inf, dtype=torch.float64, device="cuda")
    acc = torch.zeros((st["B"], st["max_len"]), dtype=torch.float64, device="cuda")
    for b, (n, length) in enumerate(zip(rows, lens)):
        at = [int(table[b, t // ps]) * ps + t % ps for t in range(length)]
        kv = pool[torch.tensor(at, dtype=torch.int64, device="cuda")].to(torch.float64)
        if case["op"] == "weight":
            acc[b, :length] = st["acc"][b, :length].to(torch.float64) * float(torch.tensor(0.9, dtype=torch.float32))
        step = max(1, (1 << 28) // (H * length))
        for i0 in range(0, n, step):
            m = min(step, n - i0)
            pos = torch.arange(length - n + i0, length - n + i0 + m, device="cuda").view(m, 1, 1)
            tok = torch.arange(length, device="cuda").view(1, 1, length)
            hidden = tok > pos
            if case["window"]:
                hidden = hidden | ((pos - tok >= case["window"]) & (tok >= case["sink"]))
            here = slice(first + i0, first + i0 + m)
            sc = (q[here].reshape(m * H, ROW) @ kv.t()).view(m, H, length) * float(torch.tensor(SCALE, dtype=torch.float32))
            sc = sc.masked_fill(hidden, -math.inf)
            if case["op"] == "weight":
                acc[b, :length] += torch.exp(sc - st["lse"][here].to(torch.float64).unsqueeze(-1)).sum((0, 1))
            else:
                lse[here] = torch.logsumexp(sc, -1)
                out[here] = (torch.softmax(sc, -1).view(m * H, length) @ kv[:, :VAL]).view(m, H, VAL)
        first += n
    return acc if case["op"] == "weight" else (out, lse)
