"""What the operators for drafted tokens and for the pages of a cache cost: cases, plain forms
and 64-bit values.

Four operators around per-head variable-length pages: the attention of a tree of drafted
tokens per sequence (``tree``), the accepted path of a draft moved together (``accept``),
sequences that go on as several (``fork``) and the pages that no row names any more taken
back (``reclaim``).  With ``own`` false ``run`` computes them from elementary torch operations
in 32 bits; with ``own`` true it makes the library's calls.

Row r = (l * H_kv + hk) * B + b of a cache is KV head hk of layer l of sequence b.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one user's chat turn: 8 drafted tokens, one layer, a pruned prompt of about 600 tokens a
        # head; latency
        dict(name="tree_one_short", op="tree", L=1, B=1, H_q=32, H_kv=8, d=128, T=2048,
             keep_lo=0.2, keep_hi=0.4, w=0, page=16, m_lo=8, m_hi=8, chain=False),
        # 64 sequences with 1 to 16 drafted tokens each, prompts of up to 2048 tokens
        dict(name="tree_batch", op="tree", L=1, B=64, H_q=32, H_kv=8, d=128, T=2048,
             keep_lo=0.3, keep_hi=0.7, w=0, page=16, m_lo=1, m_hi=16, chain=False),
        # drafts in a line, six query heads per KV head, an odd page size, the window ring of 128
        dict(name="tree_chain_g6_ring", op="tree", L=1, B=33, H_q=12, H_kv=2, d=128, T=2048,
             keep_lo=0.3, keep_hi=0.7, w=128, page=13, m_lo=5, m_hi=5, chain=True),
        # one long document of 131072 tokens pruned to 10 to 50 % per head, 64 drafted tokens
        dict(name="tree_one_long", op="tree", L=1, B=1, H_q=32, H_kv=8, d=128, T=131072,
             keep_lo=0.1, keep_hi=0.5, w=0, page=16, m_lo=64, m_hi=64, chain=False),
        # wide trees at head dimension 64: 150 to 256 tokens, two query heads per KV head
        dict(name="tree_wide_d64", op="tree", L=2, B=8, H_q=16, H_kv=8, d=64, T=16384,
             keep_lo=0.1, keep_hi=1.0, w=0, page=16, m_lo=150, m_hi=256, chain=False),
        # a full serving batch: 96 sequences of 16384 tokens, heads kept at 25 to 75 %, 16 drafts
        dict(name="tree_batch_long", op="tree", L=1, B=96, H_q=32, H_kv=8, d=128, T=16384,
             keep_lo=0.25, keep_hi=0.75, w=0, page=16, m_lo=16, m_hi=16, chain=False),
        # the accepted paths of four users' drafts, all 36 layers at once
        dict(name="accept_few", op="accept", L=36, B=4, H_kv=8, d=128, T=512, page=16, m_lo=16,
             m_hi=16, most=6),
        # the same of 64 sequences, ragged drafts of up to 64 tokens, 8 layers
        dict(name="accept_batch", op="accept", L=8, B=64, H_kv=8, d=128, T=300, page=16, m_lo=1,
             m_hi=64, most=32),
        # one prompt sampled four times, 4 layers
        dict(name="fork_one", op="fork", L=4, B=4, forks=3, H_kv=8, d=128, T=2048, page=16, w=0),
        # half of the beams of a batch replaced by copies of others, with their window rings
        dict(name="fork_beams", op="fork", L=8, B=64, forks=31, H_kv=8, d=128, T=300, page=16, w=128),
        # after a step of speculation: every row has a page or two too many
        dict(name="reclaim_step", op="reclaim", L=4, B=8, H_kv=8, d=128, T=600, page=16, gone=0.0,
             spare=2),
        # a third of a batch has finished: their pages come free, the others move to the front
        dict(name="reclaim_third", op="reclaim", L=4, B=32, H_kv=8, d=128, T=1024, page=16,
             gone=0.34, spare=1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "accept", "fork", "reclaim"])
    d = rng.choice([64, 128, 128])
    H_kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([1, 8, 13, 16, 16, 64])
    L = rng.choice([1, 1, 2, 4])
    if op == "tree":
        B, T = _log_int(rng, 1, 96), _log_int(rng, 64, 131072)
        T = max(1, min(T, 96 * 16384 * 4 // (L * B * H_kv)))
        H_q = H_kv * rng.choice([1, 2, 4, 6, 8])
        most = max(1, min(256, 96 * 16384 * 128 // (L * B * T * H_q)))  # fewer products than the largest
        m_hi = _log_int(rng, 1, most)
        lo = rng.uniform(0.0, 0.6)
        return dict(op=op, L=L, B=B, H_q=H_q, H_kv=H_kv, d=d, T=T, keep_lo=lo,
                    keep_hi=rng.uniform(lo, 0.75), w=rng.choice([0, 0, 16, 128]), page=page,
                    m_lo=rng.randint(1, m_hi), m_hi=m_hi, chain=rng.random() < 0.25)
    B = _log_int(rng, 2, 64)
    if op == "accept":
        m_hi = _log_int(rng, 1, 256)
        return dict(op=op, L=L, B=B, H_kv=H_kv, d=d, T=_log_int(rng, 16, 1024), page=page,
                    m_lo=rng.randint(0, m_hi), m_hi=m_hi, most=rng.randint(1, m_hi))
    if op == "fork":
        return dict(op=op, L=L, B=B, forks=rng.randint(1, B // 2), H_kv=H_kv, d=d,
                    T=_log_int(rng, 16, 1024), page=page, w=rng.choice([0, 0, 16, 128]))
    return dict(op=op, L=L, B=B, H_kv=H_kv, d=d, T=_log_int(rng, 16, 2048), page=page,
                gone=rng.choice([0.0, 0.2, 0.5, 0.9]), spare=rng.randint(0, 3))


# ----------------------------------------------------------------------------- inputs

def _scales(gen, *shape):
    """Per-channel scales, log-uniform in [0.5, 4]."""
    u = torch.rand(*shape, generator=gen, device=DEV)
    return torch.exp(math.log(0.5) + u * (math.log(4.0) - math.log(0.5)))


def _drafts(c):
    """The drafted tokens of each sequence, from the case alone."""
    rng = np.random.RandomState(c["T"] * 3 + c["B"])
    m = rng.randint(c["m_lo"], c["m_hi"] + 1, size=c["B"])
    m[0] = c["m_hi"]
    return m


def _lengths(c):
    """The tokens of each row (drafts included) and those in its ring, from the case alone."""
    rng = np.random.RandomState(c["T"] * 7 + c["B"])
    shape = (c["L"], c["H_kv"], c["B"])
    if c["op"] == "tree":
        share = rng.uniform(c["keep_lo"], c["keep_hi"], size=shape)
        span = rng.randint((c["T"] + 1) // 2, c["T"] + 1, size=c["B"])
        span[0] = c["T"]
        n = np.floor(share * span) + _drafts(c)
    else:
        n = rng.randint(0, c["T"] + 1, size=shape)
        if c["op"] == "accept":
            n = n + _drafts(c)
        if c["op"] == "reclaim":  # the sequences that have finished
            n = n * (rng.uniform(size=c["B"]) >= c["gone"])
    pos = rng.randint(0, 3 * c.get("w", 0) + 1, size=c["B"]).astype(np.int32)
    return n.astype(np.int32), pos


def _paths(c):
    """How many drafted tokens of each sequence are accepted, and which."""
    rng = np.random.RandomState(c["T"] * 11 + c["B"])
    m = _drafts(c)
    count = np.minimum(rng.randint(0, c["most"] + 1, size=c["B"]), m)
    which = [np.sort(rng.permutation(x)[:k]) for x, k in zip(m, count)]
    return m, count, which


def _forks(c):
    """Sources and targets of the forks: no target is a source or another's target."""
    rng = np.random.RandomState(c["T"] * 13 + c["B"])
    order = rng.permutation(c["B"])
    dst = order[: c["forks"]]
    return rng.choice(order[c["forks"]:], size=c["forks"]), dst


def _in_use(c):
    """Pages of a row, the pages handed out for it (spare ones and the finished rows' own
    among them), and their sum."""
    n, _ = _lengths(c)
    need = -(-n // c["page"])
    if c["op"] != "reclaim":
        return need, need, int(need.sum())
    rng = np.random.RandomState(c["T"] * 17 + c["B"])
    had = np.where(n > 0, need, -(-c["T"] // c["page"] // 2))
    handed = had + rng.randint(0, c["spare"] + 1, size=n.shape)
    return need, handed, int(handed.sum())


def _ids(c):
    """The page ids of every row, [rows, widest], -1 behind them: from the case alone."""
    need, handed, total = _in_use(c)
    mp = max(1, int(need.max()) + (2 if c["op"] == "fork" else 0))
    flat_need, flat = need.reshape(-1), handed.reshape(-1)
    # in the order in which a running server hands them out: scattered
    ids = np.random.RandomState(c["T"] * 19 + c["B"]).permutation(total).astype(np.int32)
    start = np.concatenate([[0], np.cumsum(flat)])[:-1]
    at = np.arange(mp)[None] < flat_need[:, None]
    bt = np.full((flat_need.size, mp), -1, dtype=np.int32)
    bt[at] = ids[(start[:, None] + np.arange(mp)[None])[at]]
    return bt, mp, total


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 29)
    s = dict(c)
    L, H_kv, B, d, ps = c["L"], c["H_kv"], c["B"], c["d"], c["page"]
    bf = lambda *shape: torch.randn(*shape, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
    i32 = lambda x: torch.from_numpy(np.asarray(x).astype(np.int32)).to(DEV)  # noqa: E731
    n, pos = _lengths(c)
    bt, mp, total = _ids(c)
    rows = L * H_kv * B
    cap = total + 3 + (L * H_kv * c["forks"] if c["op"] == "fork" else 0)
    s.update(mp=mp, cap=cap, total=total, n_seq=i32(n), bt=torch.from_numpy(bt).to(DEV).view(L, H_kv, B, mp),
             k_pages=bf(cap, ps, d), v_pages=bf(cap, ps, d),
             next=torch.full((1,), total, dtype=torch.int32, device=DEV))
    if own:
        from kv_cache_eviction_lse_gb300 import capi
        s["capi"], s["dm"] = capi, capi.dims(L, c.get("H_q", H_kv), H_kv, d)
    size = 0
    if c["op"] == "tree":
        H_q, w, m = c["H_q"], c["w"], _drafts(c)
        N = int(m.sum())
        s.update(N=N, max_draft=c["m_hi"], tok_start=i32(np.concatenate([[0], np.cumsum(m)])), pos=i32(pos))
        own_index = torch.arange(N, device=DEV) - s["tok_start"][:-1].long().repeat_interleave(i32(m).long())
        u = torch.rand(N, generator=gen, device=DEV, dtype=torch.float64)
        s["parent"] = None if c["chain"] else ((u * (own_index + 1)).floor().int() - 1)
        sk, sq = _scales(gen, d), _scales(gen, L, H_q, 1, d)
        s["q"] = (torch.randn(L, H_q, N, d, generator=gen, device=DEV) * sq).to(torch.bfloat16)
        s["k_pages"].mul_(sk.to(torch.bfloat16))
        s["ring_k"] = bf(L, H_kv, B, w, d).mul_(sk.to(torch.bfloat16)) if w else None
        s["ring_v"] = bf(L, H_kv, B, w, d) if w else None
        s["o"] = torch.empty(L, H_q, N, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(L, H_q, N, dtype=torch.float32, device=DEV)
        if own:
            size = capi.kvs_attn_tree_workspace_size(s["dm"], B, N)
    elif c["op"] == "accept":
        m, count, which = _paths(c)
        start = np.concatenate([[0], np.cumsum(m)])
        path = np.zeros(max(1, int(start[-1])), dtype=np.int32)
        for b in range(B):
            path[start[b]:start[b] + count[b]] = which[b]
        s.update(N=int(start[-1]), tok_start=i32(start), count=i32(count), path=i32(path),
                 n_out=torch.empty(L, H_kv, B, dtype=torch.int32, device=DEV))
    elif c["op"] == "fork":
        src, dst = _forks(c)
        w = c["w"]
        s.update(src=i32(src), dst=i32(dst), pos=i32(pos), next_out=torch.empty_like(s["next"]))
        s["ring_score"] = torch.randn(L, H_kv, B, w, generator=gen, device=DEV) if w else None
        s["ring_k"] = bf(L, H_kv, B, w, d) if w else None
        s["ring_v"] = bf(L, H_kv, B, w, d) if w else None
        if own:
            size = capi.kvs_fork_paged_workspace_size(s["dm"], B, c["forks"])
    else:
        s.update(bt_out=torch.empty_like(s["bt"]), next_out=torch.empty_like(s["next"]))
        if own:
            size = capi.kvs_reclaim_paged_workspace_size(s["dm"], B, cap)
    if size:
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    s["rows"] = rows
    return s


# ----------------------------------------------------------------------------- plain forms

def _plain_tree(s):
    L, H_q, N, d = s["q"].shape
    B, H_kv, ps, w, M = s["B"], s["H_kv"], s["page"], s["w"], s["max_draft"]
    rows, g = L * H_kv * B, H_q // H_kv
    start = s["tok_start"].long()
    m = start[1:] - start[:-1]
    # [B, M]: each sequence's tokens, its last one again behind them
    idx = torch.arange(M, device=DEV)
    tok = start[:-1, None] + torch.minimum(idx[None], (m[:, None] - 1).clamp(min=0))
    real = idx[None] < m[:, None]
    # which drafted tokens a token sees: itself and those above it, by squaring "itself or parent"
    parent = tok - start[:-1, None] - 1 if s["parent"] is None else s["parent"].long()[tok]
    sees = (idx[None, None] == idx[None, :, None]) | (idx[None, None] == parent[:, :, None])
    sees = sees.float()
    for _ in range(8):  # M <= 256
        sees = torch.bmm(sees, sees).clamp(max=1)
    n = s["n_seq"].reshape(rows)
    base = (s["n_seq"] - m.int()).reshape(rows).long()
    ids = s["bt"].reshape(rows, -1).clamp(min=0).long()
    k = s["k_pages"][ids].reshape(rows, -1, d)
    v = s["v_pages"][ids].reshape(rows, -1, d)
    key = torch.arange(k.shape[1], device=DEV)
    live = key[None] < n[:, None]
    if w:
        k = torch.cat([k, s["ring_k"].reshape(rows, w, d)], 1)
        v = torch.cat([v, s["ring_v"].reshape(rows, w, d)], 1)
        held = s["pos"].clamp(max=w).expand(L, H_kv, B).reshape(rows, 1)
        live = torch.cat([live, torch.arange(w, device=DEV)[None] < held], 1)
    k = k.masked_fill_(~live[..., None], 0.0).float()
    v = v.masked_fill_(~live[..., None], 0.0).float()
    q = s["q"].view(L, H_kv, g, N, d)[:, :, :, tok]               # [L, H_kv, g, B, M, d]
    q = q.permute(0, 1, 3, 4, 2, 5).reshape(rows, M * g, d).float()
    x = torch.bmm(q, k.transpose(1, 2)) / math.sqrt(d)
    del k
    # the drafts' columns: [rows, M, M] from slot base on
    col = base[:, None] + idx[None]
    seen = torch.ones(rows, M, v.shape[1] + M, dtype=torch.bool, device=DEV)
    seen.scatter_(2, col[:, None].expand(rows, M, M), sees.bool().repeat(L * H_kv, 1, 1))
    # columns behind a sequence's last draft belong to the ring again
    seen[:, :, : v.shape[1]] |= (torch.arange(v.shape[1], device=DEV)[None] >= n[:, None])[:, None]
    seen = seen[:, :, : v.shape[1]] & live[:, None]
    x = x.view(rows, M, g, -1).masked_fill_(~seen[:, :, None], -math.inf).view(rows, M * g, -1)
    del seen
    top = x.amax(-1, keepdim=True).clamp(min=-3.4e38)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p, v)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).to(torch.bfloat16)
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(top, -math.inf))
    back = lambda y: y.view(L, H_kv, B, M, g, -1).permute(0, 1, 4, 2, 3, 5)[:, :, :, real].reshape(L, H_q, N, -1)  # noqa: E731,E501
    return {"o": back(o), "lse": back(lse)[..., 0]}


def _slots(s, seq, slot):
    """Rows of the pool of slots [L, H_kv, X] of sequences [X]."""
    ps = s["page"]
    page = torch.gather(s["bt"][:, :, seq], 3, (slot // ps)[..., None])[..., 0].long()
    return (page * ps + slot % ps).reshape(-1)


def _plain_accept(s):
    d, start = s["d"], s["tok_start"].long()
    m = start[1:] - start[:-1]
    base = s["n_seq"].long() - m
    tok = torch.arange(s["N"], device=DEV)
    seq = torch.searchsorted(start[1:], tok, right=True)
    j = tok - start[seq]
    kept = j < s["count"].long()[seq]
    seq, j, path = seq[kept], j[kept], s["path"].long()[: s["N"]][kept]
    frm, to = _slots(s, seq, base[..., seq] + path), _slots(s, seq, base[..., seq] + j)
    pools = (s["k_pages"].view(-1, d), s["v_pages"].view(-1, d))
    pools[0][to] = pools[0][frm]
    pools[1][to] = pools[1][frm]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "seq_lens": (base + s["count"]).int()}


def _plain_fork(s):
    d, ps, mp = s["d"], s["page"], s["mp"]
    src, dst = s["src"].long(), s["dst"].long()
    n = s["n_seq"].long()[:, :, src]                              # [L, H_kv, forks]
    part = (n % ps > 0).reshape(-1)
    fresh = (s["next"].long() + part.long().cumsum(0) - part.long()).view_as(n)
    bt = s["bt"][:, :, src].long()
    page, last = torch.arange(mp, device=DEV), n // ps
    part = part.view_as(n)
    old = torch.gather(bt, 3, last.clamp(max=mp - 1)[..., None])[..., 0]
    bt = torch.where(page < -(-n // ps)[..., None], bt, torch.full_like(bt, -1))
    bt = torch.where((page == last[..., None]) & part[..., None], fresh[..., None], bt)
    row = torch.arange(ps, device=DEV)
    used = (row < (n % ps)[..., None])[part][..., None]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[fresh[part]] = torch.where(used, pool[old[part]], torch.zeros((), dtype=pool.dtype, device=DEV))
    s["bt"][:, :, dst] = bt.int()
    s["n_seq"][:, :, dst] = n.int()
    out = {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "block_table": s["bt"],
           "seq_lens": s["n_seq"], "next_page": (s["next"] + part.sum()).int()}
    if s["w"]:
        for name in ("ring_score", "ring_k", "ring_v"):
            s[name][:, :, dst] = s[name][:, :, src]
            out[name] = s[name]
        s["pos"][dst] = s["pos"][src]
        out["pos"] = s["pos"]
    return out


def _plain_reclaim(s):
    ps, cap = s["page"], s["cap"]
    need = -(-s["n_seq"] // ps)
    used = torch.arange(s["mp"], device=DEV) < need[..., None]
    live = torch.zeros(cap + 1, dtype=torch.bool, device=DEV)
    live[torch.where(used, s["bt"], cap).long().reshape(-1)] = True
    live = live[:cap]
    count = live.sum()
    at = torch.arange(cap, device=DEV)
    hole, mover = ~live & (at < count), live & (at >= count)
    new = at.clone()
    new[mover] = at[hole]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[new[mover]] = pool[mover]
    bt = torch.where(used, new[s["bt"].clamp(min=0).long()], torch.full((), -1, device=DEV))
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "block_table": bt.int(),
            "next_page": count.int().view(1)}


# ----------------------------------------------------------------------------- one pass

def run(state):
    s = state
    if not own:
        return {"tree": _plain_tree, "accept": _plain_accept, "fork": _plain_fork,
                "reclaim": _plain_reclaim}[s["op"]](s)
    C, pools = s["capi"], {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["op"] == "tree":
        C.kvs_attn_tree(s["dm"], s["B"], s["N"], s["max_draft"], s["tok_start"], s["parent"], s["q"],
                        s["page"], s["k_pages"], s["v_pages"], s["cap"], s["bt"], s["mp"], s["n_seq"],
                        s["w"], s["pos"], s["ring_k"], s["ring_v"], s["o"], s["lse"], s["ws"],
                        s["ws"].numel())
        return {"o": s["o"], "lse": s["lse"]}
    if s["op"] == "accept":
        C.kvs_accept_paged(s["dm"], s["B"], s["N"], s["tok_start"], s["count"], s["path"], s["page"],
                           s["k_pages"], s["v_pages"], s["cap"], s["bt"], s["mp"], s["n_seq"], s["n_out"])
        return {**pools, "seq_lens": s["n_out"]}
    if s["op"] == "fork":
        C.kvs_fork_paged(s["dm"], s["B"], s["forks"], s["src"], s["dst"], s["page"], s["k_pages"],
                         s["v_pages"], s["cap"], s["next"], s["next_out"], s["bt"], s["mp"], s["n_seq"],
                         s["w"], s["pos"] if s["w"] else None, s["ring_score"], s["ring_k"], s["ring_v"],
                         s["ws"], s["ws"].numel())
        out = {**pools, "block_table": s["bt"], "seq_lens": s["n_seq"], "next_page": s["next_out"]}
        if s["w"]:
            out.update(ring_score=s["ring_score"], ring_k=s["ring_k"], ring_v=s["ring_v"], pos=s["pos"])
        return out
    C.kvs_reclaim_paged(s["dm"], s["B"], s["page"], s["k_pages"], s["v_pages"], s["cap"], s["next"],
                        s["next_out"], s["bt"], s["bt_out"], s["mp"], s["n_seq"], s["ws"],
                        s["ws"].numel())
    return {**pools, "block_table": s["bt_out"], "next_page": s["next_out"]}


def work(case):
    c = case
    L, H_kv, B, d, ps = c["L"], c["H_kv"], c["B"], c["d"], c["page"]
    n, pos = _lengths(c)
    token = 2 * d * 2  # K and V
    pages = -(-n // ps)
    if c["op"] == "tree":
        m, g = _drafts(c).astype(np.int64), c["H_q"] // H_kv
        keys = n.sum((0, 1)) + L * H_kv * np.minimum(pos, c["w"])
        tokens = int(m.sum())
        io = L * c["H_q"] * tokens * (2 * d * 2 + 4) + n.size * 4 + int(pages.sum()) * 4 + 8 * tokens
        return {"bytes": int(keys.sum()) * token + io, "flops": int((keys * m).sum()) * 4 * d * g}
    if c["op"] == "accept":
        _, count, which = _paths(c)
        moved = sum(int((x != np.arange(x.size)).sum()) for x in which)
        return {"bytes": L * H_kv * (2 * moved * token + 8 * B) + 4 * int(count.sum()), "flops": 0}
    if c["op"] == "fork":
        src, _ = _forks(c)
        of = n[:, :, src]
        rest = of % ps
        fill = np.where(rest > 0, ps - rest, 0)
        ring = L * H_kv * c["forks"] * c["w"] * (token + 4)
        return {"bytes": int(2 * rest.sum() + fill.sum()) * token + 2 * ring + 8 * int(pages[:, :, src].sum())
                + 8 * of.size, "flops": 0}
    bt, _, _ = _ids(c)
    live = np.unique(bt[bt >= 0])
    moved = int((live >= live.size).sum())
    return {"bytes": 2 * moved * ps * token + 8 * int(pages.sum()) + 4 * n.size, "flops": 0}


# ----------------------------------------------------------------------------- 64 bits

def _exact_tree(s, case):
    n, pos = _lengths(case)
    m = _drafts(case)
    L, H_kv, B, ps, d = s["L"], s["H_kv"], s["B"], s["page"], s["d"]
    g, N = s["H_q"] // H_kv, s["N"]
    if n.size > 2048 or float((n.astype(np.float64) * m).sum()) * g > 4e9:
        return None
    o = torch.zeros(L, s["H_q"], N, d, dtype=torch.float64, device=DEV)
    lse = torch.full((L, s["H_q"], N), -math.inf, dtype=torch.float64, device=DEV)
    start = np.concatenate([[0], np.cumsum(m)])
    parents = None if s["parent"] is None else s["parent"].cpu().numpy()
    for b in range(B):
        mb, t0 = int(m[b]), int(start[b])
        path = np.zeros((mb, mb), dtype=bool)  # row i: the tokens on i's way up
        for i in range(mb):
            up = i - 1 if parents is None else int(parents[t0 + i])
            if up >= 0:
                path[i] = path[up]
            path[i, i] = True
        path = torch.from_numpy(path).to(DEV)
        for l in range(L):
            for h in range(H_kv):
                size = int(n[l, h, b])
                ids = s["bt"][l, h, b, : -(-size // ps)].long()
                k = s["k_pages"][ids].reshape(-1, d)[:size].double()
                v = s["v_pages"][ids].reshape(-1, d)[:size].double()
                held = min(int(pos[b]), s["w"])
                if held:
                    k = torch.cat([k, s["ring_k"][l, h, b, :held].double()])
                    v = torch.cat([v, s["ring_v"][l, h, b, :held].double()])
                heads = slice(h * g, (h + 1) * g)
                x = s["q"][l, heads, t0:t0 + mb].double() @ k.t() * d ** -0.5
                x[:, :, size - mb:size] = torch.where(path, x[:, :, size - mb:size], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[l, heads, t0:t0 + mb] = z
                o[l, heads, t0:t0 + mb] = torch.exp(x - z[..., None]) @ v
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "tree":
        return _exact_tree(s, case)
    if s["rows"] > 5000 or s["k_pages"].numel() > 1 << 27:
        return None
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    n, _ = _lengths(case)
    bt = s["bt"].cpu().numpy()
    ps, cells = s["page"], list(np.ndindex(s["L"], s["H_kv"]))
    if s["op"] == "accept":
        m, count, which = _paths(case)
        out = n.copy()
        for l, h in cells:
            for b in range(s["B"]):
                base = int(n[l, h, b]) - int(m[b])
                out[l, h, b] = base + count[b]
                if not count[b]:
                    continue
                frm, to = base + which[b], base + np.arange(count[b])
                frm = (torch.from_numpy(bt[l, h, b, frm // ps]).long(), torch.from_numpy(frm % ps).long())
                to = (torch.from_numpy(bt[l, h, b, to // ps]).long(), torch.from_numpy(to % ps).long())
                kp[to], vp[to] = kp[frm].clone(), vp[frm].clone()
        return {"k_pages": kp, "v_pages": vp, "seq_lens": torch.from_numpy(out)}
    if s["op"] == "fork":
        src, dst = _forks(case)
        nxt, lens = int(s["next"]), n.copy()
        for l, h in cells:
            for a, b in zip(src, dst):
                size = int(n[l, h, a])
                full, rest = size // ps, size % ps
                bt[l, h, b] = -1
                bt[l, h, b, :full] = bt[l, h, a, :full]
                lens[l, h, b] = size
                if rest:
                    bt[l, h, b, full] = nxt
                    for pool in (kp, vp):
                        pool[nxt] = 0.0
                        pool[nxt, :rest] = pool[bt[l, h, a, full], :rest]
                    nxt += 1
        out = {"k_pages": kp, "v_pages": vp, "block_table": torch.from_numpy(bt),
               "seq_lens": torch.from_numpy(lens), "next_page": torch.tensor([nxt], dtype=torch.int32)}
        if s["w"]:
            order = np.arange(s["B"])
            order[dst] = src
            order = torch.from_numpy(order).to(DEV)
            for name in ("ring_score", "ring_k", "ring_v"):
                out[name] = s[name][:, :, order].double()
            out["pos"] = s["pos"][order]
        return out
    need = -(-n // ps)
    flat, rows = bt.reshape(-1, s["mp"]), need.reshape(-1)
    live = sorted({int(p) for r in range(rows.size) for p in flat[r, : rows[r]]})
    holes = sorted(set(range(len(live))) - set(live))
    to = dict(zip([p for p in live if p >= len(live)], holes))
    for a, b in to.items():
        kp[b], vp[b] = kp[a].clone(), vp[a].clone()
    table = np.full_like(flat, -1)
    for r in range(rows.size):
        table[r, : rows[r]] = [to.get(int(p), int(p)) for p in flat[r, : rows[r]]]
    return {"k_pages": kp, "v_pages": vp, "block_table": torch.from_numpy(table.reshape(bt.shape)),
            "next_page": torch.tensor([len(live)], dtype=torch.int32)}
