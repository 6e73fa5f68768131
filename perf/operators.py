"""What the serving operators over the paged cache cost: cases, plain forms and 64-bit values.

Three operators of a decode loop over per-head variable-length pages: the position
rotation of queries and keys (``rope``), the append of new tokens to the paged cache with
that rotation on the way (``append``) and the attention of one new token per sequence over
the cache (``attend``).  With ``own`` false ``run`` computes them from elementary torch
operations in 32 bits (rotation angles in 64); with ``own`` true it makes the library's
calls.

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
        # one user's chat turn: one sequence, one layer, a pruned prompt of about 600 tokens a
        # head; latency
        dict(name="attend_one_short", op="attend", L=1, B=1, H_q=32, H_kv=8, d=128, T=2048,
             keep_lo=0.2, keep_hi=0.4, w=0, page=16),
        # a batch of 64 short decodes whose tokens still sit mostly in the window ring of 128
        # (the ring sizes of the decode workload), all 4 layers of one pipeline stage at once
        dict(name="attend_ring_batch", op="attend", L=4, B=64, H_q=32, H_kv=8, d=128, T=200,
             keep_lo=0.0, keep_hi=0.5, w=128, page=16),
        # six query heads per KV head, two KV heads, a ragged batch and an odd page size: prompts
        # of up to 2048 tokens at the keep ratios 0.3 to 0.7
        dict(name="attend_g6_odd_page", op="attend", L=1, B=33, H_q=12, H_kv=2, d=128, T=2048,
             keep_lo=0.3, keep_hi=0.7, w=0, page=13),
        # one long document of 131072 tokens pruned to 10 to 50 % per head: few rows, long axis
        dict(name="attend_one_long", op="attend", L=1, B=1, H_q=32, H_kv=8, d=128, T=131072,
             keep_lo=0.1, keep_hi=0.5, w=128, page=16),
        # head dimension 64 with two query heads per KV head, batch of 24
        dict(name="attend_d64", op="attend", L=2, B=24, H_q=16, H_kv=8, d=64, T=4096,
             keep_lo=0.1, keep_hi=1.0, w=16, page=16),
        # a full serving batch: 96 sequences of 16384 tokens, heads kept at 25 to 75 %
        dict(name="attend_batch_long", op="attend", L=1, B=96, H_q=32, H_kv=8, d=128, T=16384,
             keep_lo=0.25, keep_hi=0.75, w=128, page=16),
        # one new token of each of 64 sequences into one layer's cache
        dict(name="append_token_batch", op="append", L=1, B=64, N=64, single=True, H_q=32, H_kv=8,
             d=128, n_max=4096, rot=128, interleaved=False, page=16),
        # one chunk of prompts of several users, ragged (empty and one-token ones among them),
        # over 4 layers
        dict(name="append_chunk_ragged", op="append", L=4, B=7, N=8192, single=False, H_q=32,
             H_kv=8, d=128, n_max=1000, rot=128, interleaved=False, page=16),
        # a short prompt, half of each head rotated in interleaved pairs, odd page size
        dict(name="append_partial_d64", op="append", L=1, B=3, N=517, single=False, H_q=16, H_kv=8,
             d=64, n_max=300, rot=32, interleaved=True, page=13),
        # one new token of each of 64 sequences before a pruning decode step
        dict(name="rope_token_batch", op="rope", L=1, N=64, H_q=32, H_kv=8, d=128, rot=128,
             interleaved=False),
        # a prompt of 16384 tokens, two layers
        dict(name="rope_prompt", op="rope", L=2, N=16384, H_q=32, H_kv=8, d=128, rot=128,
             interleaved=False),
        # interleaved pairs, odd length, twelve and two heads
        dict(name="rope_interleaved_odd", op="rope", L=1, N=2079, H_q=12, H_kv=2, d=128, rot=128,
             interleaved=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "append", "rope"])
    d = rng.choice([64, 128, 128])
    H_kv = rng.choice([1, 2, 4, 8])
    H_q = H_kv * rng.choice([1, 2, 4, 6, 8])
    page = rng.choice([1, 8, 13, 16, 16, 64])
    if op == "attend":
        B, T, L = _log_int(rng, 1, 96), _log_int(rng, 64, 131072), rng.choice([1, 1, 2, 4])
        T = max(1, min(T, 96 * 16384 * 4 // (L * B * H_kv)))
        lo = rng.uniform(0.0, 0.6)
        return dict(op=op, L=L, B=B, H_q=H_q, H_kv=H_kv, d=d, T=T, keep_lo=lo,
                    keep_hi=rng.uniform(lo, 0.75), w=rng.choice([0, 0, 16, 128]), page=page)
    rot = rng.choice([d, d, d // 2])
    N, L = _log_int(rng, 1, 8192), rng.choice([1, 1, 2, 4])
    if op == "append":
        B = _log_int(rng, 1, 64)
        single = rng.random() < 0.3
        return dict(op=op, L=L, B=B, N=B if single else N, single=single, H_q=H_q, H_kv=H_kv, d=d,
                    n_max=_log_int(rng, 1, 2048), rot=rot, interleaved=rng.random() < 0.3, page=page)
    return dict(op=op, L=L, N=N, H_q=H_q, H_kv=H_kv, d=d, rot=rot, interleaved=rng.random() < 0.4)


# ----------------------------------------------------------------------------- inputs

def _inv_freq(rot):
    """The usual geometric frequencies, base 1e6, as the 32-bit buffer that a model keeps."""
    f = 1e6 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot) if rot else np.zeros(0)
    return torch.from_numpy(f.astype(np.float32).astype(np.float64))


def _scales(gen, *shape):
    """Per-channel scales, log-uniform in [0.5, 4]."""
    u = torch.rand(*shape, generator=gen, device=DEV)
    return torch.exp(math.log(0.5) + u * (math.log(4.0) - math.log(0.5)))


def _lengths(c):
    """The kept tokens of each row of an attend case, and of its rings: from the case alone."""
    rng = np.random.RandomState(c["T"] * 7 + c["B"])
    share = rng.uniform(c["keep_lo"], c["keep_hi"], size=(c["L"], c["H_kv"], c["B"]))
    span = rng.randint((c["T"] + 1) // 2, c["T"] + 1, size=c["B"])
    span[0] = c["T"]
    n = np.floor(share * span[None, None]).astype(np.int32)
    pos = rng.randint(0, 3 * c["w"] + 1, size=c["B"]).astype(np.int32)
    return n, pos


def _chunks(c):
    """The first token of each sequence of an append case, and the rows' lengths before it."""
    rng = np.random.RandomState(c["N"] * 5 + c["B"])
    if c["single"]:
        m = np.ones(c["B"], dtype=np.int64)
    else:
        cut = np.sort(rng.randint(0, c["N"] + 1, size=c["B"] - 1))
        m = np.diff(np.concatenate([[0], cut, [c["N"]]]))
    n = rng.randint(0, c["n_max"] + 1, size=(c["L"], c["H_kv"], c["B"])).astype(np.int32)
    return m, n


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 17)
    s = dict(c)
    if own:
        from kv_cache_eviction_lse_gb300 import capi
        s["capi"], s["dm"] = capi, capi.dims(c["L"], c["H_q"], c["H_kv"], c["d"])
    bf = lambda *shape: torch.randn(*shape, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
    L, H_q, H_kv, d = c["L"], c["H_q"], c["H_kv"], c["d"]
    if c["op"] == "attend":
        B, w, ps = c["B"], c["w"], c["page"]
        n, pos = _lengths(c)
        need = -(-n // ps)
        total, mp = int(need.sum()), max(1, int(need.max()))
        cap = total + 3
        s.update(n_seq=torch.from_numpy(n).to(DEV), pos=torch.from_numpy(pos).to(DEV), mp=mp, cap=cap)
        # pages in the order in which a running server hands them out: scattered
        ids = torch.randperm(cap, generator=gen, device=DEV)[:total].to(torch.int32)
        at = torch.arange(mp, device=DEV)[None] < torch.from_numpy(need.reshape(-1, 1)).to(DEV)
        bt = torch.full((L * H_kv * B, mp), -1, dtype=torch.int32, device=DEV)
        bt[at] = ids
        s["bt"] = bt.view(L, H_kv, B, mp)
        sk, sq = _scales(gen, d), _scales(gen, L, H_q, 1, d)
        s["q"] = (torch.randn(L, H_q, B, d, generator=gen, device=DEV) * sq).to(torch.bfloat16)
        s["k_pages"], s["v_pages"] = bf(cap, ps, d), bf(cap, ps, d)
        s["k_pages"].mul_(sk.to(torch.bfloat16))
        s["ring_k"] = bf(L, H_kv, B, w, d).mul_(sk.to(torch.bfloat16)) if w else None
        s["ring_v"] = bf(L, H_kv, B, w, d) if w else None
        s["o"] = torch.empty(L, H_q, B, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(L, H_q, B, dtype=torch.float32, device=DEV)
        if own:
            size = capi.kvs_attn_decode_workspace_size(s["dm"], B)
            s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        return s
    N = c["N"]
    s["inv_freq"] = _inv_freq(c["rot"])
    s["q"], s["k"] = bf(L, H_q, N, d), bf(L, H_kv, N, d)
    s["q_out"] = torch.empty_like(s["q"])
    if c["op"] == "rope":
        s["k_out"] = torch.empty_like(s["k"])
        s["pos"] = torch.randint(0, 131072, (N,), generator=gen, device=DEV, dtype=torch.int32)
        return s
    B, ps = c["B"], c["page"]
    m, n = _chunks(c)
    have, end = -(-n // ps), -(-(n + m[None, None]) // ps)
    total, mp = int(have.sum()), int(end.max()) + 2
    cap = int(end.sum()) + 3
    s.update(mp=mp, cap=cap, v=bf(L, H_kv, N, d))
    s["tok_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(m)]).astype(np.int32)).to(DEV)
    s["n_seq"] = torch.from_numpy(n).to(DEV)
    bt = torch.full((L * H_kv * B, mp), -1, dtype=torch.int32, device=DEV)
    at = torch.arange(mp, device=DEV)[None] < torch.from_numpy(have.reshape(-1, 1)).to(DEV)
    bt[at] = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    s["bt"] = bt.view(L, H_kv, B, mp)
    s["next"] = torch.full((1,), total, dtype=torch.int32, device=DEV)
    # a token's position is past its row's length: the cache was pruned
    first = torch.randint(4096, 100000, (B,), generator=gen, device=DEV)
    tok = torch.arange(N, device=DEV)
    seq = torch.searchsorted(s["tok_start"][1:].long(), tok, right=True)
    s["pos"] = (first[seq] + tok - s["tok_start"].long()[seq]).to(torch.int32)
    s["k_pages"], s["v_pages"] = bf(cap, ps, d), bf(cap, ps, d)
    s["n_out"], s["next_out"] = torch.empty_like(s["n_seq"]), torch.empty_like(s["next"])
    if own:
        size = capi.kvs_append_paged_workspace_size(s["dm"], B)
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s


# ----------------------------------------------------------------------------- plain forms

def _plain_rotate(x, pos, inv_freq, rot, interleaved):
    """x [..., N, d] rotated at pos [N]; angles in 64 bits, the products in 32."""
    angle = pos.double()[:, None] * inv_freq.to(x.device)[None]
    cos, sin = angle.cos().float(), angle.sin().float()
    y = x.float()
    r, rest = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., : rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1).to(torch.bfloat16)


def _plain_attend(s):
    L, H_q, B, d = s["q"].shape
    H_kv, ps, w = s["H_kv"], s["page"], s["w"]
    rows, g = L * H_kv * B, H_q // H_kv
    n = s["n_seq"].reshape(rows)
    ids = s["bt"].reshape(rows, -1).clamp(min=0).long()
    k = s["k_pages"][ids].reshape(rows, -1, d)
    v = s["v_pages"][ids].reshape(rows, -1, d)
    live = torch.arange(k.shape[1], device=DEV)[None] < n[:, None]
    if w:
        k = torch.cat([k, s["ring_k"].reshape(rows, w, d)], 1)
        v = torch.cat([v, s["ring_v"].reshape(rows, w, d)], 1)
        held = s["pos"].clamp(max=w).expand(L, H_kv, B).reshape(rows, 1)
        live = torch.cat([live, torch.arange(w, device=DEV)[None] < held], 1)
    k = k.masked_fill_(~live[..., None], 0.0).float()
    q = s["q"].view(L, H_kv, g, B, d).transpose(2, 3).reshape(rows, g, d).float()
    x = torch.bmm(q, k.transpose(1, 2)) / math.sqrt(d)
    del k
    x.masked_fill_(~live[:, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3.4e38)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p, v.masked_fill_(~live[..., None], 0.0).float())
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).to(torch.bfloat16)
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(top, -math.inf))
    back = lambda y: y.view(L, H_kv, B, g, -1).transpose(2, 3).reshape(L, H_q, B, -1).contiguous()  # noqa: E731
    return {"o": back(o), "lse": back(lse)[..., 0]}


def _plain_append(s):
    L, H_kv, N, d = s["k"].shape
    ps, mp = s["page"], s["mp"]
    q = _plain_rotate(s["q"], s["pos"], s["inv_freq"], s["rot"], s["interleaved"])
    k = _plain_rotate(s["k"], s["pos"], s["inv_freq"], s["rot"], s["interleaved"])
    n, start = s["n_seq"].long(), s["tok_start"].long()
    m = start[1:] - start[:-1]
    have, end = (n + ps - 1) // ps, (n + m + ps - 1) // ps
    need = (end - have).reshape(-1)
    first = (s["next"].long() + need.cumsum(0) - need).view_as(n)
    page = torch.arange(mp, device=DEV)
    fresh = (page >= have[..., None]) & (page < end[..., None])
    bt = torch.where(fresh, first[..., None] + page - have[..., None], s["bt"].long())
    # the slots of the tokens, and the unused rows of the rows' last new pages
    tok = torch.arange(N, device=DEV)
    seq = torch.searchsorted(start[1:], tok, right=True)
    slot = n[..., seq] + tok - start[seq]
    at = torch.gather(bt[:, :, seq], 3, (slot // ps)[..., None])[..., 0] * ps + slot % ps
    tail = (n + m)[..., None] + torch.arange(ps, device=DEV)
    clear = (tail < (end * ps)[..., None]) & (end > have)[..., None]
    last = torch.gather(bt, 3, (end - 1).clamp(min=0)[..., None]) * ps + tail % ps
    clear_at = last[clear]
    pools = (s["k_pages"].view(-1, d), s["v_pages"].view(-1, d))
    pools[0][at.reshape(-1)] = k.reshape(-1, d)
    pools[1][at.reshape(-1)] = s["v"].reshape(-1, d)
    pools[0][clear_at] = 0.0
    pools[1][clear_at] = 0.0
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"], "block_table": bt.int(),
            "seq_lens": (n + m).int(), "next_page": (s["next"] + need.sum()).int()}


# ----------------------------------------------------------------------------- one pass

def run(state):
    s = state
    if own:
        C = s["capi"]
        if s["op"] == "attend":
            C.kvs_attn_decode(s["dm"], s["B"], s["q"], s["page"], s["k_pages"], s["v_pages"],
                              s["cap"], s["bt"], s["mp"], s["n_seq"], s["w"], s["pos"],
                              s["ring_k"], s["ring_v"], s["o"], s["lse"], s["ws"], s["ws"].numel())
            return {"o": s["o"], "lse": s["lse"]}
        if s["op"] == "append":
            C.kvs_append_paged(s["dm"], s["B"], s["N"], None if s["single"] else s["tok_start"],
                               s["pos"], s["rot"], s["inv_freq"], s["interleaved"], s["q"],
                               s["q_out"], s["k"], s["v"], s["page"], s["k_pages"], s["v_pages"],
                               s["cap"], s["next"], s["next_out"], s["bt"], s["mp"], s["n_seq"],
                               s["n_out"], s["ws"], s["ws"].numel())
            return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"],
                    "block_table": s["bt"], "seq_lens": s["n_out"], "next_page": s["next_out"]}
        C.kvs_rope(s["dm"], s["N"], s["pos"], s["rot"], s["inv_freq"], s["interleaved"], s["q"],
                   s["q_out"], s["k"], s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if s["op"] == "attend":
        return _plain_attend(s)
    if s["op"] == "append":
        return _plain_append(s)
    return {"q": _plain_rotate(s["q"], s["pos"], s["inv_freq"], s["rot"], s["interleaved"]),
            "k": _plain_rotate(s["k"], s["pos"], s["inv_freq"], s["rot"], s["interleaved"])}


def work(case):
    c = case
    L, H_q, H_kv, d = c["L"], c["H_q"], c["H_kv"], c["d"]
    if c["op"] == "attend":
        n, pos = _lengths(c)
        keys = int(n.sum()) + L * H_kv * int(np.minimum(pos, c["w"]).sum())
        pages = int((-(-n // c["page"])).sum())
        io = L * H_q * c["B"] * (2 * d * 2 + 4) + n.size * 4 + pages * 4
        return {"bytes": keys * 2 * d * 2 + io, "flops": 4 * d * keys * (H_q // H_kv)}
    N = c["N"]
    angles = 6 * L * N * c["rot"] // 2
    if c["op"] == "rope":
        return {"bytes": 2 * L * (H_q + H_kv) * N * d * 2 + 4 * N, "flops": angles * (H_q + H_kv)}
    m, n = _chunks(c)
    ps = c["page"]
    end, have = -(-(n + m[None, None]) // ps), -(-n // ps)
    clear = np.where(end > have, end * ps - n - m[None, None], 0)
    tables = n.size * 8 + int((end - have).sum()) * 4 + N * 4
    return {"bytes": 2 * L * (H_q + 2 * H_kv) * N * d * 2 + int(clear.sum()) * d * 4 + tables,
            "flops": angles * (H_q + H_kv)}


# ----------------------------------------------------------------------------- 64 bits

def _exact_rotate(x, pos, inv_freq, rot, interleaved):
    """Every pair as a complex number times exp(i angle)."""
    y = x.double().clone()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       torch.outer(pos.double(), inv_freq.to(DEV)))
    re = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    im = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    z = torch.complex(y[..., re].contiguous(), y[..., im].contiguous()) * turn
    y[..., re], y[..., im] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    L, H_kv = s["L"], s["H_kv"]
    if s["op"] == "rope":
        return {n: _exact_rotate(s[n], s["pos"], s["inv_freq"], s["rot"], s["interleaved"])
                for n in ("q", "k")}
    B, ps = s["B"], s["page"]
    if s["op"] == "append":
        k = _exact_rotate(s["k"], s["pos"], s["inv_freq"], s["rot"], s["interleaved"])
        q = _exact_rotate(s["q"], s["pos"], s["inv_freq"], s["rot"], s["interleaved"])
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        bt, n = s["bt"].cpu().numpy(), s["n_seq"].cpu().numpy()
        start, nxt = s["tok_start"].cpu().numpy(), int(s["next"])
        out = n.copy()
        for l in range(L):
            for h in range(H_kv):
                for b in range(B):
                    t0, t1, at = int(start[b]), int(start[b + 1]), int(n[l, h, b])
                    out[l, h, b] += t1 - t0
                    while t0 < t1:  # one page at a time
                        if at % ps == 0:
                            bt[l, h, b, at // ps] = nxt
                            kp[nxt], vp[nxt] = 0.0, 0.0
                            nxt += 1
                        page, lo = bt[l, h, b, at // ps], at % ps
                        step = min(ps - lo, t1 - t0)
                        kp[page, lo:lo + step] = k[l, h, t0:t0 + step]
                        vp[page, lo:lo + step] = s["v"][l, h, t0:t0 + step].double()
                        t0, at = t0 + step, at + step
        return {"q": q, "k_pages": kp, "v_pages": vp, "block_table": torch.from_numpy(bt),
                "seq_lens": torch.from_numpy(out), "next_page": torch.tensor([nxt], dtype=torch.int32)}
    n, pos = _lengths(case)
    if n.size > 4096:
        return None
    g, d = s["H_q"] // H_kv, s["d"]
    o = torch.zeros(L, s["H_q"], B, d, dtype=torch.float64, device=DEV)
    lse = torch.full((L, s["H_q"], B), -math.inf, dtype=torch.float64, device=DEV)
    for l in range(L):
        for h in range(H_kv):
            for b in range(B):
                m = int(n[l, h, b])
                ids = s["bt"][l, h, b, : -(-m // ps)].long()
                k = s["k_pages"][ids].reshape(-1, d)[:m].double()
                v = s["v_pages"][ids].reshape(-1, d)[:m].double()
                held = min(int(pos[b]), s["w"])
                if held:
                    k = torch.cat([k, s["ring_k"][l, h, b, :held].double()])
                    v = torch.cat([v, s["ring_v"][l, h, b, :held].double()])
                if not k.shape[0]:
                    continue
                heads = slice(h * g, (h + 1) * g)
                x = s["q"][l, heads, b].double() @ k.t() * d ** -0.5
                z = torch.logsumexp(x, -1)
                lse[l, heads, b] = z
                o[l, heads, b] = torch.exp(x - z[:, None]) @ v
    return {"o": o, "lse": lse}
