"""fp64 oracle of the operators for drafted tokens and for the pages of a cache: attention of a
tree of drafted tokens per sequence, the accepted path of a draft, forks of sequences and the
pages that come free.  Plain loops from the definitions; the storage is that of compact_paged
and append_paged (reading: the pages name paged storage for heads of different lengths
[KVzap limitation 3] without specifying it)."""
import numpy as np

from .kvs_oracle import _group, attention_logits


def way_up(parent, i):
    """Token i of a sequence and the tokens above it (parent None: a chain)."""
    path = []
    while i >= 0:
        path.append(i)
        i = i - 1 if parent is None else int(parent[i])
    return path


def attn_tree(q, tok_start, parent, k_pages, v_pages, page_size, block_table, seq_lens, ring_k=None,
              ring_v=None, pos=None):
    """Attention of the drafted tokens tok_start[b] .. tok_start[b + 1] - 1 of every sequence.
    They are the last tokens of its rows; token i sees the tokens before them, the ring's, and
    those on its way up the tree.  q [L][H_q][N][d]; parent [N] (index among the sequence's own,
    -1 for none) or None.  Returns (o, lse, spread) as attn_decode."""
    L, H_q, N, d = q.shape
    H_kv = block_table.shape[1]
    g = _group(H_q, H_kv)
    o, lse_, spread = np.zeros(q.shape), np.full(q.shape[:3], -np.inf), np.zeros(q.shape)
    for b in range(len(tok_start) - 1):
        t0, m = int(tok_start[b]), int(tok_start[b + 1] - tok_start[b])
        up = None if parent is None else np.asarray(parent)[t0:t0 + m]
        for l in range(L):
            for hk in range(H_kv):
                n = int(seq_lens[l, hk, b])
                at = [(block_table[l, hk, b, s // page_size], s % page_size) for s in range(n)]
                K, V = [k_pages[p, r] for p, r in at], [v_pages[p, r] for p, r in at]
                for i in range(m):
                    see = list(range(n - m)) + [n - m + j for j in way_up(up, i) if n - m + j >= 0]
                    Ki, Vi = [K[s] for s in see], [V[s] for s in see]
                    if ring_k is not None:
                        held = min(int(pos[b]), ring_k.shape[3])
                        Ki += list(ring_k[l, hk, b, :held])
                        Vi += list(ring_v[l, hk, b, :held])
                    if not Ki:
                        continue
                    Ki, Vi = np.array(Ki), np.array(Vi)
                    for hq in range(hk * g, (hk + 1) * g):
                        x = attention_logits(q[l, hq, t0 + i][None], Ki)[0]
                        top = x.max()
                        w = np.exp(x - top)
                        a = w / w.sum()
                        o[l, hq, t0 + i], spread[l, hq, t0 + i] = a @ Vi, a @ np.abs(Vi)
                        lse_[l, hq, t0 + i] = top + np.log(w.sum())
    return o, lse_, spread


def accept_paged(tok_start, n_accept, accept, page_size, k_pages, v_pages, block_table, seq_lens):
    """The accepted tokens of every row's draft one behind the other; the new lengths."""
    kp, vp, sl = k_pages.copy(), v_pages.copy(), seq_lens.copy()
    for l, h, b in np.ndindex(*seq_lens.shape):
        t0, m = int(tok_start[b]), int(tok_start[b + 1] - tok_start[b])
        base = int(seq_lens[l, h, b]) - m
        at = [(block_table[l, h, b, s // page_size], s % page_size) for s in range(base + m)]
        for j in range(int(n_accept[b])):
            new, old = at[base + j], at[base + int(accept[t0 + j])]
            kp[new], vp[new] = k_pages[old], v_pages[old]
        sl[l, h, b] = base + int(n_accept[b])
    return kp, vp, sl


def fork_paged(src, dst, page_size, k_pages, v_pages, next_page, block_table, seq_lens):
    """Sequence dst[i] becomes a copy of sequence src[i]: full pages shared, the last one copied
    to a new page, rows in the order (layer, head, fork).  "pool" if the pool is too small."""
    kp, vp, bt, sl = k_pages.copy(), v_pages.copy(), block_table.copy(), seq_lens.copy()
    nxt = int(next_page)
    L, H = seq_lens.shape[:2]
    for l, h, i in np.ndindex(L, H, len(src)):
        n = int(seq_lens[l, h, src[i]])
        full = n // page_size
        bt[l, h, dst[i]] = -1
        bt[l, h, dst[i], :full] = block_table[l, h, src[i], :full]
        sl[l, h, dst[i]] = n
        if n > full * page_size:
            if nxt >= len(kp):
                return "pool"
            kp[nxt], vp[nxt] = 0, 0
            for s in range(full * page_size, n):
                old = block_table[l, h, src[i], full]
                kp[nxt, s % page_size], vp[nxt, s % page_size] = k_pages[old, s % page_size], \
                    v_pages[old, s % page_size]
            bt[l, h, dst[i], full] = nxt
            nxt += 1
    return kp, vp, nxt, bt, sl


def reclaim_paged(page_size, k_pages, v_pages, block_table, seq_lens):
    """Pages in use to the front: the i-th one with an id from their number on to the i-th id
    below that is not in use."""
    kp, vp, bt = k_pages.copy(), v_pages.copy(), np.full_like(block_table, -1)
    need = {r: -(-int(seq_lens[r]) // page_size) for r in np.ndindex(*seq_lens.shape)}
    use = sorted({int(p) for r in need for p in block_table[r][:need[r]]})
    free = [i for i in range(len(use)) if i not in use]
    new = {p: p for p in use}
    for p, hole in zip([p for p in use if p >= len(use)], free):
        new[p] = hole
        kp[hole], vp[hole] = k_pages[p], v_pages[p]
    for r in need:
        for i in range(need[r]):
            bt[r][i] = new[int(block_table[r][i])]
    return kp, vp, len(use), bt
