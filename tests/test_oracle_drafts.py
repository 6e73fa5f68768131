"""Pins of the oracle's tree attention, accepted paths, forks and reclaimed pages (closed forms,
hand-worked cases, agreement with the other oracle functions), and one-line slips planted in a
copy that the pins must catch.  CPU only."""
import inspect
import math
import types

import numpy as np
import pytest

import oracle as O
import oracle.drafts_oracle as real


def tree_closed_forms(M):
    rng = np.random.default_rng(2)
    d, ps = 4, 3
    kp, vp = rng.standard_normal((5, ps, d)), rng.standard_normal((5, ps, d))
    bt = np.array([[[[4, 1, 0]], [[2, 3, -1]]]])
    sl = np.array([[[7], [4]]])
    # four drafted tokens: two roots, 0 -> 2 -> 3, 1
    parent, ts = [-1, -1, 0, 2], [0, 4]
    q = rng.standard_normal((1, 4, 4, d))
    o, lse, spread = M.attn_tree(q * 0, ts, parent, kp, vp, ps, bt, sl)
    # q = 0: ln of the number of visible keys, the mean of their values
    assert np.allclose(lse[0, 0], np.log([4, 4, 5, 6])) and np.allclose(lse[0, 3], np.log([1, 1, 2, 3]))
    seq = [(4, 0), (4, 1), (4, 2), (1, 0), (1, 1), (1, 2), (0, 0)]
    v = np.array([vp[p] for p in seq])
    assert np.allclose(o[0, 0, 3], v[[0, 1, 2, 3, 5, 6]].mean(0))
    assert np.allclose(o[0, 1, 1], v[[0, 1, 2, 4]].mean(0))
    assert np.allclose(o[0, 2, 1], vp[2, 1]) and np.allclose(spread[0, 2, 1], np.abs(vp[2, 1]))
    # a chain: token i is the decode of a cache that ends with it
    o, lse, _ = M.attn_tree(q, ts, None, kp, vp, ps, bt, sl)
    same = M.attn_tree(q, ts, [-1, 0, 1, 2], kp, vp, ps, bt, sl)
    assert np.array_equal(o, same[0]) and np.array_equal(lse, same[1])
    rk, rv = rng.standard_normal((1, 2, 1, 2, d)), rng.standard_normal((1, 2, 1, 2, d))
    for i in range(4):
        for ring in ((), (rk, rv, [1])):
            want = O.attn_decode(q[:, :, i:i + 1], kp, vp, ps, bt, sl - 3 + i, *ring)
            o, lse, spread = M.attn_tree(q, ts, None, kp, vp, ps, bt, sl, *ring)
            assert np.allclose(o[:, :, i], want[0][:, :, 0]) and np.allclose(lse[:, :, i], want[1][:, :, 0])
            assert np.allclose(spread[:, :, i], want[2][:, :, 0])
    # a tree without a branch that is taken is a shorter tree: what a token does not see, is not there
    a = M.attn_tree(q[:, :, [0, 2]], [0, 2], [-1, 0], kp, vp, 1, np.array([[[[0, 1, 2]], [[0, 1, 2]]]]), sl * 0 + 3)
    kp2, vp2 = kp[:4, :1].copy(), vp[:4, :1].copy()
    kp2[3], vp2[3] = kp2[2], vp2[2]
    kp2[2], vp2[2] = np.nan, np.nan
    # pools of one-row pages: keys 0, 1 before and 1 again as the draft's
    b = M.attn_tree(q[:, :, [0, 1, 2]], [0, 3], [-1, -1, 0], kp2, vp2, 1,
                    np.array([[[[0, 1, 2, 3]], [[0, 1, 2, 3]]]]), sl * 0 + 4)
    assert np.allclose(a[0], b[0][:, :, [0, 2]]) and np.allclose(a[1], b[1][:, :, [0, 2]])
    # two sequences: the second's indices are its own; one without drafts; a row without keys
    q2 = rng.standard_normal((1, 4, 3, d))
    bt2 = np.concatenate([bt, bt, bt], 2)
    sl2 = np.array([[[4, 0, 6], [2, 1, 4]]])
    o, lse, _ = M.attn_tree(q2, [0, 1, 1, 3], [-1, -1, 0], kp, vp, ps, bt2, sl2)
    alone = M.attn_tree(q2[:, :, 1:], [0, 2], [-1, 0], kp, vp, ps, bt, np.array([[[6], [4]]]))
    assert np.allclose(o[:, :, 1:], alone[0]) and np.allclose(lse[:, :, 1:], alone[1])
    o, lse, _ = M.attn_tree(q2[:, :, :1], [0, 1], None, kp, vp, ps, bt, sl * 0)
    assert (o == 0).all() and (lse == -np.inf).all()
    # large logits
    x = M.attn_tree(q * 1e3, ts, parent, kp, vp, ps, bt, sl)
    assert np.isfinite(x[0]).all() and np.isfinite(x[1]).all()
    assert math.isclose(float(x[1][0, 2, 1]), float(q[0, 2, 1] @ kp[2, 1] * 1e3 / 2), rel_tol=1e-12)


def accept_by_hand(M):
    ps = 2
    kp = np.arange(8.0).reshape(4, ps, 1)
    vp = kp + 50
    bt = np.array([[[[3, 0, 1], [2, -1, -1]]]])
    sl = np.array([[[5, 2]]])
    # row 0: 6 7 | 0 1 | 2 with four drafted: 7 0 1 2 at slots 1 .. 4; keep 1 and 3: 0 and 2
    k, v, n = M.accept_paged([0, 4, 6], [2, 0], [1, 3, 9, 9, 9, 9], ps, kp, vp, bt, sl)
    assert n.tolist() == [[[3, 0]]]
    assert k[3, :, 0].tolist() == [6, 0] and k[0, :, 0].tolist() == [2, 1]
    assert k[1, :, 0].tolist() == [2, 3] and k[2, :, 0].tolist() == [4, 5]
    assert np.array_equal(v, k + 50)
    k, v, n = M.accept_paged([0, 4, 6], [4, 2], [0, 1, 2, 3, 0, 1], ps, kp, vp, bt, sl)
    assert np.array_equal(k, kp) and np.array_equal(n, sl)


def fork_by_hand(M):
    ps = 2
    kp = np.arange(12.0).reshape(6, ps, 1)
    vp = kp + 50
    bt = np.array([[[[3, 0, -1], [1, 4, 5], [-1, -1, -1]], [[2, -1, -1], [-1, -1, -1], [-1, -1, -1]]]])
    sl = np.array([[[3, 5, 0], [2, 0, 0]]])
    kp = np.concatenate([kp, kp * 0 + 99])
    vp = np.concatenate([vp, vp * 0 + 99])
    k, v, nxt, b, n = M.fork_paged([0, 0], [2, 1], ps, kp, vp, 6, bt, sl)
    assert nxt == 8 and n.tolist() == [[[3, 3, 3], [2, 2, 2]]]
    assert b[0, 0].tolist() == [[3, 0, -1], [3, 7, -1], [3, 6, -1]]
    assert b[0, 1].tolist() == [[2, -1, -1]] * 3
    for p in (6, 7):
        assert k[p, :, 0].tolist() == [0, 0] and v[p, :, 0].tolist() == [50, 0]
    assert (k[8:] == 99).all() and np.array_equal(k[:6], kp[:6])
    assert M.fork_paged([0, 0], [2, 1], ps, kp[:7], vp[:7], 6, bt, sl) == "pool"
    assert M.fork_paged([0, 0], [2, 1], ps, kp[:8], vp[:8], 6, bt, sl)[2] == 8
    k, _, nxt, b, _ = M.fork_paged([1], [0], ps, kp, vp, 6, bt, sl)
    assert nxt == 7 and b[0, 0, 0].tolist() == [1, 4, 6] and k[6, :, 0].tolist() == [10, 0]
    # the copies attend alike
    rng = np.random.default_rng(3)
    kp, vp = rng.standard_normal((12, ps, 4)), rng.standard_normal((12, ps, 4))
    k, v, _, b, n = M.fork_paged([1], [2], ps, kp, vp, 6, bt, sl)
    q = np.repeat(rng.standard_normal((1, 2, 1, 4)), 3, 2)
    o, lse, _ = O.attn_decode(q, k, v, ps, b, n)
    assert np.allclose(o[:, :, 1], o[:, :, 2]) and np.allclose(lse[:, :, 1], lse[:, :, 2])


def reclaim_by_hand(M):
    ps = 2
    kp = np.arange(14.0).reshape(7, ps, 1)
    vp = kp + 50
    # in use: 5 (twice), 1, 6, 3; ids 0 .. 3 hold four pages: 5 -> 0, 6 -> 2
    bt = np.array([[[[5, 1, 2], [5, 6, 0], [3, 4, -1], [0, 2, 4]]]])
    sl = np.array([[[3, 4, 2, 0]]])
    k, v, n, b = M.reclaim_paged(ps, kp, vp, bt, sl)
    assert n == 4 and b[0, 0].tolist() == [[0, 1, -1], [0, 2, -1], [3, -1, -1], [-1, -1, -1]]
    assert k[:, 0, 0].tolist() == [10, 2, 12, 6, 8, 10, 12] and np.array_equal(v, k + 50)
    # nothing to do, and nothing in use
    k2, _, n, b2 = M.reclaim_paged(ps, k, v, b, sl)
    assert n == 4 and np.array_equal(b2, b) and np.array_equal(k2, k)
    k, _, n, b = M.reclaim_paged(ps, kp, vp, bt, sl * 0)
    assert n == 0 and (b == -1).all() and np.array_equal(k, kp)


PINS = [tree_closed_forms, accept_by_hand, fork_by_hand, reclaim_by_hand]


@pytest.mark.parametrize("pin", PINS, ids=lambda p: p.__name__)
def test_pin(pin):
    pin(real)


MUTATIONS = [
    ("sees no parent", "i = i - 1 if parent is None else int(parent[i])", "i = i - 1 if parent is None else -1"),
    ("chain skips", "i = i - 1 if parent is None", "i = i - 2 if parent is None"),
    ("not itself", "path.append(i)\n        i = ", "path.append(i) if path else None\n        i = "),
    ("parents of the batch", "np.asarray(parent)[t0:t0 + m]", "np.asarray(parent)"),
    ("sees every draft", "for j in way_up(up, i) if", "for j in range(m) if"),
    ("one key too few", "see = list(range(n - m)) +", "see = list(range(n - m - 1)) +"),
    ("first head's keys", "for hq in range(hk * g, (hk + 1) * g):", "for hq in range(hk, H_q, H_kv):"),
    ("whole ring", "held = min(int(pos[b]), ring_k.shape[3])", "held = ring_k.shape[3]"),
    ("no maximum", "top = x.max()", "top = 0.0"),
    ("pages in order", "at = [(block_table[l, hk, b, s // page_size], s % page_size)", "at = [(s // page_size, s % page_size)"),
    ("path in place", "at[base + int(accept[t0 + j])]", "at[base + j]"),
    ("path from the row's start", "at[base + int(accept[t0 + j])]", "at[int(accept[t0 + j])]"),
    ("length keeps the draft", "sl[l, h, b] = base + int(n_accept[b])", "sl[l, h, b] = base + m"),
    ("reads what it wrote", "kp[new], vp[new] = k_pages[old], v_pages[old]", "kp[new], vp[new] = kp[old], kp[old]"),
    ("last page shared", "if n > full * page_size:", "if n > full * page_size + page_size:"),
    ("page not cleared", "kp[nxt], vp[nxt] = 0, 0", "pass"),
    ("pool one short", "if nxt >= len(kp):", "if nxt >= len(kp) - 1:"),
    ("old table behind", "bt[l, h, dst[i]] = -1", "pass"),
    ("source's length kept", "sl[l, h, dst[i]] = n", "pass"),
    ("holes from the back", "free = [i for i in range(len(use)) if i not in use]", "free = [i for i in range(len(use)) if i not in use][::-1]"),
    ("rounds down", "need = {r: -(-int(seq_lens[r]) // page_size)", "need = {r: int(seq_lens[r]) // page_size"),
    ("moves one too few", "if p >= len(use)], free):", "if p > len(use) + 1], free):"),
]


@pytest.mark.parametrize("name,old,new", MUTATIONS, ids=[m[0] for m in MUTATIONS])
def test_planted_slip_is_caught(name, old, new):
    src = inspect.getsource(real)
    assert src.count(old) == 1, name
    mod = types.ModuleType("oracle.mutated")
    mod.__package__ = "oracle"
    exec(compile(src.replace(old, new), "mutated", "exec"), mod.__dict__)
    for pin in PINS:
        try:
            pin(mod)
        except Exception:
            return
    raise AssertionError(f"no pin caught: {name}")
