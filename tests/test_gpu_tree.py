"""GPU parity of the attention of drafted tokens (kvs_attn_tree) with a plain implementation in 64
bits, at the sizes, trees and states where it can go wrong, and its use with the calls around it.

Tolerances, from the arithmetic (u = 2^-24, an fp32 rounding; 2^-8, a bf16 rounding):
  logits: |dx| <= delta = (d + 8) u max_k sum_e |q_e k_ke| / sqrt(d) + 2^-20 |x|max (fp32 sums in any
          order, the scale by log2 e, ex2 to 2^-22)
  lse:    delta + 2^-20 (1 + |lse|) + (n + 32) u (sums of n positive terms in any order)
  o:      2^-8 |o| (output) + (2^-8 + 2.1 delta + (n + 32) u) sum a |v| (weights rounded to bf16, their
          error from the logits in numerator and denominator, the sums)
"""
import threading

import numpy as np
import pytest
import torch

import oracle as O
from .gpu_util import f64, need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def C():
    need_gpu()
    from kv_cache_eviction_lse_gb300 import build
    build.build()
    from kv_cache_eviction_lse_gb300 import capi
    return capi


def tree(rng, m, kind):
    """Parents of m tokens."""
    i = np.arange(m)
    if kind == "chain":
        return i - 1
    if kind == "star":
        return np.full(m, -1)
    if kind == "levels":  # four children each, level by level
        return i // 4 - 1
    return np.floor(rng.uniform(size=m) * (i + 1)).astype(int) - 1


def case(seed, L=1, Hq=4, H=2, B=2, d=128, ps=16, w=0, n=100, m=(5, 3), kind="random", pad=0, scale=1.0,
         mp_extra=1, n_lo=0):
    """Rows of n_lo to n tokens below the m[b] drafted ones."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    m = np.array(m)
    sl = rng.integers(n_lo, n + 1, size=(L, H, B)) + m
    need = -(-sl // ps)
    mp, cap = max(1, int(need.max()) + mp_extra), int(need.sum()) + 2
    bt = rng.integers(-3, cap + 3, size=(L, H, B, mp)).astype(np.int32)  # anything behind the pages
    ids, i = rng.permutation(cap), 0
    for r in np.ndindex(L, H, B):
        bt[r][:need[r]] = ids[i:i + need[r]]
        i += int(need[r])
    ts = np.concatenate([[0], np.cumsum(m)])
    N = int(ts[-1]) + pad
    bf = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16)  # noqa: E731
    parent = np.concatenate([tree(rng, x, kind) for x in m] + [np.full(pad, 77)]).astype(np.int32)
    return dict(L=L, Hq=Hq, H=H, B=B, d=d, ps=ps, w=w, N=N, cap=cap, mp=mp, m=m, sl=sl.astype(np.int32), bt=bt,
                ts=ts.astype(np.int32), parent=parent, q=(bf(L, Hq, N, d).float() * scale).to(torch.bfloat16),
                kp=bf(cap, ps, d), vp=bf(cap, ps, d), pos=rng.integers(0, 3 * w + 1, size=B).astype(np.int32),
                rk=bf(L, H, B, w, d), rv=bf(L, H, B, w, d), md=max(1, int(m.max())))


def expected(c):
    """o, lse, sum a |v| and the tolerance of the logits, in 64 bits; padding stays NaN."""
    L, Hq, N, d, H, B, ps = c["L"], c["Hq"], c["N"], c["d"], c["H"], c["B"], c["ps"]
    g = Hq // H
    q, kp, vp, rk, rv = (f64(c[k]) for k in ("q", "kp", "vp", "rk", "rv"))
    o, sp = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, delta = np.full(q.shape[:3], np.nan), np.zeros(q.shape[:3])
    for b in range(B):
        t0, m = int(c["ts"][b]), int(c["m"][b])
        sees = np.zeros((m, m), dtype=bool)
        for i in range(m):
            p = i - 1 if c["parent"] is None else int(c["parent"][t0 + i])
            if p >= 0:
                sees[i] = sees[p]
            sees[i, i] = True
        for l in range(L):
            for h in range(H):
                n = int(c["sl"][l, h, b])
                ids = c["bt"][l, h, b, : -(-n // ps)]
                K, V = kp[ids].reshape(-1, d)[:n], vp[ids].reshape(-1, d)[:n]
                held = min(int(c["pos"][b]), c["w"])
                K, V = np.concatenate([K, rk[l, h, b, :held]]), np.concatenate([V, rv[l, h, b, :held]])
                see = np.ones((m, n + held), dtype=bool)
                see[:, n - m:n] = sees
                for hq in range(h * g, (h + 1) * g):
                    qs = q[l, hq, t0:t0 + m]
                    if not m:
                        continue
                    with np.errstate(invalid="ignore", over="ignore"):
                        x = np.where(see, qs @ K.T / np.sqrt(d), -np.inf)
                        top = x.max(1, keepdims=True)
                        e = np.exp(x - top)
                        z = e.sum(1, keepdims=True)
                        a = e / z
                        o[l, hq, t0:t0 + m] = np.stack([(a[i][see[i]] @ V[see[i]]) for i in range(m)])
                        sp[l, hq, t0:t0 + m] = np.stack([(a[i][see[i]] @ np.abs(V[see[i]])) for i in range(m)])
                        lse[l, hq, t0:t0 + m] = (top + np.log(z))[:, 0]
                        size = np.where(see, np.abs(qs) @ np.abs(K).T, 0).max(1) / np.sqrt(d)
                        delta[l, hq, t0:t0 + m] = (d + 8) * U * size + 2.0 ** -20 * np.abs(np.where(see, x, 0)).max(1)
    return o, lse, sp, delta


def call(C, c, lse=True, stream=None, fill=7.0):
    dev = lambda x: None if x is None else (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).cuda()  # noqa: E731
    g = {k: dev(c[k]) for k in ("q", "kp", "vp", "bt", "sl", "ts", "parent", "pos", "rk", "rv")}
    g["o"] = torch.full_like(g["q"], fill)
    g["lse"] = torch.full(c["q"].shape[:3], fill, device="cuda") if lse else None
    dm = C.dims(c["L"], c["Hq"], c["H"], c["d"])
    nb = C.kvs_attn_tree_workspace_size(dm, c["B"], c["N"])
    g["ws"] = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    ring = (g["pos"], g["rk"], g["rv"]) if c["w"] else (None, None, None)
    torch.cuda.synchronize()
    g["go"] = lambda: C.kvs_attn_tree(dm, c["B"], c["N"], c["md"], g["ts"], g["parent"], g["q"], c["ps"], g["kp"],
                                      g["vp"], c["cap"], g["bt"], c["mp"], g["sl"], c["w"], *ring, g["o"],
                                      g["lse"], g["ws"], nb, stream=stream)
    g["go"]()
    return g


def check(c, r, what="", want=None):
    o, lse, sp, delta = expected(c) if want is None else want
    used, n = int(c["ts"][-1]), int(c["sl"].max()) + c["w"]
    got, got_lse = f64(r["o"])[:, :, :used], r["lse"].double().cpu().numpy()[:, :, :used]
    o, lse, sp, delta = o[:, :, :used], lse[:, :, :used], sp[:, :, :used], delta[:, :, :used]
    err = np.abs(got_lse - lse)
    assert (err <= delta + 2.0 ** -20 * (1 + np.abs(lse)) + (n + 32) * U).all(), (what, err.max())
    err = np.abs(got - o)
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.1 * delta[..., None] + (n + 32) * U) * sp
    assert (err <= tol).all(), (what, err.max(), np.nanmax(err / tol))
    assert (r["o"][:, :, used:] == 7.0).all() and (r["lse"][:, :, used:] == 7.0).all()  # padding as it was


CASES = {
    "one token": dict(B=1, m=[1], n=40),
    "one token each, as a decode": dict(B=3, m=[1, 1, 1], n=300, Hq=8, H=2),
    "only drafts": dict(B=2, m=[9, 1], n=0),
    "drafts across a tile's end": dict(B=4, m=[20, 7, 130, 2], n=130, n_lo=118),
    "pages of one": dict(B=2, m=[17, 4], n=50, ps=1, d=64),
    "odd pages, six heads": dict(B=3, m=[12, 0, 33], n=400, ps=13, Hq=12, H=2),
    "large pages": dict(B=2, m=[12, 31], n=700, ps=300, d=64),
    "page of 4096": dict(B=1, m=[6], n=5000, ps=4096, H=1),
    "a ring": dict(B=4, m=[3, 8, 1, 2], n=90, w=16),
    "a ring of more than a tile": dict(B=3, m=[3, 8, 40], n=30, w=300, d=64),
    "a ring alone below": dict(B=3, m=[3, 8, 5], n=0, w=7),
    "padding, empty sequences": dict(B=5, m=[0, 4, 0, 0, 6], n=60, pad=9),
    "one head each": dict(Hq=3, H=3, B=2, m=[128, 129], n=70, d=64),
    "eight heads, two query tiles": dict(Hq=16, H=2, B=2, m=[17, 31], n=300),
    "sixteen heads and more": dict(Hq=40, H=2, B=1, m=[20], n=200, d=64),
    "256 drafts": dict(Hq=2, H=1, B=2, m=[256, 200], n=500, d=64),
    "256 drafts in a line": dict(Hq=2, H=1, B=2, m=[256, 255], n=100, kind="chain"),
    "256 roots": dict(Hq=1, H=1, B=1, m=[256], n=300, kind="star"),
    "levels": dict(Hq=4, H=1, B=2, m=[85, 64], n=300, kind="levels"),
    "split over many blocks": dict(Hq=4, H=1, B=1, m=[9], n=30000, n_lo=30000),
    "few rows, few blocks each": dict(Hq=4, H=4, B=3, m=[9, 30, 70], n=9000, d=64),
    "many short rows": dict(L=5, Hq=8, H=8, B=33, m=[3] * 33, n=60, d=64),
    "more rows than threads": dict(L=9, Hq=8, H=8, B=20, m=[i % 4 for i in range(20)], n=20, d=64, ps=4),
    "large logits": dict(B=2, m=[8, 30], n=500, scale=300.0),
    "equal logits": dict(B=2, m=[8, 30], n=500, scale=0.0),
}


@pytest.mark.parametrize("name", CASES)
def test_tree(C, name):
    c = case(len(name), **CASES[name])
    r = call(C, c)
    torch.cuda.synchronize()
    assert C.kvs_device_error() == 0
    check(c, r, name)
    first, first_lse = r["o"].clone(), r["lse"].clone()
    r["go"]()  # the same bits again
    assert torch.equal(r["o"], first) and torch.equal(r["lse"], first_lse)
    no_lse = call(C, c, lse=False)
    assert torch.equal(no_lse["o"], first)
    assert C.kvs_device_error() == 0


def test_plain_implementation_agrees_with_the_oracle():
    for w, kind in ((0, "random"), (3, "levels"), (0, "chain")):
        c = case(3, B=3, m=[4, 0, 9], n=30, d=64, ps=5, w=w, kind=kind, Hq=4, H=2)
        c["parent"] = None if kind == "chain" else c["parent"]
        o, lse, sp, _ = expected(c)
        ring = (f64(c["rk"]), f64(c["rv"]), c["pos"]) if w else ()
        want = O.attn_tree(f64(c["q"]), c["ts"], c["parent"], f64(c["kp"]), f64(c["vp"]), c["ps"], c["bt"], c["sl"], *ring)
        assert np.allclose(o, want[0]) and np.allclose(lse, want[1]) and np.allclose(sp, want[2])


def test_no_parents_is_a_chain(C):
    c = case(5, B=3, m=[70, 1, 256], n=200, kind="chain", Hq=4, H=2)
    a = call(C, c)
    b = call(C, dict(c, parent=None))
    assert torch.equal(a["o"], b["o"]) and torch.equal(a["lse"], b["lse"])


def test_one_token_is_the_decode(C):
    """A tree of one token each is what kvs_attn_decode computes."""
    c = case(6, B=5, m=[1] * 5, n=600, Hq=12, H=2, w=16)
    r = call(C, c)
    dm = C.dims(1, 12, 2, 128)
    o, lse = torch.empty_like(r["o"]), torch.empty_like(r["lse"])
    ws = torch.empty(C.kvs_attn_decode_workspace_size(dm, 5), dtype=torch.uint8, device="cuda")
    C.kvs_attn_decode(dm, 5, r["q"], 16, r["kp"], r["vp"], c["cap"], r["bt"], c["mp"], r["sl"], 16, r["pos"], r["rk"],
                      r["rv"], o, lse, ws, ws.numel())
    check(c, dict(o=o, lse=lse))
    check(c, r)


# ----------------------------------------------------------------------------- what is not seen

@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan"), 3.38e38])
@pytest.mark.parametrize("d", [64, 128])
def test_unseen_drafts_leave_no_trace(C, bad, d):
    """Infinities, NaN and the largest number in K and V of drafted tokens that others do not see,
    behind the rows' ends and in pages of no row: the others' results are those of finite ones, to
    the bit, the tokens that see them get what the formula gives."""
    for m, kind, n in (([6, 40], "star", 100), ([130, 256], "random", 60), ([33, 3], "chain", 5000)):
        c = case(7, B=2, m=m, n=n, n_lo=n, d=d, kind=kind)
        clean = call(C, c)
        want = expected(c)
        kp, vp = c["kp"].clone(), c["vp"].clone()
        owned = torch.zeros(c["cap"], c["ps"], dtype=torch.bool)
        who = [2, m[1] - 2]  # the bad token of each sequence
        for l, h, b in np.ndindex(1, 2, 2):
            s = np.arange(int(c["sl"][l, h, b]))
            owned[c["bt"][l, h, b, s // 16], s % 16] = True
            slot = int(c["sl"][l, h, b]) - m[b] + who[b]
            page, row = c["bt"][l, h, b, slot // 16], slot % 16
            kp[page, row], vp[page, row, ::3] = bad, bad
            if h:
                kp[page, row] = c["kp"][page, row]  # the second head: in V alone
        kp[~owned], vp[~owned] = bad, bad
        c2 = dict(c, kp=kp, vp=vp)
        r = call(C, c2)
        torch.cuda.synchronize()
        assert C.kvs_device_error() == 0
        o, lse, sp, delta = expected(c2)
        for b in range(2):
            t0 = int(c["ts"][b])
            up = [set() for _ in range(m[b])]
            for i in range(m[b]):
                p = int(c["parent"][t0 + i])
                up[i] = {i} | (up[p] if p >= 0 else set())
            blind = [t0 + i for i in range(m[b]) if who[b] not in up[i]]
            seeing = [t0 + i for i in range(m[b]) if who[b] in up[i]]
            assert torch.equal(r["o"][:, :, blind], clean["o"][:, :, blind])
            assert torch.equal(r["lse"][:, :, blind], clean["lse"][:, :, blind])
            if abs(bad) < 1e38 or np.isnan(bad) or np.isinf(bad):
                # the second head's tokens that see it: not finite where its values are not, the
                # same elsewhere
                got, exp = f64(r["o"])[0, 2:][:, seeing], o[0, 2:][:, seeing]
                if np.isinf(bad) or np.isnan(bad):
                    assert np.array_equal(np.isnan(got), np.isnan(exp))
                    assert np.array_equal(got[np.isinf(exp)], exp[np.isinf(exp)])
                    fine = np.isfinite(exp)
                    assert np.array_equal(np.isfinite(got), fine)
                    base = f64(clean["o"])[0, 2:][:, seeing]
                    assert np.array_equal(got[fine], base[fine])
        del want


def test_bad_values_of_several_drafts_add_up(C):
    """+inf and -inf on one way up make NaN, each alone stays an infinity."""
    c = case(8, B=1, m=[4], n=40, H=1, Hq=2, kind="chain")
    for i, x in ((1, float("inf")), (3, float("-inf"))):
        slot = int(c["sl"][0, 0, 0]) - 4 + i
        c["vp"][c["bt"][0, 0, 0, slot // 16], slot % 16, 5] = x
    r = call(C, c)
    col = r["o"][0, :, :, 5].float().cpu()
    assert col[:, 0].isfinite().all() and (col[:, 1:3] == float("inf")).all() and col[:, 3].isnan().all()
    rest = r["o"].float().cpu().clone()
    rest[..., 5] = 0
    assert rest.isfinite().all()
    # in the cache below the drafts, all see it
    page = c["bt"][0, 0, 0, 0]
    c["vp"][page, 0, 9] = float("inf")
    assert (call(C, c)["o"][0, :, :, 9] == float("inf")).all()


# ----------------------------------------------------------------------------- refusals on the device

def test_bad_states_are_bounded_and_reported(C):
    base = dict(B=3, m=[5, 4, 9], n=150, d=64, Hq=4, H=2, w=0)

    def code(c):
        r = call(C, c)
        torch.cuda.synchronize()
        assert C.kvs_device_error() == 10 and C.kvs_device_error() == 0
        return r

    # page ids: their keys are left out
    for page in (-1, 2 ** 31 - 1, -2 ** 31, None):
        c = case(9, **base, n_lo=60)
        ok = call(C, c)
        c["bt"][0, 1, 1, 1] = c["cap"] if page is None else page
        r = code(c)
        keep = [i for i in range(c["N"]) if not c["ts"][1] <= i < c["ts"][2]]
        assert torch.equal(r["o"][:, :, keep], ok["o"][:, :, keep])
        assert torch.equal(r["o"][:, :2], ok["o"][:, :2])
        # 16 keys fewer: the row's table without that page
        c2 = dict(c, sl=c["sl"].copy(), bt=c["bt"].copy())
        c2["bt"][0, 1, 1, 1:-1], c2["sl"][0, 1, 1] = c["bt"][0, 1, 1, 2:], c["sl"][0, 1, 1] - 16
        o, lse, _, delta = expected(c2)
        t = slice(c["ts"][1], c["ts"][2])
        err = np.abs(r["lse"].double().cpu().numpy() - lse)[:, 2:, t]
        assert (err <= delta[:, 2:, t] + 2.0 ** -18).all()
    # lengths: the nearest bound; drafted tokens before slot 0 are not there
    for n in (-1, -2 ** 31):
        c = case(10, **base)
        c["sl"][0, 0, 0] = n
        r = code(c)
        assert (r["o"][0, :2, :5] == 0).all() and (r["lse"][0, :2, :5] == -np.inf).all()
    c = case(10, **base)
    c["sl"][0, 0, 0] = 2  # of five drafted tokens, the last two
    c["parent"][:5] = [-1, 0, 1, 0, 3]
    r = code(c)
    lse = r["lse"][0, :2, :5].cpu().numpy()
    assert (lse[:, :3] == -np.inf).all() and (r["o"][0, :2, :3] == 0).all()
    o, v = f64(r["o"])[0, :2], f64(c["vp"])[c["bt"][0, 0, 0, 0]]
    assert np.abs(o[:, 3] - v[0]).max() <= 2.0 ** -7 * np.abs(v[0]).max()
    assert np.isfinite(lse[:, 3:]).all()
    c = case(10, **base, n_lo=60)
    room = c["mp"] * c["ps"]
    c["sl"][0, 0, 0] = room + 1
    c["bt"][0, 0, 0] = np.clip(c["bt"][0, 0, 0], 0, c["cap"] - 1)
    r = code(c)
    assert r["lse"][0, :2, :5].isfinite().all()
    # token starts: no results for the sequence
    for ts in ([0, 5, 4, 18], [-1, 5, 9, 18], [0, 5, 9, 19], [0, 5, 2 ** 31 - 1, 18]):
        c = case(11, **base)
        c["ts"] = np.array(ts, dtype=np.int32)
        code(c)
    c = case(11, **base)
    c["md"] = 8  # the last sequence has nine
    r = code(c)
    assert (r["o"][:, :, 9:] == 7.0).all() and (r["lse"][:, :, 9:] == 7.0).all()
    o, lse, sp, delta = (x[:, :, :9] for x in expected(c))
    assert (np.abs(f64(r["o"])[:, :, :9] - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.1 * delta[..., None] + 2.0 ** -16) * sp).all()
    # parents: as roots
    for p in (-2, 3, 7, 2 ** 31 - 1, -2 ** 31):
        c = case(12, **base)
        c["parent"][3] = -1
        ok = call(C, c)
        c = dict(c, parent=c["parent"].copy())
        c["parent"][3] = p
        r = code(c)
        assert torch.equal(r["o"], ok["o"])


def test_a_pool_of_no_pages(C):
    """Rings alone: nothing of the pool is read, whatever came for it."""
    c = case(13, B=2, m=[0, 0], n=0, w=5, pad=3)
    r = call(C, c)
    torch.cuda.synchronize()
    assert C.kvs_device_error() == 0 and (r["o"] == 7.0).all()


# ----------------------------------------------------------------------------- streams, graphs, threads

def test_captured_and_replayed(C):
    """Replays with other lengths, tokens and parents in the same tensors."""
    c = case(14, B=4, m=[8, 3, 20, 1], n=800, Hq=8, H=2, pad=40)
    r = call(C, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r["go"]()
    for m, sub in (([8, 3, 20, 1], 0), ([1, 1, 1, 1], 37), ([20, 20, 20, 12], 300)):
        sl = np.maximum(c["sl"] - sub, np.array(m))
        ts = np.concatenate([[0], np.cumsum(m)]).astype(np.int32)
        rng = np.random.default_rng(sub)
        parent = np.concatenate([tree(rng, x, "random") for x in m] + [np.zeros(c["N"] - ts[-1])]).astype(np.int32)
        c2 = dict(c, sl=sl.astype(np.int32), ts=ts, m=np.array(m), parent=parent)
        for k in ("sl", "ts", "parent"):
            r[k].copy_(torch.from_numpy(c2[k]))
        r["o"].fill_(7.0)
        r["lse"].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert C.kvs_device_error() == 0
        check(c2, r, m)


def test_two_streams_and_two_threads(C):
    cs = [case(15, B=3, m=[8, 3, 20], n=3000, Hq=8, H=2), case(16, B=2, m=[100, 7], n=900, d=64, Hq=8, H=2)]
    want = [expected(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    rs = [call(C, c, stream=s) for c, s in zip(cs, streams)]
    torch.cuda.synchronize()

    raised = []

    def work(r):
        try:
            for _ in range(20):
                r["go"]()
        except Exception as e:  # an exception of a thread fails no test by itself
            raised.append(e)

    threads = [threading.Thread(target=work, args=(r,)) for r in rs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not raised
    torch.cuda.synchronize()
    assert C.kvs_device_error() == 0
    for c, r, x in zip(cs, rs, want):
        check(c, r, want=x)
