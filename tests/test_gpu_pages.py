"""GPU parity of the accepted paths, forks and reclaimed pages with the oracle, to the bit (no
value is computed), at the sizes and states where they can go wrong, and their use together."""
import numpy as np
import pytest
import torch

import oracle as O
from .gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def C():
    need_gpu()
    from kv_cache_eviction_lse_gb300 import build
    build.build()
    from kv_cache_eviction_lse_gb300 import capi
    return capi


def pages(rng, n, ps, spare=0, mp_extra=1, cap_extra=0, shared=0):
    """A cache of rows of n [L][H][B] tokens whose pages lie scattered below the counter, with
    `spare` pages handed out and not named, and pages of `shared` rows those of the row before."""
    need = -(-n // ps)
    total = int(need.sum()) + spare
    mp = max(1, int(need.max()) + mp_extra)
    ids = rng.permutation(total)
    bt = rng.integers(-5, total + 5, size=n.shape + (mp,)).astype(np.int32)  # anything behind the pages
    i = 0
    for r in np.ndindex(*n.shape):
        bt[r][:need[r]] = ids[i:i + need[r]]
        i += int(need[r])
    for _ in range(shared):
        a, b = rng.integers(0, n.shape[2], size=2)
        n[:, :, a] = n[:, :, b]
        if mp:
            bt[:, :, a] = bt[:, :, b]
    return bt, mp, total, total + cap_extra


def pool(rng, cap, ps, d):
    return torch.from_numpy(rng.integers(-32768, 32767, size=(cap, ps, d)).astype(np.int16))


def dev(x):
    x = torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)) if isinstance(x, np.ndarray) else x
    return (x.view(torch.bfloat16) if x.dtype == torch.int16 else x).cuda()


def raw(t):
    t = t.detach().cpu()
    return (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).numpy()


def no_error(C):
    torch.cuda.synchronize()
    assert C.kvs_device_error() == 0


# ----------------------------------------------------------------------------- accept

ACCEPT = {
    "one row": dict(L=1, H=1, B=1, d=128, ps=16, m=[8], count=[3], n=20),
    "all kept, none kept, none drafted": dict(L=2, H=2, B=4, d=64, ps=4, m=[7, 9, 0, 1], count=[7, 0, 0, 1], n=9),
    "pages of one": dict(L=1, H=3, B=3, d=64, ps=1, m=[5, 20, 3], count=[2, 9, 1], n=3),
    "odd pages, odd rows": dict(L=3, H=1, B=5, d=64, ps=13, m=[40, 1, 33, 17, 64], count=[11, 0, 33, 1, 20], n=50),
    "long drafts": dict(L=1, H=2, B=3, d=128, ps=16, m=[256, 700, 90], count=[131, 600, 40], n=30),
    "empty cache below": dict(L=1, H=2, B=2, d=128, ps=16, m=[30, 5], count=[9, 5], n=0),
    "large pages": dict(L=1, H=2, B=2, d=128, ps=300, m=[30, 5], count=[9, 4], n=290),
    "many rows": dict(L=5, H=8, B=33, d=64, ps=16, m=[6] * 33, count=[i % 7 for i in range(33)], n=40),
}


def accept_case(rng, L, H, B, d, ps, m, count, n, cap_extra=2):
    m, count = np.array(m), np.array(count)
    sl = rng.integers(0, n + 1, size=(L, H, B)) + m
    bt, mp, _, cap = pages(rng, sl, ps, cap_extra=cap_extra)
    ts = np.concatenate([[0], np.cumsum(m)])
    path = rng.integers(-9, 9, size=ts[-1])
    for b in range(B):
        path[ts[b]:ts[b] + count[b]] = np.sort(rng.permutation(m[b])[:count[b]])
    return dict(L=L, H=H, B=B, d=d, ps=ps, ts=ts, count=count, path=path, sl=sl, bt=bt, mp=mp, cap=cap,
                kp=pool(rng, cap, ps, d), vp=pool(rng, cap, ps, d))


def call_accept(C, c, in_place=False):
    g = {k: dev(c[k]) for k in ("ts", "count", "path", "sl", "bt", "kp", "vp")}
    out = g["sl"] if in_place else torch.full_like(g["sl"], -7)
    C.kvs_accept_paged(C.dims(c["L"], c["H"], c["H"], c["d"]), c["B"], len(c["path"]), g["ts"], g["count"],
                       g["path"] if len(c["path"]) else None, c["ps"], g["kp"], g["vp"], c["cap"], g["bt"],
                       c["mp"], g["sl"], out)
    return dict(g, out=out)


@pytest.mark.parametrize("name", ACCEPT)
def test_accept(C, name):
    c = accept_case(np.random.default_rng(len(name)), **ACCEPT[name])
    kp, vp, sl = O.accept_paged(c["ts"], c["count"], c["path"], c["ps"], c["kp"].numpy(), c["vp"].numpy(),
                                c["bt"], c["sl"])
    for in_place in (False, True):
        r = call_accept(C, c, in_place)
        no_error(C)
        assert np.array_equal(raw(r["kp"]), kp) and np.array_equal(raw(r["vp"]), vp)
        assert np.array_equal(raw(r["out"]), sl) and np.array_equal(raw(r["bt"]), c["bt"])


def test_accept_refused_on_the_device(C):
    """A row that cannot be right stays as it is, the others go on."""
    base = dict(L=1, H=2, B=3, d=64, ps=4, m=[6, 5, 9], count=[3, 2, 4], n=9)

    def check(c, rows):
        r = call_accept(C, c)
        torch.cuda.synchronize()
        assert C.kvs_device_error() == 11 and C.kvs_device_error() == 0
        good = dict(c, count=c["count"].copy(), path=c["path"].copy(), ts=c["ts0"], bt=c["bt0"], sl=c["sl0"])
        want = [O.accept_paged(good["ts"], c["count0"], c["path0"], c["ps"], c[p].numpy(), c[p].numpy(),
                               good["bt"], good["sl"]) for p in ("kp", "vp")]
        out = want[0][2].copy()
        for p, (x, _, _) in zip(("kp", "vp"), want):
            x = x.copy()
            for l, h, b in rows:  # the pages of a row that stays
                ids = good["bt"][l, h, b][: -(-int(good["sl"][l, h, b]) // c["ps"])]
                x[ids] = c[p].numpy()[ids]
            assert np.array_equal(raw(r[p]), x), p
        for l, h, b in rows:
            out[l, h, b] = c["sl"][l, h, b]
        assert np.array_equal(raw(r["out"]), out)

    def fresh():
        c = accept_case(np.random.default_rng(4), **base)
        c.update({k + "0": c[k].copy() for k in ("ts", "count", "path", "sl", "bt")})
        return c

    both = [(0, 0, 1), (0, 1, 1)]
    for count in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        c = fresh()
        c["count"][1] = count
        check(c, both)
    for path in ([1, 1], [3, 2], [-1, 2], [0, 5], [0, 2 ** 31 - 1], [-2 ** 31, 0]):
        c = fresh()
        c["path"][6:8] = path
        check(c, both)
    for n in (4, -1, 2 ** 31 - 1, -2 ** 31, 4 * 100):
        c = fresh()
        c["sl"][0, 1, 1] = n
        check(c, [(0, 1, 1)])
    for page in (-1, 10 ** 6, 2 ** 31 - 1):
        c = fresh()
        base1 = int(c["sl"][0, 1, 1]) - 5
        c["bt"][0, 1, 1, base1 // 4] = page  # of the first slot that is written
        check(c, [(0, 1, 1)])
    for ts in ([0, 6, 11, 21], [0, 6, 11, 2 ** 31 - 1]):
        c = fresh()
        c["ts"] = np.array(ts)
        check(c, [(0, 0, 2), (0, 1, 2)])
    c = fresh()
    c["ts"] = np.array([-1, 6, 11, 20])
    check(c, [(0, 0, 0), (0, 1, 0)])


# ----------------------------------------------------------------------------- fork

FORK = {
    "one": dict(L=1, H=1, B=2, d=128, ps=16, src=[0], dst=[1], n=40, w=0),
    "one to many": dict(L=2, H=2, B=6, d=64, ps=4, src=[2] * 5, dst=[0, 5, 1, 4, 3], n=30, w=3),
    "pages of one": dict(L=1, H=2, B=4, d=64, ps=1, src=[0, 3], dst=[2, 1], n=9, w=0),
    "odd pages": dict(L=3, H=2, B=5, d=128, ps=13, src=[4, 0], dst=[1, 2], n=70, w=16),
    "a ring of several pieces": dict(L=1, H=2, B=3, d=128, ps=16, src=[1], dst=[0], n=5, w=129),
    "large pages": dict(L=1, H=2, B=3, d=64, ps=300, src=[1, 1], dst=[0, 2], n=900, w=1),
    "exactly as many pages": dict(L=2, H=2, B=3, d=64, ps=4, src=[0], dst=[2], n=17, w=0, room=0),
    "thousands of rows": dict(L=17, H=8, B=40, d=64, ps=2, src=list(range(20)), dst=list(range(20, 40)), n=7, w=1),
}


def fork_case(rng, L, H, B, d, ps, src, dst, n, w, room=3, empty=True):
    sl = rng.integers(0, n + 1, size=(L, H, B))
    if empty:
        sl.reshape(-1)[rng.integers(0, sl.size)] = 0
    sl[0, 0, src[0]] = n // ps * ps  # no page of its own
    src, dst = np.array(src), np.array(dst)
    new = int((sl[:, :, src] % ps > 0).sum())
    bt, mp, total, cap = pages(rng, sl, ps, spare=1, cap_extra=new + room)
    ring = lambda *s: torch.from_numpy(rng.standard_normal((L, H, B, w) + s).astype(np.float32))  # noqa: E731
    return dict(L=L, H=H, B=B, d=d, ps=ps, w=w, src=src, dst=dst, sl=sl, bt=bt, mp=mp, cap=cap, new=new,
                nxt=np.array([total]), kp=pool(rng, cap, ps, d), vp=pool(rng, cap, ps, d),
                pos=rng.integers(0, 3 * w + 1, size=B), rs=ring(), rk=ring(d).to(torch.bfloat16),
                rv=ring(d).to(torch.bfloat16))


def call_fork(C, c, in_place=False):
    g = {k: dev(c[k]) for k in ("src", "dst", "sl", "bt", "kp", "vp", "nxt", "pos", "rs", "rk", "rv")}
    out = g["nxt"] if in_place else torch.full_like(g["nxt"], -7)
    dm, w = C.dims(c["L"], c["H"], c["H"], c["d"]), c["w"]
    nb = C.kvs_fork_paged_workspace_size(dm, c["B"], len(c["src"]))
    ws = torch.full((nb,), 171, dtype=torch.uint8, device="cuda")
    C.kvs_fork_paged(dm, c["B"], len(c["src"]), g["src"], g["dst"], c["ps"], g["kp"], g["vp"], c["cap"],
                     g["nxt"], out, g["bt"], c["mp"], g["sl"], w, *((g["pos"], g["rs"], g["rk"], g["rv"])
                                                                   if w else [None] * 4), ws, nb)
    return dict(g, out=out)


@pytest.mark.parametrize("name", FORK)
def test_fork(C, name):
    c = fork_case(np.random.default_rng(len(name)), **FORK[name])
    kp, vp, nxt, bt, sl = O.fork_paged(c["src"], c["dst"], c["ps"], c["kp"].numpy(), c["vp"].numpy(),
                                       c["nxt"][0], c["bt"], c["sl"])
    order = np.arange(c["B"])
    order[c["dst"]] = c["src"]
    if not c["w"]:
        order = np.arange(c["B"])
    for in_place in (False, True):
        r = call_fork(C, c, in_place)
        no_error(C)
        assert np.array_equal(raw(r["kp"]), kp) and np.array_equal(raw(r["vp"]), vp)
        assert int(r["out"]) == nxt == c["nxt"][0] + c["new"]
        assert np.array_equal(raw(r["bt"]), bt) and np.array_equal(raw(r["sl"]), sl)
        assert np.array_equal(raw(r["pos"]), c["pos"][order])
        for k in ("rs", "rk", "rv"):
            assert torch.equal(r[k].cpu(), c[k][:, :, order]), k


def test_fork_refused_on_the_device(C):
    """All or nothing, and the error word tells why."""
    base = dict(L=2, H=2, B=6, d=64, ps=4, src=[0, 1], dst=[3, 5], n=30, w=3)

    def check(code, seed=5, **change):
        c = fork_case(np.random.default_rng(seed), **base)
        if "cap" in change:
            c["cap"] -= c["cap"] - int(c["nxt"][0]) - c["new"] + 1
            c["kp"], c["vp"] = c["kp"][:c["cap"]], c["vp"][:c["cap"]]
        for k, v in change.items():
            if k == "sl":
                c["sl"][1, 1, 1] = v
            elif k != "cap":
                c[k] = np.array(v)
        r = call_fork(C, c)
        torch.cuda.synchronize()
        assert C.kvs_device_error() == code and C.kvs_device_error() == 0
        for k in ("kp", "vp", "bt", "sl", "pos", "rs", "rk", "rv"):
            want = c[k] if isinstance(c[k], np.ndarray) else c[k].view(torch.int16).numpy() \
                if c[k].dtype == torch.bfloat16 else c[k].numpy()
            assert np.array_equal(raw(r[k]), want), (k, change)
        assert int(r["out"]) == c["nxt"][0]

    check(4, cap=None)
    check(4, nxt=[2 ** 31 - 1])
    check(11, nxt=[-1])
    for dst in ([3, 3], [3, 1], [0, 3], [3, 6], [-1, 3], [2 ** 31 - 1, 3]):
        check(11, dst=dst)
    for src in ([0, 6], [-1, 0], [0, 5], [-2 ** 31, 1]):
        check(11, src=src)
    for n in (-1, 2 ** 31 - 1, 4 * 100):
        check(11, sl=n)


def test_fork_of_a_row_with_a_bad_page(C):
    c = fork_case(np.random.default_rng(6), L=1, H=1, B=2, d=64, ps=4, src=[0], dst=[1], n=30, w=0, empty=False)
    c["sl"][0, 0, 0] = 7
    c["bt"][0, 0, 0, 1] = -1
    nxt = int(c["nxt"][0])
    c["cap"] = nxt + 1
    c["kp"], c["vp"] = (torch.ones(nxt + 1, 4, 64, dtype=torch.int16) for _ in range(2))
    r = call_fork(C, c)
    torch.cuda.synchronize()
    assert C.kvs_device_error() == 11
    assert (raw(r["kp"])[nxt] == 0).all() and (raw(r["kp"])[:nxt] == 1).all()
    assert raw(r["bt"])[0, 0, 1, :2].tolist() == [c["bt"][0, 0, 0, 0], nxt] and raw(r["sl"])[0, 0, 1] == 7


# ----------------------------------------------------------------------------- reclaim

RECLAIM = {
    "one row": dict(L=1, H=1, B=1, d=128, ps=16, n=100, spare=5),
    "nothing in use": dict(L=1, H=2, B=2, d=64, ps=4, n=0, spare=9),
    "nothing handed out": dict(L=1, H=2, B=2, d=64, ps=4, n=0, spare=0, cap_extra=3),
    "nothing to do": dict(L=2, H=2, B=3, d=64, ps=4, n=30, spare=0),
    "pages of one": dict(L=1, H=2, B=3, d=64, ps=1, n=40, spare=17),
    "odd pages, shared": dict(L=2, H=3, B=9, d=128, ps=13, n=300, spare=40, shared=4),
    "several chunks of bits": dict(L=2, H=8, B=40, d=64, ps=1, n=12, spare=1500, shared=5),
    "large pages": dict(L=1, H=2, B=3, d=64, ps=150, n=900, spare=7),
    "half finished": dict(L=2, H=4, B=16, d=64, ps=4, n=60, spare=20, gone=0.5, cap_extra=100),
}


def reclaim_case(rng, L, H, B, d, ps, n, spare, shared=0, gone=0.0, cap_extra=0):
    sl = rng.integers(0, n + 1, size=(L, H, B))
    bt, mp, total, cap = pages(rng, sl, ps, spare=spare, cap_extra=cap_extra, shared=shared)
    sl *= rng.uniform(size=B) >= gone
    return dict(L=L, H=H, B=B, d=d, ps=ps, sl=sl, bt=bt, mp=mp, cap=cap, nxt=np.array([total]),
                kp=pool(rng, cap, ps, d), vp=pool(rng, cap, ps, d))


def call_reclaim(C, c, in_place=False):
    g = {k: dev(c[k]) for k in ("sl", "bt", "kp", "vp", "nxt")}
    nxo = g["nxt"] if in_place else torch.full_like(g["nxt"], -7)
    bto = g["bt"] if in_place else torch.full_like(g["bt"], -7)
    dm = C.dims(c["L"], c["H"], c["H"], c["d"])
    nb = C.kvs_reclaim_paged_workspace_size(dm, c["B"], c["cap"])
    ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    C.kvs_reclaim_paged(dm, c["B"], c["ps"], g["kp"], g["vp"], c["cap"], g["nxt"], nxo, g["bt"], bto,
                        c["mp"], g["sl"], ws, nb)
    return dict(g, nxo=nxo, bto=bto)


@pytest.mark.parametrize("name", RECLAIM)
def test_reclaim(C, name):
    c = reclaim_case(np.random.default_rng(len(name)), **RECLAIM[name])
    kp, vp, n, bt = O.reclaim_paged(c["ps"], c["kp"].numpy(), c["vp"].numpy(), c["bt"], c["sl"])
    for in_place in (False, True):
        r = call_reclaim(C, c, in_place)
        no_error(C)
        assert int(r["nxo"]) == n and np.array_equal(raw(r["bto"]), bt)
        assert np.array_equal(raw(r["kp"]), kp) and np.array_equal(raw(r["vp"]), vp)
        assert in_place or np.array_equal(raw(r["bt"]), c["bt"])


def test_reclaim_refused_on_the_device(C):
    base = dict(L=2, H=2, B=4, d=64, ps=4, n=40, spare=6, cap_extra=5)

    def check(change):
        c = reclaim_case(np.random.default_rng(7), **base)
        change(c)
        r = call_reclaim(C, c)
        torch.cuda.synchronize()
        assert C.kvs_device_error() == 11 and C.kvs_device_error() == 0
        assert np.array_equal(raw(r["bto"]), c["bt"]) and int(r["nxo"]) == c["nxt"][0]
        assert np.array_equal(raw(r["kp"]), c["kp"].numpy()) and np.array_equal(raw(r["vp"]), c["vp"].numpy())

    def put(c, key, at, v):
        c[key][at] = v

    for v in (-1, 2 ** 31 - 1, -2 ** 31, "next", "cap"):
        def page(c, v=v):
            c["sl"][1, 1, 2] = 5
            c["bt"][1, 1, 2, 1] = {"next": c["nxt"][0], "cap": c["cap"]}.get(v, v)
        check(page)
    for v in (-1, 2 ** 31 - 1, -2 ** 31, 4 * 100):
        check(lambda c, v=v: put(c, "sl", (0, 1, 3), v))
    for v in (-1, -2 ** 31, 2 ** 31 - 1):
        check(lambda c, v=v: put(c, "nxt", 0, v))
    check(lambda c: put(c, "nxt", 0, c["cap"] + 1))


@pytest.mark.parametrize("cap", [250_000, 2_200_000])  # a word a chunk, 60 KB of them; more words a chunk
def test_reclaim_of_a_large_pool(C, cap):
    """Rows name the last of the pages and move to the front."""
    B, ps, d = 64, 1, 64
    dm = C.dims(1, 1, 1, d)
    kp = torch.zeros(cap, ps, d, dtype=torch.bfloat16, device="cuda")
    ids = torch.cat([torch.tensor([0, 5, 31, 32, 1024]), torch.arange(cap - 59, cap)]).int()
    kp[ids.long().cuda(), 0, 0] = torch.arange(B, device="cuda").to(torch.bfloat16)
    order = torch.randperm(B, generator=torch.Generator().manual_seed(1))
    bt = ids[order].view(1, 1, B, 1).cuda()
    nxt = torch.tensor([cap], dtype=torch.int32, device="cuda")
    nb = C.kvs_reclaim_paged_workspace_size(dm, B, cap)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    C.kvs_reclaim_paged(dm, B, ps, kp, kp.clone(), cap, nxt, nxt, bt, bt, 1,
                        torch.ones(1, 1, B, dtype=torch.int32, device="cuda"), ws, nb)
    no_error(C)
    assert int(nxt) == B and sorted(bt.flatten().tolist()) == list(range(B))
    assert kp[bt.flatten().long(), 0, 0].float().cpu().int().tolist() == order.tolist()
    stay = {0: 0, 1: 5, 2: 31, 3: 32}
    for i, page in stay.items():
        assert int(bt.flatten()[int((order == i).nonzero())]) == page


# ----------------------------------------------------------------------------- together

def test_calls_are_captured_and_replayed(C):
    """One graph of all three on its own stream; each replay on new contents of the same tensors
    gives what the calls give."""
    c = accept_case(np.random.default_rng(8), L=2, H=2, B=4, d=64, ps=4, m=[6, 5, 9, 2], count=[3, 2, 4, 1], n=30,
                    cap_extra=30)
    dm = C.dims(2, 2, 2, 64)
    g = {k: dev(c[k]) for k in ("ts", "count", "path", "sl", "bt", "kp", "vp")}
    used = int((-(-c["sl"] // 4)).sum())
    g["nxt"] = dev(np.array([used]))
    src, dst = dev(np.array([0])), dev(np.array([2]))
    first = {k: g[k].clone() for k in g}
    w1 = torch.empty(C.kvs_fork_paged_workspace_size(dm, 4, 1), dtype=torch.uint8, device="cuda")
    w2 = torch.empty(C.kvs_reclaim_paged_workspace_size(dm, 4, c["cap"]), dtype=torch.uint8, device="cuda")

    def step():
        C.kvs_accept_paged(dm, 4, len(c["path"]), g["ts"], g["count"], g["path"], 4, g["kp"], g["vp"], c["cap"],
                           g["bt"], c["mp"], g["sl"], g["sl"])
        C.kvs_fork_paged(dm, 4, 1, src, dst, 4, g["kp"], g["vp"], c["cap"], g["nxt"], g["nxt"], g["bt"], c["mp"],
                         g["sl"], 0, None, None, None, None, w1, w1.numel())
        C.kvs_reclaim_paged(dm, 4, 4, g["kp"], g["vp"], c["cap"], g["nxt"], g["nxt"], g["bt"], g["bt"], c["mp"],
                            g["sl"], w2, w2.numel())

    def want(s, d):
        kp, vp, sl = O.accept_paged(c["ts"], c["count"], c["path"], 4, c["kp"].numpy(), c["vp"].numpy(), c["bt"],
                                    c["sl"])
        kp, vp, nxt, bt, sl = O.fork_paged([s], [d], 4, kp, vp, used, c["bt"], sl)
        kp, vp, n, bt = O.reclaim_paged(4, kp, vp, bt, sl)
        return kp, vp, n, bt, sl

    def check(s, d):
        kp, vp, n, bt, sl = want(s, d)
        no_error(C)
        assert np.array_equal(raw(g["sl"]), sl) and np.array_equal(raw(g["bt"]), bt) and int(g["nxt"]) == n
        for r in np.ndindex(*sl.shape):
            ids = bt[r][: -(-int(sl[r]) // 4)]
            assert np.array_equal(raw(g["kp"])[ids], kp[ids]) and np.array_equal(raw(g["vp"])[ids], vp[ids])

    step()
    check(0, 2)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            step()
    for s, d in ((0, 2), (3, 1), (1, 0)):
        for k in g:
            g[k].copy_(first[k])
        src.fill_(s)
        dst.fill_(d)
        torch.cuda.synchronize()
        graph.replay()
        check(s, d)
