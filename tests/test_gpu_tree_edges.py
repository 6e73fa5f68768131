"""Edges of kvs_attn_tree: tables with room for more keys than L2 holds (whose keys are copied with
a policy of their own), no pages at all, sequences with bad token starts, and large finite values
in drafted tokens.  Tolerances as in test_gpu_tree.py."""
import numpy as np
import pytest
import torch

from .gpu_util import f64, need_gpu
from .test_gpu_tree import U, call, case, check, expected

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def C():
    need_gpu()
    from kv_cache_eviction_lse_gb300 import build
    build.build()
    from kv_cache_eviction_lse_gb300 import capi
    return capi


def fine(C):
    torch.cuda.synchronize()
    assert C.kvs_device_error() == 0


# ----------------------------------------------------------------------------- wide tables

# A query tile a row and tables with room for more than 64.5 MB of keys and values in all: the room
# counts, not what is in it.
WIDE = {
    "pages of 16": dict(B=3, m=[9, 1, 32], n=2000, ps=16),
    "pages of 32, d = 64": dict(B=3, m=[9, 1, 32], n=2000, ps=32, d=64),
    "pages of 8, ring": dict(B=3, m=[5, 12, 2], n=700, ps=8, w=40),
    "pages of 128, ring, d = 64": dict(B=2, m=[64, 3], n=900, ps=128, w=129, d=64),
    "odd pages, six heads": dict(B=3, m=[12, 0, 21], n=800, ps=13, Hq=12, H=2),
    "odd pages, ring, d = 64": dict(B=4, m=[3, 8, 1, 2], n=300, ps=7, w=16, d=64),
    "pages of one": dict(B=2, m=[17, 4], n=300, ps=1),
    "split over many blocks": dict(Hq=4, H=1, B=1, m=[9], n=30000, n_lo=30000),
    "split, d = 64, chain": dict(Hq=8, H=4, B=2, m=[16, 60], n=9000, d=64, kind="chain"),
    "only drafts, padding": dict(B=4, m=[9, 0, 1, 33], n=0, pad=5),
    "many short rows": dict(L=2, Hq=8, H=8, B=16, m=[3] * 16, n=60, d=64),
}


@pytest.mark.parametrize("name", WIDE)
def test_wide_tables(C, name):
    c = case(len(name) + 40, **WIDE[name])
    rows, tile = c["L"] * c["H"] * c["B"], 2 * 128 * c["d"] * 2
    assert c["md"] * (c["Hq"] // c["H"]) <= 128
    room = (129 << 19) // (rows * tile) + 2  # tiles of 128 keys a row
    mp = max(c["mp"], -(-room * 128 // c["ps"]))
    wide = dict(c, mp=mp, bt=np.full((c["L"], c["H"], c["B"], mp), -9, dtype=np.int32))
    wide["bt"][..., :c["mp"]] = c["bt"]
    assert rows * -(-mp * c["ps"] // 128) * tile > 129 << 19
    r = call(C, wide)
    fine(C)
    check(wide, r, name)
    narrow = call(C, c)  # shares go by the rows' keys, so the bits are the same
    fine(C)
    assert torch.equal(r["o"], narrow["o"]) and torch.equal(r["lse"], narrow["lse"])
    first = r["o"].clone()
    for _ in range(3):
        r["go"]()
    assert torch.equal(r["o"], first)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("d, ps", [(64, 16), (128, 16), (128, 13), (64, 5)])
def test_unseen_drafts_leave_no_trace_in_wide_tables(C, bad, d, ps):
    """Every other root of a star holds infinities or NaN: the others are as without, to the bit."""
    c = case(50, B=2, m=[6, 32], n=3000, n_lo=3000, d=d, ps=ps, kind="star")
    mp = max(c["mp"], (129 << 19) // (4 * 4 * d * ps) + 2)
    bt = np.full((1, 2, 2, mp), -9, dtype=np.int32)
    bt[..., :c["mp"]] = c["bt"]
    c = dict(c, mp=mp, bt=bt)
    clean = call(C, c)
    fine(C)
    kp, vp = c["kp"].clone(), c["vp"].clone()
    for l, h, b in np.ndindex(1, 2, 2):
        for i in range(1, int(c["m"][b]), 2):
            slot = int(c["sl"][l, h, b]) - int(c["m"][b]) + i
            at = c["bt"][l, h, b, slot // ps], slot % ps
            kp[at], vp[at] = bad, bad
    r = call(C, dict(c, kp=kp, vp=vp))
    fine(C)
    even = [int(c["ts"][b]) + i for b in range(2) for i in range(0, int(c["m"][b]), 2)]
    assert torch.equal(r["o"][:, :, even], clean["o"][:, :, even])
    assert torch.equal(r["lse"][:, :, even], clean["lse"][:, :, even])


# ----------------------------------------------------------------------------- no pages

def over_the_ring(c):
    """o, lse, sum a |v| and the tolerance of the logits of tokens that see the ring alone."""
    g = c["Hq"] // c["H"]
    q, rk, rv = (f64(c[k]) for k in ("q", "rk", "rv"))
    o, sp = np.zeros(q.shape), np.zeros(q.shape)
    lse, delta = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    for b in range(c["B"]):
        held, t = min(int(c["pos"][b]), c["w"]), slice(int(c["ts"][b]), int(c["ts"][b + 1]))
        if not held:
            continue
        for l, hq in np.ndindex(c["L"], c["Hq"]):
            K, V = rk[l, hq // g, b, :held], rv[l, hq // g, b, :held]
            x = q[l, hq, t] @ K.T / np.sqrt(c["d"])
            top = x.max(1, keepdims=True)
            a = np.exp(x - top)
            z = a.sum(1, keepdims=True)
            o[l, hq, t], sp[l, hq, t], lse[l, hq, t] = a / z @ V, a / z @ np.abs(V), (top + np.log(z))[:, 0]
            size = (np.abs(q[l, hq, t]) @ np.abs(K).T).max(1) / np.sqrt(c["d"])
            delta[l, hq, t] = (c["d"] + 8) * U * size + 2.0 ** -20 * np.abs(x).max(1)
    return o, lse, sp, delta


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [0, 50])
def test_no_pages_at_all(C, d, n):
    """capacity_pages = 0 and no pointers: the drafted tokens lie before slot 0 (n = 0) or on pages
    that are not there, which sets the error word, and tokens see the ring alone, if it holds any."""
    c = case(51, B=3, m=[4, 1, 9], n=n, n_lo=n, d=d, w=5, pad=2)
    c["pos"] = np.array([2, 0, 17], dtype=np.int32)
    c = dict(c, kp=None, vp=None, cap=0, sl=np.full_like(c["sl"], n))
    r = call(C, c)
    torch.cuda.synchronize()
    assert C.kvs_device_error() == 10 and C.kvs_device_error() == 0
    o, lse, sp, delta = (x[:, :, :14] for x in over_the_ring(c))
    got, got_lse = f64(r["o"])[:, :, :14], r["lse"].double().cpu().numpy()[:, :, :14]
    none = np.isinf(lse)
    assert np.array_equal(got_lse[none], lse[none]) and (got[none] == 0).all() and none.any()
    err = np.abs(got_lse[~none] - lse[~none])
    assert (err <= delta[~none] + 2.0 ** -20 * (1 + np.abs(lse[~none])) + 40 * U).all()
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.1 * delta[..., None] + 40 * U) * sp
    assert (np.abs(got - o) <= tol).all()
    assert (r["o"][:, :, 14:] == 7.0).all() and (r["lse"][:, :, 14:] == 7.0).all()


def test_no_pages_and_no_ring(C):
    """Nothing is there to see: zeros and -inf."""
    c = case(52, B=2, m=[4, 130], n=40, n_lo=40, d=64)
    c = dict(c, kp=None, vp=None, cap=0)
    r = call(C, c)
    torch.cuda.synchronize()
    assert C.kvs_device_error() == 10
    assert (r["o"] == 0).all() and (r["lse"] == -np.inf).all()


# ----------------------------------------------------------------------------- bad states

@pytest.mark.parametrize("ts, good", [
    ([0, 5, 4, 18], [0]), ([-1, 5, 9, 18], [1, 2]), ([0, 5, 9, 19], [0, 1]), ([0, 5, 2 ** 31 - 1, 18], [0]),
    ([0, 5, 9, 2 ** 31 - 1], [0, 1]), ([-2 ** 31, 5, 9, 18], [1, 2])])
@pytest.mark.parametrize("d", [64, 128])
def test_sequences_with_bad_starts_get_no_results(C, ts, good, d):
    """Theirs stay as they were, the others' are right."""
    c = case(53, B=3, m=[5, 4, 9], n=150, d=d, Hq=4, H=2)
    want = expected(c)
    r = call(C, dict(c, ts=np.array(ts, dtype=np.int32)))
    torch.cuda.synchronize()
    assert C.kvs_device_error() == 10 and C.kvs_device_error() == 0
    theirs = np.zeros(c["N"], dtype=bool)
    for b in good:
        theirs[c["ts"][b]:c["ts"][b + 1]] = True
    assert (r["o"][:, :, ~theirs] == 7.0).all() and (r["lse"][:, :, ~theirs] == 7.0).all()
    o, lse, sp, delta = (x[:, :, theirs] for x in want)
    n = int(c["sl"].max())
    err = np.abs(r["lse"].double().cpu().numpy()[:, :, theirs] - lse)
    assert (err <= delta + 2.0 ** -20 * (1 + np.abs(lse)) + (n + 32) * U).all()
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.1 * delta[..., None] + (n + 32) * U) * sp
    assert (np.abs(f64(r["o"])[:, :, theirs] - o) <= tol).all()


@pytest.mark.parametrize("d", [64, 128])
def test_large_finite_values_of_drafts_count_where_they_are_seen(C, d):
    """2^100 in V of one drafted token a sequence (2^8 of a weight and the keys' number above it stay
    finite): nothing is taken for an infinity, and who does not see it has no part of it."""
    for m, kind, n in (([6, 40], "star", 100), ([130, 256], "random", 60), ([33, 3], "chain", 3000)):
        c = case(54, B=2, m=m, n=n, n_lo=n, d=d, kind=kind)
        clean = call(C, c)
        vp = c["vp"].clone()
        who = [2, m[1] - 2]
        for l, h, b in np.ndindex(1, 2, 2):
            slot = int(c["sl"][l, h, b]) - m[b] + who[b]
            vp[c["bt"][l, h, b, slot // 16], slot % 16, ::3] = 2.0 ** 100
        c2 = dict(c, vp=vp)
        r = call(C, c2)
        fine(C)
        check(c2, r, (m, kind))
        for b in range(2):
            t0 = int(c["ts"][b])
            up = []
            for i in range(m[b]):
                p = int(c["parent"][t0 + i])
                up.append({i} | (up[p] if p >= 0 else set()))
            blind = [t0 + i for i in range(m[b]) if who[b] not in up[i]]
            assert torch.equal(r["o"][:, :, blind], clean["o"][:, :, blind])
