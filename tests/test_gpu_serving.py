"""GPU parity of the rotation, the paged append and the paged decode attention against the
fp64 oracle, at the sizes and states where they can go wrong, and their use together.

Tolerances, from the arithmetic (u = 2^-24, an fp32 rounding; 2^-8, a bf16 rounding):
  rotation   |err| <= 2^-8 |y| + 2^-20 (|a| + |b|): the output's rounding; the angle is good
             to 2^-22, the hardware's cosine and sine of it to 2^-21.2, and the two products
             and their sum add three fp32 roundings (together below 2^-20 of the pair's size)
  attention  logits: |dx| <= delta = (d + 8) u max_i sum_e |q_e k_ie| / sqrt(d) + 2^-20 |x|max
             (fp32 sums in any order, the scale by log2 e, ex2 to 2^-22)
             lse: delta + 2^-20 (1 + |lse|) + (n / 8 + 16) u (sums of positive terms: at most
             n / 8 of them in sequence, and the join)
             o: 2^-8 |o| (output) + (2^-8 + 2.1 delta + (n + 32) u) sum a |v| (weights rounded
             to bf16, their error from the logits in numerator and denominator, the sums)
"""
import threading

import numpy as np
import pytest
import torch

import oracle as O
from .gpu_util import f64, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def C():
    need_gpu()
    from kv_cache_eviction_lse_gb300 import build
    build.build()
    from kv_cache_eviction_lse_gb300 import capi
    return capi


def freqs(rot, base=1e6):
    return base ** (-np.arange(0, rot, 2, dtype=np.float64) / max(rot, 1))


def bits(t):
    return t.detach().contiguous().cpu().view(torch.int16).numpy()


def check_rotated(got, x, pos, rot, f, il, what):
    x64 = f64(x)
    want = O.rope(x64, pos, f, rot, il)
    size = np.abs(x64).copy()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if il else (slice(0, rot // 2), slice(rot // 2, rot))
    size[..., a] = size[..., b] = np.abs(x64[..., a]) + np.abs(x64[..., b])
    err = np.abs(f64(got) - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size).all(), (what, err.max())
    assert np.array_equal(bits(got)[..., rot:], bits(x)[..., rot:]), what


# ----------------------------------------------------------------------------- rotation

ROPE = [
    # L, Hq, Hkv, N, d, rot, interleaved
    (1, 4, 2, 1, 128, 128, False),
    (2, 12, 2, 77, 128, 128, False),
    (1, 3, 1, 1025, 64, 64, True),
    (1, 32, 8, 64, 128, 128, True),
    (3, 2, 2, 33, 128, 64, False),
    (1, 5, 5, 31, 64, 32, True),
    (1, 2, 1, 9, 128, 16, False),
    (1, 2, 1, 9, 64, 48, False),
    (1, 2, 2, 40, 128, 0, False),
    (7, 64, 8, 5, 64, 64, False),
]


@pytest.mark.parametrize("shape", ROPE, ids=str)
def test_rope(C, shape):
    L, Hq, Hkv, N, d, rot, il = shape
    gen = torch.Generator().manual_seed(N + rot)
    q = torch.randn(L, Hq, N, d, generator=gen).to(torch.bfloat16)
    k = torch.randn(L, Hkv, N, d, generator=gen).to(torch.bfloat16)
    pos = torch.randint(-50, 1 << 20, (N,), generator=gen, dtype=torch.int32)
    pos[0] = 0
    f = freqs(rot)
    dm = C.dims(L, Hq, Hkv, d)
    qg, kg, pg = q.cuda(), k.cuda(), pos.cuda()
    qo, ko = torch.full_like(qg, 9.0), torch.full_like(kg, 9.0)
    C.kvs_rope(dm, N, pg, rot, f, il, qg, qo, kg, ko)
    check_rotated(qo, q, pos.numpy(), rot, f, il, "q")
    check_rotated(ko, k, pos.numpy(), rot, f, il, "k")
    assert torch.equal(qg.cpu(), q) and torch.equal(kg.cpu(), k)
    # in place, one at a time, the same bits
    C.kvs_rope(dm, N, pg, rot, f, il, qg, qg, None, None)
    C.kvs_rope(dm, N, pg, rot, f, il, None, None, kg, kg)
    assert np.array_equal(bits(qg), bits(qo)) and np.array_equal(bits(kg), bits(ko))


def test_rope_far_positions_and_whole_turns(C):
    """Whole turns come off without loss: positions at both ends of 32 bits, a frequency of
    one turn a position and of none.  Frequencies up to 1e-3, so that the oracle's own fp64
    product is good to 2^-30 there."""
    d = 64
    f = np.minimum(freqs(d), 1e-3)
    f[:5] = [1e-3, -1e-3, 2 * np.pi, 0.0, 5e-4]
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 123456789, -1, 1], dtype=np.int32)
    x = torch.ones(1, 1, len(pos), d, dtype=torch.bfloat16)
    y = torch.empty_like(x, device="cuda")
    C.kvs_rope(C.dims(1, 1, 1, d), len(pos), torch.from_numpy(pos).cuda(), d, f, False, x.cuda(), y,
               None, None)
    got, p = f64(y)[0, 0], pos.astype(np.float64)
    for i in range(32):
        t = np.zeros_like(p) if i == 2 else p * f[i]
        tol = 2.0 ** -8 * 1.42 + 2.0 ** -19
        assert (np.abs(got[:, i] - (np.cos(t) - np.sin(t))) <= tol).all(), i
        assert (np.abs(got[:, i + 32] - (np.cos(t) + np.sin(t))) <= tol).all(), i


def test_rope_backward_is_the_rotation_back(C):
    """The gradient of sum(y z) with respect to x is z rotated by negated frequencies: against
    the formula's, and against differences of the kernel itself (y is linear in x, so steps
    are exact up to the roundings of the two outputs)."""
    L, H, N, d = 1, 2, 6, 64
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(L, H, N, d, generator=gen).to(torch.bfloat16)
    z = torch.randn(L, H, N, d, generator=gen).to(torch.bfloat16)
    pos, f = torch.arange(5, 5 + N, dtype=torch.int32), freqs(d, 100.0)
    for il in (False, True):
        dm, grad = C.dims(L, H, H, d), torch.empty_like(z, device="cuda")
        C.kvs_rope(dm, N, pos.cuda(), d, -f, il, z.cuda(), grad, None, None)
        check_rotated(grad, z, pos.numpy(), d, -f, il, "gradient")
        g = f64(grad)
        for dim in (0, 1, 17, 31, 32, 63):
            step = torch.zeros(d)
            step[dim] = 2.0
            out = []
            for sgn in (1, -1):
                xs = (x.float() + sgn * step).to(torch.bfloat16)
                y = torch.empty_like(xs, device="cuda")
                C.kvs_rope(dm, N, pos.cuda(), d, f, il, xs.cuda(), y, None, None)
                out.append((f64(xs), f64(y)))
            h = out[0][0][..., dim] - out[1][0][..., dim]
            diff = ((out[0][1] - out[1][1]) * f64(z)).sum(-1) / h
            # two of the outputs of each side are off by 2^-8 of at most |a| + |b|
            touched = np.abs(out[0][1]) + np.abs(out[1][1])
            tol = (2.0 ** -8 * touched * np.abs(f64(z))).sum(-1) / h + 2.0 ** -8 * np.abs(g[..., dim])
            assert (np.abs(diff - g[..., dim]) <= tol + 1e-4).all()


# ----------------------------------------------------------------------------- append

def cache(gen, L, H, B, d, ps, n, cap, mp, scatter=True):
    """Pools of `cap` pages with rows of n [L][H][B] tokens, every page handed out so far at
    a random place below the counter."""
    need = -(-n // ps)
    total = int(need.sum())
    assert total <= cap and int(need.max()) <= mp
    bt = torch.full((L, H, B, mp), -1, dtype=torch.int32)
    ids = torch.randperm(total, generator=gen) if scatter else torch.arange(total)
    i = 0
    for r in np.ndindex(L, H, B):
        for p in range(int(need[r])):
            bt[r][p] = ids[i]
            i += 1
    kp = torch.randn(cap, ps, d, generator=gen).to(torch.bfloat16)
    vp = torch.randn(cap, ps, d, generator=gen).to(torch.bfloat16)
    return dict(kp=kp, vp=vp, bt=bt, sl=torch.from_numpy(n.astype(np.int32)),
                nxt=torch.tensor([total], dtype=torch.int32))


def append_case(C, L, Hq, H, B, d, ps, m, nmax, rot=None, il=False, pad=0, single=False, extra=0,
                seed=0, mp_extra=1):
    gen = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    m = np.asarray(m)
    n = rng.integers(0, nmax + 1, size=(L, H, B))
    have, end = -(-n // ps), -(-(n + m) // ps)
    mp, cap = int(end.max()) + mp_extra, int(end.sum()) + extra
    st = cache(gen, L, H, B, d, ps, n, max(cap, int(have.sum())), max(mp, 1))
    N = int(m.sum()) + pad
    ts = np.concatenate([[0], np.cumsum(m)]).astype(np.int32)
    rot = d if rot is None else rot
    return dict(st, C=C, dm=C.dims(L, Hq, H, d), L=L, H=H, B=B, d=d, ps=ps, N=N, rot=rot, il=il,
                f=freqs(rot), ts=ts, single=single, mp=st["bt"].shape[-1], cap=st["kp"].shape[0],
                q=torch.randn(L, Hq, N, d, generator=gen).to(torch.bfloat16),
                k=torch.randn(L, H, N, d, generator=gen).to(torch.bfloat16),
                v=torch.randn(L, H, N, d, generator=gen).to(torch.bfloat16),
                pos=torch.randint(0, 100000, (N,), generator=gen, dtype=torch.int32))


def call_append(c, in_place=False, with_q=True):
    C = c["C"]
    g = {n: c[n].cuda() for n in ("kp", "vp", "bt", "sl", "nxt", "q", "k", "v", "pos")}
    ts = None if c["single"] else torch.from_numpy(c["ts"]).cuda()
    slo, nxo = (g["sl"], g["nxt"]) if in_place else (torch.full_like(g["sl"], -7),
                                                     torch.full_like(g["nxt"], -7))
    qo = g["q"] if in_place else torch.full_like(g["q"], 9.0)
    nb = C.kvs_append_paged_workspace_size(c["dm"], c["B"])
    ws = torch.full((nb,), 171, dtype=torch.uint8, device="cuda")
    C.kvs_append_paged(c["dm"], c["B"], c["N"], ts, g["pos"], c["rot"], c["f"], c["il"],
                       g["q"] if with_q else None, qo if with_q else None, g["k"], g["v"], c["ps"],
                       g["kp"], g["vp"], c["cap"], g["nxt"], nxo, g["bt"], c["mp"], g["sl"], slo,
                       ws, nb)
    torch.cuda.synchronize()
    return dict(g, slo=slo, nxo=nxo, qo=qo)


def check_append(c, r):
    used = int(c["ts"][-1])
    if used:
        k = O.rope(f64(c["k"]), c["pos"].numpy(), c["f"], c["rot"], c["il"])
    else:
        k = np.zeros((c["L"], c["H"], 0, c["d"]))
    k16 = torch.from_numpy(k)
    want = O.append_paged(k16.numpy(), f64(c["v"]), c["ts"], c["ps"], f64(c["kp"]), f64(c["vp"]),
                          int(c["nxt"]), c["bt"].numpy(), c["sl"].numpy())
    assert not isinstance(want, str)
    kp, vp, nxt, bt, sl = want
    assert int(r["nxo"]) == nxt
    assert np.array_equal(r["slo"].cpu().numpy(), sl)
    assert np.array_equal(r["bt"].cpu().numpy(), bt)
    assert np.array_equal(f64(r["vp"]), vp)
    # K pages: the appended rows to the rotation's tolerance, all others to the bit
    got = f64(r["kp"])
    mag = np.abs(f64(c["k"])).max() if used else 0.0
    err = np.abs(got - kp)
    assert (err <= 2.0 ** -8 * np.abs(kp) + 2.0 ** -19 * mag).all(), err.max()
    for l, h, b in np.ndindex(c["L"], c["H"], c["B"]):
        for t in range(c["ts"][b], c["ts"][b + 1]):
            s = int(c["sl"][l, h, b]) + t - c["ts"][b]
            row = r["kp"][bt[l, h, b, s // c["ps"]], s % c["ps"]]
            check_rotated(row[None], c["k"][l, h, t][None], c["pos"][t:t + 1].numpy(), c["rot"],
                          c["f"], c["il"], (l, h, b, t))
            kp[bt[l, h, b, s // c["ps"]], s % c["ps"]] = f64(row)
    assert np.array_equal(got, kp)


APPENDS = {
    "one token each": dict(L=1, Hq=4, H=2, B=5, d=128, ps=16, m=[1] * 5, nmax=40, single=True),
    "one token, starts given": dict(L=2, Hq=4, H=2, B=3, d=64, ps=4, m=[1] * 3, nmax=9),
    "pages of one": dict(L=1, Hq=2, H=2, B=2, d=64, ps=1, m=[3, 2], nmax=5),
    "ragged with empty sequences": dict(L=2, Hq=6, H=3, B=6, d=128, ps=13, m=[0, 17, 1, 0, 40, 0],
                                        nmax=30),
    "padded batch": dict(L=1, Hq=2, H=1, B=3, d=128, ps=16, m=[5, 0, 7], nmax=20, pad=21),
    "all padding": dict(L=1, Hq=2, H=1, B=2, d=64, ps=16, m=[0, 0], nmax=20, pad=5),
    "empty cache, whole prompt": dict(L=1, Hq=4, H=2, B=1, d=128, ps=16, m=[133], nmax=0),
    "exactly full pages": dict(L=1, Hq=2, H=2, B=2, d=64, ps=8, m=[16, 8], nmax=0, mp_extra=0),
    "large pages": dict(L=1, Hq=2, H=2, B=3, d=64, ps=300, m=[3, 310, 1], nmax=400),
    "partly rotated, interleaved": dict(L=1, Hq=4, H=4, B=2, d=64, ps=5, m=[9, 4], nmax=11, rot=32,
                                        il=True),
    "not rotated": dict(L=1, Hq=4, H=4, B=2, d=128, ps=16, m=[9, 4], nmax=11, rot=0),
    "many rows": dict(L=9, Hq=16, H=16, B=24, d=64, ps=4, m=[1] * 24, nmax=9, single=True),
}


@pytest.mark.parametrize("name", APPENDS)
def test_append(C, name):
    c = append_case(C, seed=len(name), **APPENDS[name])
    r = call_append(c)
    assert C.kvs_device_error(clear=True) == 0
    check_append(c, r)
    used = int(c["ts"][-1])
    if used:
        check_rotated(r["qo"][:, :, :used], c["q"][:, :, :used], c["pos"][:used].numpy(), c["rot"],
                      c["f"], c["il"], "q")
    assert (r["qo"][:, :, used:] == 9.0).all()          # padding left as it was
    # in place, the same; without queries, the same pages
    p = call_append(c, in_place=True)
    for n in ("kp", "vp", "bt"):
        assert torch.equal(p[n], r[n]), n
    assert torch.equal(p["sl"], r["slo"]) and torch.equal(p["nxt"], r["nxo"])
    assert torch.equal(p["q"][:, :, :used], r["qo"][:, :, :used])
    w = call_append(c, with_q=False)
    assert torch.equal(w["kp"], r["kp"]) and torch.equal(w["vp"], r["vp"])


def refused(C, c, code):
    r = call_append(c)
    assert C.kvs_device_error(clear=True) == code
    for n in ("kp", "vp", "bt", "sl", "nxt"):
        assert torch.equal(r[n].cpu(), c[n]), n
    assert torch.equal(r["slo"], r["sl"]) and torch.equal(r["nxo"], r["nxt"])
    assert (r["qo"] == 9.0).all()


def test_append_refused_on_the_device(C):
    """Everything the kernel itself has to check: the call leaves all state as it was and
    the error word tells why."""
    base = dict(L=2, Hq=4, H=2, B=3, d=64, ps=4, m=[5, 0, 9], nmax=9, seed=5)
    c = append_case(C, extra=-1, **base)                  # pool one page short
    refused(C, c, 4)
    c = append_case(C, mp_extra=-1, **base)               # one row's table one page short
    refused(C, c, 5)
    for ts in ([0, 5, 4, 14], [1, 5, 5, 14], [0, 5, 5, 15], [0, -3, 5, 14], [0, 2 ** 31 - 1, -5, 14]):
        c = append_case(C, **base)
        c["ts"] = np.array(ts, dtype=np.int32)
        refused(C, c, 8)
    for n in (-1, -2 ** 31, 2 ** 31 - 1, 4 * 100):
        c = append_case(C, **base)
        c["sl"][1, 1, 2] = n
        refused(C, c, 8)
    for page in (-1, 2 ** 31 - 1, None):
        c = append_case(C, **base)
        c["sl"][0, 1, 0] = 6                              # in the middle of its second page
        c["bt"][0, 1, 0, 1] = c["cap"] if page is None else page
        refused(C, c, 8)
    c = append_case(C, **base)
    c["nxt"][0] = -1
    refused(C, c, 8)
    # thousands of rows, planned by several blocks: a short pool, a bad length in the last row
    many = dict(L=5, Hq=16, H=16, B=30, d=64, ps=2, m=[1] * 30, nmax=5, single=True, seed=6)
    refused(C, append_case(C, extra=-1, **many), 4)
    c = append_case(C, **many)
    c["sl"][4, 15, 29] = -1
    refused(C, c, 8)
    # and the same call with a pool that is large enough goes through
    c = append_case(C, **base)
    check_append(c, call_append(c))
    assert C.kvs_device_error(clear=True) == 0


def test_append_to_more_rows_than_plan_threads(C):
    """135168 rows, more than one a thread of the plan: every row's first token takes the page
    of the row's number; the next two calls fill it and take another."""
    L, H, B, d, ps = 33, 64, 64, 64, 2
    rows, dm = L * H * B, C.dims(L, H, H, d)
    kp = torch.zeros(2 * rows, ps, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    bt = torch.full((L, H, B, 2), -1, dtype=torch.int32, device="cuda")
    sl = torch.zeros(L, H, B, dtype=torch.int32, device="cuda")
    nxt = torch.zeros(1, dtype=torch.int32, device="cuda")
    nb = C.kvs_append_paged_workspace_size(dm, B)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    toks = []
    for i in range(3):
        k = torch.randn(L, H, B, d, generator=gen, device="cuda").to(torch.bfloat16)
        toks.append(k)
        C.kvs_append_paged(dm, B, B, None, None, 0, None, False, None, None, k, -k, ps, kp, vp,
                           2 * rows, nxt, nxt, bt, 2, sl, sl, ws, nb)
    assert C.kvs_device_error(clear=True) == 0
    first = torch.arange(rows, dtype=torch.int32, device="cuda").view(L, H, B)
    assert torch.equal(bt[..., 0], first) and torch.equal(bt[..., 1], first + rows)
    assert (sl == 3).all() and int(nxt) == 2 * rows
    got = kp.view(2, L, H, B, ps, d)
    for i, (page, r) in enumerate(((0, 0), (0, 1), (1, 0))):
        assert torch.equal(got[page, :, :, :, r], toks[i])
    assert not got[1, :, :, :, 1].any() and torch.equal(vp, -kp)


def test_append_taken_back(C):
    """A draft appended out of place and dropped: the next append from the old state gives
    what it gives without the draft."""
    c = append_case(C, L=1, Hq=2, H=2, B=2, d=64, ps=4, m=[3, 6], nmax=10, seed=8)
    plain = call_append(c)
    draft = dict(c, k=c["k"] + 1, v=c["v"] * 2)
    d = call_append(draft)
    again = call_append(dict(c, kp=d["kp"].cpu(), vp=d["vp"].cpu(), bt=d["bt"].cpu()))
    for n in ("kp", "vp", "bt", "slo", "nxo"):
        assert torch.equal(again[n], plain[n]), n


def test_append_and_attend_captured_and_replayed(C):
    """A captured pair of calls with the state in place: every replay appends the next token
    behind the last and attends over all of them, as the same calls do without a graph; on
    the legacy default stream too."""
    L, Hq, H, B, d, ps, steps = 1, 8, 2, 3, 128, 4, 11
    gen = torch.Generator().manual_seed(21)
    dm, f, mp = C.dims(L, Hq, H, d), freqs(d), 8
    rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16)  # noqa: E731
    toks = [(rnd(L, Hq, B, d), rnd(L, H, B, d), rnd(L, H, B, d)) for _ in range(steps)]
    runs = {}
    for how in ("graph", "eager", "default stream"):
        g = dict(kp=torch.zeros(L * H * B * mp, ps, d, dtype=torch.bfloat16, device="cuda"),
                 vp=torch.zeros(L * H * B * mp, ps, d, dtype=torch.bfloat16, device="cuda"),
                 bt=torch.full((L, H, B, mp), -1, dtype=torch.int32, device="cuda"),
                 sl=torch.zeros(L, H, B, dtype=torch.int32, device="cuda"),
                 nxt=torch.zeros(1, dtype=torch.int32, device="cuda"),
                 pos=torch.full((B,), 100, dtype=torch.int32, device="cuda"))
        q, k, v = (t.cuda() for t in toks[0])
        qo, o = torch.empty_like(q), torch.empty_like(q)
        na, nd = C.kvs_append_paged_workspace_size(dm, B), C.kvs_attn_decode_workspace_size(dm, B)
        wa = torch.empty(na, dtype=torch.uint8, device="cuda")
        wd = torch.empty(nd, dtype=torch.uint8, device="cuda")
        stream = 0 if how == "default stream" else None

        def step():
            C.kvs_append_paged(dm, B, B, None, g["pos"], d, f, False, q, qo, k, v, ps, g["kp"],
                               g["vp"], len(g["kp"]), g["nxt"], g["nxt"], g["bt"], mp, g["sl"],
                               g["sl"], wa, na, stream=stream)
            C.kvs_attn_decode(dm, B, qo, ps, g["kp"], g["vp"], len(g["kp"]), g["bt"], mp, g["sl"], 0,
                              None, None, None, o, None, wd, nd, stream=stream)
        if how == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        outs = []
        for t in toks:
            for x, y in zip((q, k, v), t):
                x.copy_(y)
            torch.cuda.synchronize()
            graph.replay() if how == "graph" else step()
            torch.cuda.synchronize()
            g["pos"] += 1
            outs.append(o.cpu())
        assert (g["sl"] == steps).all() and int(g["nxt"]) == L * H * B * -(-steps // ps)
        runs[how] = outs
    assert C.kvs_device_error(clear=True) == 0
    for how in ("eager", "default stream"):
        assert all(torch.equal(a, b) for a, b in zip(runs["graph"], runs[how])), how
    # the first token attends to itself alone
    first = toks[0][2].repeat_interleave(Hq // H, 1)
    assert torch.equal(runs["graph"][0], first)


def test_offsets_past_32_bits(C):
    """A pool of over 2^31 elements with the row's pages at its end: appended there, and read
    back by the attention."""
    ps, d, cap = 256, 128, 66000                          # 2.16e9 elements, 4.3 GB a pool
    kp = torch.zeros(cap, ps, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros(cap, ps, d, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(1)
    N = 300
    k = torch.randn(1, 1, N, d, generator=gen).to(torch.bfloat16)
    v = torch.randn(1, 1, N, d, generator=gen).to(torch.bfloat16)
    q = torch.randn(1, 2, 1, d, generator=gen).to(torch.bfloat16)
    dm = C.dims(1, 2, 1, d)
    bt = torch.full((1, 1, 1, 4), -1, dtype=torch.int32, device="cuda")
    sl = torch.zeros(1, 1, 1, dtype=torch.int32, device="cuda")
    nxt = torch.tensor([cap - 2], dtype=torch.int32, device="cuda")
    ts = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    nb = C.kvs_append_paged_workspace_size(dm, 1)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    C.kvs_append_paged(dm, 1, N, ts, None, 0, None, False, None, None, k.cuda(), v.cuda(), ps, kp, vp,
                       cap, nxt, nxt, bt, 4, sl, sl, ws, nb)
    assert bt.flatten().tolist() == [cap - 2, cap - 1, -1, -1] and int(nxt) == cap
    assert torch.equal(kp[-2:].reshape(-1, d)[:N].cpu(), k[0, 0])
    assert torch.equal(vp[-2:].reshape(-1, d)[:N].cpu(), v[0, 0])
    assert not kp[:-2].any() and not kp[-2:].reshape(-1, d)[N:].any()
    o = torch.empty(1, 2, 1, d, dtype=torch.bfloat16, device="cuda")
    nb = C.kvs_attn_decode_workspace_size(dm, 1)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    C.kvs_attn_decode(dm, 1, q.cuda(), ps, kp, vp, cap, bt, 4, sl, 0, None, None, None, o, None, ws, nb)
    assert C.kvs_device_error(clear=True) == 0
    want, _, spread = O.attn_decode(f64(q), f64(k)[0], f64(v)[0], N, np.zeros((1, 1, 1, 1), int),
                                    np.full((1, 1, 1), N))
    assert (np.abs(f64(o) - want) <= 2.0 ** -8 * np.abs(want) + 1.1 * 2.0 ** -8 * spread).all()


# ----------------------------------------------------------------------------- attention

def attend_case(C, L, Hq, H, B, d, ps, n, w=0, pos=None, seed=0, scale=1.0, room=0):
    """room: tokens that a row's table has place for at least (the kernel is chosen by it)."""
    gen = torch.Generator().manual_seed(seed)
    n = np.broadcast_to(np.asarray(n), (L, H, B)).copy()
    need = -(-n // ps)
    mp, cap = max(max(1, int(need.max())) + 1, -(-room // ps)), int(need.sum()) + 2
    st = cache(gen, L, H, B, d, ps, n, cap, mp)
    # what no row owns must not be read: NaN rows behind every length, NaN pages, and table
    # entries past the end that point at them
    own = torch.zeros(cap, ps, dtype=torch.bool)
    for r in np.ndindex(L, H, B):
        for i in range(int(n[r])):
            own[st["bt"][r][i // ps], i % ps] = True
    for p in ("kp", "vp"):
        st[p][~own] = float("nan")
    st["bt"][st["bt"] < 0] = 2 ** 31 - 1
    q = (torch.randn(L, Hq, B, d, generator=gen) * scale).to(torch.bfloat16)
    c = dict(st, C=C, dm=C.dims(L, Hq, H, d), L=L, H=H, B=B, d=d, ps=ps, mp=mp, cap=cap, w=w, q=q, n=n)
    if w:
        c["pos"] = torch.tensor(np.broadcast_to(np.asarray(pos), (B,)).copy(), dtype=torch.int32)
        c["rk"] = torch.randn(L, H, B, w, d, generator=gen).to(torch.bfloat16)
        c["rv"] = torch.randn(L, H, B, w, d, generator=gen).to(torch.bfloat16)
        for b in range(B):
            c["rk"][:, :, b, max(0, int(c["pos"][b])):] = float("nan")
            c["rv"][:, :, b, max(0, int(c["pos"][b])):] = float("nan")
    return c


def call_attend(c, lse=True, stream=None):
    C = c["C"]
    g = {n: c[n].cuda() for n in ("q", "kp", "vp", "bt", "sl")}
    for n in ("pos", "rk", "rv"):
        g[n] = c[n].cuda() if c["w"] else None
    o = torch.full_like(g["q"], 9.0)
    z = torch.full(o.shape[:3], 9.0, device="cuda") if lse else None
    nb = C.kvs_attn_decode_workspace_size(c["dm"], c["B"])
    ws = torch.full((nb,), 171, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    C.kvs_attn_decode(c["dm"], c["B"], g["q"], c["ps"], g["kp"], g["vp"], c["cap"], g["bt"], c["mp"],
                      g["sl"], c["w"], g["pos"], g["rk"], g["rv"], o, z, ws, nb, stream=stream)
    torch.cuda.synchronize()
    return o.cpu(), None if z is None else z.cpu()


def check_attend(c, o, z, but=None):
    """but: an index of o and z that is left out."""
    ring = (f64(c["rk"]), f64(c["rv"]), np.maximum(c["pos"].numpy(), 0)) if c["w"] else (None,) * 3
    q, kp = f64(c["q"]), f64(c["kp"])
    want, lse, spread = O.attn_decode(q, kp, f64(c["vp"]), c["ps"], c["bt"].numpy(), c["n"], *ring)
    d, g = c["d"], q.shape[1] // c["H"]
    keys = np.concatenate([np.abs(kp).reshape(-1, d)] +
                          ([np.abs(ring[0]).reshape(-1, d)] if c["w"] else []))
    kmax = np.nanmax(keys, axis=0) if np.isfinite(keys).any() else np.zeros(d)
    x = (np.abs(q) * np.nan_to_num(kmax)).sum(-1) / np.sqrt(d)
    delta = (d + 8) * 2.0 ** -24 * x + 2.0 ** -20 * x
    n = np.repeat(c["n"], g, axis=1).astype(float) + c["w"]
    u = 2.0 ** -24
    if but is not None:
        o, z = o.clone(), z.clone()
        o[but], z[but] = torch.from_numpy(want[but]).to(o.dtype), torch.from_numpy(lse[but]).to(z.dtype)
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(z.numpy()), empty)
    err = np.abs(np.where(empty, 0, z.double().numpy()) - np.where(empty, 0, lse))
    tol = delta + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, lse))) + (n / 8 + 16) * u
    assert (err <= tol).all(), (err.max(), (err / tol).max())
    err = np.abs(f64(o) - want)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.1 * delta + (n + 32) * u)[..., None] * spread
    assert (err <= tol + 1e-30).all(), (err.max(), (err / (tol + 1e-30)).max())
    assert (f64(o)[empty] == 0).all()


ATTEND = {
    "one key": dict(L=1, Hq=4, H=2, B=1, d=128, ps=16, n=1),
    "lengths around a tile": dict(L=1, Hq=8, H=8, B=9, d=128, ps=16,
                                  n=[0, 1, 15, 16, 17, 31, 32, 33, 64]),
    "lengths around a tile, d 64": dict(L=1, Hq=8, H=4, B=9, d=64, ps=16,
                                        n=[0, 1, 15, 16, 17, 31, 32, 33, 65]),
    "no keys at all": dict(L=2, Hq=4, H=2, B=3, d=64, ps=16, n=0),
    "odd pages": dict(L=1, Hq=12, H=2, B=5, d=128, ps=13, n=[100, 13, 0, 77, 12]),
    "pages of one": dict(L=1, Hq=4, H=2, B=3, d=128, ps=1, n=[50, 3, 17]),
    "one large page": dict(L=1, Hq=4, H=2, B=2, d=64, ps=4096, n=[200, 4097]),
    "groups of 1": dict(L=1, Hq=3, H=3, B=2, d=128, ps=16, n=[70, 200]),
    "groups of 5": dict(L=2, Hq=10, H=2, B=3, d=64, ps=8, n=[70, 200, 9]),
    "groups of 9": dict(L=1, Hq=18, H=2, B=2, d=128, ps=16, n=[70, 133]),
    "groups of 16": dict(L=1, Hq=16, H=1, B=2, d=128, ps=16, n=[70, 133]),
    "groups of 17": dict(L=1, Hq=17, H=1, B=3, d=64, ps=16, n=[0, 133, 40]),
    "groups of 40": dict(L=1, Hq=40, H=1, B=2, d=128, ps=16, n=[20, 133]),
    "ring alone": dict(L=1, Hq=4, H=2, B=4, d=128, ps=16, n=0, w=20, pos=[0, 1, 20, 500]),
    "ring and pages": dict(L=2, Hq=8, H=2, B=4, d=128, ps=16, n=[0, 5, 48, 100], w=33,
                           pos=[3, 32, 33, 34]),
    "ring of one, d 64": dict(L=1, Hq=2, H=2, B=3, d=64, ps=16, n=[16, 0, 7], w=1, pos=[0, 1, 2]),
    "negative ring position": dict(L=1, Hq=2, H=2, B=2, d=64, ps=16, n=[16, 3], w=4, pos=[-5, 2]),
    "long row": dict(L=1, Hq=4, H=1, B=1, d=128, ps=16, n=5003),
    "long among short": dict(L=1, Hq=8, H=2, B=6, d=64, ps=16, n=[3, 4000, 0, 1, 0, 700]),
    "many rows": dict(L=3, Hq=32, H=16, B=40, d=64, ps=16, n=np.arange(40) % 19),
    "many rows, groups of 9": dict(L=1, Hq=144, H=16, B=60, d=128, ps=16, n=np.arange(60) % 37),
    "large logits": dict(L=1, Hq=4, H=2, B=2, d=128, ps=16, n=[300, 40], scale=30.0),
}


@pytest.mark.parametrize("room", [0, 100000], ids=["tight", "wide"])
@pytest.mark.parametrize("name", ATTEND)
def test_attend(C, name, room):
    """With tables as narrow as the lengths allow (a block or cluster per row), and with
    tables that hold long rows (shares of one stream of tiles)."""
    c = attend_case(C, seed=len(name), room=room, **ATTEND[name])
    o, z = call_attend(c)
    assert C.kvs_device_error(clear=True) == 0
    check_attend(c, o, z)
    # again, on another stream and without the lse: the same bits
    side = torch.cuda.Stream()
    o2, _ = call_attend(c, lse=False, stream=side)
    assert np.array_equal(bits(o2), bits(o))


@pytest.mark.parametrize("room", [1, 100000], ids=["tight", "wide"])
def test_attend_with_an_empty_pool(C, room):
    """No pool at all (NULL pages, capacity 0): the ring's keys alone, or none."""
    c = attend_case(C, L=1, Hq=4, H=2, B=3, d=128, ps=16, n=0, w=7, pos=[0, 3, 9], seed=3, room=room)
    g = {n: c[n].cuda() for n in ("q", "bt", "sl", "pos", "rk", "rv")}
    o, z = torch.full_like(g["q"], 9.0), torch.full(c["q"].shape[:3], 9.0, device="cuda")
    nb = C.kvs_attn_decode_workspace_size(c["dm"], c["B"])
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    C.kvs_attn_decode(c["dm"], c["B"], g["q"], c["ps"], None, None, 0, g["bt"], c["mp"], g["sl"], 7,
                      g["pos"], g["rk"], g["rv"], o, z, ws, nb)
    torch.cuda.synchronize()
    assert C.kvs_device_error(clear=True) == 0
    check_attend(c, o.cpu(), z.cpu())


def test_binding_refuses_strided_tensors(C):
    """The layouts are dense: a transposed or sliced tensor is refused by name."""
    dm = C.dims(1, 2, 2, 64)
    x = torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        C.kvs_rope(dm, 4, pos, 0, None, False, x[..., :64], y, None, None)
    with pytest.raises(ValueError, match="contiguous"):
        C.kvs_rope(dm, 4, pos[::2], 64, [1.0] * 32, False, y, y, None, None)


@pytest.mark.parametrize("room", [0, 100000], ids=["tight", "wide"])
def test_attend_minus_infinity_and_nan_stay_in_their_row(C, room):
    """Logits of -inf weigh nothing (a row of nothing else is an empty one); a NaN key gives
    its own row NaN and no other."""
    c = attend_case(C, L=1, Hq=2, H=1, B=3, d=64, ps=16, n=[40, 40, 40], seed=4, room=room)
    big = torch.finfo(torch.bfloat16).max
    c["q"][:, :, 0] = big
    kp = c["kp"]
    for i in range(40):
        pg, r = c["bt"][0, 0, 0, i // 16], i % 16
        kp[pg, r] = -big
    pg = c["bt"][0, 0, 1, 1]
    kp[pg, 3, 5] = float("nan")
    o, z = call_attend(c)
    assert (z[:, :, 0] == -float("inf")).all() and (o[:, :, 0] == 0).all()
    assert torch.isnan(z[:, :, 1]).all() and torch.isnan(o[:, :, 1]).all()
    assert torch.isfinite(z[:, :, 2]).all() and torch.isfinite(o[:, :, 2]).all()


@pytest.mark.parametrize("room", [0, 100000], ids=["tight", "wide"])
def test_attend_bad_pages_and_lengths_are_reported(C, room):
    """A page id outside the pool leaves its keys out; a length outside the table is taken as
    the nearest bound.  Nothing outside the buffers is read and the error word is set."""
    base = dict(L=1, Hq=4, H=2, B=2, d=128, ps=16, n=[60, 40], seed=6, room=room)
    for bad in (-1, 2 ** 31 - 1, None, -2 ** 31):
        c = attend_case(C, **base)
        c["bt"][0, 1, 0, 1] = c["cap"] if bad is None else bad
        o, z = call_attend(c)
        assert C.kvs_device_error(clear=True) == 9
        # the row without keys 16..31
        bt = c["bt"].numpy().copy()
        bt[0, 1, 0, 1:-1], c2 = bt[0, 1, 0, 2:].copy(), dict(c)
        n = c["n"].copy()
        n[0, 1, 0] = 44
        c2.update(bt=torch.from_numpy(bt), n=n)
        check_attend(c2, o, z)
    c = attend_case(C, **base)
    c["sl"][0, 0, 1] = -3
    c["n"][0, 0, 1] = 0
    o, z = call_attend(c)
    assert C.kvs_device_error(clear=True) == 9
    check_attend(c, o, z)
    c = attend_case(C, **base)
    c["sl"][0, 0, 1] = 2 ** 31 - 1                        # its table's last entries are bad pages
    o, z = call_attend(c)
    assert C.kvs_device_error(clear=True) == 9
    check_attend(c, o, z, but=(0, slice(0, 2), 1))        # that row also meets unwritten (NaN) keys


@pytest.mark.parametrize("room", [0, 100000], ids=["tight", "wide"])
def test_attend_graph_replays_follow_the_state(C, room):
    """A captured call reads lengths, tables and positions when it runs: replayed after they
    change, it answers for the new ones."""
    c = attend_case(C, L=1, Hq=8, H=2, B=3, d=128, ps=16, n=[200, 90, 33], w=8, pos=[3, 8, 9],
                    seed=2, room=room)
    g = {n: c[n].cuda() for n in ("q", "kp", "vp", "bt", "sl", "pos", "rk", "rv")}
    o = torch.zeros_like(g["q"])
    z = torch.zeros(o.shape[:3], device="cuda")
    nb = C.kvs_attn_decode_workspace_size(c["dm"], c["B"])
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")

    def call():
        C.kvs_attn_decode(c["dm"], c["B"], g["q"], c["ps"], g["kp"], g["vp"], c["cap"], g["bt"],
                          c["mp"], g["sl"], c["w"], g["pos"], g["rk"], g["rv"], o, z, ws, nb)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n, pos in (([200, 90, 33], [3, 8, 9]), ([0, 1, 17], [0, 1, 2]), ([199, 16, 0], [3, 7, 0])):
        c["n"] = np.broadcast_to(np.array(n), (1, 2, 3)).copy()
        c["pos"] = torch.tensor(pos, dtype=torch.int32)
        g["sl"].copy_(torch.from_numpy(c["n"]))
        g["pos"].copy_(c["pos"])
        ws.fill_(171)
        graph.replay()
        torch.cuda.synchronize()
        check_attend(c, o.cpu(), z.cpu())
    assert C.kvs_device_error(clear=True) == 0


@pytest.mark.parametrize("room", [0, 100000], ids=["tight", "wide"])
def test_two_calls_at_once(C, room):
    """Calls on two streams with workspaces of their own do not disturb each other."""
    cases = [attend_case(C, L=1, Hq=8, H=2, B=4, d=128, ps=16, n=[2000, 5, 900, 64], seed=s,
                         room=room) for s in (1, 2)]
    alone = [call_attend(c) for c in cases]
    runs = []
    for c in cases:
        g = {n: c[n].cuda() for n in ("q", "kp", "vp", "bt", "sl")}
        nb = C.kvs_attn_decode_workspace_size(c["dm"], c["B"])
        runs.append((c, g, torch.empty_like(g["q"]), torch.empty(nb, dtype=torch.uint8, device="cuda"),
                     nb, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, g, o, ws, nb, s in runs:
            C.kvs_attn_decode(c["dm"], c["B"], g["q"], c["ps"], g["kp"], g["vp"], c["cap"], g["bt"],
                              c["mp"], g["sl"], 0, None, None, None, o, None, ws, nb, stream=s)
    torch.cuda.synchronize()
    for (o, _), run in zip(alone, runs):
        assert torch.equal(run[2].cpu(), o)


def test_calls_of_two_threads(C):
    """Host threads that launch rows of one block and rows of clusters, each on a stream of its
    own: neither changes the other's launch."""
    cases = [attend_case(C, L=1, Hq=2, H=2, B=150, d=128, ps=16, n=9, seed=1, room=600),
             attend_case(C, L=1, Hq=2, H=2, B=2, d=128, ps=16, n=100, seed=2, room=1500)]
    alone = [call_attend(c)[0] for c in cases]
    outs, failed = [], []

    def calls(c, g, o, ws, nb, s):
        try:
            for _ in range(400):
                C.kvs_attn_decode(c["dm"], c["B"], g["q"], c["ps"], g["kp"], g["vp"], c["cap"],
                                  g["bt"], c["mp"], g["sl"], 0, None, None, None, o, None, ws, nb,
                                  stream=s)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = []
    for c in cases:
        g = {n: c[n].cuda() for n in ("q", "kp", "vp", "bt", "sl")}
        nb = C.kvs_attn_decode_workspace_size(c["dm"], c["B"])
        outs.append(torch.empty_like(g["q"]))
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        threads.append(threading.Thread(target=calls, args=(c, g, outs[-1], ws, nb,
                                                            torch.cuda.Stream())))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for o, want in zip(outs, alone):
        assert torch.equal(o.cpu(), want)


@pytest.mark.parametrize("room", [0, 100000], ids=["tight", "wide"])
def test_chain_without_gaps_gives_what_separate_calls_give(C, room):
    """Rotation in place, append and attention behind one another on the same few buffers, each
    starting while the one before it ends: the same bits as with a synchronisation between."""
    L, Hq, H, B, d, ps, steps = 2, 8, 2, 6, 128, 16, 40
    gen = torch.Generator().manual_seed(21)
    dm, f = C.dims(L, Hq, H, d), freqs(d)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    mp = max(8, -(-room // ps))
    cap = L * H * B * (steps // ps + 1)
    q0, k0, v = rnd(L, Hq, B, d), rnd(L, H, B, d), rnd(L, H, B, d)
    pos = torch.arange(1, B + 1, dtype=torch.int32, device="cuda") * 37
    na, nd = C.kvs_append_paged_workspace_size(dm, B), C.kvs_attn_decode_workspace_size(dm, B)
    wa = torch.empty(na, dtype=torch.uint8, device="cuda")
    wd = torch.empty(nd, dtype=torch.uint8, device="cuda")

    def run(between):
        q, k = q0.clone(), k0.clone()
        kp = torch.zeros(cap, ps, d, dtype=torch.bfloat16, device="cuda")
        vp = torch.zeros_like(kp)
        bt = torch.full((L, H, B, mp), -1, dtype=torch.int32, device="cuda")
        sl = torch.zeros(L, H, B, dtype=torch.int32, device="cuda")
        nxt = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = torch.empty(steps, *q0.shape, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        for i in range(steps):  # queries and keys turn on from step to step
            C.kvs_rope(dm, B, pos, d, f, False, q, q, k, k)
            between()
            C.kvs_append_paged(dm, B, B, None, None, 0, None, False, None, None, k, v, ps, kp, vp,
                               cap, nxt, nxt, bt, mp, sl, sl, wa, na)
            between()
            C.kvs_attn_decode(dm, B, q, ps, kp, vp, cap, bt, mp, sl, 0, None, None, None, o[i], None,
                              wd, nd)
            between()
        torch.cuda.synchronize()
        return o, kp, vp, bt, sl, nxt, k, q

    want = run(torch.cuda.synchronize)
    assert (want[4] == steps).all() and C.kvs_device_error(clear=True) == 0
    for _ in range(3):
        for x, y in zip(run(lambda: None), want):
            assert torch.equal(x, y)
    assert C.kvs_device_error(clear=True) == 0


def test_calls_that_follow_other_streams(C):
    """Rotations on two streams that a third joins by events, then the append and the attention
    there, eager and captured, after a memset and a library kernel of torch's: every call
    starts from what came before it, wherever that ran (the kernels may start early)."""
    L, Hq, H, B, d, ps, n = 1, 8, 2, 3, 128, 16, 700
    gen = torch.Generator().manual_seed(12)
    dm, f = C.dims(L, Hq, H, d), freqs(d)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    c = attend_case(C, L=L, Hq=Hq, H=H, B=B, d=d, ps=ps, n=n, seed=12, room=5000)
    src = {"kp": c["kp"].cuda(), "vp": c["vp"].cuda(), "bt": c["bt"].cuda(), "sl": c["sl"].cuda()}
    src["kp"] = torch.cat([src["kp"], torch.zeros_like(src["kp"])])
    src["vp"] = torch.cat([src["vp"], torch.zeros_like(src["vp"])])
    cap, nxt0 = len(src["kp"]), int(c["nxt"])
    q0, k0, v0 = rnd(L, Hq, B, d), rnd(L, H, B, d), rnd(L, H, B, d)
    pos = torch.tensor([900, 5, 70000], dtype=torch.int32, device="cuda")
    g = {k: v.clone() for k, v in src.items()}
    nxt = torch.full((1,), nxt0, dtype=torch.int32, device="cuda")
    q, k, o = torch.empty_like(q0), torch.empty_like(k0), torch.empty_like(q0)
    na, nd = C.kvs_append_paged_workspace_size(dm, B), C.kvs_attn_decode_workspace_size(dm, B)
    wa = torch.empty(na, dtype=torch.uint8, device="cuda")
    wd = torch.empty(nd, dtype=torch.uint8, device="cuda")
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()

    def work():
        main = torch.cuda.current_stream()
        for x in g:
            g[x].copy_(src[x])
        nxt.fill_(nxt0)
        o.zero_()
        for s, (x, y, which) in zip(sides, ((q0, q, 0), (k0, k, 1))):
            s.wait_stream(main)
            with torch.cuda.stream(s):
                y.copy_(x * 2)                    # a kernel of torch's before the early starter
                a = (y, y, None, None) if which == 0 else (None, None, y, y)
                C.kvs_rope(dm, B, pos, d, f, False, *a)
        for s in sides:
            main.wait_stream(s)
        C.kvs_append_paged(dm, B, B, None, None, 0, None, False, None, None, k, v0, ps, g["kp"],
                           g["vp"], cap, nxt, nxt, g["bt"], c["mp"], g["sl"], g["sl"], wa, na)
        C.kvs_attn_decode(dm, B, q, ps, g["kp"], g["vp"], cap, g["bt"], c["mp"], g["sl"], 0, None,
                          None, None, o, None, wd, nd)
        return o + 0                              # and one behind it

    def check(out):
        torch.cuda.synchronize()
        assert C.kvs_device_error(clear=True) == 0
        assert (g["sl"] == n + 1).all()
        want, _, spread = O.attn_decode(f64(q), f64(g["kp"]), f64(g["vp"]), ps, g["bt"].cpu().numpy(),
                                        g["sl"].cpu().numpy())
        err = np.abs(f64(out) - want)
        assert (err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 1e-3) * spread).all()
        check_rotated(q, (q0 * 2).cpu(), pos.cpu().numpy(), d, f, False, "q")

    first = work()
    check(first)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = work()
    for _ in range(3):
        for x in (q, k, o, *g.values()):
            x.zero_()
        graph.replay()
        check(out)
        assert torch.equal(out, first)


# ----------------------------------------------------------------------------- together

def test_prompt_pruned_then_decoded(C):
    """A prompt is rotated, pruned and compacted; then tokens are appended one at a time and
    attend over the pruned cache.  Every step against the oracle on the kept tokens."""
    L, Hq, H, d, T, ps, steps = 1, 4, 2, 64, 90, 16, 20
    gen = torch.Generator().manual_seed(0)
    dm, f = C.dims(L, Hq, H, d), freqs(d, 1e4)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    k, v, score = rnd(L, H, T, d), rnd(L, H, T, d), torch.randn(L, H, T, generator=gen).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    C.kvs_rope(dm, T, pos, d, f, False, None, None, k, k)
    mask = torch.empty(L, H, T, dtype=torch.uint8, device="cuda")
    keep = torch.empty(L, H, dtype=torch.int32, device="cuda")
    C.kvs_prune_mask(dm, score, T, C.KVS_THRESHOLD, 0.3, 0, 8, mask, keep)
    mp = -(-(T + steps) // ps)
    cap = L * H * mp
    kp = torch.full((cap, ps, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    bt = torch.empty(L, H, 1, mp, dtype=torch.int32, device="cuda")
    sl = torch.empty(L, H, 1, dtype=torch.int32, device="cuda")
    nxt = torch.empty(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(C.kvs_compact_workspace_size(dm, T), C.kvs_append_paged_workspace_size(dm, 1),
                         C.kvs_attn_decode_workspace_size(dm, 1)), dtype=torch.uint8, device="cuda")
    C.kvs_compact_paged(dm, k, v, T, mask, ps, kp, vp, cap, bt, mp, sl, nxt, ws, ws.numel())
    m = mask.cpu().bool().numpy()
    K = [f64(k)[0, h][m[0, h]] for h in range(H)]
    V = [f64(v)[0, h][m[0, h]] for h in range(H)]
    o = torch.empty(L, Hq, 1, d, dtype=torch.bfloat16, device="cuda")
    for t in range(T, T + steps):
        q1, k1, v1 = rnd(L, Hq, 1, d), rnd(L, H, 1, d), rnd(L, H, 1, d)
        p = torch.tensor([t], dtype=torch.int32, device="cuda")
        x = f64(k1)
        C.kvs_append_paged(dm, 1, 1, None, p, d, f, False, q1, q1, k1, v1, ps, kp, vp, cap, nxt, nxt,
                           bt, mp, sl, sl, ws, ws.numel())
        C.kvs_attn_decode(dm, 1, q1, ps, kp, vp, cap, bt, mp, sl, 0, None, None, None, o, None, ws,
                          ws.numel())
        y = O.rope(x, [t], f, d, False)
        q = f64(q1)
        for h in range(H):
            # the stored key is the rotated one, rounded
            n = int(sl[0, h, 0]) - 1
            got = f64(kp[bt[0, h, 0, n // ps].long(), n % ps])
            assert (np.abs(got - y[0, h, 0]) <= 2.0 ** -8 * np.abs(y[0, h, 0]) + 1e-5).all()
            K[h] = np.concatenate([K[h], got[None]])
            V[h] = np.concatenate([V[h], f64(v1)[0, h]])
            for hq in range(h * 2, h * 2 + 2):
                a = np.exp(K[h] @ q[0, hq, 0] / np.sqrt(d))
                a /= a.sum()
                want = a @ V[h]
                tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2e-5) * (a @ np.abs(V[h]))
                assert (np.abs(f64(o)[0, hq, 0] - want) <= tol).all()
    assert C.kvs_device_error(clear=True) == 0


def test_pruning_decode_with_attention(C):
    """Decode steps that prune at the window boundary, each followed by the attention over
    appended pages and ring: the keys are exactly the kept tokens plus the last w."""
    L, Hq, H, B, d, w, ps, steps, tau = 1, 6, 2, 3, 128, 5, 4, 40, 0.0
    gen = torch.Generator().manual_seed(7)
    dm, f = C.dims(L, Hq, H, d), freqs(d, 1e4)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    mp = steps // ps + 1
    cap = L * H * B * mp
    kp, vp = rnd(cap, ps, d), rnd(cap, ps, d)
    bt = torch.full((L, H, B, mp), -1, dtype=torch.int32, device="cuda")
    sl = torch.zeros(L, H, B, dtype=torch.int32, device="cuda")
    nxt = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    rs = torch.full((L, H, B, w), float("nan"), device="cuda")
    rk, rv = rnd(L, H, B, w, d), rnd(L, H, B, w, d)
    ws = torch.empty(C.kvs_attn_decode_workspace_size(dm, B), dtype=torch.uint8, device="cuda")
    o = torch.empty(L, Hq, B, d, dtype=torch.bfloat16, device="cuda")
    z = torch.empty(L, Hq, B, device="cuda")
    K, V, S = [], [], []
    for t in range(steps):
        q1, k1, v1 = rnd(L, Hq, B, d), rnd(L, H, B, d), rnd(L, H, B, d)
        s1 = torch.randn(L, H, B, generator=gen).cuda()
        C.kvs_rope(dm, B, pos, d, f, False, q1, q1, k1, k1)
        C.kvs_decode_step(dm, B, w, pos, s1, k1, v1, rs, rk, rv, tau, ps, kp, vp, cap, nxt, bt, mp, sl)
        C.kvs_attn_decode(dm, B, q1, ps, kp, vp, cap, bt, mp, sl, w, pos, rk, rv, o, z, ws, ws.numel())
        K.append(f64(k1)), V.append(f64(v1)), S.append(s1.cpu().double().numpy())
        kept, window = O.decode_prune(np.stack(S, -1).reshape(-1, t + 1), tau, w)
        q = f64(q1)
        for h, b in np.ndindex(H, B):
            at = kept[h * B + b] + window[h * B + b]
            Kr = np.array([K[i][0, h, b] for i in at])
            Vr = np.array([V[i][0, h, b] for i in at])
            for hq in range(h * 3, h * 3 + 3):
                x = Kr @ q[0, hq, b] / np.sqrt(d)
                lse = np.log(np.exp(x).sum())
                a = np.exp(x - lse)
                assert abs(float(z[0, hq, b]) - lse) <= 1e-4
                tol = 2.0 ** -8 * np.abs(a @ Vr) + (2.0 ** -8 + 2e-5) * (a @ np.abs(Vr))
                assert (np.abs(f64(o)[0, hq, b] - a @ Vr) <= tol).all()
    assert C.kvs_device_error(clear=True) == 0


def test_decode_pipeline_with_attention(C):
    """The decode pipeline's own path: rotated keys in ring and pages, decided by the
    surrogate, attended over; a captured step replays like the eager one."""
    from kv_cache_eviction_lse_gb300 import pipeline, workloads as W
    wl = W.WORKLOADS["c7"].scaled(L=2, H_q=4, H_kv=2, D_h=512, batch=3, w=6, tau=-4.0)
    x = W.generate(wl, device="cuda")
    x["q"] = W.decode_queries(wl, device="cuda")
    p = pipeline.make_pipeline(wl, x, max_steps=64, attention=True)
    f, steps = p.inv_freq.numpy(), 30
    outs, keys = [], []
    for t in range(steps):
        p.step()
        torch.cuda.synchronize()
        outs.append((p.o.clone(), p.lse.clone()))
        check_rotated(p.q_rot, x["q"], np.full(wl.batch, t), wl.d, f, False, "q")
        check_rotated(p.k_rot, x["k"], np.full(wl.batch, t), wl.d, f, False, "k")
        assert torch.equal(p.ring_k[:, :, :, t % wl.w], p.k_rot)
        keys.append(p.k_rot.clone())
        if t in (0, 4, 5, 6, 7, steps - 1):
            want, lse, spread = O.attn_decode(
                f64(p.q_rot), f64(p.k_pages), f64(p.v_pages), wl.page_size,
                p.block_table.cpu().numpy(), p.seq_lens.cpu().numpy(), f64(p.ring_k), f64(p.ring_v),
                p.pos.cpu().numpy())
            assert np.isfinite(lse).all()
            assert np.abs(p.lse.cpu().double().numpy() - lse).max() <= 1e-4
            err = np.abs(f64(p.o) - want)
            assert (err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 1e-4) * spread).all()
    assert C.kvs_device_error(clear=True) == 0
    # rows that pass the threshold hold every token that left the ring, rotated at its own place
    kept = (p.score >= wl.tau).cpu().numpy()
    n = p.seq_lens.cpu().numpy()
    assert 0 < kept.sum() < kept.size and np.array_equal(n, np.where(kept, steps - wl.w, 0))
    for r in zip(*np.nonzero(kept)):
        ids = p.block_table[r][: -(-int(n[r]) // wl.page_size)].long()
        got = p.k_pages[ids].reshape(-1, wl.d)[: int(n[r])]
        assert torch.equal(got, torch.stack([k[r] for k in keys[: int(n[r])]]))
    p.reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.step()
    p.reset()
    for t in range(steps):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.o, outs[t][0]) and torch.equal(p.lse, outs[t][1]), t
    with pytest.raises(ValueError):
        pipeline.make_pipeline(wl.scaled(w=0), x, attention=True)
