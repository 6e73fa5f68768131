"""Drafting as a server does it: drafted trees appended to the pages, attention over them, the accepted
paths, forks and pages given back, step after step on one state.  Every step is checked: attention
against 64 bits, the tokens of every row to the bit."""
import numpy as np
import pytest
import torch

from oracle.drafts_oracle import way_up
from .gpu_util import need_gpu
from .test_gpu_tree import call, case, check, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def C():
    need_gpu()
    from kv_cache_eviction_lse_gb300 import build
    build.build()
    from kv_cache_eviction_lse_gb300 import capi
    return capi


def bits(t):
    return t.detach().cpu().view(torch.int16).numpy()


class Server:
    """The state on the device, and what each row holds as lists of key and value bits."""

    def __init__(self, C, L, Hq, H, B, d, ps, m_max, steps, prompt, seed):
        self.C, self.L, self.Hq, self.H, self.B, self.d, self.ps = C, L, Hq, H, B, d, ps
        self.dm, self.N, self.m_max = C.dims(L, Hq, H, d), B * m_max, m_max
        self.gen, self.rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        self.mp = -(-(prompt + (steps + 1) * m_max) // ps)
        self.cap = L * H * B * self.mp
        z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        self.kp, self.vp = (z(self.cap, ps, d, t=torch.bfloat16) for _ in range(2))
        self.bt, self.sl, self.nxt = z(L, H, B, self.mp), z(L, H, B), z(1)
        self.inv = torch.from_numpy(1e4 ** (-np.arange(0, d, 2) / d))
        self.ts, self.pos, self.parent = z(B + 1), z(self.N), z(self.N)
        self.count, self.path = z(B), z(self.N)
        self.q, self.qr, self.o = (z(L, Hq, self.N, d, t=torch.bfloat16) for _ in range(3))
        self.k, self.v = (z(L, H, self.N, d, t=torch.bfloat16) for _ in range(2))
        self.lse = z(L, Hq, self.N, t=torch.float32)
        byte = lambda n: torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.wa = byte(C.kvs_append_paged_workspace_size(self.dm, B))
        self.wt = byte(C.kvs_attn_tree_workspace_size(self.dm, B, self.N))
        self.wr = byte(C.kvs_reclaim_paged_workspace_size(self.dm, B, self.cap))
        self.rows = {r: ([], []) for r in np.ndindex(L, H, B)}
        self.len = np.zeros(B, dtype=int)  # tokens of a sequence, those of pruned heads included

    def draft(self, m, kind):
        """m[b] tokens for every sequence, and a path through each tree that is kept."""
        C, N = self.C, self.N
        ts = np.concatenate([[0], np.cumsum(m)])
        up = np.concatenate([tree(self.rng, x, kind) for x in m]).astype(int)
        depth, path, count = np.zeros(N, dtype=np.int32), np.zeros(N, dtype=np.int32), np.zeros(self.B, dtype=np.int32)
        for b in range(self.B):
            u = up[ts[b]:ts[b + 1]]
            for i in range(m[b]):
                depth[ts[b] + i] = self.len[b] + len(way_up(u, i)) - 1
            if m[b]:
                way = way_up(u, int(self.rng.integers(0, m[b])))[::-1]
                count[b] = self.rng.integers(0, len(way) + 1)
                path[ts[b]:ts[b] + len(way)] = way
        put = lambda t, x: t[:len(x)].copy_(torch.from_numpy(np.asarray(x, dtype=np.int32)))  # noqa: E731
        put(self.ts, ts), put(self.pos, depth), put(self.parent, up), put(self.count, count), put(self.path, path)
        for t in (self.q, self.k, self.v):
            t.copy_(torch.randn(t.shape, generator=self.gen).to(torch.bfloat16))
        self.o.fill_(7.0)
        self.lse.fill_(7.0)
        return ts, up, path, count

    def append(self):
        self.C.kvs_append_paged(self.dm, self.B, self.N, self.ts, self.pos, self.d, self.inv, False, self.q,
                                self.qr, self.k, self.v, self.ps, self.kp, self.vp, self.cap, self.nxt, self.nxt,
                                self.bt, self.mp, self.sl, self.sl, self.wa, self.wa.numel())

    def attend(self):
        self.C.kvs_attn_tree(self.dm, self.B, self.N, self.m_max, self.ts, self.parent, self.qr, self.ps, self.kp,
                             self.vp, self.cap, self.bt, self.mp, self.sl, 0, None, None, None, self.o, self.lse,
                             self.wt, self.wt.numel())

    def accept(self):
        self.C.kvs_accept_paged(self.dm, self.B, self.N, self.ts, self.count, self.path, self.ps, self.kp, self.vp,
                                self.cap, self.bt, self.mp, self.sl, self.sl)

    def reclaim(self):
        self.C.kvs_reclaim_paged(self.dm, self.B, self.ps, self.kp, self.vp, self.cap, self.nxt, self.nxt, self.bt,
                                 self.bt, self.mp, self.sl, self.wr, self.wr.numel())

    def fork(self, src, dst):
        n = len(src)
        ws = torch.full((self.C.kvs_fork_paged_workspace_size(self.dm, self.B, n),), 255, dtype=torch.uint8,
                        device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.C.kvs_fork_paged(self.dm, self.B, n, i32(src), i32(dst), self.ps, self.kp, self.vp, self.cap, self.nxt,
                              self.nxt, self.bt, self.mp, self.sl, 0, None, None, None, None, ws, ws.numel())
        for (l, h, b), _ in list(self.rows.items()):
            if b in dst:
                k, v = self.rows[l, h, src[dst.index(b)]]
                self.rows[l, h, b] = (list(k), list(v))
        for s, t in zip(src, dst):
            self.len[t] = self.len[s]

    def appended(self, ts):
        """The lists with the new tokens; their keys as kvs_rope turns them."""
        kr = torch.empty_like(self.k)
        self.C.kvs_rope(self.dm, self.N, self.pos, self.d, self.inv, False, self.q, self.qr.clone(), self.k, kr)
        torch.cuda.synchronize()
        kr, v = bits(kr), bits(self.v)
        for l, h, b in self.rows:
            for t in range(ts[b], ts[b + 1]):
                self.rows[l, h, b][0].append(kr[l, h, t])
                self.rows[l, h, b][1].append(v[l, h, t])

    def accepted(self, ts, path, count):
        for (l, h, b), (k, v) in self.rows.items():
            base = len(k) - (ts[b + 1] - ts[b])
            keep = list(range(base)) + [base + int(path[ts[b] + j]) for j in range(count[b])]
            self.rows[l, h, b] = ([k[i] for i in keep], [v[i] for i in keep])
        self.len += count

    def same(self):
        torch.cuda.synchronize()
        assert self.C.kvs_device_error() == 0
        bt, sl, kp, vp = self.bt.cpu().numpy(), self.sl.cpu().numpy(), bits(self.kp), bits(self.vp)
        for r, (k, v) in self.rows.items():
            n = int(sl[r])
            assert n == len(k), r
            ids = bt[r][:-(-n // self.ps)]
            assert (ids >= 0).all() and (ids < int(self.nxt)).all()
            if n:
                assert np.array_equal(kp[ids].reshape(-1, self.d)[:n], np.stack(k)), r
                assert np.array_equal(vp[ids].reshape(-1, self.d)[:n], np.stack(v)), r

    def attended(self, m, ts, up):
        c = dict(L=self.L, Hq=self.Hq, H=self.H, B=self.B, d=self.d, ps=self.ps, w=0, N=self.N, m=np.array(m),
                 sl=self.sl.cpu().numpy(), bt=self.bt.cpu().numpy(), ts=ts, parent=up, q=self.qr.cpu(),
                 kp=self.kp.cpu(), vp=self.vp.cpu(), pos=np.zeros(self.B, dtype=int),
                 rk=torch.zeros(self.L, self.H, self.B, 0, self.d, dtype=torch.bfloat16),
                 rv=torch.zeros(self.L, self.H, self.B, 0, self.d, dtype=torch.bfloat16))
        check(c, dict(o=self.o, lse=self.lse))

    def named(self):
        bt, sl = self.bt.cpu().numpy(), self.sl.cpu().numpy()
        return len({int(p) for r in self.rows for p in bt[r][:-(-int(sl[r]) // self.ps)]})

    def prompts(self, n):
        """n[b] tokens each, by the call that drafts use too, in pieces of m_max."""
        left = np.array(n)
        while left.any():
            m = np.minimum(left, self.m_max)
            ts, _, _, _ = self.draft(m, "chain")
            self.append()
            self.appended(ts)
            self.len += m
            left -= m


STEPS = [("random", [5, 0, 8, 1]), ("levels", [8, 7, 0, 3]), ("chain", [1, 6, 2, 8]), ("star", [4, 8, 8, 0]),
         ("random", [8, 8, 8, 8])]


@pytest.mark.parametrize("size", [dict(d=128, ps=16, Hq=8, H=2), dict(d=64, ps=5, Hq=3, H=1)],
                         ids=["d128", "d64, pages of five"])
def test_drafts_step_after_step(C, size):
    s = Server(C, L=2, B=4, m_max=8, steps=5, prompt=150, seed=3, **size)
    s.prompts([150, 3, 40, 0])
    s.same()
    for i, (kind, m) in enumerate(STEPS):
        ts, up, path, count = s.draft(m, kind)
        s.append()
        s.attend()
        s.appended(ts)
        s.same()
        s.attended(m, ts, up)
        s.accept()
        s.accepted(ts, path, count)
        s.same()
        if i == 1:
            s.fork([0], [3])  # what sequence 3 held is dropped
            s.same()
        if i == 2:
            s.fork([2, 2], [0, 1])
            s.same()
        if i % 2:
            s.reclaim()
            s.same()
            assert int(s.nxt) == s.named()


def test_a_captured_step_is_the_eager_one(C):
    """Append, attention, accepted paths and reclaimed pages as one graph; every replay on new drafts leaves
    the state and the outputs that the calls leave."""
    size = dict(L=2, Hq=8, H=2, B=4, d=128, ps=16, m_max=8, steps=5, prompt=60, seed=9)
    a, b = Server(C, **size), Server(C, **size)
    for s in (a, b):
        s.prompts([60, 1, 33, 0])

    def step(s):
        s.append()
        s.attend()
        s.accept()
        s.reclaim()

    keep = {k: t.clone() for k, t in vars(b).items() if isinstance(t, torch.Tensor)}
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            step(b)
    for k, t in keep.items():
        getattr(b, k).copy_(t)
    for kind, m in STEPS:
        for s in (a, b):
            ts, up, path, count = s.draft(m, kind)
            s.appended(ts)
            s.accepted(ts, path, count)
        step(a)
        torch.cuda.synchronize()
        graph.replay()
        a.same()
        b.same()
        for x, y in ((a.o, b.o), (a.lse, b.lse), (a.bt, b.bt), (a.sl, b.sl), (a.nxt, b.nxt)):
            assert torch.equal(x.cpu(), y.cpu())


@pytest.mark.parametrize("ps", [16, 13])
def test_a_pool_of_more_than_32_bit_offsets(C, ps):
    """The last pages of a pool of 2^32 elements and more hold what a small pool holds: the same results, and
    pages given back move from there to the front."""
    c = case(5, L=2, Hq=8, H=2, B=3, d=128, ps=ps, n=300, m=(8, 1, 20))
    small = call(C, c)
    cap = 2 ** 32 // (ps * 128) + c["cap"] + 7
    far = cap - c["cap"]
    dm, B, N = C.dims(2, 8, 2, 128), 3, c["N"]
    kp, vp = (torch.empty(cap, ps, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kp[far:], vp[far:] = small["kp"], small["vp"]
    bt = small["bt"] + far
    o, lse = torch.full_like(small["o"], 7.0), torch.full_like(small["lse"], 7.0)
    nb = max(C.kvs_attn_tree_workspace_size(dm, B, N), C.kvs_reclaim_paged_workspace_size(dm, B, cap))
    ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    C.kvs_attn_tree(dm, B, N, c["md"], small["ts"], small["parent"], small["q"], ps, kp, vp, cap, bt, c["mp"],
                    small["sl"], 0, None, None, None, o, lse, ws, nb)
    torch.cuda.synchronize()
    assert C.kvs_device_error() == 0
    assert torch.equal(o, small["o"]) and torch.equal(lse, small["lse"])
    ts, i32 = c["ts"], lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    path = np.zeros(N, dtype=np.int32)
    for b, p in enumerate(([1, 4, 7], [0], [0, 3, 9, 19])):
        path[ts[b]:ts[b] + len(p)] = p
    count, path, sl = i32([3, 1, 4]), i32(path.tolist()), small["sl"].clone()
    C.kvs_accept_paged(dm, B, N, small["ts"], count, path, ps, small["kp"], small["vp"], c["cap"], small["bt"],
                       c["mp"], small["sl"], small["sl"])
    C.kvs_accept_paged(dm, B, N, small["ts"], count, path, ps, kp, vp, cap, bt, c["mp"], sl, sl)
    nxt = i32([cap])
    C.kvs_reclaim_paged(dm, B, ps, kp, vp, cap, nxt, nxt, bt, bt, c["mp"], sl, ws, nb)
    torch.cuda.synchronize()
    assert C.kvs_device_error() == 0 and torch.equal(sl, small["sl"])
    lens, near = sl.cpu().numpy(), small["bt"].cpu().numpy()
    used = 0
    for r in np.ndindex(*lens.shape):
        n = -(-int(lens[r]) // ps)
        ids, was = bt[r][:n].long(), torch.from_numpy(near[r][:n]).long().cuda()
        assert int(ids.max()) < int(nxt)
        for new, old in ((kp, small["kp"]), (vp, small["vp"])):
            a, b = new[ids].reshape(-1, 128)[:lens[r]], old[was].reshape(-1, 128)[:lens[r]]
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        used += n
    assert int(nxt) == used
