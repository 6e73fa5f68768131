"""Edges of the calls that move pages: pools that a decode step has filled, counters apart from
their inputs in calls that move nothing, counters out of range, pools of different sizes from two
host threads, and the pool of a whole model."""
import threading

import numpy as np
import pytest
import torch

from .gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def C():
    need_gpu()
    from kv_cache_eviction_lse_gb300 import build
    build.build()
    from kv_cache_eviction_lse_gb300 import capi
    return capi


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bytes_of(n):
    return torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")


# ----------------------------------------------------------------------------- full pools

class Decode:
    """A cache without a ring that kvs_decode_step fills: every token is kept, and its keys hold
    the step that brought it."""

    def __init__(self, C, L, H, B, ps, cap, mp=8, d=64):
        self.C, self.dm, self.shape, self.ps, self.cap, self.mp, self.d = C, C.dims(L, H, H, d), (L, H, B), ps, cap, mp, d
        self.kp = torch.zeros(cap, ps, d, dtype=torch.bfloat16, device="cuda")
        self.vp = torch.zeros_like(self.kp)
        self.nxt, self.pos = i32([0]), torch.zeros(B, dtype=torch.int32, device="cuda")
        self.bt = torch.full((L, H, B, mp), -1, dtype=torch.int32, device="cuda")
        self.sl = torch.zeros(L, H, B, dtype=torch.int32, device="cuda")
        self.steps = 0

    def step(self):
        L, H, B = self.shape
        self.steps += 1
        x = torch.full((L, H, B, self.d), float(self.steps), device="cuda").to(torch.bfloat16)
        self.C.kvs_decode_step(self.dm, B, 0, self.pos, torch.zeros(L, H, B, device="cuda"), x, x, None, None, None,
                               -1.0, self.ps, self.kp, self.vp, self.cap, self.nxt, self.bt, self.mp, self.sl)
        torch.cuda.synchronize()
        return self.C.kvs_device_error()

    def tokens(self, r):
        n = int(self.sl[r])
        return self.kp[self.bt[r][: -(-n // self.ps)].long()].reshape(-1, self.d)[:n, 0].int().tolist()

    def reclaim(self, nxt_out=None, bt_out=None):
        ws = bytes_of(self.C.kvs_reclaim_paged_workspace_size(self.dm, self.shape[2], self.cap))
        self.C.kvs_reclaim_paged(self.dm, self.shape[2], self.ps, self.kp, self.vp, self.cap, self.nxt,
                                 self.nxt if nxt_out is None else nxt_out, self.bt,
                                 self.bt if bt_out is None else bt_out, self.mp, self.sl, ws, ws.numel())
        torch.cuda.synchronize()
        return self.C.kvs_device_error()


def test_pages_come_back_after_a_decode_step_filled_the_pool(C):
    """Four rows, five pages: a step that asks for more leaves the counter at the pool's end, and
    with a sequence ended its pages serve the other."""
    s = Decode(C, 1, 2, 2, ps=4, cap=5)
    codes = [s.step() for _ in range(7)]
    assert codes == [0] * 4 + [4] * 3  # step 5 asks for four pages and gets one
    assert int(s.nxt) == 5
    assert sorted(s.sl.flatten().tolist()) == [4, 4, 4, 7]
    before = [s.tokens((0, h, 0)) for h in range(2)]
    s.sl[:, :, 1] = 0
    for _ in range(2):  # a second call finds nothing to do
        assert s.reclaim() == 0
        assert int(s.nxt) == sum(-(-len(x) // 4) for x in before)
        assert [s.tokens((0, h, 0)) for h in range(2)] == before
    assert s.step() in (0, 4)  # the ended sequence's rows ask for pages too
    assert [s.tokens((0, h, 0))[:len(x)] for h, x in enumerate(before)] == before
    assert int(s.nxt) <= 5


@pytest.mark.parametrize("cap", [1, 700, 959, 960, 2500])
def test_a_full_pool_keeps_its_counter(C, cap):
    """960 rows ask at once, and again."""
    s = Decode(C, 4, 8, 30, ps=1, cap=cap)
    for asked in (960, 1920, 2880):
        assert s.step() == (4 if asked > cap else 0)
        assert int(s.nxt) == min(asked, cap)
    pages = torch.cat([s.bt[r][: int(s.sl[r])] for r in np.ndindex(4, 8, 30)]).tolist()
    assert sorted(pages) == list(range(cap))


# ----------------------------------------------------------------------------- counters

def fork(C, forks, nxt, out, B=2, cap=6, sl=(8, 4), L=1):
    """Forks of sequence 0 to sequence 1, pages of four tokens."""
    dm = C.dims(L, 1, 1, 64)
    kp = torch.zeros(cap, 4, 64, dtype=torch.bfloat16, device="cuda")
    bt, lens = i32([0, 1, -1, 2, -1, -1]), i32(list(sl))
    ws = bytes_of(C.kvs_fork_paged_workspace_size(dm, 2, max(forks, 1)))
    C.kvs_fork_paged(dm, B, forks, i32([0]), i32([1]), 4, kp, kp.clone(), cap, nxt, out, bt, 3, lens, 0, None, None,
                     None, None, ws, ws.numel())
    torch.cuda.synchronize()
    return C.kvs_device_error(), bt.tolist(), lens.tolist()


def test_calls_that_move_nothing_hand_the_counter_on(C):
    """Separate counters alternate from call to call: one that is skipped would hand out pages that
    are in use."""
    for B, forks in ((2, 0), (0, 0)):
        nxt, out = i32([3]), i32([-7])
        assert fork(C, forks, nxt, out, B=B) == (0, [0, 1, -1, 2, -1, -1], [8, 4])
        assert int(out) == 3 and int(nxt) == 3
        assert fork(C, forks, nxt, nxt, B=B)[0] == 0 and int(nxt) == 3  # in place
    # a batch of no sequences: nothing is counted
    dm = C.dims(1, 1, 1, 64)
    nxt, out, ws, x = i32([3]), i32([-7]), bytes_of(1 << 16), torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    C.kvs_reclaim_paged(dm, 0, 4, x, x, 6, nxt, out, i32([]), i32([]), 3, i32([]), ws, ws.numel())
    assert int(out) == 3
    nxt, out = i32([4]), i32([-7])
    C.kvs_append_paged(dm, 0, 0, None, None, 0, None, False, None, None, x, x, 4, x, x, 6, nxt, out, i32([]), 3, i32([]),
                       i32([]), ws, ws.numel())
    assert int(out) == 4
    torch.cuda.synchronize()
    assert C.kvs_device_error() == 0


def test_a_counter_handed_on_in_a_graph(C):
    nxt, out = i32([3]), i32([-7])
    graph = torch.cuda.CUDAGraph()
    dm = C.dims(1, 1, 1, 64)
    kp, bt, lens = torch.zeros(6, 4, 64, dtype=torch.bfloat16, device="cuda"), i32([0, 1, 2]), i32([4])
    with torch.cuda.graph(graph):
        C.kvs_fork_paged(dm, 1, 0, None, None, 4, kp, kp, 6, nxt, out, bt, 3, lens, 0, None, None, None, None, None, 0)
    assert int(out) == -7
    for v in (5, 0):
        nxt.fill_(v)
        graph.replay()
        assert int(out) == v


def test_fork_refuses_a_counter_above_the_capacity(C):
    """Also where no page is needed (the source's rows end with a page); at the capacity it goes on."""
    for v in (7, 2 ** 31 - 1, -1):
        nxt, out = i32([v]), i32([-7])
        assert fork(C, 1, nxt, out) == (11, [0, 1, -1, 2, -1, -1], [8, 4])
        assert int(out) == v
    nxt, out = i32([6]), i32([-7])
    assert fork(C, 1, nxt, out) == (0, [0, 1, -1, 0, 1, -1], [8, 8])
    assert int(out) == 6
    for v in (6, 7, 2 ** 31 - 1):  # too small a pool where one is
        nxt, out = i32([v]), i32([-7])
        assert fork(C, 1, nxt, out, sl=(7, 4)) == (4, [0, 1, -1, 2, -1, -1], [7, 4])
        assert int(out) == v


# ----------------------------------------------------------------------------- sizes

def model_case(L, H, B, most, ps, d, gone, seed, spare=1000):
    """Rows of up to `most` tokens, scattered pages of which each holds its id; some sequences end."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows = L * H * B
    n = torch.randint(0, most + 1, (rows,), generator=gen, device="cuda")
    need = (n + ps - 1) // ps
    total = int(need.sum()) + spare
    mp = int(need.max())
    ids = torch.randperm(total, generator=gen, device="cuda").int()
    bt = torch.full((rows, mp), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(mp, device="cuda") < need[:, None]
    bt[used] = ids[: int(need.sum())]
    n = (n.view(L * H, B) * (torch.rand(B, generator=gen, device="cuda") >= gone)).view(-1)
    bt.view(L * H, B, mp)[:, 0] = bt.view(L * H, B, mp)[:, 1]  # two sequences share their pages
    n.view(L * H, B)[:, 0] = n.view(L * H, B)[:, 1]
    kp = torch.zeros(total, ps, d, dtype=torch.int16, device="cuda")
    kp[:, 0, :2] = torch.arange(total, dtype=torch.int32, device="cuda").view(torch.int16).view(-1, 2)
    kp[:, -1, -2:] = kp[:, 0, :2]
    return dict(L=L, H=H, B=B, ps=ps, d=d, mp=mp, cap=total, n=n.int(), bt=bt, kp=kp.view(torch.bfloat16))


def expected_reclaim(c):
    """The new table, where each page goes, and their number, from the definition."""
    need = (c["n"].long() + c["ps"] - 1) // c["ps"]
    used = torch.arange(c["mp"], device="cuda") < need[:, None]
    live = torch.zeros(c["cap"], dtype=torch.bool, device="cuda")
    live[c["bt"][used].long()] = True
    count = int(live.sum())
    at = torch.arange(c["cap"], device="cuda")
    new = at.clone()
    new[live & (at >= count)] = at[~live & (at < count)]
    bt = torch.full_like(c["bt"], -1)
    bt[used] = new[c["bt"][used].long()].int()
    return bt, live, new, count


@pytest.mark.parametrize("gone", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("L, H, B, most, ps, spare", [
    (3, 8, 16, 1200, 1, 7),       # 230 thousand pages: a word a chunk, in shared memory
    (4, 8, 64, 3000, 1, 1000),    # 3 million: several words a chunk
    (36, 8, 24, 3000, 4, 50000),  # 2.6 million in rows of a whole model
])
def test_reclaim_of_a_models_pool(C, L, H, B, most, ps, spare, gone):
    c = model_case(L, H, B, most, ps, 64, gone, seed=B, spare=spare)
    bt, live, new, count = expected_reclaim(c)
    dm = C.dims(L, H, H, 64)
    ws = bytes_of(C.kvs_reclaim_paged_workspace_size(dm, B, c["cap"]))
    kp, vp = c["kp"].clone(), c["kp"].clone()
    nxt, out, bt_out = i32([c["cap"]]), i32([-7]), torch.full_like(c["bt"], -7)
    C.kvs_reclaim_paged(dm, B, ps, kp, vp, c["cap"], nxt, out, c["bt"], bt_out, c["mp"], c["n"], ws, ws.numel())
    torch.cuda.synchronize()
    assert C.kvs_device_error() == 0
    assert int(out) == count and torch.equal(bt_out, bt)
    want = c["kp"].view(torch.int16).clone()  # what moves, and all else as it was
    want[new[live]] = c["kp"].view(torch.int16)[live]
    assert torch.equal(kp.view(torch.int16), want) and torch.equal(vp.view(torch.int16), want)


def test_two_threads_reclaim_pools_of_different_sizes(C):
    """Calls that need more than 48 KB of shared memory a block, 50 KB and 62, at once."""
    dm = C.dims(1, 1, 1, 64)

    class Pool:
        def __init__(self, cap, seed):
            self.cap, self.B = cap, 64
            self.kp = torch.zeros(cap, 1, 64, dtype=torch.bfloat16, device="cuda")
            self.vp = torch.zeros_like(self.kp)
            gen = torch.Generator().manual_seed(seed)
            self.bt0 = torch.randperm(cap, generator=gen)[: self.B].int().view(1, 1, self.B, 1).cuda()
            self.bt = self.bt0.clone()
            self.nxt, self.out, self.sl = i32([cap]), i32([-7]), torch.ones(1, 1, self.B, dtype=torch.int32, device="cuda")
            self.ws = bytes_of(C.kvs_reclaim_paged_workspace_size(dm, self.B, cap))
            self.stream = torch.cuda.Stream()
            self.raised = []

        def go(self):
            C.kvs_reclaim_paged(dm, self.B, 1, self.kp, self.vp, self.cap, self.nxt, self.out, self.bt0, self.bt, 1,
                                self.sl, self.ws, self.ws.numel(), stream=self.stream)

        def work(self):
            for i in range(3000):
                try:
                    self.go()
                except Exception as e:  # an exception of a thread fails no test by itself
                    self.raised.append((i, e))
                if i % 500 == 499:
                    self.stream.synchronize()

    pools = [Pool(200_000, 1), Pool(250_000, 2)]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=p.work) for p in pools]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not pools[0].raised and not pools[1].raised, [p.raised[:3] for p in pools]
    assert C.kvs_device_error() == 0
    for p in pools:
        ids = p.bt0.flatten().tolist()
        high, holes = sorted(x for x in ids if x >= p.B), [i for i in range(p.B) if i not in ids]
        new = dict(zip(high, holes))
        assert int(p.out) == p.B and p.bt.flatten().tolist() == [new.get(x, x) for x in ids]


def test_graphs_that_share_a_workspace(C):
    """Forks and reclaims of two caches of different sizes in graphs with one workspace, replayed in
    turn on one stream, give what calls with workspaces of their own give."""
    dm = [C.dims(2, 3, 3, 64), C.dims(5, 2, 2, 64)]
    cs = [model_case(2, 3, 9, 60, 4, 64, 0.3, seed=1), model_case(5, 2, 40, 90, 1, 64, 0.0, seed=2)]
    room = 3000  # pages behind the counter, for the forks

    def tensors(c):
        pad = torch.zeros(room, c["ps"], c["d"], dtype=torch.bfloat16, device="cuda")
        kp = torch.cat([c["kp"], pad])
        return dict(kp=kp, vp=kp.clone(), bt=c["bt"].clone(), sl=c["n"].clone(), nxt=i32([c["cap"]]))

    def step(i, t, ws):
        c = cs[i]
        C.kvs_fork_paged(dm[i], c["B"], 2, src, dst, c["ps"], t["kp"], t["vp"], c["cap"] + room, t["nxt"], t["nxt"],
                         t["bt"], c["mp"], t["sl"], 0, None, None, None, None, ws, ws.numel())
        C.kvs_reclaim_paged(dm[i], c["B"], c["ps"], t["kp"], t["vp"], c["cap"] + room, t["nxt"], t["nxt"], t["bt"],
                            t["bt"], c["mp"], t["sl"], ws, ws.numel())

    src, dst = i32([2, 3]), i32([5, 7])
    need = [max(C.kvs_fork_paged_workspace_size(d, c["B"], 2),
                C.kvs_reclaim_paged_workspace_size(d, c["B"], c["cap"] + room)) for d, c in zip(dm, cs)]
    want = [tensors(c) for c in cs]
    for i, t in enumerate(want):
        step(i, t, bytes_of(need[i]))
    ws, first, got, graphs = bytes_of(max(need)), [tensors(c) for c in cs], [tensors(c) for c in cs], []
    for i, t in enumerate(got):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(i, t, ws)
        graphs.append(g)
    for _ in range(3):
        for t, f in zip(got, first):
            for k in t:
                t[k].copy_(f[k])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert C.kvs_device_error() == 0
        for t, w in zip(got, want):
            for k in t:
                x, y = (v.view(torch.int16) if v.dtype == torch.bfloat16 else v for v in (t[k], w[k]))
                assert torch.equal(x, y), k
