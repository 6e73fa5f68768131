"""GPU parity of the rotation, the paged append and the paged decode attention where more than
the sizes of tests/test_gpu_serving.py is needed to see a fault.

Attention, near-equal weights: with queries of 0.02 the logits' own error (delta, as there) is
below 1e-5, and what is left of the weights' is seen.  A weight is held in two bf16 parts: the
first cut off (at most 2^-7 of it is left), the second rounded (2^-8 of that) and made of
p (1 + 2^-20).  So o is off by 2^-8 |o| (output) + (2^-15 + 2^-19 + 2.1 delta + (n + 32) u)
sum a |v|, u = 2^-24.
"""
import numpy as np
import pytest
import torch

import oracle as O
from .gpu_util import f64
from .test_gpu_serving import ATTEND, C, attend_case, call_attend  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def check_attend_closely(c, o, z):
    ring = (f64(c["rk"]), f64(c["rv"]), np.maximum(c["pos"].numpy(), 0)) if c["w"] else (None,) * 3
    q, kp = f64(c["q"]), f64(c["kp"])
    want, lse, spread = O.attn_decode(q, kp, f64(c["vp"]), c["ps"], c["bt"].numpy(), c["n"], *ring)
    d, g = c["d"], q.shape[1] // c["H"]
    keys = np.concatenate([np.abs(kp).reshape(-1, d)] +
                          ([np.abs(ring[0]).reshape(-1, d)] if c["w"] else []))
    kmax = np.where(np.isnan(keys), 0, keys).max(axis=0)
    x = (np.abs(q) * kmax).sum(-1) / np.sqrt(d)
    delta = (d + 8) * U * x + 2.0 ** -20 * x
    n = np.repeat(c["n"], g, axis=1).astype(float) + c["w"]
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(z.numpy()), empty)
    err = np.abs(np.where(empty, 0, z.double().numpy()) - np.where(empty, 0, lse))
    assert (err <= delta + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, lse))) + (n / 8 + 16) * U).all()
    err = np.abs(f64(o) - want)
    weights = 2.0 ** -15 + 2.0 ** -19 + 2.1 * delta + (n + 32) * U
    tol = 2.0 ** -8 * np.abs(want) + weights[..., None] * spread + 1e-30
    assert (err <= tol).all(), (err.max(), (err / tol).max())


# ----------------------------------------------------------------------------- attention

@pytest.mark.parametrize("room", [0, 100000], ids=["tight", "wide"])
@pytest.mark.parametrize("name", ATTEND)
def test_attend_weights_keep_their_bits(C, name, room):  # noqa: F811
    c = attend_case(C, seed=len(name), room=room, **dict(ATTEND[name], scale=0.02))
    o, z = call_attend(c)
    assert C.kvs_device_error(clear=True) == 0
    check_attend_closely(c, o, z)


def plan(c):
    """Which kernels take a case, by the rules of their launch: ("row", warps, cluster), or
    ("stream", "few" or "general", the most blocks that share a row and group of heads)."""
    d, g, rows = c["d"], c["q"].shape[1] // c["H"], c["n"].size
    groups, tile = 1 if g <= 8 else -(-g // 16), 16 if d == 128 else 32
    vrows, room = rows * groups, -(-(c["mp"] * c["ps"] + c["w"]) // tile)
    if vrows > 456 and room <= 32:
        return "row", 2, 1
    cluster = 1
    while cluster < 8 and vrows * cluster * 2 <= 456:
        cluster *= 2
    if room <= cluster * 4 * (16 if vrows * cluster >= 152 else 6):
        return "row", 4, cluster
    warps = {(64, 1): 12, (64, 2): 10, (128, 1): 10, (128, 2): 8}[d, 1 if g <= 8 else 2]
    sms = min(160, torch.cuda.get_device_properties(0).multi_processor_count)
    blocks = min(sms, -(-vrows * room // warps))
    held = np.minimum(c["pos"].numpy(), c["w"]) if c["w"] else np.zeros(c["B"], int)
    tiles = np.repeat(-(-(c["n"] + held) // tile), groups)       # row by row, its groups in turn
    each, more = divmod(int(tiles.sum()), blocks * warps)
    if not each:
        each, more = 1, 0
    first = np.concatenate([[0], np.cumsum(tiles)])
    warp = lambda t: t // (each + 1) if t < more * (each + 1) else more + (t - more * (each + 1)) // each  # noqa: E731
    spans = [warp(b - 1) // warps - warp(a) // warps + 1 for a, b in zip(first[:-1], first[1:]) if b > a]
    return "stream", "few" if vrows * 8 <= blocks else "general", max(spans)


SPANS = [  # lengths of 40 rows, and how many blocks the longest one takes at least
    ([6000, 2500, 900, 400, 0, 200] + [3, 0, 40, 17] * 8 + [1300, 64], 16),
    ([700, 5, 1100, 0] * 10, 4),
    ([2900 + 7 * i for i in range(40)], 3),
    ([25000] + [100] * 38 + [9000], 34),
]


@pytest.mark.parametrize("lengths,span", SPANS, ids=["one long", "some", "even", "two long"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [3, 12, 24])
def test_attend_rows_over_many_blocks(C, g, d, lengths, span):  # noqa: F811
    """More rows than the join of few rows takes, the longest over three and more blocks."""
    c = attend_case(C, L=1, Hq=g, H=1, B=40, d=d, ps=16, n=lengths, seed=g + d, room=100000)
    kind, join, most = plan(c)
    assert (kind, join) == ("stream", "general") and most >= span
    o, z = call_attend(c)
    assert C.kvs_device_error(clear=True) == 0
    check_attend_closely(c, o, z)
    o2, z2 = call_attend(c)                                # the same bits again
    assert torch.equal(o2, o) and torch.equal(z2, z)


SHAPES = {  # B sequences of H KV heads: the four warps' clusters of 1, 2, 4 and 8, and two warps
    ("row", 4, 1): dict(B=150, H=2), ("row", 4, 2): dict(B=75, H=2), ("row", 4, 4): dict(B=39, H=2),
    ("row", 4, 8): dict(B=9, H=2), ("row", 2, 1): dict(B=231, H=2),
}


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [2, 9, 17])
def test_attend_shapes_of_a_row(C, g, d, shape):  # noqa: F811
    """Every shape of the kernel that takes a block or cluster per row."""
    B, H = SHAPES[shape]["B"], SHAPES[shape]["H"]
    if g == 17:                                            # two groups of heads a row
        H = 1
    n = (np.arange(B) * 37) % 301
    n[[1, B // 2]] = 0
    c = attend_case(C, L=1, Hq=g * H, H=H, B=B, d=d, ps=16, n=n, w=11, pos=np.arange(B) % 14,
                    seed=g + d, room=320)
    assert plan(c) == shape
    o, z = call_attend(c)
    assert C.kvs_device_error(clear=True) == 0
    check_attend_closely(c, o, z)


@pytest.mark.parametrize("d", [64, 128])
def test_attend_more_rows_than_a_scan_step(C, d):  # noqa: F811
    """Over 8192 rows in one stream: chunks of several steps, with a number of sequences that
    divides none of them, ring positions among them."""
    L, H, B, w = 3, 16, 173, 5
    n = (np.arange(B)[None, None] * 5 + np.arange(H)[None, :, None] + np.arange(L)[:, None, None]) % 23
    c = attend_case(C, L=L, Hq=H, H=H, B=B, d=d, ps=16, n=n, w=w, pos=np.arange(B) * 7 % 9, seed=d,
                    room=3000)
    assert plan(c)[:2] == ("stream", "general")
    o, z = call_attend(c)
    assert C.kvs_device_error(clear=True) == 0
    check_attend_closely(c, o, z)


@pytest.mark.parametrize("room", [0, 100000], ids=["tight", "wide"])
@pytest.mark.parametrize("g,d", [(4, 128), (12, 128), (4, 64), (12, 64)])
def test_attend_infinite_values_stay_infinite(C, g, d, room):  # noqa: F811
    """An infinite value of a key that is there makes its dimension infinite, with its sign,
    and no other; of both signs, NaN."""
    c = attend_case(C, L=1, Hq=g, H=1, B=3, d=d, ps=16, n=[40, 700, 33], seed=g, room=room)
    pages = c["bt"][0, 0, :, 1].tolist()
    c["vp"][pages[0], 3, 5] = float("inf")
    c["vp"][pages[0], 7, d - 1] = -float("inf")
    c["vp"][pages[1], 2, 0] = float("inf")
    c["vp"][pages[2], 2, 9] = float("inf")
    c["vp"][pages[2], 5, 9] = -float("inf")
    o, z = call_attend(c)
    assert C.kvs_device_error(clear=True) == 0
    assert torch.isfinite(z).all()
    inf = torch.full_like(o, 0.0)
    inf[:, :, 0, 5], inf[:, :, 0, d - 1], inf[:, :, 1, 0] = float("inf"), -float("inf"), float("inf")
    inf[:, :, 2, 9] = float("nan")
    assert torch.equal(torch.isnan(o), torch.isnan(inf))
    assert torch.equal(torch.where(torch.isinf(o), o, 0.0), torch.where(torch.isinf(inf), inf, 0.0))


@pytest.mark.parametrize("room", [0, 100000], ids=["tight", "wide"])
def test_attend_does_not_touch_what_is_not_used(C, room):  # noqa: F811
    """A ring of no slots and a pool of no pages may be anything: no tensor, one of the two, an
    address that is not aligned."""
    odd = 2 ** 20 + 2
    c = attend_case(C, L=1, Hq=4, H=2, B=3, d=128, ps=16, n=[40, 0, 7], seed=1, room=room)
    o, z = call_attend(c)
    g = {n: c[n].cuda() for n in ("q", "kp", "vp", "bt", "sl")}
    nb = C.kvs_attn_decode_workspace_size(c["dm"], c["B"])
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    for rk, rv in ((None, None), (g["q"], None), (None, g["q"]), (odd, odd + 4), (odd, None)):
        o2 = torch.full_like(g["q"], 9.0)
        C.kvs_attn_decode(c["dm"], c["B"], g["q"], c["ps"], g["kp"], g["vp"], c["cap"], g["bt"],
                          c["mp"], g["sl"], 0, None, rk, rv, o2, None, ws, nb)
        assert torch.equal(o2.cpu(), o)
    c = attend_case(C, L=1, Hq=4, H=2, B=3, d=128, ps=16, n=0, w=7, pos=[0, 3, 9], seed=3, room=room)
    o, z = call_attend(c)
    g = {n: c[n].cuda() for n in ("q", "bt", "sl", "pos", "rk", "rv")}
    for kp, vp in ((None, None), (g["q"], None), (None, g["q"]), (odd, odd + 4), (odd, None)):
        o2 = torch.full_like(g["q"], 9.0)
        C.kvs_attn_decode(c["dm"], c["B"], g["q"], c["ps"], kp, vp, 0, g["bt"], c["mp"], g["sl"], 7,
                          g["pos"], g["rk"], g["rv"], o2, None, ws, nb)
        assert torch.equal(o2.cpu(), o)
    assert C.kvs_device_error(clear=True) == 0


# ----------------------------------------------------------------------------- frequencies

def test_frequencies_on_the_gpu_are_refused(C):  # noqa: F811
    """... by name, and a model's float32 buffer on the host gives what its float64 copy does."""
    dm, pos = C.dims(1, 2, 1, 64), torch.arange(5, dtype=torch.int32, device="cuda")
    x = torch.randn(1, 2, 5, 64, device="cuda").to(torch.bfloat16)
    f = torch.logspace(0, -3, 32)
    outs = []
    for g in (f.double(), f, f.tolist(), f.double().flip(0).flip(0)[::1]):
        outs.append(torch.empty_like(x))
        C.kvs_rope(dm, 5, pos, 64, g, False, x, outs[-1], None, None)
        assert torch.equal(outs[-1], outs[0])
    for g in (f.cuda(), f.double().cuda()):
        with pytest.raises(ValueError, match="inv_freq must be in host memory"):
            C.kvs_rope(dm, 5, pos, 64, g, False, x, outs[0], None, None)
