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
