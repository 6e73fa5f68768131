"""Host-side checks of kvs_rope, kvs_append_paged and kvs_attn_decode: refusals with their
status codes, empty calls, workspace sizes.  No GPU: every call fails validation, or is an
empty call, before anything is enqueued."""
import ctypes

import pytest
import torch

FAKE = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def C():
    from kv_cache_eviction_lse_gb300 import build
    build.build()
    from kv_cache_eviction_lse_gb300 import capi
    return capi


def freqs(n=64, bad=None):
    f = [10000.0 ** (-i / n) for i in range(n)]
    if bad is not None:
        f[n - 1] = bad
    return (ctypes.c_double * n)(*f)


def rope(C, dm=None, N=4, pos=FAKE, rot=128, f="f", il=0, q=FAKE, qo=FAKE, k=FAKE, ko=FAKE):
    dm = dm or C.dims(1, 4, 2, 128)
    f = freqs() if f == "f" else f
    return C._lib.kvs_rope(ctypes.byref(dm), N, pos, rot, f, il, q, qo, k, ko, None)


def test_rope_refusals(C):
    assert rope(C, dm=C.dims(1, 5, 2, 128)) == C.KVS_ERR_SHAPE
    assert rope(C, dm=C.dims(1, 4, 2, 96)) == C.KVS_ERR_UNSUPPORTED
    assert rope(C, N=-1) == C.KVS_ERR_ARG
    for rot in (-16, 8, 20, 144):
        assert rope(C, rot=rot) == C.KVS_ERR_UNSUPPORTED
    assert rope(C, dm=C.dims(1, 4, 2, 64), rot=128) == C.KVS_ERR_UNSUPPORTED
    assert rope(C, f=None) == C.KVS_ERR_ARG
    for bad in (float("nan"), float("inf"), -float("inf")):
        assert rope(C, f=freqs(64, bad)) == C.KVS_ERR_ARG
    assert rope(C, pos=None) == C.KVS_ERR_ARG
    assert rope(C, pos=FAKE + 4) == C.KVS_ERR_ALIGN
    assert rope(C, q=None) == C.KVS_ERR_ARG and rope(C, qo=None) == C.KVS_ERR_ARG
    assert rope(C, k=None) == C.KVS_ERR_ARG and rope(C, ko=None) == C.KVS_ERR_ARG
    assert rope(C, qo=FAKE + 8) == C.KVS_ERR_ALIGN
    # outputs that overlap their input without being it: 4 heads of 4 tokens of 256 bytes
    assert rope(C, qo=FAKE + 4096 - 16) == C.KVS_ERR_ARG
    assert rope(C, q=FAKE + 16) == C.KVS_ERR_ARG
    assert rope(C, ko=FAKE + 2048 - 16) == C.KVS_ERR_ARG
    # nothing to do
    assert rope(C, N=0, pos=None) == C.KVS_OK
    assert rope(C, q=None, qo=None, k=None, ko=None) == C.KVS_OK


APPEND = dict(B=2, N=6, tok=FAKE, pos=FAKE, rot=128, f="f", il=0, q=None, qo=None, k=FAKE, v=FAKE,
              ps=16, kp=FAKE, vp=FAKE, cap=8, nxt=FAKE, nxo=FAKE, bt=FAKE, mp=4, sl=FAKE, slo=FAKE,
              ws=FAKE, wsb=1 << 20)


def append(C, dm=None, **kw):
    a = dict(APPEND, **kw)
    dm = dm or C.dims(1, 4, 2, 128)
    f = freqs() if isinstance(a["f"], str) else a["f"]
    return C._lib.kvs_append_paged(
        ctypes.byref(dm), a["B"], a["N"], a["tok"], a["pos"], a["rot"], f, a["il"], a["q"], a["qo"],
        a["k"], a["v"], a["ps"], a["kp"], a["vp"], a["cap"], a["nxt"], a["nxo"], a["bt"], a["mp"],
        a["sl"], a["slo"], a["ws"], a["wsb"], None)


def test_append_refusals(C):
    assert append(C, C.dims(1, 3, 2, 128)) == C.KVS_ERR_SHAPE
    assert append(C, C.dims(1, 4, 2, 80)) == C.KVS_ERR_UNSUPPORTED
    for kw in (dict(B=-1), dict(N=-1), dict(cap=-1), dict(tok=None), dict(pos=None), dict(f=None)):
        assert append(C, **kw) == C.KVS_ERR_ARG, kw
    for name in ("k", "v", "kp", "vp", "nxt", "nxo", "bt", "sl", "slo", "ws"):
        assert append(C, **{name: None}) == C.KVS_ERR_ARG, name
        assert append(C, **{name: FAKE + 4}) == C.KVS_ERR_ALIGN, name
    assert append(C, q=FAKE) == C.KVS_ERR_ARG and append(C, qo=FAKE) == C.KVS_ERR_ARG
    assert append(C, q=FAKE, qo=FAKE + 32) == C.KVS_ERR_ARG
    assert append(C, tok=FAKE + 8) == C.KVS_ERR_ALIGN
    assert append(C, ps=0) == C.KVS_ERR_UNSUPPORTED
    assert append(C, ps=4097) == C.KVS_ERR_UNSUPPORTED
    assert append(C, mp=0) == C.KVS_ERR_SHAPE
    assert append(C, rot=24) == C.KVS_ERR_UNSUPPORTED
    dm = C.dims(40000, 40000, 40000, 128)
    assert append(C, dm) == C.KVS_ERR_UNSUPPORTED
    # lengths of 40 rows, 16 bytes apart: an overlap that is not the same tensor
    assert append(C, C.dims(10, 4, 2, 128), slo=FAKE + 16) == C.KVS_ERR_ARG
    need = C.kvs_append_paged_workspace_size(C.dims(1, 4, 2, 128), 2)
    assert append(C, wsb=need - 1) == C.KVS_ERR_CAPACITY
    assert append(C, B=0, N=0, tok=None, pos=None) == C.KVS_OK


def attend(C, dm=None, B=2, q=FAKE, ps=16, kp=FAKE, vp=FAKE, cap=8, bt=FAKE, mp=4, sl=FAKE, w=4,
           pos=FAKE, rk=FAKE, rv=FAKE, o=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 30):
    dm = dm or C.dims(1, 4, 2, 128)
    return C._lib.kvs_attn_decode(ctypes.byref(dm), B, q, ps, kp, vp, cap, bt, mp, sl, w, pos, rk,
                                  rv, o, lse, ws, wsb, None)


def test_attend_refusals(C):
    assert attend(C, C.dims(0, 4, 2, 128)) == C.KVS_ERR_SHAPE
    assert attend(C, C.dims(1, 4, 3, 128)) == C.KVS_ERR_SHAPE
    assert attend(C, C.dims(1, 4, 2, 256)) == C.KVS_ERR_UNSUPPORTED
    for kw in (dict(B=-1), dict(w=-1), dict(cap=-1)):
        assert attend(C, **kw) == C.KVS_ERR_ARG, kw
    for name in ("q", "kp", "vp", "bt", "sl", "pos", "rk", "rv", "o", "ws"):
        assert attend(C, **{name: None}) == C.KVS_ERR_ARG, name
        assert attend(C, **{name: FAKE + 2}) == C.KVS_ERR_ALIGN, name
    assert attend(C, lse=FAKE + 4) == C.KVS_ERR_ALIGN
    assert attend(C, ps=0) == C.KVS_ERR_UNSUPPORTED
    assert attend(C, ps=5000) == C.KVS_ERR_UNSUPPORTED
    assert attend(C, mp=0) == C.KVS_ERR_SHAPE
    assert attend(C, mp=1 << 27, ps=16) == C.KVS_ERR_UNSUPPORTED
    assert attend(C, C.dims(40000, 40000, 40000, 128)) == C.KVS_ERR_UNSUPPORTED
    need = C.kvs_attn_decode_workspace_size(C.dims(1, 4, 2, 128), 2)
    assert need > 0 and attend(C, wsb=need - 1) == C.KVS_ERR_CAPACITY
    assert attend(C, B=0, q=None, o=None, ws=None) == C.KVS_OK


def test_workspace_sizes_of_empty_or_refused_shapes(C):
    for dm, B in ((C.dims(1, 4, 2, 128), 0), (C.dims(0, 4, 2, 128), 2),
                  (C.dims(40000, 40000, 40000, 128), 2)):
        assert C.kvs_append_paged_workspace_size(dm, B) == 0
        assert C.kvs_attn_decode_workspace_size(dm, B) == 0
    assert C.kvs_append_paged_workspace_size(C.dims(2, 8, 4, 128), 3) >= 2 * 4 * 3 * 8


def test_binding_checks_types_and_sizes(C):
    """A tensor of another type, or too small for the sizes given with it, is refused by
    name before the library is called; so are host tensors and short frequency lists."""
    dm = C.dims(1, 2, 1, 64)
    bf, i32 = torch.zeros(2 * 3 * 64, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="pos"):
        C.kvs_rope(dm, 3, i32.long(), 64, [1.0] * 32, False, bf, bf, None, None, stream=0)
    with pytest.raises(ValueError, match="q must"):
        C.kvs_rope(dm, 3, FAKE, 64, [1.0] * 32, False, bf[:-1], FAKE, None, None, stream=0)
    with pytest.raises(ValueError, match="frequencies"):
        C.kvs_rope(dm, 3, FAKE, 64, [1.0] * 31, False, FAKE, FAKE, None, None, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        C.kvs_rope(dm, 3, FAKE, 64, [1.0] * 32, False, bf, bf, None, None, stream=0)
    with pytest.raises(ValueError, match="block_table"):
        C.kvs_attn_decode(dm, 3, FAKE, 16, FAKE, FAKE, 4, i32, 4, FAKE, 0, None, None, None, FAKE,
                          None, FAKE, 1 << 20, stream=0)
    with pytest.raises(ValueError, match="tok_start"):
        C.kvs_append_paged(dm, 8, 9, i32, FAKE, 0, None, False, None, None, FAKE, FAKE, 16, FAKE,
                           FAKE, 4, FAKE, FAKE, FAKE, 4, FAKE, FAKE, FAKE, 1 << 20, stream=0)


def test_binding_refuses_what_is_not_an_argument(C):
    """Numbers that do not fit, things that are neither tensors nor addresses, other dims,
    frequencies that are no numbers: Python errors that name the argument, no call."""
    dm = C.dims(1, 2, 1, 64)
    f = [1.0] * 32

    def call(dm=dm, N=0, pos=FAKE, rot=64, f=f, q=None, stream=0):
        C.kvs_rope(dm, N, pos, rot, f, False, q, q, None, None, stream=stream)

    call()
    for kw in (dict(N=1 << 31), dict(N=-(1 << 40)), dict(rot=1 << 32), dict(N=1 << 70)):
        with pytest.raises(OverflowError, match="out of range"):
            call(**kw)
    for kw in (dict(N="4"), dict(N=1.5), dict(pos="x"), dict(q=[1.0]), dict(dm=b"abc"),
               dict(f=["a"] * 32), dict(f=3.0)):
        with pytest.raises((TypeError, ValueError)):
            call(**kw)
    with pytest.raises(AttributeError):
        call(stream="s")
    with pytest.raises(OverflowError):
        C.kvs_attn_decode(dm, 0, FAKE, 16, FAKE, FAKE, 4, FAKE, 4, FAKE, 0, None, None, None, FAKE,
                          None, FAKE, -1, stream=0)
    with pytest.raises(C.KvsError) as e:   # the library's own refusals keep status and message
        call(N=-1)
    assert e.value.status == C.KVS_ERR_ARG and "N = -1" in str(e.value)


def test_binding_takes_frequencies_of_any_kind(C):
    """float64 CPU tensors, other tensors, arrays, lists and iterators; the library refuses a
    value that is not finite, so that it shows which ones were read."""
    import numpy as np
    dm = C.dims(1, 2, 1, 64)
    good = [10000.0 ** (-i / 32) for i in range(32)]
    for bad in (False, True):
        v = good[:31] + [float("nan")] if bad else good
        kinds = [torch.tensor(v, dtype=torch.float64), torch.tensor(v), np.array(v), v, tuple(v),
                 iter(v), torch.tensor(v + v, dtype=torch.float64)[:32],
                 torch.tensor([v, v], dtype=torch.float64).t().contiguous().t()[0]]
        for f in kinds:
            if bad:
                with pytest.raises(C.KvsError, match="not finite"):
                    C.kvs_rope(dm, 0, None, 64, f, False, None, None, None, None, stream=0)
            else:
                C.kvs_rope(dm, 0, None, 64, f, False, None, None, None, None, stream=0)


def test_binding_sizes_that_pass_64_bits(C):
    """The sizes that tensors are checked against do not wrap."""
    dm = C.dims(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 128)
    bf = torch.zeros(8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q must"):
        C.kvs_rope(dm, 2 ** 31 - 1, FAKE, 0, None, False, bf, bf, None, None, stream=0)
