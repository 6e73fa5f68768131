"""Host-side checks of kvs_attn_tree, kvs_accept_paged, kvs_fork_paged and kvs_reclaim_paged: refusals with
their status codes, empty calls, workspace sizes, and what the binding refuses.  No GPU: every
call fails validation, or is an empty call, before anything is enqueued."""
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


def tree(C, dm=None, B=2, N=6, md=8, tok=FAKE, up=FAKE, q=FAKE, ps=16, kp=FAKE, vp=FAKE, cap=8, bt=FAKE, mp=4,
         sl=FAKE, w=3, pos=FAKE, rk=FAKE, rv=FAKE, o=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 30):
    dm = dm or C.dims(1, 4, 2, 128)
    return C._lib.kvs_attn_tree(ctypes.byref(dm), B, N, md, tok, up, q, ps, kp, vp, cap, bt, mp, sl, w, pos,
                                rk, rv, o, lse, ws, wsb, None)


def accept(C, dm=None, B=2, N=6, tok=FAKE, n=FAKE, path=FAKE, ps=16, kp=FAKE, vp=FAKE, cap=8, bt=FAKE,
           mp=4, sl=FAKE, slo=FAKE):
    dm = dm or C.dims(1, 4, 2, 128)
    return C._lib.kvs_accept_paged(ctypes.byref(dm), B, N, tok, n, path, ps, kp, vp, cap, bt, mp, sl, slo,
                                   None)


def fork(C, dm=None, B=4, forks=2, src=FAKE, dst=FAKE, ps=16, kp=FAKE, vp=FAKE, cap=8, nxt=FAKE, nxo=FAKE,
         bt=FAKE, mp=4, sl=FAKE, w=3, pos=FAKE, rs=FAKE, rk=FAKE, rv=FAKE, ws=FAKE, wsb=1 << 20):
    dm = dm or C.dims(1, 4, 2, 128)
    return C._lib.kvs_fork_paged(ctypes.byref(dm), B, forks, src, dst, ps, kp, vp, cap, nxt, nxo, bt, mp,
                                 sl, w, pos, rs, rk, rv, ws, wsb, None)


def reclaim(C, dm=None, B=4, ps=16, kp=FAKE, vp=FAKE, cap=8, nxt=FAKE, nxo=FAKE, bt=FAKE, bto=FAKE, mp=4,
            sl=FAKE, ws=FAKE, wsb=1 << 20):
    dm = dm or C.dims(1, 4, 2, 128)
    return C._lib.kvs_reclaim_paged(ctypes.byref(dm), B, ps, kp, vp, cap, nxt, nxo, bt, bto, mp, sl, ws,
                                    wsb, None)


@pytest.mark.parametrize("call", [tree, accept, fork, reclaim], ids=lambda f: f.__name__)
def test_what_they_share(C, call):
    assert call(C, C.dims(0, 4, 2, 128)) == C.KVS_ERR_SHAPE
    assert call(C, C.dims(1, 3, 2, 128)) == C.KVS_ERR_SHAPE
    assert call(C, C.dims(1, 4, 2, 96)) == C.KVS_ERR_UNSUPPORTED
    assert call(C, C.dims(40000, 40000, 40000, 128)) == C.KVS_ERR_UNSUPPORTED
    assert call(C, B=-1) == C.KVS_ERR_ARG and call(C, cap=-1) == C.KVS_ERR_ARG
    assert call(C, ps=0) == C.KVS_ERR_UNSUPPORTED and call(C, ps=4097) == C.KVS_ERR_UNSUPPORTED
    assert call(C, mp=0) == C.KVS_ERR_SHAPE
    names = dict(tree=("tok", "q", "kp", "vp", "bt", "sl", "pos", "rk", "rv", "o", "ws"),
                 accept=("tok", "n", "path", "kp", "vp", "bt", "sl", "slo"),
                 fork=("src", "dst", "kp", "vp", "nxt", "nxo", "bt", "sl", "pos", "rs", "rk", "rv", "ws"),
                 reclaim=("kp", "vp", "nxt", "nxo", "bt", "bto", "sl", "ws"))[call.__name__]
    for name in names:
        assert call(C, **{name: None}) == C.KVS_ERR_ARG, name
        assert call(C, **{name: FAKE + 4}) == C.KVS_ERR_ALIGN, name


def test_tree_refusals(C):
    dm = C.dims(1, 4, 2, 128)
    assert tree(C, N=-1) == C.KVS_ERR_ARG and tree(C, w=-1) == C.KVS_ERR_ARG
    for md in (0, -1, 257):
        assert tree(C, md=md) == C.KVS_ERR_UNSUPPORTED
    assert tree(C, up=FAKE + 4) == C.KVS_ERR_ALIGN and tree(C, lse=FAKE + 8) == C.KVS_ERR_ALIGN
    assert tree(C, mp=1 << 27) == C.KVS_ERR_UNSUPPORTED
    # tiles of all rows: 64 x 8 x 128 KV heads' rows, 8 query tiles each, keys for 2^22 / 128 tiles
    deep = C.dims(64, 64, 8, 128)
    big = dict(B=128, N=128 * 128, md=128, mp=1 << 18)
    assert tree(C, deep, **big) == C.KVS_ERR_UNSUPPORTED and b"tiles" in C._lib.kvs_last_error()
    # few drafted tokens in all, so a query tile a row (no workspace either way): 2^31 tiles with
    # ((2^18 - 8) * 16 + 3 + 127) / 128 = 2^15 of keys, 2^31 - 2^16 with one less
    assert tree(C, deep, B=128, N=15, md=128, mp=(1 << 18) - 8, wsb=0) == C.KVS_ERR_UNSUPPORTED
    assert tree(C, deep, B=128, N=15, md=128, mp=(1 << 18) - 16, wsb=0) == C.KVS_ERR_CAPACITY
    for d in (64, 128):
        need = C.kvs_attn_tree_workspace_size(C.dims(1, 4, 2, d), 2, 6)
        assert need > 0 and tree(C, C.dims(1, 4, 2, d), wsb=need - 1) == C.KVS_ERR_CAPACITY
    assert C.kvs_attn_tree_workspace_size(dm, 0, 6) == C.kvs_attn_tree_workspace_size(dm, 2, 0) == 0
    assert tree(C, B=0, tok=None, q=None, bt=None, sl=None, o=None, ws=None) == C.KVS_OK
    assert tree(C, N=0, tok=None, q=None, bt=None, sl=None, o=None, ws=None) == C.KVS_OK


def test_accept_refusals(C):
    assert accept(C, N=-1) == C.KVS_ERR_ARG
    # lengths of 40 rows, 16 bytes apart: an overlap that is not the same tensor
    assert accept(C, C.dims(10, 4, 2, 128), slo=FAKE + 16) == C.KVS_ERR_ARG
    assert accept(C, B=0, tok=None, n=None, path=None, bt=None, sl=None, slo=None) == C.KVS_OK


def test_fork_refusals(C):
    dm = C.dims(1, 4, 2, 128)
    assert fork(C, forks=-1) == C.KVS_ERR_ARG and fork(C, w=-1) == C.KVS_ERR_ARG
    assert fork(C, forks=5) == C.KVS_ERR_SHAPE
    assert fork(C, B=131073, forks=1) == C.KVS_ERR_UNSUPPORTED
    assert fork(C, w=2 ** 30) == C.KVS_ERR_UNSUPPORTED
    need = C.kvs_fork_paged_workspace_size(dm, 4, 2)
    assert need > 0 and fork(C, wsb=need - 1) == C.KVS_ERR_CAPACITY
    assert fork(C, forks=0, src=None, dst=None, ws=None) == C.KVS_OK
    assert fork(C, B=0, forks=0, src=None, bt=None, sl=None, ws=None) == C.KVS_OK
    for bad in ((C.dims(1, 4, 2, 128), 0, 0), (dm, 4, 5), (dm, 4, 0), (C.dims(40000, 4, 40000, 128), 64, 1)):
        assert C.kvs_fork_paged_workspace_size(*bad) == 0


def test_reclaim_refusals(C):
    dm = C.dims(1, 4, 2, 128)
    assert reclaim(C, bto=FAKE + 16) == C.KVS_ERR_ARG
    for cap in (0, 1, 1024, 1025, 3_000_000):
        need = C.kvs_reclaim_paged_workspace_size(dm, 4, cap)
        assert need >= 16 + cap / 8 and reclaim(C, cap=cap, wsb=need - 1) == C.KVS_ERR_CAPACITY
    assert reclaim(C, B=0, bt=None, bto=None, sl=None, ws=None) == C.KVS_OK
    assert C.kvs_reclaim_paged_workspace_size(dm, 0, 5) == C.kvs_reclaim_paged_workspace_size(dm, 4, -1) == 0


def test_binding_checks_types_and_sizes(C):
    """What the compiled binding refuses before the library sees it."""
    dm = C.dims(1, 2, 1, 64)
    meta = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="meta")  # noqa: E731
    with pytest.raises(ValueError, match="parent must hold at least 6 elements of torch.int32, got 6 of torch.int64"):
        C.kvs_attn_tree(dm, 2, 6, 8, FAKE, meta(6, dtype=torch.int64), FAKE, 16, FAKE, FAKE, 8, FAKE, 4, FAKE, 0,
                        None, None, None, FAKE, None, FAKE, 1 << 30, stream=0)
    with pytest.raises(ValueError, match="o must hold at least 768 elements of torch.bfloat16"):
        C.kvs_attn_tree(dm, 2, 6, 8, FAKE, None, FAKE, 16, FAKE, FAKE, 8, FAKE, 4, FAKE, 0, None, None, None,
                        meta(767, dtype=torch.bfloat16), None, FAKE, 1 << 30, stream=0)
    with pytest.raises(ValueError, match="accept must hold at least 6 elements of torch.int32"):
        C.kvs_accept_paged(dm, 2, 6, FAKE, FAKE, meta(5), 16, FAKE, FAKE, 8, FAKE, 4, FAKE, FAKE, stream=0)
    with pytest.raises(ValueError, match="n_accept must hold .* torch.int64"):
        C.kvs_accept_paged(dm, 2, 6, FAKE, meta(2, dtype=torch.int64), FAKE, 16, FAKE, FAKE, 8, FAKE, 4,
                           FAKE, FAKE, stream=0)
    with pytest.raises(ValueError, match="CUDA tensors on the current device"):
        C.kvs_accept_paged(dm, 2, 6, torch.zeros(3, dtype=torch.int32), FAKE, FAKE, 16, FAKE, FAKE, 8, FAKE,
                           4, FAKE, FAKE, stream=0)
    with pytest.raises(ValueError, match="ring_score must hold at least 12"):
        C.kvs_fork_paged(dm, 4, 2, FAKE, FAKE, 16, FAKE, FAKE, 8, FAKE, FAKE, FAKE, 4, FAKE, 3, FAKE,
                         meta(11, dtype=torch.float32), FAKE, FAKE, FAKE, 1 << 20, stream=0)
    with pytest.raises(ValueError, match="block_table_out must hold at least 16"):
        C.kvs_reclaim_paged(dm, 4, 16, FAKE, FAKE, 8, FAKE, FAKE, FAKE, meta(15), 4, FAKE, FAKE, 1 << 20,
                            stream=0)
    with pytest.raises(C.KvsError, match="kvs_fork_paged: n_forks = 5 above B = 4"):
        C.kvs_fork_paged(dm, 4, 5, FAKE, FAKE, 16, FAKE, FAKE, 8, FAKE, FAKE, FAKE, 4, FAKE, 0, None, None,
                         None, None, FAKE, 1 << 20, stream=0)
    with pytest.raises(TypeError, match="arguments"):
        C._binding.reclaim_paged(dm, 4)
