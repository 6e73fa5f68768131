"""Pins of the oracle's rotation, paged append and paged decode attention (closed forms,
invariants, hand-worked cases), and one-line slips planted in a copy of the oracle that
the pins must catch.  CPU only."""
import inspect
import math
import types

import numpy as np
import pytest

import oracle.kvs_oracle as real

FREQ = 10000.0 ** (-np.arange(0, 16, 2) / 16.0)


def rotation_closed_forms(O):
    x = np.zeros((1, 16))
    x[0, 1] = 1.0
    # a quarter turn of pair 1: (1, 0) -> (0, 1), halves and neighbours
    f = np.zeros(8)
    f[1] = math.pi / 2
    y = O.rope(x, [1], f, 16, False)
    assert abs(y[0, 9] - 1) < 1e-15 and abs(y[0, 1]) < 1e-15
    f = np.zeros(8)
    f[0] = math.pi / 2
    y = O.rope(x, [1], f, 16, True)          # dimension 1 is the second of pair 0
    assert abs(y[0, 0] + 1) < 1e-15 and abs(y[0, 1]) < 1e-15


def rotation_invariants(O):
    rng = np.random.default_rng(0)
    x, z = rng.standard_normal((5, 24)), rng.standard_normal((5, 24))
    pos = np.array([0, 1, 7, 1000, -3])
    for il in (False, True):
        y = O.rope(x, pos, FREQ, 16, il)
        assert np.array_equal(y[0], x[0])                           # position 0
        assert np.array_equal(y[:, 16:], x[:, 16:])                 # past rot_dim
        assert np.allclose((y ** 2).sum(1), (x ** 2).sum(1))        # a rotation
        assert np.allclose(O.rope(y, pos, -FREQ, 16, il), x)        # and back
        # the product of a query and a key depends on the difference of positions alone
        q1, k1 = O.rope(x, pos, FREQ, 16, il), O.rope(z, pos - 5, FREQ, 16, il)
        q2, k2 = O.rope(x, pos + 11, FREQ, 16, il), O.rope(z, pos + 6, FREQ, 16, il)
        assert np.allclose((q1 * k1).sum(1), (q2 * k2).sum(1))
        # the adjoint, by differences: d(y . z)/dx is the rotation back of z
        grad = O.rope(z, pos, -FREQ, 16, il)
        e = 1e-6
        for dim in (0, 3, 9, 15, 20):
            xp, xm = x.copy(), x.copy()
            xp[:, dim] += e
            xm[:, dim] -= e
            diff = ((O.rope(xp, pos, FREQ, 16, il) - O.rope(xm, pos, FREQ, 16, il)) * z).sum(1)
            assert np.allclose(diff / (2 * e), grad[:, dim], atol=1e-8)


def append_by_hand(O):
    # two rows (two heads) of one sequence, pages of 2, lengths 3 and 0; three tokens
    kp = np.arange(7 * 2 * 1, dtype=float).reshape(7, 2, 1) + 100
    vp = kp + 100
    bt = np.full((1, 2, 1, 3), -1)
    bt[0, 0, 0, :2] = [1, 0]
    k = np.array([[[[1.0], [2.0], [3.0]], [[4.0], [5.0], [6.0]]]])
    kp2, vp2, nxt, bt2, sl2 = O.append_paged(k, -k, [0, 3], 2, kp, vp, 2, bt,
                                             np.array([[[3], [0]]]))
    assert bt2[0, 0, 0].tolist() == [1, 0, 2] and bt2[0, 1, 0].tolist() == [3, 4, -1]
    assert nxt == 5 and sl2.ravel().tolist() == [6, 3]
    assert kp2[:, :, 0].tolist() == [[100, 1], [102, 103], [2, 3], [4, 5], [6, 0], [110, 111],
                                     [112, 113]]
    assert vp2[2, :, 0].tolist() == [-2, -3] and vp2[0, :, 0].tolist() == [200, -1]
    # five pages are in use: a pool of five holds them, one of four and a table of two do not
    assert O.append_paged(k, -k, [0, 3], 2, kp[:5], vp[:5], 2, bt, np.array([[[3], [0]]]))[2] == 5
    assert O.append_paged(k, k, [0, 3], 2, kp[:4], vp[:4], 2, bt, np.array([[[3], [0]]])) == "pool"
    assert O.append_paged(k, k, [0, 3], 2, kp, vp, 2, bt[..., :2], np.array([[[3], [0]]])) == "table"


def attend_closed_forms(O):
    rng = np.random.default_rng(1)
    L, Hq, Hkv, B, d, ps = 1, 4, 2, 2, 8, 3
    kp, vp = rng.standard_normal((6, ps, d)), rng.standard_normal((6, ps, d))
    bt = np.array([[[[5, 0], [2, -1]], [[1, 4], [-1, -1]]]])
    sl = np.array([[[4, 2], [6, 0]]])
    o, lse, spread = O.attn_decode(np.zeros((L, Hq, B, d)), kp, vp, ps, bt, sl)
    # q = 0: the mean of the values, ln n; a row without keys
    assert np.allclose(o[0, 0, 0], np.concatenate([vp[5], vp[0, :1]]).mean(0))
    assert np.allclose(o[0, 1, 1], vp[2, :2].mean(0)) and np.allclose(lse[0, 2, 0], math.log(6))
    assert np.array_equal(o[0, 3, 1], np.zeros(d)) and lse[0, 3, 1] == -np.inf
    # the paged cache laid out densely is the attention forward's last query
    q = rng.standard_normal((L, Hq, B, d))
    o, lse, _ = O.attn_decode(q, kp, vp, ps, bt, sl)
    K, V = kp[[1, 4]].reshape(1, 1, 6, d), vp[[1, 4]].reshape(1, 1, 6, d)
    want, want_lse = O.attention_forward(q[:, 2:, :1], K, None, V, None)
    assert np.allclose(o[:, 2:, :1], want) and np.allclose(lse[:, 2:, :1], want_lse)
    # ring tokens count as keys, as many as have come
    rk, rv = rng.standard_normal((L, Hkv, B, 3, d)), rng.standard_normal((L, Hkv, B, 3, d))
    o, lse, _ = O.attn_decode(q * 0, kp, vp, ps, bt, sl, rk, rv, [2, 9])
    assert np.allclose(lse[0, 0], np.log([6, 5]))
    assert np.allclose(o[0, 3, 1], rv[0, 1, 1].mean(0))
    assert np.allclose(o[0, 0, 0], np.concatenate([vp[5], vp[0, :1], rv[0, 0, 0, :2]]).mean(0))
    # one key: its value, whatever the query; spread bounds |o|
    o, _, spread = O.attn_decode(q, kp, vp, ps, bt, np.minimum(sl, 1))
    assert np.allclose(o[0, 0, 0], vp[5, 0]) and np.allclose(spread[0, 0, 0], np.abs(vp[5, 0]))


PINS = [rotation_closed_forms, rotation_invariants, append_by_hand, attend_closed_forms]


@pytest.mark.parametrize("pin", PINS, ids=lambda p: p.__name__)
def test_pin(pin):
    pin(real)


MUTATIONS = [
    ("turns the other way", "x[..., a] * np.cos(t) - x[..., b]", "x[..., a] * np.cos(t) + x[..., b]"),
    ("pairs swapped", "if interleaved else (i, i + rot_dim // 2)",
     "if not interleaved else (i, i + rot_dim // 2)"),
    ("rotates rotated values", "out[..., b] = x[..., b] * np.cos(t) + x[..., a]",
     "out[..., b] = x[..., b] * np.cos(t) + out[..., a]"),
    ("angle off by one", "t = np.asarray(pos, dtype=np.float64) *",
     "t = (np.asarray(pos, dtype=np.float64) + 1) *"),
    ("new page too late", "if n % page_size == 0:\n                        if nxt",
     "if n % page_size == 1:\n                        if nxt"),
    ("page not cleared", "kp[nxt], vp[nxt] = 0, 0", "vp[nxt] = 0"),
    ("values are keys", "] = v_new[l, h, t]", "] = k_new[l, h, t]"),
    ("table one short", "if n // page_size >= max_pages:", "if n // page_size > max_pages - 2:"),
    ("pool one short", "if nxt >= len(kp):", "if nxt >= len(kp) - 1:"),
    ("first head's tokens", "] = k_new[l, h, t]", "] = k_new[l, 0, t]"),
    ("modulo group", "hk, n = hq // g, int(", "hk, n = hq % H_kv, int("),
    ("drops the ring's last", "held = min(int(pos[b]), ring_k.shape[3])",
     "held = min(int(pos[b]), ring_k.shape[3] - 1)"),
    ("whole ring", "held = min(int(pos[b]), ring_k.shape[3])", "held = ring_k.shape[3]"),
    ("no normaliser", "o[l, hq, b], lse_[l, hq, b], spread[l, hq, b] = a @ V",
     "o[l, hq, b], lse_[l, hq, b], spread[l, hq, b] = np.exp(x) @ V"),
    ("pages in order", "at = [(block_table[l, hk, b, i // page_size], i % page_size)",
     "at = [(i // page_size, i % page_size)"),
    ("lse without the maximum", "z = m + np.log(np.exp(x - m).sum())",
     "z = np.log(np.exp(x - m).sum())"),
]


@pytest.mark.parametrize("name,old,new", MUTATIONS, ids=[m[0] for m in MUTATIONS])
def test_planted_slip_is_caught(name, old, new):
    src = inspect.getsource(real)
    assert src.count(old) == 1, name
    mod = types.ModuleType("mutated")
    exec(compile(src.replace(old, new), "mutated", "exec"), mod.__dict__)
    for pin in PINS:
        try:
            pin(mod)
        except Exception:
            return
    raise AssertionError(f"no pin caught: {name}")
