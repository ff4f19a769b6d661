"""The cache oracle against closed forms, and the plain rules it states."""

import numpy as np
import pytest

import oracle
from cache_util import Batch, to_bf16

C = oracle.cache


@pytest.mark.parametrize("amax,e", [(0.0, -48), (448.0, 0), (448.5, 1), (224.0, -1), (1.0, -8), (2.0 ** -70, -48),
                                    (float("inf"), 48), (1e-40, -48)])
def test_scale_exponent(amax, e):
    assert C.scale_exponent(np.float32(amax)) == e


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_an_angle(interleaved):
    d, rd = 64, 32
    ang = np.linspace(0.1, 3.0, rd // 2)
    table = np.concatenate([np.cos(ang), np.sin(ang)]).astype(np.float32)
    x = np.random.default_rng(0).standard_normal((3, d)).astype(np.float32)
    y = C.rope_rotate(x, table, interleaved)
    z = (x[:, 0:rd:2] + 1j * x[:, 1:rd:2] if interleaved else x[:, :rd // 2] + 1j * x[:, rd // 2:rd]) * np.exp(1j * ang)
    w = y[:, 0:rd:2] + 1j * y[:, 1:rd:2] if interleaved else y[:, :rd // 2] + 1j * y[:, rd // 2:rd]
    assert np.abs(w - z).max() < 1e-6 and np.array_equal(y[:, rd:], x[:, rd:])


def test_appending_one_by_one_or_at_once():
    """Power-of-two scales make the codes of a page independent of how its
    tokens arrived, except codes that were subnormal before the scale grew."""
    b = Batch(5, [70, 33], [70, 33], 2, 1, 64, 32, filled=False)
    one = {k: v.copy() for k, v in b.cache.items()}
    C.append(one, b.k_new, b.v_new, b.table, b.q_start, b.kv_len)
    step = {k: v.copy() for k, v in b.cache.items()}
    for i in range(70):
        live = [s for s in range(2) if i < b.lens[s]]
        rows = np.array([b.q_start[s] + i for s in live])
        C.append(step, b.k_new[rows], b.v_new[rows], b.table[live], np.arange(len(live) + 1),
                 np.full(len(live), i + 1))
    for name in ("k", "v"):
        assert np.array_equal(one[name + "_scale"], step[name + "_scale"])
        x, y = oracle.e4m3_decode(one[name]), oracle.e4m3_decode(step[name])
        big = np.abs(x) >= 2.0 ** -6
        assert np.array_equal(x[big], y[big])
        small = np.abs(x) < 2.0 ** -6
        assert np.abs(x[small] - y[small]).max() <= 2.0 ** -9   # one subnormal step
    k, v = C.cached_values(one, b.table[1], 33)
    ref = b.v_new[70:103].transpose(1, 0, 2)
    assert np.abs(v - ref).max() <= 2.0 ** -4 * np.abs(ref).max()


def test_bounds_bound_the_scores():
    b = Batch(7, [200], [3], 2, 3, 64, 32)
    for h in range(2):
        k, _ = C.cached_values(b.cache, b.table[0], 200)
        for p in range(6):
            bd = b.cache["bounds"][b.table[0, p], h].astype(float) * 448 / 127 * b.cache["k_scale"][b.table[0, p], h]
            kp = k[h, p * 32:(p + 1) * 32]
            assert (kp >= bd[0] - 1e-9).all() and (kp <= bd[1] + 1e-9).all()


def test_attend_matches_dense_oracle():
    b = Batch(11, [50], [50], 1, 1, 64, 32)
    O, L, _, _ = C.attend(b.q, b.cache, b.table, b.q_start, b.kv_len, True, 0.125)
    k, v = C.cached_values(b.cache, b.table[0], 50)
    o, l = oracle.attention_forward(b.q[:, 0][None, None], k[None], v[None], True, 0.125)
    assert np.abs(O[:, 0] - o[0, 0]).max() < 1e-12 and np.abs(L[:, 0] - l[0, 0]).max() < 1e-12
    every = np.broadcast_to(np.arange(2, dtype=np.int32), (50, 1, 2))
    O2, L2, _, _ = C.attend(b.q, b.cache, b.table, b.q_start, b.kv_len, True, 0.125, selected=every)
    assert np.array_equal(O, O2) and np.array_equal(L, L2)


def test_select_prefers_the_page_that_holds_the_key():
    b = Batch(13, [320], [1], 1, 1, 64, 32)
    b.cache["k"][:] = 0
    b.cache["bounds"][:] = 0
    b.cache["k_scale"][:] = 1
    target = int(b.table[0, 4])
    q = b.q[0, 0]
    code = oracle.e4m3_encode(np.where(q > 0, 100.0, -100.0).astype(np.float32))
    b.cache["k"][target, 0, 3] = code
    lo, hi = C._bound_units(oracle.e4m3_decode(code))
    b.cache["bounds"][target, 0] = np.stack([np.minimum(lo, 0), np.maximum(hi, 0)]).astype(np.int8)
    sel = C.select(b.q, b.cache, b.table, b.q_start, b.kv_len, 3, 1, 1)
    assert sel[0, 0].tolist() == [0, 4, 9]
    assert np.array_equal(to_bf16(b.q), b.q)
