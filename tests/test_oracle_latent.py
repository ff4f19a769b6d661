"""Pins of the oracles of rotary positions, the latent cache and shared pages:
closed forms, invariants, and an independent formula each."""

import numpy as np
import pytest
import torch

import oracle
from cache_util import to_bf16
from exact_attention_fattn_gb300 import cache


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(interleaved):
    r = np.random.default_rng(1)
    x, y = r.standard_normal((5, 40)), r.standard_normal((5, 40))
    ang = r.uniform(-9, 9, (5, 16))
    rx, ry = oracle.rope.rotate(x, ang, interleaved), oracle.rope.rotate(y, ang, interleaved)
    # lengths and inner products stay, columns from rope_dim on too; angles add up
    assert np.allclose((rx * ry).sum(1), (x * y).sum(1)) and (rx[:, 32:] == x[:, 32:]).all()
    assert np.allclose(oracle.rope.rotate(rx, -ang, interleaved), x)
    two = oracle.rope.rotate(oracle.rope.rotate(x, ang, interleaved), 0.5 * ang, interleaved)
    assert np.allclose(two, oracle.rope.rotate(x, 1.5 * ang, interleaved))
    # the stepwise fp32 form agrees: two products and a sum, three roundings of 2^-24 and the table's
    t = np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)
    x32 = x.astype(np.float32)
    got = oracle.rope.rotate_fp32(x32, t, interleaved)
    assert np.abs(got - oracle.rope.rotate(x32, ang, interleaved)).max() <= 4 * 2.0 ** -24 * 2 * np.abs(x32).max()
    back = oracle.rope.rotate_fp32(x32, t, interleaved, transposed=True)
    assert np.abs(back - oracle.rope.rotate(x32, -ang, interleaved)).max() <= 4 * 2.0 ** -24 * 2 * np.abs(x32).max()
    assert not np.allclose(back[:, :32], got[:, :32])


def test_layouts_of_pairs_differ_by_a_permutation():
    r = np.random.default_rng(2)
    x, ang = r.standard_normal((3, 32)), r.uniform(-3, 3, (3, 16))
    perm = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2)])
    assert np.allclose(oracle.rope.rotate(x, ang, True)[:, perm], oracle.rope.rotate(x[:, perm], ang, False))


def test_frequencies():
    f = oracle.rope.frequencies(64, factor=8.0, original=4096)
    plain = oracle.rope.frequencies(64)
    turns = 4096 * plain / (2 * np.pi)
    assert (f[turns >= 32] == plain[turns >= 32]).all() and np.allclose(f[turns <= 1], plain[turns <= 1] / 8)
    assert ((f >= plain / 8 * (1 - 1e-15)) & (f <= plain)).all() and (np.diff(f) < 0).all()
    assert np.allclose(oracle.rope.frequencies(64, factor=4.0), plain / 4)


@pytest.mark.parametrize("kw", [{}, {"factor": 4.0}, {"factor": 8.0, "original": 4096}, {"theta": 500000.0},
                                {"factor": 16.0, "original": 2048, "ramp": (2.0, 20.0), "magnitude": 1.0}])
def test_tables(kw):
    """The table against the oracle's angles: cosines and sines taken in 64 bits,
    one rounding to fp32 (2^-24 of values up to the magnitude)."""
    t = cache.fattn_rope_table(5000, 64, device="cpu", **kw).numpy()
    f = oracle.rope.frequencies(64, **{k: v for k, v in kw.items() if k != "magnitude"})
    mag = kw.get("magnitude", 0.1 * np.log(kw["factor"]) + 1.0 if "original" in kw else 1.0)
    ang = np.arange(5000)[:, None] * f
    # the angles' own rounding: 2^-53 of 5000
    err = np.abs(t - mag * np.concatenate([np.cos(ang), np.sin(ang)], axis=1)).max()
    assert err <= mag * (2.0 ** -24 + 4 * 5000 * 2.0 ** -53)


def test_tables_refuse():
    for kw in (dict(factor=0.5), dict(factor=float("inf")), dict(factor=2.0, original=-1),
               dict(factor=2.0, original=100, ramp=(3.0, 3.0)), dict(factor=2.0, original=100, ramp=(-1.0, 3.0))):
        with pytest.raises(ValueError):
            cache.fattn_rope_table(8, 32, device="cpu", **kw)


def test_bf16_rounding():
    r = np.random.default_rng(3)
    x = np.concatenate([r.standard_normal(1000) * 10.0 ** r.integers(-30, 30, 1000), [0.0, -0.0, np.inf, -np.inf, 3.4e38]])
    x = x.astype(np.float32)
    assert np.array_equal(oracle.latent._bf16(x), torch.from_numpy(x).to(torch.bfloat16).float().numpy())


def _batch(rank=8):
    r = np.random.default_rng(4)
    lens, news, page = [5, 9, 1, 0], [2, 9, 1, 1], 4
    data = to_bf16(r.standard_normal((9, page, rank + oracle.latent.ROPE)))
    table = np.array([[7, 1, 99], [0, 3, 8], [2, -1, 5], [-1, -1, -1]])
    q = to_bf16(r.standard_normal((14, 3, rank + oracle.latent.ROPE)))
    return data, table, np.array([0, 2, 11, 12, 13]), np.array(lens), q


def test_attention_against_one_softmax_over_all():
    """One masked softmax over the sequence, by an independent library."""
    data, table, q_start, kv_len, q = _batch()
    for causal in (True, False):
        O, L, A, D = oracle.latent.attend(q, data, 8, table, q_start, kv_len, causal, 0.3)
        for b, (r0, r1) in enumerate(zip(q_start[:-1], q_start[1:])):
            k = torch.from_numpy(oracle.latent.tokens(data, table[b], kv_len[b]))
            x = 0.3 * torch.einsum("thc,kc->thk", torch.from_numpy(q[r0:r1]).double(), k)
            if causal:
                pos = torch.arange(kv_len[b] - (r1 - r0), kv_len[b])
                x = x.masked_fill((torch.arange(kv_len[b])[None, :] > pos[:, None])[:, None], -torch.inf)
            want = torch.logsumexp(x, dim=2).numpy()
            assert np.allclose(L[r0:r1], want, equal_nan=False)
            p = torch.softmax(x, dim=2).nan_to_num(nan=0.0)
            assert np.allclose(O[r0:r1], torch.einsum("thk,kc->thc", p, k[:, :8]).numpy())
        assert np.isnan(L[13]).all() and np.isneginf(L[12]).all()    # padding; a row that sees nothing
        assert (A >= np.abs(O) - 1e-12).all() and (D >= 0).all()


def test_absorbed_and_expanded_forms_agree():
    """Heads with keys W_k c and values W_v c, and the absorbed queries q W_k."""
    r = np.random.default_rng(5)
    rank, heads, d = 8, 3, 6
    data, table, q_start, kv_len, _ = _batch(rank)
    wk, wv = r.standard_normal((heads, d, rank)), r.standard_normal((heads, d, rank))
    qn, qr = r.standard_normal((14, heads, d)), r.standard_normal((14, heads, oracle.latent.ROPE))
    q = np.concatenate([np.einsum("thd,hdr->thr", qn, wk), qr], axis=2)
    O, L, _, _ = oracle.latent.attend(q, data, rank, table, q_start, kv_len, True, 0.2)
    k = oracle.latent.tokens(data, table[1], 9)
    for h in range(heads):
        x = 0.2 * (qn[2:11, h] @ (k[:, :rank] @ wk[h].T).T + qr[2:11, h] @ k[:, rank:].T)
        x[np.triu_indices(9, 1)] = -np.inf
        p = np.exp(x - x.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        assert np.allclose(p @ (k[:, :rank] @ wv[h].T), O[2:11, h] @ wv[h].T)


def test_append_then_read():
    data, table, q_start, kv_len, q = _batch()
    r = np.random.default_rng(6)
    table[3, 0], kv_len[3] = 4, 1
    lat, key = to_bf16(r.standard_normal((14, 8))), to_bf16(r.standard_normal((14, 64)))
    lat[5, 2] = np.inf
    before = data.copy()
    oracle.latent.append(data, lat, key, table, q_start, kv_len)
    k = oracle.latent.tokens(data, table[1], 9)
    assert np.array_equal(k[:3, :8], lat[2:5]) and np.array_equal(k[:3, 8:], key[2:5])
    assert (k[3, :8] == 0).all() and np.isnan(k[3, 8:]).all()
    assert np.array_equal(data[7, :3], before[7, :3])   # sequence 0's first three tokens were there
    assert np.array_equal(data[7, 3], np.concatenate([lat[0], key[0]]))
    assert np.array_equal(data[1, 0], np.concatenate([lat[1], key[1]]))


def test_pages_story():
    """Fork, grow, free, compact: counts add up to the entries, and what each
    sequence reads is what it would without any sharing."""
    r = np.random.default_rng(7)
    page, pool, rows, width = 4, 40, 6, 9
    refs, table = np.zeros(pool, int), np.full((rows, width), -1)
    data, kv = np.zeros((pool, page)), np.zeros(rows, int)
    text = [[] for _ in range(rows)]

    def check():
        count = np.zeros(pool, int)
        for b in range(rows):
            ps = table[b, :oracle.pages.held(kv[b], page)]
            np.add.at(count, ps, 1)
            assert [data[p, i % page] for i, p in enumerate(np.repeat(ps, page)[:kv[b]])] == text[b]
        assert np.array_equal(count, refs)

    def grow(by):
        new = kv + by
        assert oracle.pages.extend(refs, table, [data], page, kv, new)
        for b in range(rows):
            for t in range(kv[b], new[b]):
                assert refs[table[b, t // page]] == 1 or t % page == 0
                data[table[b, t // page], t % page] = r.standard_normal()
                text[b].append(data[table[b, t // page], t % page])
        kv[:] = new
        check()

    grow(np.array([6, 9, 0, 0, 0, 0]))
    assert oracle.pages.fork(refs, table, kv, page, [0, 0, 1], [2, 3, 4])
    text[2], text[3], text[4] = list(text[0]), list(text[0]), list(text[1])
    check()
    assert (refs[table[0, 1]], refs[table[1, 0]]) == (3, 2)
    assert not oracle.pages.fork(refs, table, kv, page, [0, 1, 1, 5], [5, 5, 4, 9])   # twice; not empty; out of range
    check()
    grow(np.array([1, 2, 3, 1, 0, 5]))
    last = int(table[4, 2])
    assert refs[last] == 1                              # its parent has gone on
    oracle.pages.free(refs, table, kv, page, [0, 3, 0])
    text[0], text[3] = [], []
    check()
    oracle.pages.compact(refs, table, [data], page, kv)
    check()
    n = int((refs > 0).sum())
    assert (refs[:n] > 0).all()
    before = refs.copy()
    assert not oracle.pages.extend(refs, table, [data], page, kv, kv + 4 * 7)
    assert np.array_equal(refs, before)
