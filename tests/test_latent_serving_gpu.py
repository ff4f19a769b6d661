"""The latent cache, its pages and rotations together, as a server uses them, and
calls beyond the plain ones: captured, from several threads and streams, with a
wait budget that runs out."""

import threading

import numpy as np
import pytest
import torch

import exact_attention_fattn_gb300 as F
from exact_attention_fattn_gb300 import _lib, cache as K, latent as Lt
from latent_util import LatentBatch, check_latent

pytestmark = pytest.mark.gpu


def ok():
    assert F.fattn_check_status() == 0


@pytest.mark.parametrize("kind,page", [("latent", 32), ("latent", 64), ("latent", 128), ("fp8", 64)])
def test_serving(kind, page):
    """Two prompts are read, each is answered three times with shared pages, samples end
    and others go on, the pool is compacted in between: what every row gets is what the
    same tokens give in a cache of their own that shares nothing (bit for bit, as the
    rows of a call do not depend on their pages)."""
    torch.manual_seed(page)
    rows, heads, kvh, rank, d, maxp = 8, 4, 2, 256, 64, 12
    if kind == "latent":
        shared, alone = (F.fattn_latent_alloc(80, rank, page) for _ in range(2))
    else:
        shared, alone = (F.fattn_cache_alloc(80, kvh, d, page) for _ in range(2))
    pool = F.fattn_pages_alloc(shared)
    table = torch.full((rows, maxp), -1, dtype=torch.int32, device="cuda")
    own = torch.arange(rows * 10, dtype=torch.int32, device="cuda").view(rows, 10)
    kv = torch.zeros(rows, dtype=torch.int32, device="cuda")
    rope = F.fattn_rope_table(page * maxp, 64, factor=4.0, original=256)

    def call(c, tab, qs, lens, x):
        if kind == "latent":
            q = x["q"].clone()
            F.fattn_latent_append(x["lat"], x["key"], c, tab, qs, lens, rope=rope, q_rope=x["qr"], q=q)
            return F.fattn_latent_fwd(q, c, tab, qs, lens, scale=0.1)
        q = F.fattn_cache_append(x["k"], x["v"], c, tab, qs, lens, rope=rope, q=x["q8"])
        return F.fattn_cache_fwd(q, c, tab, qs, lens)

    def step(grow):
        """grow: new tokens of each sequence."""
        new = kv + torch.tensor(grow, dtype=torch.int32, device="cuda")
        F.fattn_pages_extend(pool, shared, table, kv, new)
        kv.copy_(new)
        T = sum(grow)
        qs = torch.tensor(np.concatenate([[0], np.cumsum(grow)]), dtype=torch.int32, device="cuda")
        rnd = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)
        x = dict(lat=rnd(T, rank), key=rnd(T, 64), q=rnd(T, heads, rank + 64), qr=rnd(T, heads, 64), k=rnd(T, kvh, d),
                 v=rnd(T, kvh, d), q8=rnd(T, heads, d))
        got, want = call(shared, table, qs, kv, x), call(alone, own, qs, kv, x)
        ok()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

    def fork(parent, child):
        i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        F.fattn_pages_fork(pool, shared, table, kv, i(parent), i(child))
        for p, c in zip(parent, child):
            n = -(-int(kv[p]) // page)
            for x in alone if kind == "fp8" else [alone.data]:
                if x is not None:
                    x[own[c, :n].long()] = x[own[p, :n].long()]
        ok()

    step([page * 2 + 7, 0, 0, 40, 0, 0, 0, 0])
    fork([0, 0, 3, 3], [1, 2, 4, 5])
    step([1, 1, 1, 1, 1, 1, 0, 0])
    step([1, 1, 1, 1, 1, 1, 0, 0])
    F.fattn_pages_free(pool, shared, table, kv, torch.tensor([0, 5], dtype=torch.int32, device="cuda"))
    step([0, 3, 1, page, 1, 0, 30, 0])
    F.fattn_pages_compact(pool, shared, table, kv)
    step([0, 1, 1, 1, 1, 0, 1, 0])
    fork([6], [7])
    step([5, 1, 1, 1, 1, 0, 1, 1])
    held = sum(-(-int(n) // page) for n in kv)
    assert int(pool.refs.sum()) == held and int((pool.refs > 0).sum()) <= held


@pytest.mark.parametrize("news,heads", [(1, 16), (1, 128), (40, 20)])
def test_captured_step_on_other_lengths(news, heads):
    """A captured append and attention, replayed on other lengths, rows and pages."""
    *_, big = LatentBatch(60, [900, 500, 300], [news] * 3, heads, 512, 64).tables()
    c, table, qs, kl = big.device()
    lat, key, qr = big.rows(big.latent), big.rows(big.k_rope), big.rows(big.q_rope)
    q = big.rows(big.q)
    t = F.fattn_rope_table(1000, 64)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        F.fattn_latent_append(lat, key, c, table, qs, kl, rope=t, q_rope=qr, q=q)
        got = F.fattn_latent_fwd(q, c, table, qs, kl, scale=0.07)
    for lens in ([900, 500, 300], [65, 499, 64], [news, news, news], [899, 0, 128]):
        n = [min(news, x) for x in lens]
        kl.copy_(torch.tensor(lens, dtype=torch.int32))
        qs.copy_(torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32))
        table.copy_(table.roll(1, 0)) if lens[0] == 65 else None
        c.data.copy_(torch.nan_to_num(c.data, nan=1.0))
        g.replay()
        want = F.fattn_latent_fwd(q, c, table, qs, kl, scale=0.07)
        ok()
        rows = sum(n)
        assert torch.equal(got[0][:rows], want[0][:rows]) and torch.equal(got[1][:rows], want[1][:rows])
        if lens[0] == 65:
            table.copy_(table.roll(-1, 0))


@pytest.mark.parametrize("heads", [64, 128])
def test_two_graphs_with_one_workspace(heads):
    *_, b = LatentBatch(61, [3000, 77], [1, 1], heads, 512, 64).tables()
    b2 = LatentBatch(62, [10, 5000, 600], [1, 2, 1], 16, 512, 64)
    ws = torch.zeros(max(F.fattn_latent_fwd_workspace_bytes(x.T, len(x.lens), x.heads, 512) for x in (b, b2)),
                     dtype=torch.uint8, device="cuda")
    graphs = []
    for x in (b, b2):
        dev, q = x.device(), x.rows(x.q)
        want = F.fattn_latent_fwd(q, *dev, scale=0.07)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = F.fattn_latent_fwd(q, *dev, scale=0.07, workspace=ws)
        graphs.append((g, got, want, dev, q))
    for _ in range(3):
        for g, got, want, *_ in graphs:
            g.replay()
            ok()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_threads_and_streams():
    """Eight host threads, a stream each, batches of different layouts at once."""
    bs = [[*LatentBatch(70 + i, [200 + 90 * i] * n, [new] * n, h, 256 if i & 1 else 512, 32).tables()][-1]
          for i, (n, new, h) in enumerate([(1, 1, 16), (90, 1, 3), (4, 1, 128), (7, 2, 40), (1, 90, 20), (3, 5, 64), (30, 1, 33), (2, 1, 1)])]
    dev, qs = [b.device() for b in bs], [b.rows(b.q) for b in bs]
    want = [F.fattn_latent_fwd(q, *d, scale=0.07) for q, d in zip(qs, dev)]
    torch.cuda.synchronize()
    got, errors = [None] * len(bs), []
    gate = threading.Barrier(len(bs))

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait()
                for _ in range(15):
                    got[i] = F.fattn_latent_fwd(qs[i], *dev[i], scale=0.07)
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(bs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    ok()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("news,heads", [(1, 16), (1, 40), (1, 128), (60, 20)])
def test_a_wait_budget_that_runs_out(news, heads, page):
    """Waits that give up are reported, and the next call, on the same memory and on
    tensor memory that the last one handed back, is right."""
    *_, b = LatentBatch(80, [3000, 700], [news, news], heads, 512, page).tables()
    dev, q = b.device(), b.rows(b.q)
    want = F.fattn_latent_fwd(q, *dev, scale=0.07)
    ok()
    try:
        for cycles in (1, 400, 1500, 4000):       # gives up at other places
            F.fattn_set_wait_budget(cycles)
            for _ in range(3):
                F.fattn_latent_fwd(q, *dev, scale=0.07)
                assert F.fattn_check_status() in (_lib.FATTN_OK, _lib.FATTN_ERR_TIMEOUT)
    finally:
        F.fattn_set_wait_budget(0)
    for _ in range(3):
        got = F.fattn_latent_fwd(q, *dev, scale=0.07)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ok()


@pytest.mark.parametrize("news", [1, 60])
def test_host_path_on_public_functions_alone(news, monkeypatch):
    b = LatentBatch(81, [500, 90], [news, news], 16, 256, 64)
    d, q = b.device(), b.rows(b.q)
    want = F.fattn_latent_fwd(q, *d, scale=0.07)
    for m in (K, Lt):
        monkeypatch.setattr(m, "_current_device", torch.cuda.current_device)
        monkeypatch.setattr(m, "_raw_stream", K._public_stream)
        monkeypatch.setattr(m, "_raw_alloc", None)
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            got = F.fattn_latent_fwd(q, *d, scale=0.07)
        s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ok()


def test_a_prompt_against_one_dense_softmax():
    """A whole prompt in one call, rotated parts zero, against a softmax over the dense
    matrix of scores in 64 bits."""
    torch.manual_seed(5)
    n, heads, rank = 130, 3, 256
    lat = torch.randn(n, rank, device="cuda").to(torch.bfloat16)
    c = F.fattn_latent_alloc(8, rank, 64)
    table = torch.tensor([[3, 0, 5]], dtype=torch.int32, device="cuda")
    qs, kl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [n]))
    zero = torch.zeros(n, 64, dtype=torch.bfloat16, device="cuda")
    F.fattn_latent_append(lat, zero, c, table, qs, kl)
    q = torch.randn(n, heads, rank + 64, device="cuda").to(torch.bfloat16)
    o, l = F.fattn_latent_fwd(q, c, table, qs, kl, scale=rank ** -0.5)
    ok()
    x = torch.einsum("thc,kc->thk", q[..., :rank].double(), lat.double()) * rank ** -0.5
    x = x.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool()[:, None], -torch.inf)
    p = torch.softmax(x, 2)
    want = (torch.einsum("thk,kc->thc", p, lat.double()), torch.logsumexp(x, 2),
            torch.einsum("thk,kc->thc", p, lat.double().abs()),
            torch.einsum("thc,kc->thk", q[..., :rank].double().abs(), lat.double().abs()).amax(2) * rank ** -0.5)
    check_latent(o.double().cpu().numpy(), l.double().cpu().numpy(), [w.cpu().numpy() for w in want], rank + 64)


def test_refusals_of_the_binding():
    b = LatentBatch(82, [70, 5], [1, 1], 3, 256, 32)
    c, table, qs, kl = b.device()
    q, lat, key, qr = b.rows(b.q), b.rows(b.latent), b.rows(b.k_rope), b.rows(b.q_rope)
    base = dict(q=q, c=c, table=table, qs=qs, kl=kl, kw=dict(scale=0.1))
    for bad in (dict(q=q.float()), dict(q=q[:, :, :300]), dict(q=q.transpose(0, 1)), dict(q=q.cpu()),
                dict(c=F.LatentCache(c.data, 512)), dict(c=F.LatentCache(c.data.float(), 256)), dict(table=table.long()),
                dict(qs=qs[:2]), dict(kl=kl[:1]), dict(kw=dict(scale=0.1, out=q)), dict(kw=dict(scale=0.1, lse=q)),
                dict(kw=dict(scale=0.1, workspace=q))):
        a = {**base, **bad}
        with pytest.raises((TypeError, ValueError)):
            F.fattn_latent_fwd(a["q"], a["c"], a["table"], a["qs"], a["kl"], **a["kw"])
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(scale=0.1, workspace=torch.empty(512, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(_lib.FattnError):
            F.fattn_latent_fwd(q, c, table, qs, kl, **kw)
    rope = F.fattn_rope_table(80, 64)
    for bad in (dict(latent=lat[:, :200]), dict(latent=lat.float()), dict(k_rope=key[:1]), dict(k_rope=key[:, ::2]),
                dict(q_rope=None), dict(q=None), dict(q=q[:, :2]), dict(q_rope=qr[:1]), dict(rope=F.fattn_rope_table(80, 32)),
                dict(rope=rope.double())):
        a = dict(latent=lat, k_rope=key, rope=rope, q_rope=qr, q=q)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            F.fattn_latent_append(a.pop("latent"), a.pop("k_rope"), c, table, qs, kl, **a)
    ok()
