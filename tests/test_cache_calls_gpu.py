"""Calls of the paged cache's entry points as programs make them beyond the
plain ones of test_cache_gpu.py: from several threads, with batches that are
partly senseless, with infinities among the queries."""

import threading

import numpy as np
import pytest
import torch

from cache_util import Batch
from exact_attention_fattn_gb300 import attention as A
from exact_attention_fattn_gb300 import cache as K

pytestmark = pytest.mark.gpu


def test_threads_with_batches_of_different_sizes():
    """Eight host threads, a stream each; the batches, and with them the
    shared memory that a call asks for, differ."""
    bs = [Batch(300 + i, [3 + i] * n, [new] * n, 1, 2, 64 if i & 1 else 128, 32)
          for i, (n, new) in enumerate([(1, 1), (900, 1), (40, 1), (1500, 1), (1, 40), (30, 50), (3, 60), (70, 45)])]
    dev = [b.device() for b in bs]
    qs = [b.rows(b.q) for b in bs]
    torch.cuda.synchronize()
    got, errors = [None] * len(bs), []
    gate = threading.Barrier(len(bs))

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait()
                for _ in range(20):
                    got[i] = K.fattn_cache_fwd(qs[i], *dev[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(bs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert A.fattn_check_status() == 0
    for i, b in enumerate(bs):
        want = K.fattn_cache_fwd(qs[i], *dev[i])
        assert torch.equal(got[i][0], want[0]) and torch.equal(got[i][1], want[1])
    assert A.fattn_check_status() == 0


@pytest.mark.parametrize("news", [1, 60])
def test_host_path_on_public_functions_alone(news, monkeypatch):
    b = Batch(310, [500, 90], [news, news], 2, 2, 128, 64)
    d, q = b.device(), b.rows(b.q)
    want = K.fattn_cache_fwd(q, *d)
    monkeypatch.setattr(K, "_current_device", torch.cuda.current_device)
    monkeypatch.setattr(K, "_raw_stream", K._public_stream)
    monkeypatch.setattr(K, "_raw_alloc", None)
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            got = K.fattn_cache_fwd(q, *d)
        s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert A.fattn_check_status() == 0
