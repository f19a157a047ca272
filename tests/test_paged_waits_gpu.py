"""Waits of the paged kernels that run out: the call returns, the status word
names the wait, and the next call is right.  ``selftest_wait_polls`` shortens
the waits; with 0 polls each gives up at once, with 1 some do and some do not."""
import time

import numpy as np
import pytest
import torch

import bit_mixed_precision_tri_b200 as tri
from bit_mixed_precision_tri_b200 import paged
from test_paged_runs_gpu import batch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture
def polls():
    """Sets the limit for one call, and the default again behind it."""
    tri.wait_status(DEV, clear=True)
    yield tri.selftest_wait_polls
    tri.selftest_wait_polls()
    tri.wait_status(DEV, clear=True)


@pytest.mark.parametrize("fp8,dh,H,Hkv,ps,M,longest", [
    (False, 64, 12, 4, 8, 200, 2500),
    (False, 64, 32, 2, 64, 300, 3000),
    (True, 64, 24, 3, 16, 300, 2500),
    (True, 64, 48, 4, 256, 200, 2500),
    (False, 128, 16, 2, 32, 300, 2000),
    (False, 128, 24, 2, 128, 200, 2000),
    (True, 128, 8, 4, 64, 200, 2500),
    (True, 128, 48, 3, 8, 200, 2500),
])
@pytest.mark.parametrize("limit", [0, 1])
def test_attention_whose_waits_run_out_returns(polls, limit, fp8, dh, H, Hkv, ps, M, longest):
    args, kw, (*_, table, pos, seq) = batch(H, Hkv, dh, ps, fp8, M, longest, H + ps)
    want = paged.attention_decode(*args, **kw)
    assert tri.wait_status(DEV) == 0
    out = torch.full_like(want, float("nan"))
    polls(limit)
    t0 = time.perf_counter()
    paged.attention_decode(*args, out=out, **kw)
    code = tri.wait_status(DEV, clear=True)
    assert time.perf_counter() - t0 < 60.0
    polls(-1)
    assert code in ((51, 52) if limit == 0 else (0, 51, 52, 53))
    empty = (pos < 0) | (seq < 0) | (seq >= len(table))
    assert empty.any() and torch.all(out[torch.from_numpy(empty).to(DEV)] == 0)
    assert torch.equal(paged.attention_decode(*args, out=out, **kw), want)
    assert tri.wait_status(DEV) == 0


def test_attention_of_one_tile_rows_whose_waits_run_out_stores_nothing(polls):
    """Tables of one tile: no row is split, nothing joins what is not there."""
    rng = np.random.default_rng(3)
    for M in (3, 700):
        k, v = (torch.from_numpy(rng.standard_normal((M, 2, 32, 64)).astype(np.float16)).to(DEV) for _ in range(2))
        table, pos = torch.arange(M, dtype=torch.int32, device=DEV)[:, None], torch.full((M,), 30, dtype=torch.int32, device=DEV)
        q = torch.from_numpy(rng.standard_normal((M, 4, 64)).astype(np.float16)).to(DEV)
        out = torch.full((M, 256), 3.0, dtype=torch.float16, device=DEV)
        polls(0)
        paged.attention_decode(q, k, v, table, pos, out=out)
        assert tri.wait_status(DEV, clear=True) in (51, 52)
        assert torch.all(out == 3.0)
        polls(-1)
        assert not torch.any(paged.attention_decode(q, k, v, table, pos, out=out) == 3.0) and tri.wait_status(DEV) == 0
