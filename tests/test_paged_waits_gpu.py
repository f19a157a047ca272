"""Waits of the paged kernels that run out: the call returns, the status word
names the wait, and the next call is right.  ``selftest_wait_polls`` shortens
the waits; with 0 nothing is loaded and each runs out, with 1 some do and some do not."""
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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("limit", [0, 1])
def test_append_whose_waits_run_out_returns(polls, limit, fp8):
    """3000 rows of 6 heads take the kernel that streams them; with no poll at all it stores nothing."""
    T, H, Hkv, dh, ps = 3000, 4, 1, 128, 64
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(T, (H + 2 * Hkv) * dh, generator=g).half().to(DEV)
    pages = -(-T // ps)
    table, pos = torch.arange(pages, dtype=torch.int32, device=DEV)[None], torch.arange(T, dtype=torch.int32, device=DEV)
    seq, cs = torch.zeros_like(pos), paged.rope_table(pages * ps, DEV)
    one = torch.full((Hkv,), 0.05, device=DEV)
    kw = dict(k_scale=one, v_scale=one) if fp8 else {}

    def call():
        k, v = (torch.full((pages, Hkv, ps, dh), 3.0, device=DEV).to(torch.float8_e4m3fn if fp8 else torch.float16)
                for _ in range(2))
        q = torch.full((T, H, dh), 3.0, dtype=torch.float16, device=DEV)
        paged.qknorm_rope_append(qkv, pos, None, None, cs, k, v, table, H, seq=seq, out=q, **kw)
        code = tri.wait_status(DEV, clear=True)
        return code, q, k.view(torch.uint8), v.view(torch.uint8)

    code, *want = call()
    assert code == 0
    polls(limit)
    code, *got = call()
    polls(-1)
    assert code in ((61, 62) if limit == 0 else (0, 61, 62, 63))
    if limit == 0:
        assert torch.all(got[0] == 3.0) and len(set(got[1].flatten().tolist())) <= 2 and torch.equal(got[1], got[2])
    code, *again = call()
    assert code == 0 and all(torch.equal(a, b) for a, b in zip(again, want))


def test_check_option(polls):
    """check=True returns as without it, and raises WaitGaveUp with the wait's code."""
    args, kw, _ = batch(8, 4, 128, 64, False, 40, 900, 1)
    want = paged.attention_decode(*args, **kw)
    assert torch.equal(paged.attention_decode(*args, check=True, **kw), want)
    polls(0)
    with pytest.raises(tri.WaitGaveUp) as e:
        paged.attention_decode(*args, check=True, **kw)
    assert e.value.code in (51, 52)
    T = 3000
    k = torch.zeros(T // 8, 1, 8, 64, dtype=torch.float16, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    rows = (torch.zeros(T, 192, dtype=torch.float16, device=DEV), pos, None, None, paged.rope_table(T, DEV, rot=16), k,
            k.clone(), torch.arange(T // 8, dtype=torch.int32, device=DEV)[None], 1, torch.zeros_like(pos))
    with pytest.raises(tri.WaitGaveUp) as e:
        paged.qknorm_rope_append(*rows, check=True)
    assert e.value.code in (61, 62)
    polls(-1)
    paged.qknorm_rope_append(*rows, check=True)
    assert torch.equal(paged.attention_decode(*args, check=True, **kw), want)


def test_first_calls_of_a_process_may_be_captured():
    """Nothing is looked up or set on first use that a capture forbids."""
    import os
    import subprocess
    import sys
    code = """
import torch
from bit_mixed_precision_tri_b200 import paged
dev = "cuda:0"
T = 2500
qkv = torch.randn(T, 6 * 64, device=dev).half()
k = torch.zeros(T // 8 + 1, 1, 8, 64, dtype=torch.float16, device=dev)
v = torch.zeros_like(k)
pos = torch.arange(T, dtype=torch.int32, device=dev)
seq = torch.zeros_like(pos)
table = torch.arange(T // 8 + 1, dtype=torch.int32, device=dev)[None]
pools = torch.zeros(4, 1, 8, 64, dtype=torch.float16, device=dev)
ids = torch.tensor([[0], [1]], dtype=torch.int32, device=dev)
pools[0] = 5.0
torch.cuda.synchronize()
def calls():
    cs = paged.rope_table(T, dev, rot=32)
    q = paged.qknorm_rope_append(qkv, pos, None, None, cs, k, v, table, 4, seq=seq)
    paged.qknorm_rope_append(qkv[:2], pos[:2], None, None, cs, k, v, table, 4, seq=seq[:2])
    paged.copy_pages(pools, ids[0], ids[1])
    return paged.attention_decode(q[-3:], k, v, table, pos[-3:], seq=seq[-3:])
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = calls()
g.replay()
torch.cuda.synchronize()
got = out.clone()
assert bool((pools[1] == 5.0).all()) and bool((got != 0).any())
assert torch.equal(calls(), got)
print("captured first")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]
