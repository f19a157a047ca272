"""Attention over pages where a worker's run of tiles is longer than its ring of
stages: slots that are filled again, the waits' parities, a row's last tile in
the middle of a run, one-tile rows between long ones.

Tolerances: ``attention_rows_f64``."""
import numpy as np
import pytest
import torch

from bit_mixed_precision_tri_b200 import paged
from oracle import decode_oracle as D
from oracle import paged_oracle as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
STAGES, CTAS_PER_SM = 5, 3           # at most, of any form of the kernel


def _t(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def tiles(pos, seq, S, width, ps, Hkv, dh, fp8):
    """Tiles of a call: 64 positions where a position takes 256 bytes, else 128."""
    n = np.where((seq >= 0) & (seq < S) & (pos >= 0), np.minimum(pos + 1, width * ps), 0)
    t = 64 if dh * (1 if fp8 else 2) > 128 else 128
    return int((-(-n // t)).sum()) * Hkv


def batch(H, Hkv, dh, ps, fp8, M, longest, seed):
    """Ragged rows of 40 sequences with holes and dropped fronts; NaN behind each
    sequence's end and in every page that no table names."""
    rng = np.random.default_rng(seed)
    S, width = 40, -(-longest // ps)
    length = rng.integers(1, longest + 1, S)
    length[:12] = rng.integers(1, 65, 12)
    length[12] = longest
    need = -(-length // ps)
    pages = int(need.sum()) + 4
    perm = rng.permutation(pages)
    table = np.full((S, width), -1, np.int32)
    at = 0
    for s in range(S):
        table[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
    pools, vals = [], []
    for _ in range(2):
        x = torch.from_numpy(rng.standard_normal((pages, Hkv, ps, dh)).astype(np.float32))
        t = (x * 16).to(E4M3) if fp8 else x.half()
        vals.append(t.float().numpy())
        raw, nan = (t.view(torch.uint8), 0x7F) if fp8 else (t.view(torch.int16), 0x7E00)
        raw[torch.from_numpy(perm[at:].copy())] = nan
        for s in range(S):
            if length[s] % ps:
                raw[int(table[s, need[s] - 1]), :, int(length[s] % ps):] = nan
        pools.append(t.to(DEV))
    table[13, need[13] // 3] = -1
    table[14, :need[14] // 2] = -1
    table[15, :] = -1
    seq = rng.integers(0, S, M).astype(np.int32)
    pos = (length[seq] - 1).astype(np.int32)
    some = rng.random(M) < 0.5
    pos[some] = (rng.random(int(some.sum())) * length[seq[some]]).astype(np.int32)
    pos[rng.random(M) < 0.04], seq[rng.random(M) < 0.02], seq[rng.random(M) < 0.02] = -1, S, -1
    q = D.rn16(rng.standard_normal((M, H, dh)) * rng.choice([0.3, 1.0, 4.0], (M, H, 1)))
    scales = [rng.uniform(0.04, 0.09, Hkv).astype(np.float32) if fp8 else None for _ in range(2)]
    if fp8:
        vals = [v * s[:, None, None] for v, s in zip(vals, scales)]
    kw = dict(seq=_t(seq, torch.int32))
    if fp8:
        kw.update(k_scale=_t(scales[0], torch.float32), v_scale=_t(scales[1], torch.float32))
    args = (_t(q, torch.float16), *pools, _t(table, torch.int32), _t(pos, torch.int32))
    return args, kw, (q, *vals, table, pos, seq)


@pytest.mark.parametrize("fp8,dh,H,Hkv,ps,M,longest", [
    (False, 64, 12, 4, 8, 300, 2500),
    (False, 64, 32, 2, 64, 500, 3000),
    (True, 64, 24, 3, 16, 500, 2500),
    (True, 64, 48, 4, 256, 320, 2500),
    (False, 128, 16, 2, 32, 450, 2000),
    (False, 128, 24, 2, 128, 350, 2000),
    (True, 128, 8, 4, 64, 300, 2500),
    (True, 128, 48, 3, 8, 400, 2500),
])
def test_runs_longer_than_the_ring(fp8, dh, H, Hkv, ps, M, longest):
    args, kw, (q, k, v, table, pos, seq) = batch(H, Hkv, dh, ps, fp8, M, longest, H + ps)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert tiles(pos, seq, len(table), table.shape[1], ps, Hkv, dh, fp8) > 2 * STAGES * CTAS_PER_SM * sms
    out = torch.full((M, H * dh), float("nan"), dtype=torch.float16, device=DEV)
    paged.attention_decode(*args, out=out, **kw)
    ref, tol = P.attention_rows_f64(q, k, v, table, pos, seq, dh ** -0.5)
    got = out.float().cpu().numpy().astype(np.float64).reshape(M, H, dh)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / tol))
    assert torch.equal(paged.attention_decode(*args, **kw), out)


def test_as_many_rows_as_a_long_list():
    """300000 rows of one sequence, a position more each row up to a page's end, then padding among them."""
    M, dh, ps = 300000, 64, 256
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(1, 1, ps, dh, generator=g).half().to(DEV) for _ in range(2))
    q = torch.randn(1, 1, dh, generator=g).half().to(DEV).expand(M, -1, -1).contiguous()
    pos = (torch.arange(M, device=DEV) % 257 - 1).int()
    table, seq = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.zeros(M, dtype=torch.int32, device=DEV)
    out = paged.attention_decode(q, k, v, table, pos, seq=seq)
    few = paged.attention_decode(q[:257], k, v, table, pos[:257], seq=seq[:257])
    ref, tol = P.attention_rows_f64(q[:257].double().cpu().numpy(), k.double().cpu().numpy(), v.double().cpu().numpy(),
                                    np.zeros((1, 1), np.int32), pos[:257].cpu().numpy(), np.zeros(257, np.int32), dh ** -0.5)
    # every row within the bound; equal rows need not be equal bit for bit, since one that two runs share is summed in two parts
    for got in (few, *out.split(257)):
        n = len(got)
        assert np.all(np.abs(got.double().cpu().numpy().reshape(n, 1, dh) - ref[:n]) <= tol[:n])


@pytest.mark.parametrize("Hkv", [1, 3])
def test_the_farthest_position_there_is(Hkv):
    """A row at position 2^30 - 1: of its 2^27 pages the first, one in the middle and the last are present."""
    dh, ps, n = 64, 8, 1 << 30
    table = torch.full((1, n // ps), -1, dtype=torch.int32, device=DEV)
    at = [0, (n // ps) // 2 + 5, n // ps - 1]
    table[0, at] = torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(3, Hkv, ps, dh, generator=g).half().to(DEV) for _ in range(2))
    q = torch.randn(1, 2 * Hkv, dh, generator=g).half().to(DEV)
    far = paged.attention_decode(q, k, v, table, torch.tensor([n - 1], dtype=torch.int32, device=DEV))
    near = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    ref, tol = P.attention_rows_f64(q.double().cpu().numpy(), k.double().cpu().numpy(), v.double().cpu().numpy(),
                                    near.cpu().numpy(), np.array([23]), np.array([0]), dh ** -0.5)
    assert np.all(np.abs(far.double().cpu().numpy().reshape(ref.shape) - ref) <= tol)
    clamped = paged.attention_decode(q, k, v, table, torch.tensor([2 ** 31 - 1], dtype=torch.int32, device=DEV))
    assert torch.equal(clamped, far)
