"""GPU parity of the paged key/value cache (rotary tables, append, attention,
page copies) against the float64 oracle (oracle/paged_oracle.py), and a run of
them together in the ternary block's decode step.

Tolerances: fp16 results round once from fp32, half a step 2^-11 of the value
(2^-25 for subnormals); e4m3 elements 2^-4 (2^-10).  Before that, RMSNorm and
the rotation are off by a few units of 2^-24 of the head's largest value (the
sum of 128 squares, one square root, one division, three products, the table's
float32 entries, off by 2^-25 each): 2^-20 of it in all.  Attention:
``attention_bound``."""
import numpy as np
import pytest
import torch

import bit_mixed_precision_tri_b200 as tri
from bit_mixed_precision_tri_b200 import decode as dec
from bit_mixed_precision_tri_b200 import paged
from oracle import decode_oracle as D
from oracle import paged_oracle as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
CODES = P.e4m3_values()


def _t(a, dtype=torch.float16):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _bits(t):
    return t.view(torch.uint8 if t.dtype == E4M3 else torch.int16).cpu().numpy()


def _pool(rng, pages, Hkv, ps, dh, fp8):
    """(device pool, its values before scaling)."""
    x = torch.from_numpy(rng.standard_normal((pages, Hkv, ps, dh)).astype(np.float32))
    t = (x * 16).to(E4M3) if fp8 else x.half()
    return t.to(DEV), t.float().numpy().astype(np.float64)


def _table(rng, lengths, ps, width, pages):
    """Shuffled distinct pages for each sequence, -1 behind them."""
    perm = list(rng.permutation(pages))
    table = np.full((len(lengths), width), -1, np.int32)
    for s, n in enumerate(lengths):
        for i in range(-(-n // ps)):
            table[s, i] = perm.pop()
    return table


# ---------------------------------------------------------------- rotary tables
@pytest.mark.parametrize("rot", [16, 48, 64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="bands", factor=8.0, context=4096.0, low=1.0, high=4.0),
                                dict(scaling="ramp", factor=16.0, context=2048.0, low=1.0, high=32.0),
                                dict(scaling="ramp", factor=1.0, context=16.0, low=1.0, high=1.5)])
def test_rope_table(rot, kw):
    for L in (1, 3001):
        cs = paged.rope_table(L, DEV, rot=rot, theta=1e4, **kw).cpu().numpy().astype(np.float64)
        ref = P.rope_table_f64(L, rot, theta=1e4, **kw)
        # float32 storage (half a step of values up to the gain < 2), angles exact to 2^-50 of up to 3001
        assert cs.shape == ref.shape and np.max(np.abs(cs - ref)) <= 2.0 ** -24


def test_rope_table_far_positions_and_default_is_the_blocks_table():
    L = 1 << 20
    cs = paged.rope_table(L, DEV, rot=16, theta=5e5)
    f, _ = P.rope_freqs(16)
    for p in (L - 1, 777777):
        a = p * f
        got = cs[p].cpu().numpy().astype(np.float64)
        assert np.max(np.abs(got - np.stack([np.cos(a), np.sin(a)], -1))) <= 2.0 ** -24
    assert torch.equal(paged.rope_table(500, DEV), dec.rope_table(500, DEV))


# ---------------------------------------------------------------- append
def _append_case(T, H, Hkv, dh, ps, rot, inter, norm, fp8, seed, S=None, wide=0):
    rng = np.random.default_rng(seed)
    S = S or T
    width = 7
    pages = S * width + 2
    table = rng.permutation(pages)[:S * width].reshape(S, width).astype(np.int32)
    # distinct places: row t takes position t // S (+ a random offset per sequence) of sequence t % S
    start = rng.integers(0, width * ps - -(-T // S) + 1, S)
    seq = np.arange(T) % S
    pos = start[seq] + np.arange(T) // S
    cols = (H + 2 * Hkv) * dh
    buf = torch.from_numpy((rng.standard_normal((T, cols + wide)) * 2).astype(np.float16)).to(DEV)
    qkv = buf[:, :cols]
    gains = [D.rn16(rng.uniform(0.5, 1.5, dh)) if norm else None for _ in range(2)]
    scales = [rng.uniform(0.01, 0.1, Hkv).astype(np.float32) if fp8 else None for _ in range(2)]
    return rng, table, seq.astype(np.int32), pos.astype(np.int32), qkv, gains, scales, pages


def _check_append(T, H, Hkv, dh, ps, rot, inter, norm, fp8, seed, S=None, wide=0, break_rows=()):
    rng, table, seq, pos, qkv, gains, scales, pages = _append_case(T, H, Hkv, dh, ps, rot, inter, norm, fp8, seed, S,
                                                                   wide)
    for what, t in break_rows:
        if what == "pad":
            pos[t] = -1
        elif what == "far":
            pos[t] = table.shape[1] * ps
        elif what == "seq":
            seq[t] = table.shape[0]
        elif what == "negseq":
            seq[t] = -3
        else:
            table[seq[t], pos[t] // ps] = {"hole": -1, "big": pages}[what]
    cs = paged.rope_table(table.shape[1] * ps, DEV, rot=rot)
    k, kv0 = _pool(rng, pages, Hkv, ps, dh, fp8)
    v, vv0 = _pool(rng, pages, Hkv, ps, dh, fp8)
    k_bits, v_bits = _bits(k).copy(), _bits(v).copy()
    q = torch.full((T, H, dh), 7.0, dtype=torch.float16, device=DEV)
    paged.qknorm_rope_append(qkv, _t(pos, torch.int32), None if gains[0] is None else _t(gains[0]),
                             None if gains[1] is None else _t(gains[1]), cs, k, v, _t(table, torch.int32), H,
                             seq=_t(seq, torch.int32), interleaved=inter,
                             k_scale=None if not fp8 else _t(scales[0], torch.float32),
                             v_scale=None if not fp8 else _t(scales[1], torch.float32), out=q)
    ref_q, writes = P.append_f64(_np(qkv), pos, seq, gains[0], gains[1], cs.cpu().numpy(), table,
                                 (pages, Hkv, ps, dh), H, inter, scales[0], scales[1])
    got = _np(q)
    for t in range(T):
        if ref_q[t] is None:
            assert np.all(got[t] == 7.0)                     # padding rows are left alone
            continue
        top = np.max(np.abs(ref_q[t]), -1, keepdims=True)
        assert np.all(np.abs(got[t] - ref_q[t]) <= 2.0 ** -11 * np.abs(ref_q[t]) + 2.0 ** -20 * top + 2.0 ** -25), t
    K, V = _np(k), _np(v)
    half, tiny = (2.0 ** -4, 2.0 ** -10) if fp8 else (2.0 ** -11, 2.0 ** -25)
    kb, vb = _bits(k), _bits(v)
    for pg, j, slot, kr, vr in writes:
        tol = half * np.abs(kr) + 2.0 ** -20 * np.max(np.abs(kr)) + tiny
        assert np.all(np.abs(K[pg, j, slot] - kr) <= tol)
        if fp8:
            assert np.all(np.abs(V[pg, j, slot] - vr) <= half * np.abs(vr) + 2.0 ** -20 * np.abs(vr) + tiny)
        else:
            assert np.array_equal(V[pg, j, slot], vr)
        kb[pg, j, slot], vb[pg, j, slot] = k_bits[pg, j, slot], v_bits[pg, j, slot]
    assert np.array_equal(kb, k_bits) and np.array_equal(vb, v_bits)   # nothing else was written
    return writes


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,H,Hkv,dh,ps,rot,inter,S", [
    (1, 1, 1, 64, 8, 16, False, 1),
    (1, 64, 8, 128, 16, 128, False, 1),
    (3, 8, 2, 128, 256, 128, True, 3),
    (5, 6, 3, 64, 32, 48, False, 2),
    (37, 5, 1, 64, 8, 64, True, 4),
    (130, 12, 12, 128, 16, 96, False, 7),
    (700, 4, 2, 64, 32, 32, True, 5),
    (1201, 1, 1, 64, 8, 16, False, 40),
    (2505, 1, 1, 64, 8, 16, False, 90),      # the many-row kernel: 32 rows an item, the last one ragged
    (2100, 3, 3, 128, 16, 80, True, 30),
    (2200, 4, 2, 64, 32, 32, True, 12),
    (301, 90, 10, 128, 64, 128, False, 3),   # a row longer than an item: two runs of heads
    (333, 60, 60, 64, 32, 64, True, 2),
])
def test_append(T, H, Hkv, dh, ps, rot, inter, S, norm, fp8):
    _check_append(T, H, Hkv, dh, ps, rot, inter, norm, fp8, T + H + rot, S)


@pytest.mark.parametrize("T", [6, 600, 2200])
def test_append_padding_rows_absent_pages_and_strided_rows(T):
    bad = [("pad", 0), ("far", 1), ("seq", 2), ("negseq", 3), ("hole", 4), ("big", T - 1)]
    w = _check_append(T, 4, 2, 128, 8, 64, False, True, False, 5, S=T, wide=24, break_rows=bad)
    assert len(w) == 2 * (T - 6)


def test_append_short_table_drops_rows_behind_it():
    """A row behind the rotary table's last position writes nothing."""
    k = torch.zeros(4, 1, 8, 64, dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    q = torch.full((2, 1, 64), 5.0, dtype=torch.float16, device=DEV)
    paged.qknorm_rope_append(torch.ones(2, 192, dtype=torch.float16, device=DEV), _t([9, 10], torch.int32), None, None,
                             paged.rope_table(10, DEV, rot=16), k, v, _t([[0, 1, 2, 3]] * 2, torch.int32), 1, out=q)
    assert torch.all(q[1] == 5.0) and not torch.any(q[0] == 5.0)
    assert int((v != 0).sum()) == 64 and torch.all(v[1, 0, 1] == 1.0)


def test_append_e4m3_clamps_rounds_to_even_and_keeps_nan():
    k = torch.zeros(1, 1, 8, 64, dtype=torch.uint8, device=DEV).view(E4M3)
    v = torch.zeros_like(k.view(torch.uint8)).view(E4M3)
    x = np.zeros(64)
    x[:10] = [1000, -1000, np.inf, -np.inf, np.nan, 17, 19, 0.0029296875, 448, 500]
    qkv = _t(np.concatenate([np.zeros(64), np.zeros(64), x])[None].astype(np.float16))
    one = torch.ones(1, device=DEV)
    paged.qknorm_rope_append(qkv, _t([0], torch.int32), None, None, paged.rope_table(8, DEV, rot=16), k, v,
                             _t([[0]], torch.int32), 1, k_scale=one, v_scale=one)
    got = _np(v)[0, 0, 0]
    assert list(got[:4]) == [448, -448, 448, -448] and np.isnan(got[4])
    assert list(got[5:10]) == [16, 20, 0.00390625, 448, 448]   # 17, 19: ties to even; 1.5 units of 2^-9 up
    assert np.all(got[10:] == 0)


def test_append_values_are_the_ieee_quotient_rounded():
    """Every fp16 value below 448 * scale, divided in float32 and rounded to the nearest code."""
    codes = torch.arange(0, 0x7C00, dtype=torch.int32).to(torch.int16).view(torch.float16)
    codes = codes[: len(codes) // 64 * 64]
    T = len(codes) // 64
    k = torch.zeros(-(-T // 8), 1, 8, 64, dtype=torch.uint8, device=DEV).view(E4M3)
    v = torch.zeros_like(k.view(torch.uint8)).view(E4M3)
    qkv = torch.zeros(T, 192, dtype=torch.float16)
    qkv[:, 128:] = codes.view(T, 64)
    scale = torch.tensor([0.37], device=DEV)
    table = torch.arange(-(-T // 8), dtype=torch.int32, device=DEV)[None]
    paged.qknorm_rope_append(qkv.to(DEV), torch.arange(T, dtype=torch.int32, device=DEV), None, None,
                             paged.rope_table(T, DEV, rot=16), k, v, table, 1,
                             seq=torch.zeros(T, dtype=torch.int32, device=DEV), k_scale=scale, v_scale=scale)
    want = (codes.float() / np.float32(0.37)).clamp(max=448).to(E4M3).float()
    assert torch.equal(v.float().cpu().view(-1)[: len(codes)], want)


# ---------------------------------------------------------------- attention
def _attention(M, H, Hkv, dh, ps, lengths, fp8, seed, width=None, table=None, seq=None, pos=None, scale=None):
    rng = np.random.default_rng(seed)
    S = len(lengths)
    width = width or max(1, max(-(-n // ps) for n in lengths))
    pages = sum(-(-n // ps) for n in lengths) + 3
    table = _table(rng, lengths, ps, width, pages) if table is None else table(rng, pages)
    k, kval = _pool(rng, pages, Hkv, ps, dh, fp8)
    v, vval = _pool(rng, pages, Hkv, ps, dh, fp8)
    scales = [rng.uniform(0.04, 0.09, Hkv).astype(np.float32) if fp8 else None for _ in range(2)]
    q = D.rn16(rng.standard_normal((M, H, dh)) * rng.choice([0.3, 1.0, 4.0], (M, H, 1)))
    seq = np.arange(M, dtype=np.int32) if seq is None else np.array(seq, np.int32)
    pos = np.array(lengths, np.int32)[:M] - 1 if pos is None else np.array(pos, np.int32)
    # what lies behind each sequence's end must not matter
    for s in range(S):
        if lengths[s] % ps and lengths[s] > 0:
            pg = int(table[s, lengths[s] // ps])
            if 0 <= pg < pages:
                for pool in (k, v):
                    raw, nan = (pool.view(torch.uint8), 0x7F) if fp8 else (pool.view(torch.int16), 0x7E00)
                    raw[pg, :, lengths[s] % ps:] = nan
    sc = dh ** -0.5 if scale is None else scale
    args = (_t(q), k, v, _t(table, torch.int32), _t(pos, torch.int32))
    kw = dict(seq=_t(seq, torch.int32), scale=scale,
              k_scale=None if not fp8 else _t(scales[0], torch.float32),
              v_scale=None if not fp8 else _t(scales[1], torch.float32))
    out = torch.full((M, H * dh), float("nan"), dtype=torch.float16, device=DEV)
    paged.attention_decode(*args, **kw, out=out)
    if fp8:
        kval, vval = kval * scales[0].astype(np.float64)[:, None, None], vval * scales[1].astype(np.float64)[:, None, None]
    ref = P.attention_f64(q, kval, vval, table, pos, seq, sc)
    tol = P.attention_bound(q, kval, vval, table, pos, seq, sc, ref)
    got = _np(out).reshape(M, H, dh)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) - tol))
    return args, kw, out, ref


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("M,H,Hkv,dh,ps,lengths", [
    (1, 1, 1, 64, 8, [1]),
    (1, 8, 1, 128, 16, [37]),
    (1, 64, 8, 128, 16, [700]),
    (4, 8, 8, 64, 8, [1, 8, 9, 333]),
    (3, 16, 1, 128, 128, [5, 64, 1000]),
    (5, 18, 2, 64, 32, [63, 64, 65, 128, 129]),
    (2, 33, 3, 128, 64, [2000, 70]),
    (3, 14, 2, 128, 256, [256, 257, 511]),
    (40, 4, 2, 64, 16, list(range(1, 41))),
    (7, 24, 2, 128, 8, [100, 1, 15, 16, 17, 200, 31]),
])
def test_attention(M, H, Hkv, dh, ps, lengths, fp8):
    _attention(M, H, Hkv, dh, ps, lengths, fp8, M + H + ps)


def test_attention_many_rows():
    """More rows than workers, every length from 0 to 299."""
    rng = np.random.default_rng(1)
    _attention(300, 2, 1, 64, 16, list(rng.permutation(300)), False, 2, width=19)


def test_attention_long():
    _attention(1, 8, 1, 128, 64, [30011], False, 3)
    _attention(2, 2, 2, 64, 256, [20000, 19], True, 4)


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_rows_with_nothing_left(fp8):
    """Padding rows, sequences outside the table, rows whose pages are all absent."""
    def table(rng, pages):
        t = _table(rng, [40, 40, 40], 8, 6, pages)
        t[1, :] = -1
        t[2, 0], t[2, 2], t[2, 4] = pages, -7, 2 ** 31 - 1
        return t
    *_, out, ref = _attention(7, 4, 2, 64, 8, [40, 40, 40], fp8, 5, width=6, table=table,
                              seq=[0, 0, 1, 2, 3, -1, 2], pos=[39, -1, 39, 39, 39, 39, 7])
    zero = [1, 2, 4, 5, 6]                                   # row 6 sees only its absent first page
    assert torch.all(out[zero] == 0) and np.all(ref[zero] == 0)
    assert torch.all(torch.any(out[[0, 3]] != 0, 1))


def test_attention_clamps_to_the_table_and_takes_rows_of_one_sequence():
    """Several rows of one sequence (a draft), one of them behind the table's last page."""
    _attention(5, 8, 2, 128, 16, [112, 48], False, 6, width=7, seq=[0, 0, 0, 1, 0], pos=[97, 98, 99, 47, 10 ** 9])


def test_attention_scale_and_large_scores():
    _attention(2, 4, 1, 64, 32, [90, 91], False, 7, scale=2.5)
    # equal keys give the mean of the values, scores of hundreds do not overflow
    k = torch.full((1, 1, 64, 64), 12.0, dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    v[0, 0, :50, 3] = torch.arange(50, device=DEV).half()
    q = torch.full((1, 1, 64), 60.0, dtype=torch.float16, device=DEV)
    o = paged.attention_decode(q, k, v, _t([[0]], torch.int32), _t([49], torch.int32))
    assert abs(float(o[0, 3]) - 24.5) <= 2.0 ** -11 * 24.5 and float(o[0, 4]) == 0.0


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_many_tiny_weights_are_not_lost(fp8):
    """One position outweighs 30000 others by e^17.5 each (2^-25.2 of its weight):
    together they are a thousandth of the output."""
    n, dh = 30001, 64
    k = np.zeros((n, dh), np.float32)
    v = np.zeros((n, dh), np.float32)
    k[777, 0], v[:, 1], v[777, 1] = 17.5, 1.0, 0.0
    pages = -(-n // 256)
    pool = lambda a: torch.from_numpy(np.pad(a, ((0, pages * 256 - n), (0, 0))).reshape(pages, 1, 256, dh))
    q = np.zeros((1, 1, dh))
    q[0, 0, 0] = 1.0
    if fp8:
        k[777, 0] = 8.75
        one, two = torch.ones(1, device=DEV), torch.full((1,), 2.0, device=DEV)
        K, V, kw = pool(k).to(E4M3), pool(v).to(E4M3), dict(k_scale=two, v_scale=one)
    else:
        K, V, kw = pool(k).half(), pool(v).half(), {}
    kr, vr = K.float().numpy().astype(np.float64) * (2 if fp8 else 1), V.float().numpy().astype(np.float64)
    table, pos = np.arange(pages, dtype=np.int32)[None], np.array([n - 1])
    o = paged.attention_decode(_t(q), K.to(DEV), V.to(DEV), _t(table, torch.int32), _t(pos, torch.int32), scale=1.0, **kw)
    ref = P.attention_f64(q, kr, vr, table, pos, [0], 1.0)[0, 0, 1]
    # score 17.5 or 18 (8.75 becomes 9 in e4m3): off by one unit of 2^-23 of it and the exponential's 2^-22 each,
    # sums of equal terms by 2^-23 a step, the output by half an fp16 step (it is above the subnormals)
    assert 2e-4 < ref < 2e-3
    assert abs(float(o[0, 1]) - ref) <= ref * (18 * 2.0 ** -22 + 2.0 ** -21 + n / 8 * 2.0 ** -23 + 2.0 ** -11)


def test_attention_without_seq_pads_rows_behind_the_table():
    args, kw, out, _ = _attention(3, 4, 2, 64, 8, [20, 9, 33], False, 14)
    q, k, v, table, pos = args
    more = torch.cat([q, q])
    o = paged.attention_decode(more, k, v, table, torch.cat([pos, pos]))
    assert torch.equal(o[:3], out) and torch.all(o[3:] == 0)
    kk, vv = k.clone(), v.clone()
    qkv = torch.randn(6, 8 * 64, device=DEV).half()
    res = torch.full((6, 4, 64), 3.0, dtype=torch.float16, device=DEV)
    cs = paged.rope_table(40, DEV, rot=32)
    paged.qknorm_rope_append(qkv, torch.cat([pos, pos]), None, None, cs, kk, vv, table, 4, out=res)
    assert torch.all(res[3:] == 3.0)
    k2, v2 = k.clone(), v.clone()
    paged.qknorm_rope_append(qkv[:3], pos, None, None, cs, k2, v2, table, 4)
    assert torch.equal(_nan0(kk), _nan0(k2)) and torch.equal(_nan0(vv), _nan0(v2))


def _nan0(t):
    return t.view(torch.int16)


def test_attention_infinities_and_nan_where_they_count():
    """A NaN or infinite value that a row does see reaches its output; other rows and heads stay clean."""
    k = torch.randn(4, 2, 8, 64, device=DEV).half()
    v = torch.randn(4, 2, 8, 64, device=DEV).half()
    q = torch.randn(2, 4, 64, device=DEV).half()
    table, pos = _t([[0, 1], [2, 3]], torch.int32), _t([15, 15], torch.int32)
    base = paged.attention_decode(q, k, v, table, pos)
    k[1, 1, 3, 5], v[2, 0, 0, 7] = float("nan"), float("inf")
    o = paged.attention_decode(q, k, v, table, pos)
    a, b = o.view(2, 4, 64), base.view(2, 4, 64)
    assert torch.all(torch.isnan(a[0, 2:])) and torch.equal(a[0, :2], b[0, :2])
    assert torch.all(torch.isinf(a[1, :2, 7])) and torch.equal(a[1, 2:], b[1, 2:])
    keep = [c for c in range(64) if c != 7]
    assert torch.equal(a[1, :2][:, keep], b[1, :2][:, keep])


def test_attention_agrees_with_the_contiguous_caches():
    rng = np.random.default_rng(8)
    M, H, Hkv, Lmax = 3, 16, 2, 320
    q = _t(D.rn16(rng.standard_normal((M, H, 128))))
    kc, vc = (_t(D.rn16(rng.standard_normal((M, Hkv, Lmax, 128)))) for _ in range(2))
    pos = _t([319, 5, 200], torch.int32)
    a = dec.attention_decode(q, kc, vc, pos, Lmax)
    perm = torch.from_numpy(rng.permutation(M * 5)).to(DEV)
    table = torch.empty(M * 5, dtype=torch.int32, device=DEV)
    table.copy_(perm)
    pool = torch.empty(2, M * 5, Hkv, 64, 128, dtype=torch.float16, device=DEV)
    for i, c in enumerate((kc, vc)):
        pool[i, perm] = c.view(M, Hkv, 5, 64, 128).transpose(1, 2).reshape(M * 5, Hkv, 64, 128)
    b = paged.attention_decode(q, pool[0], pool[1], table.view(M, 5), pos)
    # each rounds once from fp32: half a step each, and their own errors far below
    assert torch.all((a - b).abs().float() <= 2.0 ** -10 * b.abs().float() + 2.0 ** -14)


def test_attention_strided_pools_rows_and_table():
    """K and V interleaved in one pool, q a slice of a wider buffer, a table with wider rows."""
    rng = np.random.default_rng(9)
    args, kw, out, _ = _attention(4, 6, 3, 64, 16, [50, 3, 17, 90], False, 10)
    q, k, v, table, pos = args
    both = torch.stack([k, v], 1)                            # [pages][2][Hkv][ps][dh]
    wide = torch.zeros(4, 6 * 64 + 40, dtype=torch.float16, device=DEV)
    wide[:, :384] = q.view(4, 384)
    t2 = torch.full((4, 11), -1, dtype=torch.int32, device=DEV)
    t2[:, : table.shape[1]] = table
    res = torch.zeros(4, 400, dtype=torch.float16, device=DEV)
    paged.attention_decode(wide[:, :384].unflatten(1, (6, 64)), both[:, 0], both[:, 1], t2[:, : table.shape[1]], pos,
                           out=res[:, :384], **kw)
    assert torch.equal(res[:, :384], out) and torch.all(res[:, 384:] == 0)
    one = table[:1].expand(4, -1)                            # one table row for every row, no seq
    a = paged.attention_decode(q, k, v, one, pos.clamp(max=49))
    b = paged.attention_decode(q, k, v, table, pos.clamp(max=49), seq=torch.zeros_like(pos))
    assert torch.equal(a, b)


def test_attention_offsets_past_32_bits():
    """A pool of more than 2^32 elements: the pages used lie at its far end."""
    pages = (1 << 32) // (8 * 256 * 128) + 40
    k = torch.empty(pages, 8, 256, 128, dtype=torch.uint8, device=DEV).view(E4M3)
    v = torch.empty(pages, 8, 256, 128, dtype=torch.uint8, device=DEV).view(E4M3)
    rng = np.random.default_rng(11)
    small = [_pool(rng, 3, 8, 256, 128, True) for _ in range(2)]
    far = [pages - 1, pages - 3, pages - 30]
    for pool, (part, _) in zip((k, v), small):
        for i, p in enumerate(far):
            pool.view(torch.uint8)[p] = part.view(torch.uint8)[i]
    q = _t(D.rn16(rng.standard_normal((1, 8, 128))))
    sc = torch.full((8,), 0.06, device=DEV)
    pos = _t([700], torch.int32)
    a = paged.attention_decode(q, k, v, _t([far], torch.int32), pos, k_scale=sc, v_scale=sc)
    b = paged.attention_decode(q, small[0][0], small[1][0], _t([[0, 1, 2]], torch.int32), pos, k_scale=sc, v_scale=sc)
    assert torch.equal(a, b) and torch.any(a != 0)
    # appending there, and copying a page to the far end
    qkv = _t(rng.standard_normal((1, 24 * 128)).astype(np.float16))
    cs = paged.rope_table(768, DEV)
    paged.qknorm_rope_append(qkv, pos, None, None, cs, k, v, _t([far], torch.int32), 8, k_scale=sc, v_scale=sc)
    paged.qknorm_rope_append(qkv, pos, None, None, cs, small[0][0], small[1][0], _t([[0, 1, 2]], torch.int32), 8,
                             k_scale=sc, v_scale=sc)
    paged.copy_pages(k, [far[2]], [far[0] - 1])
    assert torch.equal(k.view(torch.uint8)[far[0] - 1], small[0][0].view(torch.uint8)[2])
    assert torch.equal(v.view(torch.uint8)[far[2]], small[1][0].view(torch.uint8)[2])


def test_attention_repeats_bit_for_bit_and_on_other_streams():
    args, kw, out, _ = _attention(3, 32, 4, 128, 16, [3000, 900, 17], False, 12)
    for _ in range(5):
        assert torch.equal(paged.attention_decode(*args, **kw), out)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):                                      # two calls at once, no shared scratch
        for s in (s1, s2):
            with torch.cuda.stream(s):
                got.append(paged.attention_decode(*args, **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(g, out) for g in got)


def test_two_captured_graphs_replayed_at_once_and_new_lengths():
    args, kw, out, _ = _attention(2, 16, 2, 128, 32, [2000, 500], False, 13)
    pos = args[4]
    graphs, outs, streams = [], [], []
    for _ in range(2):
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            outs.append(paged.attention_decode(*args, **kw))
        graphs.append(g), streams.append(s)
    torch.cuda.synchronize()
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, out) for o in outs)
    pos.copy_(_t([3, 450], torch.int32))                     # the same graph serves other lengths
    graphs[0].replay()
    assert torch.equal(outs[0], paged.attention_decode(*args, **kw))


# ---------------------------------------------------------------- page copies
@pytest.mark.parametrize("shape", [(40, 1, 8, 64), (3, 2, 40, 2, 16, 128), (2, 40, 5, 32, 64)])
@pytest.mark.parametrize("fp8", [False, True])
def test_copy_pages(shape, fp8):
    g = torch.Generator().manual_seed(3)
    pools = torch.randint(0, 256, (*shape[:-1], shape[-1] * (1 if fp8 else 2)), generator=g, dtype=torch.uint8)
    pools = pools.to(DEV).view(E4M3 if fp8 else torch.float16)
    perm = torch.randperm(40, generator=g).tolist()
    for n in (0, 1, 19):
        src, dst = perm[:n], perm[20:20 + n]
        want = pools.clone()
        for a, b in zip(src, dst):
            want.view(torch.uint8).view(-1, *want.view(torch.uint8).shape[-4:])[:, b] = \
                pools.view(torch.uint8).view(-1, *want.view(torch.uint8).shape[-4:])[:, a]
        if n == 1:
            paged.copy_pages(pools, src, dst)
        else:
            paged.copy_pages(pools, torch.tensor(src, dtype=torch.int32, device=DEV),
                             torch.tensor(dst, dtype=torch.int32, device=DEV))
        assert torch.equal(pools.view(torch.uint8), want.view(torch.uint8))


def test_copy_pages_skips_pairs_outside_the_pool_and_leaves_gaps_alone():
    wide = torch.arange(10 * 3 * 8 * 64, device=DEV).half().view(10, 3, 8, 64)
    pools, want = wide[:, :2], wide.clone()                  # the third head is not part of a page
    want[7, :2], want[4, :2] = wide[2, :2], wide[4, :2]
    ids = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    paged.copy_pages(pools, ids([2, 1, -1, 10, 4]), ids([7, 10, 3, 0, 4]))
    assert torch.equal(wide, want)


# ---------------------------------------------------------------- the cache and the block
def test_cache_forks_write_their_own_pages_and_survive_compaction():
    rng = np.random.default_rng(20)
    c = paged.PagedCache(24, 2, 5, 6, DEV, layers=2, page_size=8, head_dim=64)
    cs = paged.rope_table(48, DEV, rot=16)
    held = {}

    def grow(seqs, n):
        for _ in range(n):
            for s in seqs:
                c.extend(s)
            rows = torch.from_numpy(rng.standard_normal((len(seqs), 6 * 64)).astype(np.float16)).to(DEV)
            pos = _t([c.length(s) - 1 for s in seqs], torch.int32)
            for i in range(2):
                k, v, _, _ = c.layer(i)
                paged.qknorm_rope_append(rows * (i + 1), pos, None, None, cs, k, v, c.table, 2,
                                         seq=_t(seqs, torch.int32))
            for r, s in enumerate(seqs):
                held.setdefault(s, []).append(rows[r, 256:].view(2, 64).clone())

    def check():
        for s, vals in held.items():
            for i in range(2):
                v = c.layer(i)[1]
                row = c.table[s].tolist()
                for p, x in enumerate(vals):
                    if row[p // 8] >= 0:
                        assert torch.equal(v[row[p // 8], :, p % 8], x * (i + 1)), (s, p)

    a, b = c.new(), c.new()
    grow([a, b], 11)
    f = c.fork(a)
    held[f] = list(held[a])
    g = c.fork(f)
    held[g] = list(held[a])
    check()
    grow([a, f, g], 9)                                       # three owners of one half-filled page
    check()
    before = c.free_pages
    c.free(b)
    del held[b]
    c.drop_front(a, 9)
    assert c.free_pages == before + 2 + 0                    # page 0 of a is still f's and g's
    moved = c.compact()
    assert moved > 0 and int(c.table.max()) == 24 - c.free_pages - 1
    check()
    grow([a, f, g], 3)
    check()
    for s in (a, f, g):
        c.free(s)
    assert c.free_pages == 24 and int(c.table.max()) == -1


def test_cache_full_changes_nothing():
    c = paged.PagedCache(3, 1, 2, 4, DEV, page_size=8, head_dim=64)
    s = c.new(17)
    with pytest.raises(paged.CacheFull):
        c.extend(s, 8)
    with pytest.raises(paged.CacheFull):
        c.new(1)
    assert c.length(s) == 17 and c.free_pages == 0
    t = c.new()
    with pytest.raises(paged.CacheFull):
        c.new()
    with pytest.raises(paged.CacheFull):
        c.extend(s, 100)
    c.free(t)
    f = c.fork(s)
    with pytest.raises(paged.CacheFull):
        c.extend(f)                                          # the shared page would have to be copied
    c.free(s)
    c.extend(f)
    assert c.length(f) == 18


def test_entry_points_refuse_bad_tensors():
    k = torch.zeros(4, 2, 8, 64, dtype=torch.float16, device=DEV)
    table, pos = _t([[0, 1]], torch.int32), _t([3], torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.float16, device=DEV)
    ok = dict(q=q, k=k, v=k.clone(), table=table, pos=pos)
    for kw in (dict(q=q.float()), dict(q=q[..., :32]), dict(k=k[:, :, :4]), dict(v=k[:2]), dict(pos=pos.long()),
               dict(pos=_t([1, 2], torch.int32)), dict(table=table.long()), dict(k_scale=torch.ones(2, device=DEV)),
               dict(seq=_t([0, 0], torch.int32)), dict(q=q.cpu()), dict(out=torch.zeros(2, 256, device=DEV).half()),
               dict(k=k.transpose(1, 2), v=k.transpose(1, 2)), dict(k=k.bfloat16(), v=k.bfloat16())):
        with pytest.raises(ValueError):
            paged.attention_decode(**dict(ok, **kw))
    with pytest.raises(tri.TriError):                        # page size 4
        paged.attention_decode(q, k[:, :, :4].contiguous(), k[:, :, :4].contiguous(), table, pos)
    with pytest.raises(tri.TriError):                        # 20 query heads on one
        paged.attention_decode(torch.zeros(1, 20, 64, dtype=torch.float16, device=DEV), k[:, :1].contiguous(),
                               k[:, :1].contiguous(), table, pos)
    with pytest.raises(ValueError):
        paged.copy_pages(k, [0, 1], [1, 2])
    with pytest.raises(ValueError):
        paged.copy_pages(k, [0, 1], [2, 2])
    with pytest.raises(ValueError):
        paged.copy_pages(k, [0], [4])
    with pytest.raises(ValueError):
        paged.copy_pages(k[:, :, :4], [0], [1])


# ---------------------------------------------------------------- the ternary block on pages
def _block_weights(Dm, F, H, Hkv, seed):
    from bit_mixed_precision_tri_b200 import inputs
    w = {}
    shapes = {"qkv": ((H + 2 * Hkv) * 128, Dm), "o": (Dm, H * 128), "gate": (F, Dm), "up": (F, Dm), "down": (Dm, F)}
    for i, (name, (n, k)) in enumerate(shapes.items()):
        w[name] = (inputs.random_trits(n, k, 0.31, seed + i), torch.tensor([0.0159]))
    rng = np.random.default_rng(seed)
    for name, n in (("g_attn", Dm), ("g_mlp", Dm), ("gq", 128), ("gk", 128)):
        w[name] = _t(D.rn16(rng.uniform(0.5, 1.5, n)))
    return w


@pytest.mark.parametrize("fmt", ["tq2", "tq1"])
def test_block_on_pages_follows_the_contiguous_block(fmt):
    """Twelve steps of three ragged sequences on both kinds of cache.  Each step's
    attention and cache entries agree to one rounding each (2^-10 of the value);
    what follows is the same arithmetic, so the outputs stay within the block's
    own bound, 2^-9 of the value and of the row's size."""
    Dm, F, H, Hkv, M = 512, 512, 4, 2, 3
    w = _block_weights(Dm, F, H, Hkv, 3)
    flat = dec.DecodeBlock(w, Dm, H, Hkv, F, M, 64, DEV, fmt=fmt)
    cache = paged.PagedCache(30, Hkv, 5, 8, DEV, layers=2, page_size=8)
    blk = dec.DecodeBlock(w, Dm, H, Hkv, F, M, 64, DEV, fmt=fmt, cache=cache, layer=1)
    rng = np.random.default_rng(4)
    start = [0, 5, 40]
    seqs = [cache.new(n) for n in (0, 3, 0)]
    cache.free(seqs[0])
    seqs = [seqs[2], seqs[1], cache.new()]                    # handles that are not row numbers
    cache.extend(seqs[1], 2)
    cache.extend(seqs[2], 40)
    k, v, _, _ = cache.layer(1)
    for m, n in enumerate(start):                             # the same history in both
        hist = torch.from_numpy(rng.standard_normal((2, Hkv, n, 128)).astype(np.float16)).to(DEV)
        flat.kcache[m, :, :n], flat.vcache[m, :, :n] = hist[0], hist[1]
        for p in range(n):
            pg = int(cache.table[seqs[m], p // 8])
            k[pg, :, p % 8], v[pg, :, p % 8] = hist[0, :, p], hist[1, :, p]
    seq = _t(seqs, torch.int32)
    for step in range(12):
        x = _t(D.rn16(rng.standard_normal((M, Dm))))
        pos = torch.tensor([n + step for n in start], dtype=torch.int32, device=DEV)
        for s in seqs:
            cache.extend(s)
        a = _np(flat.step(x, pos, 64))
        b = _np(blk.step(x, pos, seq=seq))
        tol = 2.0 ** -9 * (np.abs(a) + np.sqrt(np.mean(a ** 2, -1, keepdims=True)))
        assert np.all(np.abs(a - b) <= tol)
        assert not torch.any(cache.pools[0])                  # the other layer is untouched


def test_block_on_pages_captured_step_serves_growth_forks_and_padding():
    """One captured step, replayed while sequences grow, fork, are dropped from
    the batch and the pool is compacted, against the same steps run eagerly on a
    cache of their own."""
    Dm, F, H, Hkv, M = 512, 512, 4, 2, 4
    w = _block_weights(Dm, F, H, Hkv, 5)
    caches = [paged.PagedCache(40, Hkv, 6, 6, DEV, page_size=8, dtype=E4M3, k_scale=torch.full((Hkv,), 0.05),
                               v_scale=torch.full((Hkv,), 0.02)) for _ in range(2)]
    cs = paged.rope_table(48, DEV, rot=64, scaling="linear", factor=2.0)
    blks = [dec.DecodeBlock(w, Dm, H, Hkv, F, M, 48, DEV, cache=c, cs=cs, interleaved=True) for c in caches]
    x = torch.zeros(M, Dm, dtype=torch.float16, device=DEV)
    pos = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    seq = torch.zeros(M, dtype=torch.int32, device=DEV)
    blks[0].step(x, pos, seq=seq)                             # first calls outside the capture
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        out = blks[0].step(x, pos, seq=seq)
    torch.cuda.synchronize()
    rng = np.random.default_rng(6)
    live = []
    for c in caches:
        a = c.new()
        b = c.new()
    live = [a, b]
    for step in range(30):
        if step == 10:
            live.append([c.fork(live[0]) for c in caches][0])
        if step == 17:
            for c in caches:
                c.free(live[1])
            live.pop(1)
            assert caches[0].compact() > 0                    # only one of the two is compacted
        if step == 20:
            for c in caches:
                c.drop_front(live[0], 9)
        for c in caches:
            for h in live:
                c.extend(h)
        n = len(live)
        x.copy_(_t(D.rn16(rng.standard_normal((M, Dm)))))
        pos.copy_(torch.tensor([caches[0].length(h) - 1 for h in live] + [-1] * (M - n), dtype=torch.int32))
        seq.copy_(torch.tensor(live + [0] * (M - n), dtype=torch.int32))
        g.replay()
        ref = blks[1].step(x, pos, seq=seq)
        assert torch.equal(out[:n], ref[:n]), step
        assert torch.all(torch.isfinite(out))


def test_block_refuses_what_its_cache_cannot_serve():
    w = _block_weights(512, 512, 4, 2, 7)
    cache = paged.PagedCache(4, 2, 2, 2, DEV)
    with pytest.raises(ValueError):
        dec.DecodeBlock(w, 512, 4, 2, 512, 1, 16, DEV, cache=cache, layer=1)
    with pytest.raises(ValueError):
        dec.DecodeBlock(w, 512, 4, 4, 512, 1, 16, DEV, cache=cache)
    with pytest.raises(ValueError):
        dec.DecodeBlock(w, 512, 4, 2, 512, 1, 16, DEV, interleaved=True)
    blk = dec.DecodeBlock(w, 512, 4, 2, 512, 1, 16, DEV)
    x, pos = torch.zeros(1, 512, dtype=torch.float16, device=DEV), _t([0], torch.int32)
    with pytest.raises(ValueError):
        blk.step(x, pos)
    with pytest.raises(ValueError):
        blk.step(x, pos, 16, seq=pos)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G", [1, 9])
@pytest.mark.parametrize("gap", [8, 16, 20, 24, 26, 27, 28, 32, 60, 120])
def test_attention_small_weights_carry_what_they_weigh(gap, G, fp8):
    """One key outweighs 131071 others by e^gap; its value is small (2^-10) beside theirs
    (96), so the others are all of the output, half of it, or nothing: where their
    weight is 0 in float32 the output is the one value."""
    n, dh, ps = 131072, 64, 256
    big = gap / 4
    k = torch.zeros(n // ps, 1, ps, dh)
    v = torch.full((n // ps, 1, ps, dh), 96.0)
    k[300, 0, 17, 0], v[300, 0, 17] = big, 2.0 ** -10
    q = torch.zeros(1, G, dh)
    q[..., 0] = 4.0
    kw = dict(k_scale=torch.ones(1, device=DEV), v_scale=torch.full((1,), 2.0 ** -1, device=DEV)) if fp8 else {}
    dt = E4M3 if fp8 else torch.float16
    if fp8:
        v *= 2
        v[300, 0, 17] = 2.0 ** -9
    gap = 4 * float(torch.tensor(big).to(dt).float())          # what the cache holds
    o = paged.attention_decode(q.half().to(DEV), k.to(dt).to(DEV), v.to(dt).to(DEV),
                               torch.arange(n // ps, dtype=torch.int32, device=DEV)[None], _t([n - 1], torch.int32),
                               scale=1.0, **kw).float().cpu().numpy().astype(np.float64)
    w = np.exp(-float(gap))
    ref = (2.0 ** -10 + (n - 1) * w * 96) / (1 + (n - 1) * w)
    # the weights' split: 2^-39 of the largest each, half of fp16's smallest step; else as attention_rows_f64
    rel = 2 * gap * 2.0 ** -22 + 2.0 ** -20 + (n / 8 + 32) * 2.0 ** -23
    tol = rel * 2 * ref + min(w, 2.0 ** -39) * n * 96 + 2.0 ** -11 * ref + 2.0 ** -25
    assert np.all(np.abs(o - ref) <= tol), (o[0, 0], ref, tol)
    if gap >= 104:                                            # e^-104 is 0 in float32
        assert np.all(o == 2.0 ** -10)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G", [1, 9])
@pytest.mark.parametrize("size", [3e3, 1e4, 3e4, 6e4])
def test_attention_scores_of_any_size(size, G, fp8):
    """Scores of 10^6 to 10^12.  Equal ones, of either sign, give the mean of the
    values; different ones are further apart than float32's error of a score, so
    the largest takes all."""
    n, dh, ps = 700, 64, 16
    rng = np.random.default_rng(int(size) + G)
    ks = torch.tensor([size / 400], device=DEV)
    kw = dict(k_scale=ks, v_scale=torch.ones(1, device=DEV)) if fp8 else {}
    dt = E4M3 if fp8 else torch.float16
    pages = -(-n // ps)
    table, pos = torch.arange(pages, dtype=torch.int32, device=DEV)[None], _t([n - 1], torch.int32)
    vals = torch.from_numpy(rng.integers(-8, 9, (pages, 1, ps, dh)).astype(np.float32))
    V = vals.numpy().astype(np.float64).reshape(-1, dh)[:n]
    kmax = 400.0 if fp8 else size
    for sign in (1.0, -1.0):
        for scale in (None, 1e20):
            k = torch.full((pages, 1, ps, dh), kmax).to(dt)
            q = torch.full((1, G, dh), sign * size).half()
            o = _np(paged.attention_decode(q.to(DEV), k.to(DEV), vals.to(dt).to(DEV), table, pos, scale=scale, **kw))
            # equal weights: sums of integers below 2^13 with a split to 2^-20, one division, one rounding to fp16
            ref = V.mean(0)
            assert np.all(np.abs(o.reshape(G, dh) - ref) <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -19 * np.abs(V).mean(0) + 2.0 ** -24), (sign, scale, o)
    k = torch.from_numpy((rng.standard_normal((pages, 1, ps, dh)) * kmax / 4).clip(-kmax, kmax).astype(np.float32)).to(dt)
    q = D.rn16((rng.standard_normal((1, G, dh)) * size / 4).clip(-size, size))
    K = k.float().numpy().astype(np.float64).reshape(-1, dh)[:n] * (float(ks) if fp8 else 1.0)
    s = q[0] @ K.T * dh ** -0.5
    two = np.sort(s, 1)[:, -2:]
    err = 2 * (dh + 4) * 2.0 ** -23 * (np.abs(q[0]) @ np.abs(K).T).max(1) * dh ** -0.5
    clear = two[:, 1] - two[:, 0] > err + 110                 # e^-110 is 0 in float32
    assert clear.any()
    o = _np(paged.attention_decode(_t(q), k.to(DEV), vals.to(dt).to(DEV), table, pos, **kw)).reshape(G, dh)
    assert np.all(np.isfinite(o)) and np.array_equal(o[clear], V[s.argmax(1)][clear])


@pytest.mark.parametrize("T", [2, 2500])
def test_append_eps_below_the_normal_numbers(T):
    """x / sqrt(mean x^2 + eps) of a head of zeros is 0 for any eps above 0."""
    k = torch.ones(-(-T // 8), 1, 8, 64, dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    qkv = torch.zeros(T, 192, dtype=torch.float16, device=DEV)
    qkv[1, :] = 2.0 ** -24                                   # the smallest number: mean x^2 is 2^-48
    table, pos = torch.arange(len(k), dtype=torch.int32, device=DEV)[None], torch.arange(T, dtype=torch.int32, device=DEV)
    one = torch.ones(64, dtype=torch.float16, device=DEV)
    q = paged.qknorm_rope_append(qkv, pos, one, one, paged.rope_table(T, DEV, rot=16), k, v, table, 1,
                                 seq=torch.zeros_like(pos), eps=1e-40)
    keep = [t for t in range(T) if t != 1]
    assert torch.all(q[keep] == 0) and not torch.any(torch.isnan(k))
    assert torch.all(k.transpose(1, 2).reshape(-1, 64)[:T][keep] == 0)
    assert torch.all((q[1, 0, 16:] - 1).abs() <= 2.0 ** -11)     # features that do not rotate


def test_block_on_pages_has_angles_for_every_position_of_its_cache():
    """A block whose Lmax is below what its cache has room for: the default table covers the cache."""
    Dm, F, H, Hkv = 512, 512, 4, 2
    w = _block_weights(Dm, F, H, Hkv, 9)
    outs = []
    for Lmax in (16, 64):
        cache = paged.PagedCache(8, Hkv, 1, 8, DEV, page_size=8)
        s = cache.new(41)
        cache.pools.view(torch.int16).copy_(torch.arange(cache.pools.numel(), device=DEV).view(cache.pools.shape) % 15000)
        blk = dec.DecodeBlock(w, Dm, H, Hkv, F, 1, Lmax, DEV, cache=cache)
        x = _t(D.rn16(np.random.default_rng(1).standard_normal((1, Dm))))
        blk.step(x * 0.5, _t([3], torch.int32), seq=_t([s], torch.int32))
        outs.append(blk.step(x, _t([40], torch.int32), seq=_t([s], torch.int32)).clone())
        assert blk.cs.shape[0] == 64
    assert torch.equal(*outs) and torch.all(torch.isfinite(outs[0]))


def test_cache_forked_before_its_room_is_written():
    """Room for 12 positions of which 5 are written at the fork: each continues with its own keys and values."""
    c = paged.PagedCache(6, 2, 2, 3, DEV, layers=2, page_size=8, head_dim=64)
    a = c.new(12)
    cs, g = paged.rope_table(24, DEV, rot=16), torch.Generator().manual_seed(4)

    def write(s, lo, hi):
        rows = torch.randn(hi - lo, 6 * 64, generator=g).half().to(DEV)
        for i in range(2):
            k, v, _, _ = c.layer(i)
            paged.qknorm_rope_append(rows * (i + 1), torch.arange(lo, hi, dtype=torch.int32, device=DEV), None, None, cs,
                                     k, v, c.table, 2, seq=torch.full((hi - lo,), s, dtype=torch.int32, device=DEV))
        return rows[:, 256:].view(-1, 2, 64)

    head = write(a, 0, 5)
    b = c.fork(a, written=5)
    assert c.free_pages == 2                                  # the half-written page and the empty one are b's own
    want = {s: torch.cat([head, write(s, 5, 12)]) for s in (a, b)}
    for s in (a, b):
        for i in range(2):
            v = c.layer(i)[1]
            got = torch.stack([v[int(c.table[s, p // 8]), :, p % 8] for p in range(12)])
            assert torch.equal(got, want[s] * (i + 1))
