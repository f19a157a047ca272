"""The paged key/value cache without a GPU: pins of its oracle, the host's book
of pages, and what the entry points refuse before they touch the device."""
import ctypes
import math
import random

import numpy as np
import pytest
import torch

from bit_mixed_precision_tri_b200 import _lib, paged
from oracle import decode_oracle as D
from oracle import paged_oracle as P

FAKE = 1 << 20        # a non-null, 256-byte-aligned address that is never dereferenced


# ---------------------------------------------------------------- the oracle's pins
def test_e4m3_codes():
    v = P.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(v, t, equal_nan=True)
    assert v[0x7E] == 448 and v[1] == 2.0 ** -9 and math.isnan(v[0x7F]) and v[0x38] == 1


def test_rope_freqs_closed_forms():
    f, g = P.rope_freqs(128)
    assert g == 1 and np.allclose(f, D.rope_angles_f64([1], 128)[0], rtol=1e-14)
    lin, _ = P.rope_freqs(64, theta=1e4, scaling="linear", factor=4.0)
    assert np.allclose(lin * 4, P.rope_freqs(64, theta=1e4)[0], rtol=1e-15)
    # ntk: the first pair keeps its frequency, the last is stretched by the factor
    ntk, _ = P.rope_freqs(64, theta=1e4, scaling="ntk", factor=8.0)
    base = P.rope_freqs(64, theta=1e4)[0]
    assert ntk[0] == 1 and math.isclose(ntk[-1] * 8, base[-1], rel_tol=1e-12)
    kw = dict(theta=1e4, factor=8.0, context=8192.0, low=1.0, high=4.0)
    bands, _ = P.rope_freqs(128, scaling="bands", **kw)
    turns = 8192.0 * P.rope_freqs(128, theta=1e4)[0] / (2 * math.pi)
    ratio = bands / P.rope_freqs(128, theta=1e4)[0]
    assert np.all(ratio[turns > 4] == 1) and np.allclose(ratio[turns < 1], 1 / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all((ratio[mid] > 1 / 8) & (ratio[mid] < 1)) and np.all(np.diff(ratio) <= 0)
    ramp, gain = P.rope_freqs(128, theta=1e4, scaling="ramp", factor=16.0, context=4096.0, low=1.0, high=32.0)
    ratio = ramp / P.rope_freqs(128, theta=1e4)[0]
    assert ratio[0] == 1 and math.isclose(ratio[-1], 1 / 16) and np.all(np.diff(ratio) <= 0)
    assert math.isclose(gain, 0.1 * math.log(16) + 1)


def test_norm_rotate_pins():
    rng = np.random.default_rng(0)
    x, g = rng.standard_normal(128), rng.uniform(0.5, 1.5, 128)
    cs = P.rope_table_f64(40, 128)
    ref = D.rope_f64(D.rmsnorm_f64(x[None], g), [37])[0]
    assert np.allclose(P.norm_rotate_f64(x, g, cs[37], False), ref, rtol=1e-12, atol=1e-12)
    # interleaved = half layout of the de-interleaved features; features past rot pass
    cs = P.rope_table_f64(40, 32)
    y = P.norm_rotate_f64(x, None, cs[5], True)
    perm = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2)])
    z = P.norm_rotate_f64(np.concatenate([x[perm], x[32:]]), None, cs[5], False)
    assert np.allclose(y[perm], z[:32]) and np.array_equal(y[32:], x[32:])
    assert np.allclose(P.norm_rotate_f64(x, None, cs[0], True), x)
    y = P.norm_rotate_f64([1.0, 0, 0, 1], None, [(0.0, 1.0), (0.0, 1.0)], True)
    assert np.array_equal(y, [0, 1, -1, 0])


def test_attention_pins():
    rng = np.random.default_rng(1)
    M, H, Hkv, L = 2, 4, 2, 24
    q, Kc, Vc = rng.standard_normal((M, H, 16)), rng.standard_normal((M, Hkv, L, 16)), rng.standard_normal((M, Hkv, L, 16))
    pool = lambda c: c.reshape(M, Hkv, 3, 8, 16).transpose(0, 2, 1, 3, 4).reshape(6, Hkv, 8, 16)
    table = np.array([[0, 1, 2], [3, 4, 5]])
    pos = np.array([23, 9])
    a = P.attention_f64(q, pool(Kc), pool(Vc), table, pos, [0, 1], 0.25)
    assert np.allclose(a.reshape(M, -1), D.attention_decode_f64(q, Kc, Vc, pos), rtol=1e-12)
    # an absent page is as if its positions were not there; nothing left gives zeros
    b = P.attention_f64(q[:1], pool(Kc), pool(Vc), np.array([[0, 6, 2]]), [23], [0], 0.25)
    keep = [*range(8), *range(16, 24)]
    assert np.allclose(b.reshape(1, -1), D.attention_decode_f64(q[:1], Kc[:1][:, :, keep], Vc[:1][:, :, keep], [15]))
    assert not P.attention_f64(q, pool(Kc), pool(Vc), np.full((2, 3), -1), pos, [0, 1], 1.0).any()
    assert not P.attention_f64(q, pool(Kc), pool(Vc), table, [-1, 3], [0, 2], 1.0).any()


def test_append_pins():
    qkv = np.arange(2 * 4 * 16, dtype=np.float64).reshape(2, 64)
    cs = P.rope_table_f64(20, 16)
    out, w = P.append_f64(qkv, [0, -1], [0, 0], None, None, cs, np.array([[2]]), (3, 1, 8, 16), 2, False)
    assert out[1] is None and np.allclose(out[0].ravel(), qkv[0, :32])
    (pg, j, slot, k, v), = w
    assert (pg, j, slot) == (2, 0, 0) and np.allclose(k, qkv[0, 32:48]) and np.array_equal(v, qkv[0, 48:])
    _, w = P.append_f64(qkv, [3, 9], [0, 0], None, None, cs, np.array([[2]]), (3, 1, 8, 16), 2, False, [0.01], [2.0])
    assert len(w) == 1 and np.all(np.abs(w[0][3]) <= 448) and np.array_equal(w[0][4], qkv[0, 48:] / 2)


# ---------------------------------------------------------------- the host's book
@pytest.mark.parametrize("seed", range(20))
def test_page_book_against_plain_lists(seed):
    """Random calls; every sequence reads back what was written to it, whoever shares its pages."""
    r, b = random.Random(seed), paged.PageBook(20, 4, 6, 9)
    ref, data = {}, [[None] * 4 for _ in range(20)]

    def copies(pair):
        for a, c in zip(*pair):
            data[c] = list(data[a])

    for _ in range(200):
        op = r.choice("neeeefdxc")
        s = r.choice(list(ref)) if ref else None
        try:
            if op == "n":
                ref[b.new()] = []
            elif op == "c":
                copies(b.compact())
                live = sum(c > 0 for c in b.count)
                assert all(c > 0 for c in b.count[:live])
            elif s is None:
                continue
            elif op == "e":
                n, L = r.randrange(0, 6), b.length[s]
                if n and L % 4 and b.pages[s][L // 4] < 0:
                    with pytest.raises(ValueError):
                        b.extend(s, n)
                    continue
                copies(b.extend(s, n))
                for p in range(L, L + n):
                    pg = b.pages[s][p // 4]
                    assert b.count[pg] == 1
                    data[pg][p % 4] = r.random()
                    ref[s].append(data[pg][p % 4])
            elif op == "f":
                ref[b.fork(s)] = list(ref[s])
            elif op == "d":
                n = r.randrange(0, len(ref[s]) + 1)
                b.drop_front(s, n)
                ref[s][: n // 4 * 4] = [None] * (n // 4 * 4)
            else:
                b.free(s)
                del ref[s]
        except paged.CacheFull:
            pass
        for s, vals in ref.items():
            assert b.length[s] == len(vals)
            for p, v in enumerate(vals):
                if v is not None:
                    assert data[b.pages[s][p // 4]][p % 4] == v
        held = [p for h in b.pages.values() for p in h if p >= 0]
        assert [held.count(p) for p in range(20)] == b.count
        assert sorted(b.free_pages) == [p for p in range(20) if b.count[p] == 0]


def test_page_book_refusals_change_nothing():
    b = paged.PageBook(2, 8, 2, 4)
    s = b.new()
    b.extend(s, 9)
    state = (list(b.pages[s]), b.length[s], list(b.count))
    for n in (8, 100):
        with pytest.raises(paged.CacheFull):
            b.extend(s, n)
    with pytest.raises(ValueError):
        b.extend(s, -1)
    with pytest.raises(ValueError):
        b.drop_front(s, 10)
    t = b.fork(s)
    with pytest.raises(paged.CacheFull):
        b.fork(s)
    with pytest.raises(paged.CacheFull):
        b.extend(t, 1)                                       # the shared page needs a free one
    b.free(t)
    assert state == (list(b.pages[s]), b.length[s], list(b.count))


def test_paged_cache_on_the_host_device():
    """Shapes, the table and refusals need no GPU."""
    c = paged.PagedCache(6, 2, 3, 4, "cpu", layers=2, page_size=8, head_dim=64)
    s = c.new(9)
    assert c.pools.shape == (2, 2, 6, 2, 8, 64) and c.table[s].tolist()[:3] == [0, 1, -1] and c.free_pages == 4
    assert [x is None for x in c.layer(1)] == [False, False, True, True]
    for kw in (dict(page_size=12), dict(head_dim=96), dict(dtype=torch.bfloat16), dict(layers=0),
               dict(dtype=paged.E4M3), dict(k_scale=torch.ones(2), v_scale=torch.ones(2))):
        with pytest.raises(ValueError):
            paged.PagedCache(6, 2, 3, 4, "cpu", **kw)
    e = paged.PagedCache(6, 2, 3, 4, "cpu", layers=2, dtype=paged.E4M3, k_scale=torch.ones(2), v_scale=torch.ones(2, 2))
    assert e.layer(1)[2].shape == (2,)


# ---------------------------------------------------------------- refusals of the C ABI
@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from bit_mixed_precision_tri_b200 import build
        build.build()
    return _lib.lib()


def _cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, table=FAKE, pages=10, page_size=16, page_stride=8 * 16 * 128,
             heads=8, head_dim=128, seqs=4, seq_pages=5, table_stride=5, dtype=0)
    d.update(kw)
    return _lib.PagedCacheDesc(*(d[n] for n, _ in _lib.PagedCacheDesc._fields_))


BAD_CACHES = [
    (1, dict(k=None)), (1, dict(v=None)), (1, dict(table=None)), (1, dict(dtype=2)), (1, dict(dtype=-1)),
    (1, dict(dtype=1)), (1, dict(dtype=1, k_scale=FAKE)), (2, dict(head_dim=96)), (2, dict(head_dim=256)),
    (2, dict(page_size=12)), (2, dict(page_size=4)), (2, dict(page_size=512, page_stride=8 * 512 * 128)),
    (2, dict(heads=0)), (2, dict(pages=0)), (2, dict(pages=1 << 31)), (2, dict(page_stride=8 * 16 * 128 - 128)),
    (2, dict(page_stride=8 * 16 * 128 + 8)), (2, dict(page_stride=1 << 39)), (2, dict(seqs=0)), (2, dict(seq_pages=0)),
    (2, dict(table_stride=-1, seqs=1)), (2, dict(seq_pages=1 << 27, table_stride=1 << 27)),
    (3, dict(k=FAKE + 8)), (3, dict(v=FAKE + 2)), (3, dict(table=FAKE + 2)),
    (3, dict(dtype=1, k_scale=FAKE + 1, v_scale=FAKE)),
]


def test_paged_attention_refusals(L):
    def call(cache=None, **kw):
        a = dict(q=FAKE, qs=64 * 128, pos=FAKE, seq=None, out=FAKE, os=64 * 128, M=2, H=64, scale=0.1, ws=FAKE, n=1 << 40)
        a.update(kw)
        c = None if cache == "null" else ctypes.byref(_cache(**(cache or {})))
        return L.tri_paged_attention(a["q"], a["qs"], a["pos"], a["seq"], c, a["out"], a["os"], a["M"], a["H"],
                                     a["scale"], a["ws"], a["n"], None)

    assert call(cache="null") == 1
    for st, kw in BAD_CACHES:
        assert call(cache=kw) == st, kw
    for st, kw in [(1, dict(q=None)), (1, dict(pos=None)), (1, dict(out=None)), (1, dict(scale=0.0)),
                   (1, dict(scale=float("nan"))), (1, dict(scale=-1.0)), (2, dict(M=0)), (2, dict(M=1 << 25)), (2, dict(H=0)),
                   (2, dict(H=12)), (2, dict(H=136, qs=136 * 128, os=136 * 128)), (2, dict(qs=64 * 128 - 8)),
                   (2, dict(qs=64 * 128 + 4)), (2, dict(os=64)), (3, dict(q=FAKE + 8)), (3, dict(out=FAKE + 2)),
                   (3, dict(pos=FAKE + 2)), (3, dict(seq=FAKE + 1))]:
        assert call(**kw) == st, kw
    assert L.tri_paged_attention_workspace_bytes(1, 64, 8, 128) > 0
    for bad in [(0, 64, 8, 128), (1, 64, 3, 128), (1, 136, 8, 128), (1, 64, 8, 32), (1 << 24, 4096, 4096, 128)]:
        assert L.tri_paged_attention_workspace_bytes(*bad) == 0


def test_paged_append_refusals(L):
    def call(cache=None, **kw):
        a = dict(qkv=FAKE, stride=80 * 128, pos=FAKE, seq=None, gq=FAKE, gk=FAKE, cs=FAKE, rows=100, rot=128, q=FAKE,
                 qs=64 * 128, T=3, H=64, eps=1e-5)
        a.update(kw)
        c = None if cache == "null" else ctypes.byref(_cache(**(cache or {})))
        return L.tri_paged_qknorm_rope(a["qkv"], a["stride"], a["pos"], a["seq"], a["gq"], a["gk"], a["cs"], a["rows"],
                                       a["rot"], 0, a["q"], a["qs"], c, a["T"], a["H"], a["eps"], None)

    assert call(cache="null") == 1
    for st, kw in BAD_CACHES:
        assert call(cache=kw) == st, kw
    for st, kw in [(1, dict(qkv=None)), (1, dict(pos=None)), (1, dict(cs=None)), (1, dict(q=None)), (1, dict(gq=None)),
                   (1, dict(gk=None)), (1, dict(eps=-1.0)), (1, dict(eps=float("nan"))), (2, dict(T=0)),
                   (2, dict(H=63)), (2, dict(H=0)), (2, dict(rot=0)), (2, dict(rot=8)), (2, dict(rot=40)),
                   (2, dict(rot=144)), (2, dict(rows=0)), (2, dict(stride=80 * 128 - 8)), (2, dict(stride=80 * 128 + 2)),
                   (2, dict(qs=8)), (3, dict(qkv=FAKE + 8)), (3, dict(q=FAKE + 8)), (3, dict(cs=FAKE + 8)),
                   (3, dict(gq=FAKE + 2)), (3, dict(pos=FAKE + 1)), (3, dict(seq=FAKE + 2))]:
        assert call(**kw) == st, kw
    assert call(cache=dict(head_dim=64), rot=128, stride=80 * 128) == 2      # more rotated features than the head has


def test_copy_pages_and_table_refusals(L):
    def copy(**kw):
        a = dict(p=FAKE, np=2, ps=1 << 20, pages=8, st=4096, b=4096, s=FAKE, d=FAKE, n=3)
        a.update(kw)
        return L.tri_copy_pages(a["p"], a["np"], a["ps"], a["pages"], a["st"], a["b"], a["s"], a["d"], a["n"], None)

    for st, kw in [(1, dict(p=None)), (1, dict(s=None)), (1, dict(d=None)), (1, dict(n=-1)), (2, dict(np=0)),
                   (2, dict(ps=8)), (2, dict(ps=4080)), (2, dict(pages=0)), (2, dict(st=4080)), (2, dict(st=4100)),
                   (2, dict(b=0)), (2, dict(b=24)), (2, dict(b=1 << 33, st=1 << 33)), (2, dict(n=1 << 31)),
                   (2, dict(n=1 << 30, np=1 << 20)), (3, dict(p=FAKE + 8)), (3, dict(s=FAKE + 2)), (3, dict(d=FAKE + 1))]:
        assert copy(**kw) == st, kw
    assert copy(n=0, s=None, d=None) == 0

    def table(scaling=None, **kw):
        a = dict(p=FAKE, n=10, rot=64, theta=1e4)
        a.update(kw)
        sc = None if scaling is None else ctypes.byref(_lib.RopeScaling(*scaling))
        return L.tri_rope_table_scaled(a["p"], a["n"], a["rot"], a["theta"], sc, None)

    for st, kw in [(1, dict(p=None)), (1, dict(theta=1.0)), (1, dict(theta=float("nan"))), (2, dict(n=0)),
                   (2, dict(n=(1 << 24) + 1)), (2, dict(rot=8)), (2, dict(rot=24)), (2, dict(rot=144)), (3, dict(p=FAKE + 8))]:
        assert table(**kw) == st, kw
    nan = float("nan")
    for bad in [(0, 2, 0, 0, 0), (5, 2, 0, 0, 0), (1, 0.5, 0, 0, 0), (1, nan, 0, 0, 0), (3, 2, 0, 1, 4), (3, 2, 100, 4, 4),
                (3, 2, 100, 0, 4), (4, 2, nan, 1, 4), (4, 2, 100, 1, float("inf"))]:
        assert table(bad) == 1, bad


def test_wrappers_refuse_host_tensors():
    k = torch.zeros(4, 2, 8, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        paged.attention_decode(torch.zeros(1, 4, 64).half(), k, k, torch.zeros(1, 2, dtype=torch.int32),
                               torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        paged.copy_pages(k, [0], [1])
    with pytest.raises(ValueError):
        paged.rope_table(4, "cpu")
    with pytest.raises(ValueError):
        paged.rope_table(4, "cuda", scaling="none")


def test_calls_make_the_tensors_device_current(monkeypatch):
    """A call for tensors of a device that is not the current one switches to it and takes its stream."""
    entered, got = [], []

    class Device:
        def __init__(self, index):
            entered.append(index)

        def __enter__(self):
            return self

        def __exit__(self, *exc):
            return False

    def entry(*args):
        got.append(args)
        return 0 if args[0] else 2

    monkeypatch.setattr(paged.torch.cuda, "device", Device)
    monkeypatch.setattr(paged, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(paged, "_current", lambda: 1)
    paged._call(entry, 0, 7)
    assert entered == [0] and got == [(7, 100)]
    paged._call(entry, 1, 8)
    assert entered == [0] and got[1] == (8, 101)
    with pytest.raises(_lib.TriError) as e:
        paged._call(entry, 1, 0)
    assert e.value.status == 2 and "entry" in str(e.value)


def test_attention_rows_is_attention():
    """The oracle for many positions agrees with the plain one, holes, padding and strangers included."""
    rng = np.random.default_rng(2)
    q, K, V = rng.standard_normal((6, 6, 64)), rng.standard_normal((9, 2, 8, 64)), rng.standard_normal((9, 2, 8, 64))
    table = np.array([[0, 1, 2, 8], [3, -1, 5, 9], [-1, -1, 11, -1]])
    pos, seq = [23, 29, 30, 100, -1, 5], [0, 1, 2, 0, 0, 3]
    a = P.attention_f64(q, K, V, table, pos, seq, 0.125)
    b, tol = P.attention_rows_f64(q, K, V, table, pos, seq, 0.125)
    assert np.allclose(a, b, rtol=1e-12, atol=1e-14) and np.all(tol >= 2.0 ** -25) and not b[2].any() and not b[4:].any()
    assert np.all(tol <= P.attention_bound(q, K, V, table, pos, seq, 0.125, a) * 2 + 2.0 ** -24)


def test_selftest_wait_polls_refusals(L):
    for bad in (-2, (1 << 18) + 1, 1 << 40):
        assert L.tri_selftest_wait_polls(bad) == 1
    for good in (0, 1 << 18, -1):
        assert L.tri_selftest_wait_polls(good) == 0


def test_block_refuses_a_rotary_table_its_cache_outgrows():
    """A row behind the table would write no key and attend with the last step's queries."""
    from bit_mixed_precision_tri_b200 import decode as dec
    cache = paged.PagedCache(6, 2, 3, 4, "cpu", page_size=8)         # 32 positions a sequence
    good = torch.zeros(32, 32, 2)
    for bad in (good[:31], torch.zeros(31, 64, 2), good.double(), good[:, :, 0], good[:, :12], torch.zeros(32, 72, 2),
                torch.zeros(32, 4, 2), torch.zeros(32, 2, 32).transpose(1, 2)):
        with pytest.raises(ValueError, match="cs "):
            dec.DecodeBlock({}, 512, 4, 2, 512, 1, 32, "cpu", cache=cache, cs=bad)
    with pytest.raises(KeyError):                                    # the table is taken; there are no weights
        dec.DecodeBlock({}, 512, 4, 2, 512, 1, 32, "cpu", cache=cache, cs=good)


@pytest.mark.parametrize("seed", range(20))
def test_cache_forked_between_room_and_write(seed, monkeypatch):
    """Room is made, sequences are forked, then each writes what it has room for: all
    read back their own, whoever shares the pages below."""
    c = paged.PagedCache(30, 1, 6, 9, "cpu", page_size=8, head_dim=64)
    flat = c.pools[0, 0, :, 0, :, 0]                                 # one number per position of K

    def copy(pools, src, dst):
        flat[dst] = flat[src]
    monkeypatch.setattr(paged, "copy_pages", copy)
    r, ref = random.Random(seed), {}                                # handle -> what it wrote
    at = lambda s, p: (int(c.table[s, p // 8]), p % 8)
    mark = 0
    for _ in range(300):
        op = r.choice("neewwwffxc")
        s = r.choice(list(ref)) if ref else None
        try:
            if op == "n":
                ref[c.new(r.randrange(0, 12))] = []
            elif op == "c":
                c.compact()
            elif s is None:
                continue
            elif op == "e":
                c.extend(s, r.randrange(0, 12))
            elif op == "w":
                for p in range(len(ref[s]), r.randint(len(ref[s]), c.length(s))):
                    mark += 1
                    flat[at(s, p)] = mark % 2000
                    ref[s].append(mark % 2000)
            elif op == "f":
                before = [list(c.book.count), c.length(s), dict(c.book.pages)]
                t = c.fork(s, written=len(ref[s]))
                ref[t] = list(ref[s])
                assert c.length(t) == c.length(s)
                if c.length(s) == len(ref[s]):
                    assert c.book.pages[t] == c.book.pages[s]       # all written: all shared
            else:
                c.free(s)
                del ref[s]
        except paged.CacheFull:
            if op == "f":
                assert before == [c.book.count, c.length(s), c.book.pages]
        for s, vals in ref.items():
            assert [float(flat[at(s, p)]) for p in range(len(vals))] == vals, (s, op)


def test_fork_refuses_more_than_there_is():
    c = paged.PagedCache(4, 1, 3, 4, "cpu", page_size=8, head_dim=64)
    s = c.new(9)
    for bad in (-1, 10):
        with pytest.raises(ValueError):
            c.fork(s, written=bad)
    assert c.free_pages == 2 and len(c.book.free_seqs) == 2 and c.book.count[:2] == [1, 1]
    t = c.fork(s)
    assert c.book.pages[t] == c.book.pages[s] and c.free_pages == 2


def test_refused_calls_take_no_row():
    c = paged.PagedCache(4, 1, 2, 4, "cpu", page_size=8, head_dim=64)
    s = c.new(3)
    for _ in range(3):
        with pytest.raises(ValueError):
            c.new(-1)
        with pytest.raises(KeyError):
            c.fork(s + 1)
        with pytest.raises(paged.CacheFull):
            c.new(100)
    assert len(c.book.free_seqs) == 1 and list(c.book.pages) == [s] and c.free_pages == 3
    assert c.fork(s) == s + 1


def test_paged_cache_takes_both_scales_or_none():
    one = torch.ones(2)
    for kw in (dict(k_scale=one), dict(v_scale=one), dict(dtype=paged.E4M3, k_scale=one), dict(dtype=paged.E4M3, v_scale=one)):
        with pytest.raises(ValueError, match="takes k_scale and v_scale"):
            paged.PagedCache(6, 2, 3, 4, "cpu", **kw)
