"""CPU oracle for the paged key/value cache -- TEST INFRASTRUCTURE ONLY.

Plain float64 statements of the rotary tables, the append of rows into pages
and attention over pages; imports nothing from the product package.  The
definitions of RMSNorm, QK-Norm, RoPE and attention are those of
``decode_oracle`` (D14-D17); what pages add:

P1  position p of sequence s lives in page table[s][p // ps], slot p % ps; a
    table entry outside [0, pages) is an absent page.
P2  a row's sequence outside the table or a negative position is padding: it
    writes nothing, and attention gives zeros, as where no page is present.
P3  e4m3 (1 sign, 4 exponent, 3 mantissa bits, bias 7, largest 448, one NaN
    code): the stored element is rn(clamp(x / scale, +-448)), its value
    element * scale.
P4  rotary frequencies theta^(-2i/rot), i < rot / 2, and their four scalings;
    pairs (i, i + rot/2) or (2i, 2i + 1); features from rot on pass.
"""
from __future__ import annotations

import math

import numpy as np


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes (P3)."""
    out = np.empty(256)
    for code in range(256):
        s, e, m = code >> 7, (code >> 3) & 15, code & 7
        v = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[code] = -v if s else v
    return out


def rope_freqs(rot: int, theta: float = 5.0e5, scaling=None, factor=1.0, context=0.0, low=1.0, high=4.0):
    """(frequencies [rot/2], gain) of P4."""
    f = []
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    gain = 1.0
    for i in range(rot // 2):
        x = theta ** (-2 * i / rot)
        if scaling == "linear":
            x /= factor
        elif scaling == "bands":
            w = 2 * math.pi / x
            if w > context / low:
                x /= factor
            elif w >= context / high:
                s = (context / w - low) / (high - low)
                x = (1 - s) * x / factor + s * x
        elif scaling == "ramp":
            def c(turns):
                return rot * math.log(context / (turns * 2 * math.pi)) / (2 * math.log(theta))
            a, b = max(math.floor(c(high)), 0), min(math.ceil(c(low)), rot - 1)
            b = a + 0.001 if a == b else b
            r = min(max((i - a) / (b - a), 0.0), 1.0)
            x = x / factor * r + x * (1 - r)
            gain = 0.1 * math.log(factor) + 1
        f.append(x)
    return np.array(f), gain


def rope_table_f64(Lmax: int, rot: int, **kw) -> np.ndarray:
    f, gain = rope_freqs(rot, **kw)
    a = np.arange(Lmax, dtype=np.float64)[:, None] * f[None]
    return gain * np.stack([np.cos(a), np.sin(a)], -1)


def norm_rotate_f64(x, gain, cs_row, interleaved: bool, eps: float = 1e-5) -> np.ndarray:
    """One head's features [dh], cs_row [rot/2][2]."""
    x = np.array(x, dtype=np.float64)
    if gain is not None:
        x = x / math.sqrt(float(np.mean(x * x)) + eps) * np.asarray(gain, np.float64)
    half = len(cs_row)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = np.asarray(cs_row, np.float64).T
    y = x.copy()
    y[a], y[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
    return y


def place(table, s: int, p: int, ps: int, pages: int) -> int:
    """The page of position p of sequence s, -1 if absent (P1, P2)."""
    if not 0 <= s < table.shape[0] or not 0 <= p < table.shape[1] * ps:
        return -1
    pg = int(table[s, p // ps])
    return pg if 0 <= pg < pages else -1


def append_f64(qkv, pos, seq, gq, gk, cs, table, shape, H: int, interleaved: bool, k_scale=None, v_scale=None):
    """(q [T][H][dh], writes): q is None for rows that write nothing; writes is
    a list of (page, head, slot, k element, v element), unrounded float64,
    divided by the scale and clamped for e4m3.  `shape` is that of a pool."""
    pages, Hkv, ps, dh = shape
    out, writes = [], []
    for t in range(len(pos)):
        p, s = int(pos[t]), int(seq[t])
        if not (0 <= s < table.shape[0] and 0 <= p < min(len(cs), table.shape[1] * ps)):
            out.append(None)
            continue
        x = np.asarray(qkv[t], np.float64).reshape(H + 2 * Hkv, dh)
        out.append(np.stack([norm_rotate_f64(x[h], gq, cs[p], interleaved) for h in range(H)]))
        pg = place(table, s, p, ps, pages)
        for j in range(Hkv if pg >= 0 else 0):
            k, v = norm_rotate_f64(x[H + j], gk, cs[p], interleaved), x[H + Hkv + j].copy()
            if k_scale is not None:
                k, v = np.clip(k / float(k_scale[j]), -448, 448), np.clip(v / float(v_scale[j]), -448, 448)
            writes.append((pg, j, p % ps, k, v))
    return out, writes


def attention_f64(q, K, V, table, pos, seq, scale: float) -> np.ndarray:
    """q [M][H][dh], pools (values) [pages][Hkv][ps][dh] -> [M][H][dh] (P1, P2)."""
    q = np.asarray(q, np.float64)
    M, H, dh = q.shape
    pages, Hkv, ps, _ = K.shape
    out = np.zeros((M, H, dh))
    for m in range(M):
        kept = [(pg, p % ps) for p in range(min(int(pos[m]) + 1, table.shape[1] * ps))
                if (pg := place(table, int(seq[m]), p, ps, pages)) >= 0]
        if not kept:
            continue
        at, slot = np.array(kept).T
        for h in range(H):
            j = h // (H // Hkv)
            s = np.asarray(K[at, j, slot], np.float64) @ q[m, h] * scale
            w = np.exp(s - s.max())
            out[m, h] = w @ np.asarray(V[at, j, slot], np.float64) / w.sum()
    return out


def attention_bound(q, K, V, table, pos, seq, scale: float, ref) -> np.ndarray:
    """How far an output computed in float32 and rounded once to fp16 may be
    from the float64 one, [M][H][dh]: a score is a sum of dh products, each
    partial sum off by at most one unit of 2^-23 of the absolute sum (tensor
    cores may truncate), so a weight is off by twice that relative to the
    others; weights carry 2^-20 more (exponential, their split into two fp16
    parts); sums over n positions add in steps of at least 8; the result rounds
    by half an fp16 step."""
    absmax = 0.0
    q = np.asarray(q, np.float64)
    M, H, dh = q.shape
    Hkv, ps = K.shape[1], K.shape[2]
    tol = np.zeros(ref.shape)
    for m in range(M):
        n = min(int(pos[m]) + 1, table.shape[1] * ps)
        kept = [(pg, p % ps) for p in range(n) if (pg := place(table, int(seq[m]), p, ps, K.shape[0])) >= 0]
        if not kept:
            continue
        at, slot = np.array(kept).T
        for h in range(H):
            j = h // (H // Hkv)
            absmax = float(np.max(np.abs(np.asarray(K[at, j, slot], np.float64)) @ np.abs(q[m, h]))) * scale
            vmax = float(np.max(np.abs(np.asarray(V[at, j, slot], np.float64))))
            tol[m, h] = (2 * (dh + 4) * 2.0 ** -23 * absmax + 2.0 ** -20 + (len(kept) / 8 + 32) * 2.0 ** -23) * vmax
    return tol + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25


def attention_rows_f64(q, K, V, table, pos, seq, scale: float):
    """(out, tolerance), both [M][H][dh]: ``attention_f64`` with the heads of a
    (row, key/value head) in one product, for batches of many positions, and a
    bound that goes by the weighted values instead of the largest one.

    A weight is off, relative to the others, by rel = 2 (dh + 4) 2^-23 of the
    scores' absolute sums (see ``attention_bound``) + 2^-20 (exponential, split
    into two fp16 parts) + (n / 8 + 32) 2^-23 (sums over n positions), and by
    2^-39 of the largest weight at least (half a step of the smaller part).  So
    the output is off by rel (sum w |V| / sum w + |out|) + n 2^-39 max |V|, then
    rounded by half an fp16 step."""
    q = np.asarray(q, np.float64)
    M, H, dh = q.shape
    pages, Hkv, ps, _ = K.shape
    G = H // Hkv
    out, tol = np.zeros((M, H, dh)), np.full((M, H, dh), 2.0 ** -25)
    for m in range(M):
        n = min(int(pos[m]) + 1, table.shape[1] * ps) if 0 <= int(seq[m]) < table.shape[0] else 0
        if n <= 0:
            continue
        p = np.arange(n)
        pg = np.asarray(table[int(seq[m])])[p // ps].astype(np.int64)
        keep = (pg >= 0) & (pg < pages)
        if not keep.any():
            continue
        at, slot, n = pg[keep], p[keep] % ps, int(keep.sum())
        for j in range(Hkv):
            k, v, qj = np.asarray(K[at, j, slot], np.float64), np.asarray(V[at, j, slot], np.float64), q[m, j * G:(j + 1) * G]
            s = qj @ k.T * scale
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            o = w @ v
            absmax = (np.abs(qj) @ np.abs(k).T).max(1, keepdims=True) * scale
            rel = 2 * (dh + 4) * 2.0 ** -23 * absmax + 2.0 ** -20 + (n / 8 + 32) * 2.0 ** -23
            out[m, j * G:(j + 1) * G] = o
            tol[m, j * G:(j + 1) * G] += rel * (w @ np.abs(v) + np.abs(o)) + n * 2.0 ** -39 * np.abs(v).max() + 2.0 ** -11 * np.abs(o)
    return out, tol
