"""What is measured of the paged key/value cache: appending rows of a fused QKV
product (QK-Norm, rotary positions, the write into pages), attention of new
tokens over the pages, and copies of pages.

``own`` false computes the plain form in float32 torch operations, true makes
the calls of ``bit_mixed_precision_tri_b200.paged`` that a decode step makes.

Layouts: a pool is [layers][2][pages][kv heads][page size][head dim] (K, then
V), fp16 or e4m3 with one float32 scale per kv head; a page table is int32
[sequences][pages of a sequence], -1 where there is no page; row t of a call
belongs to sequence seq[t] and sits at position pos[t].
"""
import math

import torch

own = False

EPS = 1e-5
THETA = 5.0e5
DEV = "cuda"


def listed():
    A, D, C = "append", "attention", "copy"
    return [
        # one token of one sequence, the 70B-like block's heads: launch latency
        dict(name="append_t1", op=A, T=1, S=1, H=64, Hkv=8, dh=128, ps=16, ctx=4096, rot=128, inter=False, norm=True,
             fp8=False, scaled=1.0),
        # one token each of 200 sequences into e4m3 pages, interleaved pairs over half of the head
        dict(name="append_t200_fp8", op=A, T=200, S=200, H=16, Hkv=2, dh=128, ps=32, ctx=2000, rot=64, inter=True,
             norm=True, fp8=True, scaled=1.0),
        # prompts of seven sequences, 64-wide heads without QK-Norm, angles stretched eightfold
        dict(name="append_prompt_d64", op=A, T=5001, S=7, H=32, Hkv=32, dh=64, ps=8, ctx=9000, rot=64, inter=False,
             norm=False, fp8=False, scaled=8.0),
        # a long prompt of the 70B-like block
        dict(name="append_prompt", op=A, T=16384, S=4, H=64, Hkv=8, dh=128, ps=64, ctx=16384, rot=128, inter=False,
             norm=True, fp8=False, scaled=1.0),
        # the first tokens of an answer: one sequence, hardly any context
        dict(name="attn_m1_short", op=D, M=1, S=1, H=64, Hkv=8, dh=128, ps=16, ctx=37, fp8=False, ragged=False,
             holes=False),
        # the 70B-like block at 4096 positions, batch 16 (the benchmark's decode step)
        dict(name="attn_m16_4k", op=D, M=16, S=16, H=64, Hkv=8, dh=128, ps=16, ctx=4096, fp8=False, ragged=False,
             holes=False),
        # one very long context
        dict(name="attn_m1_128k", op=D, M=1, S=1, H=64, Hkv=8, dh=128, ps=64, ctx=131072, fp8=False, ragged=False,
             holes=False),
        # a busy server: ragged lengths, e4m3 pages, padding rows and freed pages among them
        dict(name="attn_m128_fp8", op=D, M=128, S=100, H=64, Hkv=8, dh=128, ps=32, ctx=6000, fp8=True, ragged=True,
             holes=True),
        # one kv head per query head, 64 wide, smallest pages, odd sizes
        dict(name="attn_m37_mha_d64", op=D, M=37, S=37, H=12, Hkv=12, dh=64, ps=8, ctx=1500, fp8=False, ragged=True,
             holes=False),
        # sixteen query heads share the only kv head
        dict(name="attn_m9_mqa", op=D, M=9, S=9, H=16, Hkv=1, dh=128, ps=128, ctx=20000, fp8=True, ragged=True,
             holes=False),
        # forking a sequence: its last page, both planes of a few layers
        dict(name="copy_fork", op=C, n=1, pages=64, layers=4, Hkv=8, dh=128, ps=16, fp8=False),
        # compacting the pages of a large pool
        dict(name="copy_compact", op=C, n=1500, pages=4000, layers=2, Hkv=8, dh=128, ps=64, fp8=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "copy"])
    dh, ps, fp8 = rng.choice([64, 128]), rng.choice([8, 16, 32, 64, 128, 256]), rng.random() < 0.4
    Hkv = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    if op == "append":
        T, H = _log(rng, 1, 12000), Hkv * rng.choice([1, 2, 4, 5, 8])
        T = max(1, min(T, 16384 * 80 * 128 // ((H + 2 * Hkv) * dh)))
        S = min(T, _log(rng, 1, 64))
        return dict(op=op, T=T, S=S, H=H, Hkv=Hkv, dh=dh, ps=ps, ctx=max(-(-T // S), _log(rng, 64, 20000)),
                    rot=rng.choice([16, 32, 48, 64] + ([96, 128] if dh == 128 else [])), inter=rng.random() < 0.5,
                    norm=rng.random() < 0.7, fp8=fp8, scaled=rng.choice([1.0, 4.0, 32.0]))
    if op == "attention":
        ctx, G = _log(rng, 1, 100000), rng.choice([1, 2, 3, 5, 7, 8, 12, 16])
        most = 131072 * 8 * 128 // (ctx * Hkv * dh)
        M = max(1, min(_log(rng, 1, 300), most))
        return dict(op=op, M=M, S=max(1, M - rng.choice([0, 0, 3])), H=Hkv * G, Hkv=Hkv, dh=dh, ps=ps, ctx=ctx,
                    fp8=fp8, ragged=rng.random() < 0.6, holes=rng.random() < 0.3)
    layers, pages = rng.choice([1, 2, 3, 5]), _log(rng, 40, 3000)
    while layers * 2 * pages * Hkv * ps * dh > 4000 * 4 * 8 * 64 * 128 // 2:
        pages = max(8, pages // 2)
        ps = max(8, ps // 2)
    return dict(op=op, n=max(1, min(_log(rng, 1, 1400), pages // 2 - 1)), pages=pages, layers=layers, Hkv=Hkv, dh=dh,
                ps=ps, fp8=fp8)


# ---------------------------------------------------------------- inputs
def _pool(shape, fp8, g):
    # normal values; e4m3 pools are written in place, part by part, to keep the peak low
    out = torch.empty(shape, dtype=torch.float8_e4m3fn if fp8 else torch.float16, device=DEV)
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 27):
        b = min(flat.numel(), a + (1 << 27))
        x = torch.randn(b - a, generator=g, device=DEV)
        flat[a:b] = ((x * 16).clamp(-448, 448) if fp8 else x).to(out.dtype)
    return out


def _table(S, need, width, g, slack):
    """Pages of S sequences, need[s] of them each, in shuffled order; -1 behind them."""
    total = int(need.sum())
    perm = torch.randperm(total + slack, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    start = torch.cumsum(need, 0) - need
    col = torch.arange(width, device=DEV)
    idx = (start[:, None] + col[None]).clamp(max=total - 1)
    return torch.where(col[None] < need[:, None], perm[idx], torch.full_like(perm[idx], -1)), total + slack


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * seed + 17)
    dt = torch.float8_e4m3fn if c["fp8"] else torch.float16
    if c["op"] == "copy":
        pools = _pool((c["layers"], 2, c["pages"], c["Hkv"], c["ps"], c["dh"]), c["fp8"], g)
        perm = torch.randperm(c["pages"], generator=g, device=DEV).to(torch.int32)
        n = c["n"]
        return dict(c, pools=pools, src=perm[:n].contiguous(), dst=perm[n:2 * n].contiguous())
    Hkv, H, dh, ps, S = c["Hkv"], c["H"], c["dh"], c["ps"], c["S"]
    width = -(-c["ctx"] // ps)
    scales = [torch.rand(Hkv, generator=g, device=DEV) * 0.04 + 0.05 for _ in range(2)] if c["fp8"] else [None, None]
    if c["op"] == "append":
        T = c["T"]
        # row t belongs to sequence t * S // T; its rows sit at consecutive positions up to a random end
        seq = torch.arange(T, device=DEV) * S // T
        count = torch.bincount(seq, minlength=S)
        first = torch.cumsum(count, 0) - count
        end = (count + (torch.rand(S, generator=g, device=DEV) * (c["ctx"] - count + 1)).long()).clamp(max=c["ctx"])
        pos = end[seq] - count[seq] + torch.arange(T, device=DEV) - first[seq]
        # only the pages that the rows write are in the pool
        lo, hi = torch.div(end - count, ps, rounding_mode="floor"), torch.div(end - 1, ps, rounding_mode="floor")
        near, _ = _table(S, hi - lo + 1, width, g, 3)
        npages = int((count // ps + 2).sum()) + 3        # the same for every seed
        at = torch.arange(width, device=DEV)[None] - lo[:, None]
        table = torch.where((at >= 0) & (at <= (hi - lo)[:, None]), near.gather(1, at.clamp(min=0)),
                            torch.full_like(near, -1))
        rot = c["rot"]
        inv = THETA ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot) / c["scaled"]
        ang = torch.arange(c["ctx"], device=DEV, dtype=torch.float64)[:, None] * inv[None]
        cs = torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()
        gain = [(torch.rand(dh, generator=g, device=DEV) + 0.5).half() if c["norm"] else None for _ in range(2)]
        pools = _pool((1, 2, npages, Hkv, ps, dh), c["fp8"], g)
        qkv = (torch.randn(T, (H + 2 * Hkv) * dh, generator=g, device=DEV) * 2).half()
        return dict(c, qkv=qkv, pos=pos.to(torch.int32), seq=seq.to(torch.int32), table=table, cs=cs, gq=gain[0],
                    gk=gain[1], k=pools[0, 0], v=pools[0, 1], k_scale=scales[0], v_scale=scales[1],
                    out=torch.empty(T, H, dh, dtype=torch.float16, device=DEV))
    M, ctx = c["M"], c["ctx"]
    length = torch.full((S,), ctx, device=DEV)
    if c["ragged"]:
        length = (torch.rand(S, generator=g, device=DEV) * ctx).long() + 1
        length[int(torch.randint(S, (1,), generator=g, device=DEV))] = ctx
    need = torch.div(length + ps - 1, ps, rounding_mode="floor")
    table, npages = _table(S, need, width, g, 5)
    if c["holes"]:
        # pages freed at the front of every third sequence
        col = torch.arange(width, device=DEV)[None]
        gone = (torch.arange(S, device=DEV)[:, None] % 3 == 1) & (col < torch.div(need, 4, rounding_mode="floor")[:, None])
        table = torch.where(gone, torch.full_like(table, -1), table)
    # rows behind the last sequence are padding: no position
    seq = torch.arange(M, device=DEV).clamp(max=S - 1)
    pos = torch.where(torch.arange(M, device=DEV) < S, length[seq] - 1, torch.full_like(seq, -1))
    pools = _pool((1, 2, npages, Hkv, ps, dh), c["fp8"], g)
    q = torch.randn(M, H, dh, generator=g, device=DEV)
    q[:, ::4] *= 3                                       # some heads look at few positions, most at many
    return dict(c, q=q.half(), pos=pos.to(torch.int32), seq=seq.to(torch.int32), table=table.contiguous(),
                k=pools[0, 0], v=pools[0, 1], k_scale=scales[0], v_scale=scales[1],
                out=torch.empty(M, H * dh, dtype=torch.float16, device=DEV))


# ---------------------------------------------------------------- one pass
def run(state):
    s = state
    if own:
        from bit_mixed_precision_tri_b200 import paged
        if s["op"] == "append":
            paged.qknorm_rope_append(s["qkv"], s["pos"], s["gq"], s["gk"], s["cs"], s["k"], s["v"], s["table"],
                                     s["H"], seq=s["seq"], interleaved=s["inter"], k_scale=s["k_scale"],
                                     v_scale=s["v_scale"], out=s["out"])
            return s["out"], s["k"], s["v"]
        if s["op"] == "attention":
            return paged.attention_decode(s["q"], s["k"], s["v"], s["table"], s["pos"], seq=s["seq"],
                                          k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
        paged.copy_pages(s["pools"], s["src"], s["dst"])
        return s["pools"]
    if s["op"] == "append":
        return _append(s)
    if s["op"] == "attention":
        return _attention(s)
    src, dst = s["src"].long(), s["dst"].long()
    raw = s["pools"].view(torch.int64)
    raw[:, :, dst] = raw[:, :, src]
    return s["pools"]


def _norm_rotate(x, gain, c, sn, s):
    """float32 [T][heads][dh] -> QK-Norm and rotation in float32."""
    if gain is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.float()
    rot = s["rot"]
    r, rest = x[..., :rot], x[..., rot:]
    if s["inter"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([r, rest], -1)


def _append(s):
    H, Hkv, dh, ps = s["H"], s["Hkv"], s["dh"], s["ps"]
    T = s["qkv"].shape[0]
    x = s["qkv"].float().view(T, H + 2 * Hkv, dh)
    pos = s["pos"].long()
    cs = s["cs"][pos]
    c, sn = cs[:, None, :, 0], cs[:, None, :, 1]
    s["out"].copy_(_norm_rotate(x[:, :H], s["gq"], c, sn, s))
    k, v = _norm_rotate(x[:, H:H + Hkv], s["gk"], c, sn, s), x[:, H + Hkv:]
    if s["fp8"]:
        k = (k / s["k_scale"][None, :, None]).clamp(-448, 448)
        v = (v / s["v_scale"][None, :, None]).clamp(-448, 448)
    page = s["table"][s["seq"].long(), torch.div(pos, ps, rounding_mode="floor")].long()
    raw = torch.uint8 if s["fp8"] else torch.float16
    s["k"].view(raw)[page, :, pos % ps] = k.to(s["k"].dtype).view(raw)
    s["v"].view(raw)[page, :, pos % ps] = v.to(s["v"].dtype).view(raw)
    return s["out"], s["k"], s["v"]


def _attention(s):
    M, H, dh = s["q"].shape
    Hkv, ps, P = s["Hkv"], s["ps"], s["table"].shape[1]
    rows = s["table"][s["seq"].long()].long()                                # [M][P]
    at = rows.clamp(min=0)
    raw = torch.uint8 if s["fp8"] else torch.float16

    def gather(pool, scale):
        x = pool.view(raw)[at].view(pool.dtype).float()                       # [M][P][Hkv][ps][dh]
        x = x.transpose(1, 2).reshape(M, Hkv, P * ps, dh)
        return x if scale is None else x * scale[None, :, None, None]

    p = torch.arange(P * ps, device=rows.device)
    keep = (p[None] <= s["pos"][:, None]) & (rows >= 0).repeat_interleave(ps, 1)
    q = s["q"].float().view(M, Hkv, H // Hkv, dh)
    sc = torch.matmul(q, gather(s["k"], s["k_scale"]).transpose(2, 3)) / math.sqrt(dh)
    sc = torch.where(keep[:, None, None], sc, torch.full_like(sc, -math.inf))
    top = sc.amax(-1, keepdim=True)
    w = torch.exp(sc - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, gather(s["v"], s["v_scale"])) / torch.where(total == 0, torch.ones_like(total), total)
    s["out"].copy_(o.reshape(M, H * dh))
    return s["out"]


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "copy":
        pools = s["pools"].clone().view(torch.uint8)
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            pools[:, :, b] = s["pools"].view(torch.uint8)[:, :, a]
        return pools.view(s["pools"].dtype)
    if s["op"] == "append":
        H, Hkv, dh, ps, rot = s["H"], s["Hkv"], s["dh"], s["ps"], s["rot"]
        x = s["qkv"].double().view(-1, H + 2 * Hkv, dh)
        half = rot // 2
        one = [2 * i if s["inter"] else i for i in range(half)]
        two = [2 * i + 1 if s["inter"] else i + half for i in range(half)]
        pos = s["pos"].long()
        # the rotation as a complex product by the table's (float32) values
        turn = torch.view_as_complex(s["cs"].double())[pos][:, None]
        kd, vd = s["k"].double(), s["v"].double()
        outs = []
        for lo, hi, gain in ((0, H, s["gq"]), (H, H + Hkv, s["gk"])):
            y = x[:, lo:hi]
            if gain is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / dh + EPS) * gain.double()
            y = y.clone()
            z = torch.complex(y[..., one], y[..., two]) * turn
            y[..., one], y[..., two] = z.real, z.imag
            outs.append(y)
        v = x[:, H + Hkv:]
        if s["fp8"]:
            outs[1] = (outs[1] / s["k_scale"].double()[:, None]).clamp(-448, 448)
            v = (v / s["v_scale"].double()[:, None]).clamp(-448, 448)
        page = s["table"][s["seq"].long(), pos // ps].long()
        kd[page, :, pos % ps] = outs[1]
        vd[page, :, pos % ps] = v
        return outs[0], kd, vd
    M, H, dh = s["q"].shape
    Hkv, ps, G = s["Hkv"], s["ps"], H // s["Hkv"]
    out = torch.zeros(M, Hkv, G, dh, dtype=torch.float64, device=DEV)
    for m, (n, row) in enumerate(zip((s["pos"] + 1).tolist(), s["seq"].tolist())):
        if n <= 0:
            continue
        p = torch.arange(n, device=DEV)
        page = s["table"][row].long()[p // ps]
        p, page = p[page >= 0], page[page >= 0]
        if not len(p):
            continue
        K = s["k"].view(torch.uint8 if s["fp8"] else torch.float16)[page, :, p % ps].view(s["k"].dtype).double()
        V = s["v"].view(torch.uint8 if s["fp8"] else torch.float16)[page, :, p % ps].view(s["v"].dtype).double()
        if s["fp8"]:
            K, V = K * s["k_scale"].double()[:, None], V * s["v_scale"].double()[:, None]
        sc = torch.einsum("jgd,njd->jgn", s["q"][m].double().view(Hkv, G, dh), K) * dh ** -0.5
        out[m] = torch.einsum("jgn,njd->jgd", torch.softmax(sc, -1), V)
    return out.view(M, H * dh)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    e = 1 if c["fp8"] else 2
    if c["op"] == "copy":
        return {"bytes": 2 * c["n"] * 2 * c["layers"] * c["Hkv"] * c["ps"] * c["dh"] * e, "flops": 0}
    H, Hkv, dh = c["H"], c["Hkv"], c["dh"]
    if c["op"] == "append":
        T = c["T"]
        cols = (H + 2 * Hkv) * dh
        moved = T * cols * 2 + T * H * dh * 2 + T * 2 * Hkv * dh * e + min(T, c["ctx"]) * c["rot"] * 4 + T * 12
        return {"bytes": moved, "flops": T * (H + Hkv) * (dh * (4 if c["norm"] else 0) + 3 * c["rot"])}
    n = c["S"] * c["ctx"] * (0.5 if c["ragged"] else 1.0) * (11 / 12 if c["holes"] else 1.0)
    n = max(n, c["ctx"])
    return {"bytes": n * Hkv * dh * 2 * e + 4 * c["M"] * H * dh + 4 * n / c["ps"], "flops": 4 * n * H * dh}
