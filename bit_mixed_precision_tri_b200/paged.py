"""A paged key/value cache for decode steps, beside the contiguous caches of
``decode``.

Positions live in pages of a shared pool, [pages][kv heads][page size][head
dim] for K and for V, fp16 or e4m3 with one float32 scale per kv head; a table
[sequences][pages of a sequence] (int32, -1 where there is no page) says which
page holds which positions.  A call takes a batch of rows: row t is position
``pos[t]`` of sequence ``seq[t]`` (row t of sequence t without ``seq``); a
negative position or a sequence outside the table marks a padding row.

The functions marshal arguments for the library's entry points
(``tri_rope_table_scaled``, ``tri_paged_qknorm_rope``, ``tri_paged_attention``,
``tri_copy_pages``; include/tri.h states each in full) and run on the current
stream of the tensors' device.  ``PagedCache`` keeps the pools, the table and,
on the host, which pages are free and how many sequences share each.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .api import Workspace, _check_waits

RMS_EPS = 1e-5
ROPE_THETA = 5.0e5
E4M3 = torch.float8_e4m3fn


# A decode step makes these calls for every block and token, so the checks are
# kept to attribute reads: device indexes rather than device objects, one packed
# struct rather than a ctypes one.
_pack = _lib.PAGED_CACHE.pack
_raw_stream = torch._C._cuda_getCurrentRawStream
_current = torch.cuda.current_device
_FP16, _I32, _F32 = torch.float16, torch.int32, torch.float32
_WS_BYTES = {}


def _call(fn, index: int, *args) -> None:
    """fn(*args, stream) on the device's current stream, the device made the
    current one if it is not (the library launches on the current device)."""
    if _current() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st:
        _lib.check(st, fn.__name__)


def _device(first, *ts) -> int:
    """The index of the CUDA device that all the tensors live on."""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must live on a CUDA device")
    for t in ts:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must live on one CUDA device")
    return index


def _row_stride(t, rows, width, name) -> int:
    """The row stride of a fp16 tensor of `rows` rows, each of `width` contiguous elements."""
    st, sh = t.stride(), t.shape
    if t.dtype != _FP16:
        raise ValueError(f"{name} must be float16")
    if sh[0] != rows or not ((len(sh) == 2 and sh[1] == width and st[1] == 1) or
                             (len(sh) == 3 and sh[1] * sh[2] == width and st[2] == 1 and
                              (st[1] == sh[2] or sh[1] == 1))):
        raise ValueError(f"{name} must hold {rows} rows of {width} contiguous elements")
    return st[0] if rows > 1 else width


def _int32(t, n, name) -> int:
    if t.dtype != _I32 or t.numel() != n or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor with one element per row")
    return t.data_ptr()


def _gains(g, dh) -> int:
    if g.dtype != _FP16 or g.numel() != dh or not g.is_contiguous():
        raise ValueError("gains must be contiguous float16 [head dim]")
    return g.data_ptr()


def _scale(s, heads) -> int:
    if s is None or s.dtype != _F32 or s.shape != (heads,) or not s.is_contiguous():
        raise ValueError("an e4m3 cache needs k_scale and v_scale, float32 [kv heads]")
    return s.data_ptr()


def _cache(k, v, table, k_scale, v_scale):
    """(tri_paged_cache as bytes, kv heads, head dim) of two pools, a table and the scales."""
    shape, st, dtype = k.shape, k.stride(), k.dtype
    if len(shape) != 4 or v.shape != shape or v.stride() != st or v.dtype != dtype:
        raise ValueError("k and v must be alike: [pages][kv heads][page size][head dim]")
    pages, heads, size, dh = shape
    s0, s1, s2, s3 = st
    if s3 != 1 or s2 != dh or (s1 != size * dh and heads > 1):
        raise ValueError("the heads of a page must be contiguous")
    if table.dtype != _I32 or table.dim() != 2:
        raise ValueError("the page table must be int32 [sequences][pages] with contiguous rows")
    (seqs, width), (t0, t1) = table.shape, table.stride()
    if t1 != 1 and width > 1:
        raise ValueError("the page table must be int32 [sequences][pages] with contiguous rows")
    if dtype == _FP16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("scales belong to an e4m3 cache")
        ks, vs, code = 0, 0, _lib.CACHE_F16
    elif dtype == E4M3:
        ks, vs, code = _scale(k_scale, heads), _scale(v_scale, heads), _lib.CACHE_E4M3
    else:
        raise ValueError("a cache is float16 or float8_e4m3fn")
    return _pack(k.data_ptr(), v.data_ptr(), ks, vs, table.data_ptr(), pages, size,
                 s0 if pages > 1 else heads * size * dh, heads, dh, seqs, width, t0 if seqs > 1 else width,
                 code), heads, dh


# ---------------------------------------------------------------- operators
def rope_table(Lmax: int, device, rot: int = 128, theta: float = ROPE_THETA, scaling: str = None, factor: float = 1.0,
               context: float = 0.0, low: float = 1.0, high: float = 4.0) -> torch.Tensor:
    """(cos, sin) of the angles of `rot` rotated features, float32 [Lmax][rot/2][2].

    ``scaling`` stretches the angles for long contexts: "linear" (divided by
    ``factor``), "ntk" (theta raised so that the slowest pair is stretched by
    it), "bands" (pairs that turn more than ``high`` times in ``context``
    positions are kept, fewer than ``low`` times stretched, smooth in between)
    or "ramp" (linear in the pair's index between the pairs that turn ``high``
    and ``low`` times; cos and sin grow by 0.1 ln(factor) + 1)."""
    if scaling is not None and scaling not in _lib.ROPE_KINDS:
        raise ValueError(f"scaling is None or one of {sorted(_lib.ROPE_KINDS)}")
    # `device` may be a bare "cuda": the tensor's own device has the index
    cs = torch.empty(Lmax, rot // 2, 2, dtype=torch.float32, device=device)
    index = _device(cs)
    sc = None
    if scaling is not None:
        sc = ctypes.byref(_lib.RopeScaling(_lib.ROPE_KINDS[scaling], factor, context, low, high))
    _call(_lib.lib().tri_rope_table_scaled, index, cs.data_ptr(), Lmax, rot, float(theta), sc)
    return cs


def qknorm_rope_append(qkv: torch.Tensor, pos: torch.Tensor, gq, gk, cs: torch.Tensor, k: torch.Tensor,
                       v: torch.Tensor, table: torch.Tensor, H: int, seq: torch.Tensor = None,
                       interleaved: bool = False, k_scale: torch.Tensor = None, v_scale: torch.Tensor = None,
                       eps: float = RMS_EPS, out: torch.Tensor = None, check: bool = False) -> torch.Tensor:
    """Queries [T][H][dh] of the fused QKV rows [T][(H + 2 Hkv) dh], normed
    (unless gq and gk are None) and rotated; keys (normed, rotated) and values
    written into the pages of their rows.  ``cs`` is a table of
    ``rope_table`` ([positions][rot/2][2]); the first rot features rotate.

    ``check=True`` (for debugging; it synchronizes the stream) reads the device's
    wait status word after the call and raises WaitGaveUp if a bounded wait
    inside the kernel ran out."""
    index = _device(qkv, pos, gq, gk, cs, k, v, table, seq, k_scale, v_scale, out)
    cache, heads, dh = _cache(k, v, table, k_scale, v_scale)
    if qkv.dim() != 2:
        raise ValueError("qkv must be [rows][(H + 2 Hkv) * head dim]")
    T = len(qkv)
    stride = _row_stride(qkv, T, (H + 2 * heads) * dh, "qkv")
    angles = cs.shape
    if cs.dtype != _F32 or len(angles) != 3 or angles[2] != 2 or not cs.is_contiguous():
        raise ValueError("cs must be a contiguous float32 table [positions][rot / 2][2]")
    gq_p = None if gq is None else _gains(gq, dh)
    gk_p = None if gk is None else _gains(gk, dh)
    q = out if out is not None else torch.empty(T, H, dh, dtype=_FP16, device=qkv.device)
    q_stride = _row_stride(q, T, H * dh, "out")
    pos_p, seq_p = _int32(pos, T, "pos"), None if seq is None else _int32(seq, T, "seq")
    if T == 0:
        return q
    _call(_lib.lib().tri_paged_qknorm_rope, index, qkv.data_ptr(), stride, pos_p, seq_p, gq_p, gk_p, cs.data_ptr(),
          angles[0], 2 * angles[1], 1 if interleaved else 0, q.data_ptr(), q_stride, cache, T, H, eps)
    if check:
        _check_waits(qkv.device, _raw_stream(index), "tri_paged_qknorm_rope")
    return q


def attention_workspace_bytes(M: int, H: int, Hkv: int, head_dim: int = 128) -> int:
    """What ``attention_decode`` needs of a workspace on the current device; 0 for
    shapes that it refuses."""
    return int(_lib.lib().tri_paged_attention_workspace_bytes(M, H, Hkv, head_dim))


def attention_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, pos: torch.Tensor,
                     seq: torch.Tensor = None, k_scale: torch.Tensor = None, v_scale: torch.Tensor = None,
                     scale: float = None, out: torch.Tensor = None, workspace: Workspace = None,
                     check: bool = False) -> torch.Tensor:
    """softmax(scale K q) V over positions 0..pos[m] of sequence seq[m] whose
    page is present (zeros where nothing is left); q [M][H][dh] -> [M][H * dh].
    ``scale`` defaults to 1 / sqrt(dh).  Without ``workspace`` each call takes
    its scratch from the caching allocator, so that calls on other streams and
    in captured graphs never share one.  ``check`` as in ``qknorm_rope_append``."""
    index = _device(q, k, v, table, pos, seq, k_scale, v_scale, out)
    cache, heads, dh = _cache(k, v, table, k_scale, v_scale)
    shape = q.shape
    if len(shape) != 3 or shape[2] != dh:
        raise ValueError("q must be [rows][heads][head dim]")
    M, H, _ = shape
    stride = _row_stride(q, M, H * dh, "q")
    y = out if out is not None else torch.empty(M, H * dh, dtype=_FP16, device=q.device)
    out_stride = _row_stride(y, M, H * dh, "out")
    pos_p, seq_p = _int32(pos, M, "pos"), None if seq is None else _int32(seq, M, "seq")
    if M == 0:
        return y
    L = _lib.lib()
    key = (M, H, heads, dh, index)
    nbytes = _WS_BYTES.get(key)
    if nbytes is None:
        if len(_WS_BYTES) > 4096:
            _WS_BYTES.clear()
        with torch.cuda.device(index):
            nbytes = _WS_BYTES[key] = attention_workspace_bytes(M, H, heads, dh) or 256
    ws = workspace.get(nbytes) if workspace is not None else torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    if ws.get_device() != index:
        raise ValueError("the workspace must live on the tensors' device")
    _call(L.tri_paged_attention, index, q.data_ptr(), stride, pos_p, seq_p, cache, y.data_ptr(), out_stride, M, H,
          dh ** -0.5 if scale is None else scale, ws.data_ptr(), ws.numel())
    if check:
        _check_waits(q.device, _raw_stream(index), "tri_paged_attention")
    return y


def copy_pages(pools: torch.Tensor, src, dst) -> None:
    """Page dst[i] of every pool becomes a copy of page src[i].

    ``pools`` is [..., pages][kv heads][page size][head dim] with one or more
    leading dimensions of pools (layers, K and V).  ``src`` and ``dst`` are
    sequences of page numbers, checked here (in range, no page twice in dst or
    in both), or int32 tensors on the device, which are not looked at on the
    host: pairs outside the pool are skipped, pages named twice end up with
    unspecified bytes."""
    index = _device(pools)
    shape, strides = pools.shape, pools.stride()
    if len(shape) < 4:
        raise ValueError("pools must be [..., pages][kv heads][page size][head dim]")
    pages, heads, size, dh = shape[-4:]
    if strides[-1] != 1 or strides[-2] != dh or (strides[-3] != size * dh and heads > 1):
        raise ValueError("the heads of a page must be contiguous")
    n_pools, pool_stride = 1, 0
    for extent, stride in zip(reversed(shape[:-4]), reversed(strides[:-4])):
        if extent == 1:
            continue
        if n_pools == 1:
            pool_stride = stride
        elif stride != pool_stride * n_pools:
            raise ValueError("the pools must lie at one stride")
        n_pools *= extent
    if torch.is_tensor(src) and torch.is_tensor(dst):
        _device(pools, src, dst)
        n = src.shape[0] if src.dim() else 0
        src_p, dst_p = _int32(src, n, "src"), _int32(dst, n, "dst")
    else:
        src, dst = [int(a) for a in src], [int(b) for b in dst]
        n = len(src)
        if len(dst) != n:
            raise ValueError("src and dst must have the same length")
        if any(not 0 <= a < pages for a in src + dst):
            raise ValueError("page number out of range")
        if len(set(dst)) < n or set(src) & set(dst):
            raise ValueError("a page stands twice in dst, or in both src and dst")
        both = torch.tensor([src, dst], dtype=_I32).to(pools.device)
        src_p, dst_p = both.data_ptr(), both.data_ptr() + 4 * n
    if n == 0 or n_pools == 0 or pages == 0:
        return
    e = pools.element_size()
    page_bytes = heads * size * dh * e
    _call(_lib.lib().tri_copy_pages, index, pools.data_ptr(), n_pools, pool_stride * e, pages,
          strides[-4] * e if pages > 1 else page_bytes, page_bytes, src_p, dst_p, n)


# ---------------------------------------------------------------- the cache
class CacheFull(RuntimeError):
    """The pool has too few free pages, or the table too few rows or columns;
    nothing was changed."""


class PageBook:
    """Which pages each sequence holds (host only): pages are shared by counting.

    Rows are written at positions that ``extend`` made room for after the
    sequence was last forked, or that ``own`` was called for: no page that more
    than one sequence holds is written then.  The book cannot see writes, so
    whoever forks a sequence with positions that are not written yet says so.

    Every method that changes what the device must see returns the copies
    (source and destination pages) to be made before the next write."""

    def __init__(self, num_pages: int, page_size: int, max_seqs: int, seq_pages: int):
        self.num_pages, self.page_size, self.max_seqs, self.seq_pages = num_pages, page_size, max_seqs, seq_pages
        self.count = [0] * num_pages                       # sequences that hold each page
        self.free_pages = list(range(num_pages - 1, -1, -1))   # the lowest comes off first
        self.free_seqs = list(range(max_seqs - 1, -1, -1))
        self.pages = {}                                    # sequence -> its pages (-1: dropped)
        self.length = {}                                   # sequence -> positions

    def _take(self) -> int:
        p = self.free_pages.pop()
        self.count[p] = 1
        return p

    def _drop(self, p: int) -> None:
        if p >= 0:
            self.count[p] -= 1
            if self.count[p] == 0:
                self.free_pages.append(p)

    def new(self) -> int:
        if not self.free_seqs:
            raise CacheFull("no free row in the page table")
        s = self.free_seqs.pop()
        self.pages[s], self.length[s] = [], 0
        return s

    def extend(self, s: int, n: int):
        """Room for n more positions of s; the page that the first of them falls
        into is copied if another sequence holds it too."""
        if n < 0:
            raise ValueError("n must not be negative")
        held, L = self.pages[s], self.length[s]
        need = -(-(L + n) // self.page_size)
        if need > self.seq_pages:
            raise CacheFull("the sequence outgrows its row of the page table")
        last = L // self.page_size                          # the page of the next position
        # a page that is not full is held: drop_front gives up full ones only
        split = n > 0 and L % self.page_size > 0 and self.count[held[last]] > 1
        if max(0, need - len(held)) + split > len(self.free_pages):
            raise CacheFull("no free pages")
        src, dst = [], []
        if split:
            old = held[last]
            held[last] = self._take()
            self._drop(old)
            src, dst = [old], [held[last]]
        while len(held) < need:
            held.append(self._take())
        self.length[s] = L + n
        return src, dst

    def fork(self, s: int) -> int:
        """A new sequence that shares every page of s."""
        if not self.free_seqs:
            raise CacheFull("no free row in the page table")
        held = list(self.pages[s])                          # before the row is taken: s may not exist
        t = self.new()
        self.pages[t], self.length[t] = held, self.length[s]
        for p in self.pages[t]:
            if p >= 0:
                self.count[p] += 1
        return t

    def own(self, s: int, first: int):
        """Positions of s from `first` to its end are to be written: their pages that
        another sequence holds too are exchanged for own ones, the first of which
        is copied where it holds positions below `first`."""
        if first < 0 or first > self.length[s]:
            raise ValueError("first must be between 0 and the sequence's length")
        held = self.pages[s] if first < self.length[s] else []
        shared = [i for i in range(first // self.page_size, len(held)) if held[i] >= 0 and self.count[held[i]] > 1]
        if len(shared) > len(self.free_pages):
            raise CacheFull("no free pages")
        src, dst = [], []
        for i in shared:
            old, held[i] = held[i], self._take()
            self._drop(old)
            if i * self.page_size < first:
                src, dst = [old], [held[i]]
        return src, dst

    def drop_front(self, s: int, n: int) -> None:
        """Give up the pages that hold only positions below n."""
        if n < 0 or n > self.length[s]:
            raise ValueError("n must be between 0 and the sequence's length")
        for i in range(min(n // self.page_size, len(self.pages[s]))):
            self._drop(self.pages[s][i])
            self.pages[s][i] = -1

    def free(self, s: int) -> None:
        for p in self.pages.pop(s):
            self._drop(p)
        del self.length[s]
        self.free_seqs.append(s)

    def compact(self):
        """Move the held pages to the front of the pool."""
        live = sum(c > 0 for c in self.count)
        holes = [p for p in range(live) if self.count[p] == 0]
        src = [p for p in range(live, self.num_pages) if self.count[p] > 0]
        to = dict(zip(src, holes))
        for held in self.pages.values():
            held[:] = [to.get(p, p) for p in held]
        for a, b in to.items():
            self.count[b], self.count[a] = self.count[a], 0
        self.free_pages = list(range(self.num_pages - 1, live - 1, -1))
        return src, holes


class PagedCache:
    """Key/value pages of `layers` blocks and the sequences in them.

    ``pools`` [layers][2][pages][kv heads][page size][head dim] on the device;
    ``table`` int32 [max_seqs][seq_pages] on the device, one row per sequence
    handle.  ``new``, ``extend``, ``fork``, ``drop_front``, ``free`` and
    ``compact`` keep the host's book and bring the table (and copied pages) up to
    date on the current stream; a step in between, captured or not, reads
    them.  e4m3 pools take ``k_scale`` and ``v_scale``, float32 [layers][kv heads]."""

    def __init__(self, num_pages: int, Hkv: int, max_seqs: int, seq_pages: int, device, layers: int = 1,
                 page_size: int = 64, head_dim: int = 128, dtype=torch.float16, k_scale: torch.Tensor = None,
                 v_scale: torch.Tensor = None):
        if dtype not in (torch.float16, E4M3):
            raise ValueError("a cache is float16 or float8_e4m3fn")
        if page_size not in (8, 16, 32, 64, 128, 256) or head_dim not in (64, 128):
            raise ValueError("page_size is a power of two from 8 to 256, head_dim 64 or 128")
        if min(num_pages, Hkv, max_seqs, seq_pages, layers) < 1:
            raise ValueError("sizes must be positive")
        if [k_scale is not None, v_scale is not None] != [dtype == E4M3] * 2:
            raise ValueError("an e4m3 cache, and no other, takes k_scale and v_scale")
        self.device = torch.device(device)
        self.layers, self.page_size = layers, page_size
        self.pools = torch.zeros(layers, 2, num_pages, Hkv, page_size, head_dim, dtype=torch.float16,
                                 device=self.device) if dtype == torch.float16 else torch.zeros(
            layers, 2, num_pages, Hkv, page_size, head_dim, dtype=torch.uint8, device=self.device).view(E4M3)
        self.scales = None
        if dtype == E4M3:
            self.scales = torch.stack([k_scale.expand(layers, Hkv), v_scale.expand(layers, Hkv)]).to(
                self.device, torch.float32).contiguous()
        self.table = torch.full((max_seqs, seq_pages), -1, dtype=torch.int32, device=self.device)
        self.book = PageBook(num_pages, page_size, max_seqs, seq_pages)

    def layer(self, i: int):
        """(k, v, k_scale, v_scale) of block i."""
        if self.scales is None:
            return self.pools[i, 0], self.pools[i, 1], None, None
        return self.pools[i, 0], self.pools[i, 1], self.scales[0, i], self.scales[1, i]

    @property
    def free_pages(self) -> int:
        return len(self.book.free_pages)

    def length(self, s: int) -> int:
        return self.book.length[s]

    def _sync(self, *seqs) -> None:
        rows = torch.full((len(seqs), self.table.shape[1]), -1, dtype=torch.int32)
        for i, s in enumerate(seqs):
            held = self.book.pages.get(s, ())
            if held:
                rows[i, :len(held)] = torch.tensor(held, dtype=torch.int32)
        # pageable memory: the copies have left `rows` when these calls return
        for i, s in enumerate(seqs):
            self.table[s].copy_(rows[i])

    def new(self, n: int = 0) -> int:
        """A new sequence with room for n positions; its handle is its table row."""
        s = self.book.new()
        try:
            self.book.extend(s, n)
        except (CacheFull, ValueError):
            self.book.free(s)
            raise
        self._sync(s)
        return s

    def extend(self, s: int, n: int = 1) -> None:
        """Room for n more positions of s.  A shared page that they fall into is copied."""
        before = len(self.book.pages[s])
        src, dst = self.book.extend(s, n)
        if src:
            copy_pages(self.pools, src, dst)
        if src or len(self.book.pages[s]) != before:
            self._sync(s)

    def fork(self, s: int, written: int = None) -> int:
        """A new sequence that continues s: the two share s's pages, and ``extend``
        copies the one that they would both write into.  All positions of s must
        have been written before the fork; where room was made for more, ``written``
        says how many are, and the new sequence gets own pages for the others (the
        page that holds both kinds is copied)."""
        t = self.book.fork(s)
        if written is not None:
            try:
                src, dst = self.book.own(t, written)
            except (CacheFull, ValueError):
                self.book.free(t)
                raise
            if src:
                copy_pages(self.pools, src, dst)
        self._sync(t)
        return t

    def drop_front(self, s: int, n: int) -> None:
        """Give up the pages that hold only positions below n; attention passes over them."""
        self.book.drop_front(s, n)
        self._sync(s)

    def free(self, s: int) -> None:
        self.book.free(s)
        self._sync(s)

    def compact(self) -> int:
        """Move the held pages to the front of the pool; how many moved."""
        src, dst = self.book.compact()
        if src:
            copy_pages(self.pools, src, dst)
            self._sync(*sorted(self.book.pages))
        return len(src)
