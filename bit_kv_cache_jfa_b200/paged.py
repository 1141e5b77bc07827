"""The paged 4-bit cache and the head norms and rotary positions in front of
it: argument checks, device buffers and the host's page book-keeping over the
jfa_paged_* and jfa_qk_norm_rope calls.

    table = PageTable(batch, n_pages, max_pages)        # one for all layers
    cache = PagedKVCache(table, heads, kv_heads)        # one per layer
    ws = PagedWorkspace(cache)
    cu = table.grow([700, 1300])                        # prompts enter
    paged_append(cache, k, v, ws, cu)
    table.grow(1)                                       # then a token each
    out = paged_decode_step(cache, q, k, v, table.seq_lens - 1, plan, ws)

Unlike the calls on contiguous caches, these launch on torch's current stream
when no stream is given, and on the device that holds the cache.  What a call
allocates belongs to the stream it runs on.
"""
from __future__ import annotations

import ctypes
import heapq
import math
import numbers
import operator

import torch

from . import _lib
from ._lib import JFA_ERR_INVALID_ARG, JfaError, Paged, Rope, check

_BF16 = torch.bfloat16
_SCALE = 1.0 / math.sqrt(_lib.HEAD_DIM)
_INT_MAX = 2**31 - 1   # the library's counts are of 32 bits


def _refuse(where: str, why: str):
    raise JfaError(JFA_ERR_INVALID_ARG, f"{where}: {why}")


def _handle(dev, stream):
    """Handle of a call's stream: the given one, else torch's current one on dev."""
    if stream is None:
        return _raw_stream(dev.index) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _run(where, dev, stream, *args):
    """Call the library's ``where`` on dev and ``stream``.  These calls take
    microseconds on the device: what the host adds is kept small (one look at
    the current device and stream, no context manager when dev is current)."""
    if dev.index is None:
        _refuse(where, f"needs a CUDA device, not {dev}")
    fn = _calls.get(where)
    if fn is None:
        fn = _calls[where] = getattr(_lib.load(), where)
    st = _handle(dev, stream)
    if _current_device() == dev.index:
        status = fn(*args, st)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, st)
    if status:
        check(status, where)


_calls = {}
# The current device without the check that CUDA is up (every tensor here is on one).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
# The handle of a device's current stream without a Stream object (2 us) around it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _int32(x, n, dev, where, name):
    if x.dtype != torch.int32 or x.numel() != n or not x.is_contiguous() or x.device != dev:
        _refuse(where, f"{name} must be {n} contiguous int32 on {dev}")
    return x.data_ptr()


def _rows(x, heads, dev, where, name):
    """Address and strides of bf16 rows [T][heads][128]."""
    shape, strides = x.shape, x.stride()
    if x.dtype != _BF16 or len(shape) != 3 or shape[1] != heads or shape[2] != 128 or x.device != dev \
            or (strides[2] != 1 and x.numel()) or shape[0] > _INT_MAX:
        _refuse(where, f"{name} must be bf16 [tokens, {heads}, {_lib.HEAD_DIM}] on {dev}, channels contiguous, "
                       "of fewer than 2^31 tokens")
    # the stride of a dimension of one element means nothing
    return x.data_ptr(), strides[0] if shape[0] > 1 else 0, strides[1] if heads > 1 else 0


def _overlap(s0, n0, s1, n1):
    """Whether any two of the n0 * n1 rows of 128 elements at i s0 + j s1 share one."""
    if s0 > s1:
        s0, n0, s1, n1 = s1, n1, s0, n0
    reach = s0 * (n0 - 1) + 128           # of the rows along the smaller stride
    if n0 > 1 and s0 < 128:
        return True
    if n1 == 1 or s1 >= reach:
        return False
    if n0 == 1:
        return True
    # rows j apart along s1 are i or i + 1 strides s0 off at the nearest
    for j in range(1, n1):
        if j * s1 >= reach:
            return False
        i = j * s1 // s0
        if j * s1 - i * s0 < 128 or (i + 1 < n0 and (i + 1) * s0 - j * s1 < 128):
            return True
    return False


def _out_rows(x, like, heads, dev, where, name):
    """_rows of an output: its input's shape, no two rows in one place."""
    if x.shape != like.shape:
        _refuse(where, f"{name} must have its input's shape")
    at = _rows(x, heads, dev, where, name)
    if x.numel() and _overlap(at[1], x.shape[0], at[2], heads):
        _refuse(where, f"{name} must not overlap itself")
    return at


def _fresh(make, stream, dev):
    """make(), an output, from the memory of the call's stream."""
    if dev.index is None:
        _refuse("stream", f"needs a CUDA device, not {dev}")
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    with torch.cuda.stream(stream):
        return make()


def _like(x, stream, dev):
    """An output like x, contiguous."""
    if stream is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    return _fresh(lambda: _like(x, None, dev), stream, dev)


def _given(x, shape, dev, where, name):
    if x.shape != shape or x.dtype != _BF16 or x.device != dev or not x.is_contiguous():
        _refuse(where, f"{name} must be contiguous bf16 {list(shape)} on {dev}")


def _device(device):
    dev = torch.device(device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    return dev


def _weight(w, dev, where, name):
    if w.dtype != _BF16 or w.shape != (_lib.HEAD_DIM,) or w.device != dev or not w.is_contiguous():
        _refuse(where, f"{name} must be bf16 [{_lib.HEAD_DIM}] on {dev}")
    return w.data_ptr()


class RotaryPlan:
    """Frequencies of the rotary positions of a model, on the device.

    rotary_dim: channels that turn (even, at most 128); interleaved: pairs
    (2i, 2i + 1) instead of (i, i + rotary_dim / 2).  f_i = base^(-2i / rotary_dim),
    changed by ``scaling``:

    - "none"
    - "linear": f / factor
    - "llama3": f / factor where the wavelength is over original /
      low_freq_factor, f where it is under original / high_freq_factor, in
      between a blend that is linear in original / wavelength
    - "yarn": a blend of f / factor and f that is linear in i between the
      pairs that make beta_slow and beta_fast turns in the original context;
      rotated channels grow by amplitude = 0.1 ln(factor) + 1

    ``amplitude`` replaces the scaling's own."""

    def __init__(self, rotary_dim: int = 128, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, low_freq_factor: float = 1.0,
                 high_freq_factor: float = 4.0, original: int | None = None,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, amplitude: float | None = None,
                 device="cuda"):
        where = "RotaryPlan"
        if rotary_dim % 2 or not 2 <= rotary_dim <= _lib.HEAD_DIM:
            _refuse(where, f"rotary_dim must be even, in 2..{_lib.HEAD_DIM}")
        if not base > 1 or not factor > 0:
            _refuse(where, "base must be above 1 and factor above 0")
        if scaling not in ("none", "linear", "llama3", "yarn"):
            _refuse(where, f"unknown scaling {scaling!r}")
        if scaling in ("llama3", "yarn") and not (original and original > 0):
            _refuse(where, f"scaling {scaling!r} needs the original context length")
        if scaling == "llama3" and not high_freq_factor > low_freq_factor:
            _refuse(where, "high_freq_factor must be above low_freq_factor")
        if scaling == "yarn" and not beta_fast > beta_slow > 0:
            _refuse(where, "beta_fast must be above beta_slow, and that above 0")
        if scaling == "yarn" and not all(math.isfinite(x) for x in (base, original, beta_fast)):
            _refuse(where, "base, original and beta_fast must be finite")
        self.rotary_dim, self.interleaved = rotary_dim, bool(interleaved)
        half = rotary_dim // 2
        f = [base ** (-2.0 * i / rotary_dim) for i in range(half)]
        m = 1.0
        if scaling == "linear":
            f = [x / factor for x in f]
        elif scaling == "llama3":
            keep = [(original * x / (2 * math.pi) - low_freq_factor) / (high_freq_factor - low_freq_factor)
                    for x in f]
            keep = [min(max(u, 0.0), 1.0) for u in keep]
            f = [x * (u + (1 - u) / factor) for x, u in zip(f, keep)]
        elif scaling == "yarn":
            def pair(turns):  # that makes so many turns in the original context
                return rotary_dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo = max(math.floor(pair(beta_fast)), 0)
            hi = min(math.ceil(pair(beta_slow)), rotary_dim - 1)
            ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(half)]
            f = [x * (1 - u + u / factor) for x, u in zip(f, ramp)]
            m = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
        if not all(math.isfinite(x * 2.0**64) for x in f):
            _refuse(where, "frequencies must be finite, and below 2^960")
        self.frequencies = tuple(f)          # radians per position
        self.amplitude = float(m if amplitude is None else amplitude)
        if not math.isfinite(ctypes.c_float(self.amplitude).value):
            _refuse(where, "amplitude must be finite in 32 bits")
        turns = [round(x / (2 * math.pi) * 2.0**64) % 2**64 for x in f]   # in 2^-64 turns
        self.freq = torch.tensor([t - 2**64 if t >= 2**63 else t for t in turns], dtype=torch.int64,
                                 device=_device(device))
        self.freq_ptr = self.freq.data_ptr()


def qk_norm_rope(q, k, positions, plan: RotaryPlan, q_weight=None, k_weight=None, eps: float = 1e-6,
                 q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head (where a weight is given) and
    rotation by position, in one pass.

    q bf16 [T, H, 128], k bf16 [T, H_kv, 128] (any token and head strides that
    are multiples of 8, channels contiguous); positions int32 or int64 [T];
    weights bf16 [128].  Returns (q, k) bf16, contiguous unless given; q_out=q
    and k_out=k work in place, and otherwise an output may overlap neither an
    input nor the other output."""
    where = "qk_norm_rope"
    dev = plan.freq.device
    qs, ks = q.shape, k.shape
    if len(qs) != 3 or len(ks) != 3 or qs[0] != ks[0]:
        _refuse(where, "q and k must be [tokens, heads, 128] of the same tokens")
    t, h, hkv = qs[0], qs[1], ks[1]
    qp, q_tok, q_head = _rows(q, h, dev, where, "q")
    kp, k_tok, k_head = _rows(k, hkv, dev, where, "k")
    wide = positions.dtype == torch.int64
    if not (wide or positions.dtype == torch.int32) or positions.shape != (t,) or positions.device != dev \
            or not positions.is_contiguous():
        _refuse(where, f"positions must be {t} contiguous int32 or int64 on {dev}")
    qw = None if q_weight is None else _weight(q_weight, dev, where, "q_weight")
    kw = None if k_weight is None else _weight(k_weight, dev, where, "k_weight")
    if q_out is None:
        q_out = _like(q, stream, dev)
        qop, qo_tok, qo_head = q_out.data_ptr(), h * 128, 128
    else:
        qop, qo_tok, qo_head = _out_rows(q_out, q, h, dev, where, "q_out")
    if k_out is None:
        k_out = _like(k, stream, dev)
        kop, ko_tok, ko_head = k_out.data_ptr(), hkv * 128, 128
    else:
        kop, ko_tok, ko_head = _out_rows(k_out, k, hkv, dev, where, "k_out")
    r = Rope(t, h, hkv, plan.rotary_dim, plan.interleaved, wide, eps, plan.amplitude, qp, kp, qop, kop, q_tok,
             q_head, k_tok, k_head, qo_tok, qo_head, ko_tok, ko_head, qw, kw, positions.data_ptr(),
             plan.freq_ptr)
    _run("jfa_qk_norm_rope", dev, stream, ctypes.byref(r))
    return q_out, k_out


class PageTable:
    """Pages of the sequences of a batch: the device table and lengths that
    the kernels read, and the host's book of free and shared pages.  Layers
    with the same sequences share one table (a pool of pages each).

    A page is written when its 64 tokens are complete and never again, so
    forked sequences share it by count; it is free once no sequence lists it.
    Updates are enqueued on torch's current stream."""

    def __init__(self, batch: int, n_pages: int, max_pages: int, device="cuda"):
        if not 1 <= batch <= _lib.MAX_BATCH or not 1 <= n_pages <= _INT_MAX or not 1 <= max_pages <= _INT_MAX:
            _refuse("PageTable", f"batch must be 1..{_lib.MAX_BATCH}, n_pages and max_pages 1 or more, and below 2^31")
        self.batch, self.n_pages, self.max_pages = batch, n_pages, max_pages
        self.device = _device(device)
        self.table = torch.full((batch, max_pages), -1, dtype=torch.int32, device=self.device)
        self.seq_lens = torch.zeros(batch, dtype=torch.int32, device=self.device)
        self.lens = [0] * batch                       # as seq_lens
        self.rows = [[] for _ in range(batch)]        # pages of each sequence
        self._refs = [0] * n_pages
        self._free = list(range(n_pages))             # heap: the lowest page goes out first

    @property
    def free_pages(self) -> int:
        return len(self._free)

    @staticmethod
    def _packed(n: int) -> int:
        return 0 if n <= 0 else (n - 1) // _lib.KEY_GROUP

    def _check_row(self, row, where):
        if not 0 <= row < self.batch:
            _refuse(where, f"sequence {row} of {self.batch}")

    def _up(self, values):
        """Host ints to the device, ordered on the current stream."""
        return torch.tensor(values, dtype=torch.int32).to(self.device, non_blocking=True)

    def _store(self, cells=(), pages=()):
        """Lengths, and table cells (row * max_pages + entry) with their pages."""
        m = len(cells)
        up = self._up([*self.lens, *cells, *pages])
        self.seq_lens.copy_(up[:self.batch])
        if m:
            self.table.view(-1)[up[self.batch:self.batch + m].long()] = up[self.batch + m:]

    def grow(self, n_new):
        """Room for new tokens: n_new of every sequence that has any (int), or
        n_new[b] of sequence b.  Lengths grow and the groups that become
        complete get pages; paged_append then brings the rows.  Returns the
        rows' ranges (int32 [batch + 1] on the device) for the second form.
        Without enough free pages or room in a row nothing changes."""
        uniform = isinstance(n_new, numbers.Integral)
        n_new = int(n_new) if uniform else n_new
        counts = [n_new if n else 0 for n in self.lens] if uniform else [int(n) for n in n_new]
        if len(counts) != self.batch or min(counts) < 0:
            _refuse("PageTable.grow", f"needs {self.batch} counts, none negative")
        need = []
        for b, n in enumerate(counts):
            first, last = self._packed(self.lens[b]), self._packed(self.lens[b] + n)
            if last > self.max_pages:
                _refuse("PageTable.grow", f"sequence {b} would need {last} of {self.max_pages} pages")
            need += [(b, g) for g in range(first, last)]
        if len(need) > len(self._free):
            _refuse("PageTable.grow", f"{len(need)} pages needed, {len(self._free)} free")
        cells, pages = [], []
        for b, g in need:
            page = heapq.heappop(self._free)
            self._refs[page] = 1
            self.rows[b].append(page)
            cells.append(b * self.max_pages + g)
            pages.append(page)
        self.lens = [a + n for a, n in zip(self.lens, counts)]
        self._store(cells, pages)
        if uniform:
            return None
        return torch.cat((torch.zeros(1, dtype=torch.int32, device=self.device),
                          self._up(counts).cumsum(0, dtype=torch.int32)))

    def _release(self, row):
        for page in self.rows[row]:
            self._refs[page] -= 1
            if self._refs[page] == 0:
                heapq.heappush(self._free, page)
        self.rows[row] = []
        self.lens[row] = 0

    def free(self, rows) -> None:
        """Sequences end: their rows become idle (length 0), pages that no
        other sequence lists become free."""
        rows = [int(r) for r in rows]
        for r in rows:
            self._check_row(r, "PageTable.free")
        for r in rows:
            self._release(r)
        self._store()

    def fork(self, pairs):
        """Book (parent, child) forks; a child's earlier pages are released.
        Returns the pairs (int32 [n, 2] on the device) for paged_fork, which
        every layer's cache gets before the table changes again."""
        pairs = [(int(a), int(b)) for a, b in pairs]
        children = [b for _, b in pairs]
        for a, b in pairs:
            self._check_row(a, "PageTable.fork")
            self._check_row(b, "PageTable.fork")
        if len(set(children)) != len(children) or set(children) & {a for a, _ in pairs}:
            _refuse("PageTable.fork", "a child may be no parent and the child of one pair only")
        for _, b in pairs:
            self._release(b)
        for a, b in pairs:
            self.rows[b] = list(self.rows[a])
            self.lens[b] = self.lens[a]
            for page in self.rows[b]:
                self._refs[page] += 1
        return self._up([x for p in pairs for x in p]).view(-1, 2)

    def compact(self):
        """Book the move of the pages in use to the front of the pool.  Returns
        (moves int32 [m, 2], remap int32 [n_pages]) on the device for
        paged_move: every layer's cache gets the moves, one of them the remap,
        before the table changes again."""
        used = [p for p in range(self.n_pages) if self._refs[p]]
        holes = [p for p in range(len(used)) if not self._refs[p]]
        goes = list(range(self.n_pages))
        moves = list(zip(used[len(used) - len(holes):], holes))
        for a, b in moves:
            goes[a] = b
            self._refs[b], self._refs[a] = self._refs[a], 0
        self.rows = [[goes[p] for p in row] for row in self.rows]
        self._free = list(range(len(used), self.n_pages))
        up = self._up([*goes, *(x for m in moves for x in m)])
        return up[self.n_pages:].view(-1, 2), up[:self.n_pages]


class PagedKVCache:
    """One layer's paged 4-bit cache (device buffers owned by torch, fixed for
    its life): the pool of pages and the exact tail of each sequence."""

    def __init__(self, table: PageTable, num_heads: int, num_kv_heads: int):
        self.table, self.device = table, table.device
        self.num_heads, self.num_kv_heads = num_heads, num_kv_heads
        if max(num_heads, num_kv_heads) > _INT_MAX:
            _refuse("PagedKVCache", "num_heads and num_kv_heads must be below 2^31")
        # sizes first: a bad geometry is refused before anything is allocated
        self._struct = Paged(table.batch, num_heads, num_kv_heads, table.n_pages, table.max_pages)
        self.workspace_bytes = _lib.jfa_paged_workspace_bytes(self._struct)
        self.pages = torch.zeros(table.n_pages, num_kv_heads, _lib.PAGE_RECORD_BYTES, dtype=torch.uint8,
                                 device=self.device)
        shape = (table.batch, num_kv_heads, _lib.TAIL_MAX, _lib.HEAD_DIM)
        self.tail_k = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
        self.tail_v = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
        s = self._struct
        s.pages, s.tail_k, s.tail_v = (x.data_ptr() for x in (self.pages, self.tail_k, self.tail_v))
        s.table, s.seq_lens = table.table.data_ptr(), table.seq_lens.data_ptr()

        self._ref = ctypes.byref(s)
        self.sizes = (table.batch, num_kv_heads)

    def struct(self) -> Paged:
        return self._struct

    def record(self, page: int, head: int) -> bytes:
        """Host bytes of a page's record of one KV head (jfa_unpack_record decodes it)."""
        return self.pages[page, head].cpu().numpy().tobytes()


class PagedWorkspace:
    """Scratch of the paged calls on one cache, or on caches of as many
    sequences and KV heads on its device.  Calls that may run at the same time
    need one each."""

    def __init__(self, cache: PagedKVCache):
        self.buf = torch.zeros(cache.workspace_bytes, dtype=torch.uint8, device=cache.device)
        self.ptr, self.device = self.buf.data_ptr(), self.buf.device
        self.sizes = (cache.table.batch, cache.num_kv_heads)

    def error_flag(self, cache: PagedKVCache, stream=None) -> int:
        if cache.device.index is None:
            _refuse("jfa_paged_check_error", f"needs a CUDA device, not {cache.device}")
        with torch.cuda.device(cache.device):
            status, flag = _lib.jfa_paged_check_error(cache.struct(), self.buf, _handle(cache.device, stream))
        if status != _lib.JFA_ERR_DEVICE:
            check(status, "jfa_paged_check_error")
        return flag

    def clear_error(self, cache: PagedKVCache, stream=None) -> None:
        _run("jfa_paged_clear_error", cache.device, stream, cache._ref, self.ptr)


def _ws(cache, ws, where):
    if ws.sizes != cache.sizes or ws.device != cache.device:
        _refuse(where, "workspace is of another number of sequences or KV heads, or on another device")
    return ws.ptr


def paged_append(cache: PagedKVCache, k, v, ws: PagedWorkspace, cu=None, stream=None) -> None:
    """Append rows bf16 [T, H_kv, 128] of keys and values (any token and head
    strides that are multiples of 8).  cu (int32 [batch + 1], device): rows
    cu[b] .. cu[b + 1] - 1 are sequence b's newest tokens; without it every
    sequence has T / batch, and idle ones (length 0) are left alone.  The
    table's lengths already count the new tokens (PageTable.grow).

    Once for each growth: a group that completes is packed from what the tail
    held, and the tail is overwritten.  A second append at the same lengths (a
    warm-up before a capture, a call repeated) would pack the new rows in place
    of the old ones."""
    where = "paged_append"
    dev, batch = cache.device, cache.table.batch
    ka, va = _rows(k, cache.num_kv_heads, dev, where, "k"), _rows(v, cache.num_kv_heads, dev, where, "v")
    if k.shape[0] != v.shape[0]:
        _refuse(where, "k and v must hold the same tokens")
    cup = None if cu is None else _int32(cu, batch + 1, dev, where, "cu")
    _run("jfa_paged_append", dev, stream, cache._ref, *ka, *va, cup, k.shape[0], _ws(cache, ws, where))


def paged_gather(cache: PagedKVCache, cu, total: int, ws: PagedWorkspace, start=None, k_out=None, v_out=None,
                 stream=None):
    """Read rows back: tokens start[b] (from 0 on without start) and following
    of sequence b into rows cu[b] .. cu[b + 1] - 1 of bf16 [total, H_kv, 128];
    rows in no range are left as they are (unset in a new output).  Returns (k, v)."""
    where = "paged_gather"
    dev, batch = cache.device, cache.table.batch
    shape = (total, cache.num_kv_heads, _lib.HEAD_DIM)
    if not 0 <= total <= _INT_MAX:
        _refuse(where, "total must be 0 or more, and below 2^31")
    if k_out is None:
        k_out = cache.tail_k.new_empty(shape) if stream is None else \
            _fresh(lambda: cache.tail_k.new_empty(shape), stream, dev)
    else:
        _given(k_out, shape, dev, where, "k_out")
    if v_out is None:
        v_out = _like(k_out, stream, dev)
    else:
        _given(v_out, shape, dev, where, "v_out")
    if abs(k_out.data_ptr() - v_out.data_ptr()) < 2 * k_out.numel():
        _refuse(where, "k_out and v_out must not overlap")
    cup = _int32(cu, batch + 1, dev, where, "cu")
    stp = None if start is None else _int32(start, batch, dev, where, "start")
    _run("jfa_paged_gather", dev, stream, cache._ref, cup, stp, total, k_out.data_ptr(), v_out.data_ptr(),
         _ws(cache, ws, where))
    return k_out, v_out


def paged_attend(cache: PagedKVCache, q, ws: PagedWorkspace, scale=None, window: int = 0, sinks: int = 0,
                 out=None, lse=None, stream=None):
    """Attention of each sequence's newest token over its cached tokens, or
    (window > 0) over the last ``window`` of them and the first ``sinks``.

    q: bf16 [B, H, 128] (heads contiguous, any row stride that is a multiple
    of 8).  Returns out bf16 [B, H, 128] (which may be q), zeros for an idle
    sequence; lse (fp32 [B, H], if given) gets the natural logarithm of the
    softmax's sum."""
    where = "paged_attend"
    args = _attend_args(cache, q, out, lse, scale, window, sinks, where)
    return _attend(cache, q, ws, *args, where, stream)


def _attend_args(cache, q, out, lse, scale, window, sinks, where):
    """Checks of paged_attend's arguments but for q's memory: (out, lse, scale, window, sinks)."""
    dev, batch, heads = cache.device, cache.table.batch, cache.num_heads
    window, sinks = operator.index(window), operator.index(sinks)
    if not (0 <= window < 2**31 and 0 <= sinks < 2**31):
        _refuse(where, "window and sinks must be 0 or more, and below 2^31")
    if q.shape != (batch, heads, _lib.HEAD_DIM):
        _refuse(where, f"q must hold {batch} tokens of {heads} heads of {_lib.HEAD_DIM}")
    if out is not None:
        _given(out, q.shape, dev, where, "out")
        if out.data_ptr() % 16:
            _refuse(where, "out must be aligned to 16 bytes")
    if lse is not None and (lse.shape != (batch, heads) or lse.dtype != torch.float32 or lse.device != dev
                            or not lse.is_contiguous()):
        _refuse(where, f"lse must be contiguous fp32 [{batch}, {heads}] on {dev}")
    if scale is None:
        scale = _SCALE
    else:
        scale = ctypes.c_float(scale).value   # as the library takes it
        if not (scale > 0 and math.isfinite(scale)):
            _refuse(where, "scale must be positive and finite in 32 bits")
    return out, lse, scale, window, sinks


def _attend(cache, q, ws, out, lse, scale, window, sinks, where, stream):
    """paged_attend with arguments from _attend_args."""
    dev = cache.device
    qp, q_row, q_head = _rows(q, cache.num_heads, dev, where, "q")
    if q_head != _lib.HEAD_DIM and cache.num_heads > 1:
        _refuse(where, "the heads of q must be contiguous")
    if out is None:
        out = _like(q, stream, dev)
    _run("jfa_paged_attend", dev, stream, cache._ref, qp, q_row, scale, window, sinks, _ws(cache, ws, where),
         out.data_ptr(), None if lse is None else lse.data_ptr())
    return out


def paged_fork(cache: PagedKVCache, pairs, ws: PagedWorkspace, stream=None) -> None:
    """For each (parent, child) of pairs (int32 [n, 2], device): the child takes
    the parent's pages, length and tail.  A child may be no parent, and the
    child of one pair only (PageTable.fork books this)."""
    where = "paged_fork"
    n = pairs.shape[0]
    if n > cache.table.batch:
        _refuse(where, f"{n} pairs for {cache.table.batch} sequences")
    p = _int32(pairs, 2 * n, cache.device, where, "pairs")
    _run("jfa_paged_fork", cache.device, stream, cache._ref, p, n, _ws(cache, ws, where))


def paged_move(cache: PagedKVCache, moves, ws: PagedWorkspace, remap=None, stream=None) -> None:
    """Copy pages (from, to) of moves (int32 [n, 2], device) and, with remap
    (int32 [n_pages], device), point the table's entries to the new places.
    No page may be both source and destination, or twice a destination
    (PageTable.compact books such moves)."""
    where = "paged_move"
    n = moves.shape[0]
    if n > cache.table.n_pages:
        _refuse(where, f"{n} moves for {cache.table.n_pages} pages")
    m = _int32(moves, 2 * n, cache.device, where, "moves")
    r = None if remap is None else _int32(remap, cache.table.n_pages, cache.device, where, "remap")
    _run("jfa_paged_move", cache.device, stream, cache._ref, m if n else None, n, r, _ws(cache, ws, where))


def paged_decode_step(cache: PagedKVCache, q, k, v, positions, plan: RotaryPlan, ws: PagedWorkspace,
                      q_weight=None, k_weight=None, eps: float = 1e-6, scale=None, window: int = 0,
                      sinks: int = 0, out=None, lse=None, stream=None):
    """One decode step of a layer: norm and rotate the new token's heads,
    append its key and value, attend.  q bf16 [B, H, 128], k and v bf16
    [B, H_kv, 128] (slices of one projection's output will do), positions
    [B]; the table has grown by one token a sequence (PageTable.grow(1)).
    Three launches.  Returns out bf16 [B, H, 128].  A call that is refused has
    changed nothing; one that ran is not run again at the same lengths (see
    paged_append)."""
    where = "paged_decode_step"
    # what the attention would refuse, before the append writes
    args = _attend_args(cache, q, out, lse, scale, window, sinks, where)
    q, k = qk_norm_rope(q, k, positions, plan, q_weight, k_weight, eps, stream=stream)
    paged_append(cache, k, v, ws, stream=stream)
    return _attend(cache, q, ws, *args, where, stream)
