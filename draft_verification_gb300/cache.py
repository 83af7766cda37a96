"""Torch-facing binding of the cache operators (argument marshalling only;
include/spec_cache.h): what a verification step does to the key-value cache.

  * ``rotate_heads / RotateHeadsPlan``: rotary positions of queries (or keys);
  * ``append_cache / AppendCachePlan``: keys and values into a paged cache of
    8-bit codes, keys rotated on the way; after a tree verification, the kept
    path's rows once more;
  * ``attend_cache / AttendCachePlan``: attention of a chain's or a tree's rows
    over that cache.

``rotation_table`` and ``rotary_frequencies`` make the table that the first two
read, ``PagedCache`` holds the cache's tensors.

A plan binds its buffers once and ``run()`` launches without Python-side
allocation.  Its error bits (seq_error, error_word) are OR-ed in by every run;
``clear_errors()`` zeroes them.  The functions take one call's tensors; CPU
tensors beside a cache on the GPU are copied there and the results back
(complete on return).  With ``stream`` all of a function's work goes to that
stream, behind what the current one holds; the results belong to it.
"""

from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import _lib as L
from .api import _DTYPES, _check, _f32, _i32, _ptr, _stream_handle, _to_device
from .logits import _DevicePlan, _on, _results, _shape, _work_on, _workspace

PAGES = (16, 32, 64, 128)  # tokens per page


@dataclass(frozen=True)
class PagedCache:
    """Keys and values in 8 bits: codes uint8 [pages, H, page, D] (e4m3), exps
    int8 [pages, H]; code c of page p and head h stands for c * 2^exps[p, h]."""

    k_codes: torch.Tensor
    v_codes: torch.Tensor
    k_exps: torch.Tensor
    v_exps: torch.Tensor

    def __post_init__(self):
        if self.k_codes.dim() != 4:
            raise ValueError(f"k_codes: expected [pages, H, page, D], got {list(self.k_codes.shape)}")
        pages, H, page, D = self.k_codes.shape
        if page not in PAGES:
            raise ValueError(f"a page holds 16, 32, 64 or 128 tokens, not {page}")
        if pages < 1 or not 1 <= H <= 1024 or D % 16 or not 16 <= D <= 256 or pages * H * page > 2 ** 31 - 1:
            raise ValueError(f"cache: sizes out of range: pages={pages} H={H} page={page} D={D}")
        for name, shape, dtype in (("k_codes", (pages, H, page, D), torch.uint8),
                                   ("v_codes", (pages, H, page, D), torch.uint8),
                                   ("k_exps", (pages, H), torch.int8), ("v_exps", (pages, H), torch.int8)):
            t = getattr(self, name)
            if t.dtype != dtype or not t.is_contiguous():
                raise TypeError(f"{name}: expected a contiguous {dtype} tensor")
            _shape(t, shape, name)
            _on(self.k_codes.device, **{name: t})

    @classmethod
    def empty(cls, pages, heads, page, dim, device="cuda"):
        """A cache of `pages` pages that hold nothing (zeros)."""
        codes = [torch.zeros((pages, heads, page, dim), dtype=torch.uint8, device=device) for _ in range(2)]
        exps = [torch.zeros((pages, heads), dtype=torch.int8, device=device) for _ in range(2)]
        return cls(*codes, *exps)

    @property
    def device(self):
        return self.k_codes.device

    def values(self):
        """Keys and values as float32 [pages, H, page, D]."""
        return tuple(torch.ldexp(c.view(torch.float8_e4m3fn).float(), e.int()[..., None, None])
                     for c, e in ((self.k_codes, self.k_exps), (self.v_codes, self.v_exps)))


def rotary_frequencies(rot, base=10000.0, *, linear=1.0, bands=None):
    """float64 [rot / 2] radians per position: base^(-2 i / rot) / linear.

    bands = (factor, low, high, length): frequencies by their wavelength, for a
    context `factor` times as long as the `length` that a model was trained on.
    Of a frequency whose wavelength fits more than `high` times into length
    nothing changes, one whose wavelength fits fewer than `low` times is divided
    by factor, and between the two they are blended linearly in that number."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot: an even number of at least 2 required, got {rot}")
    if not base > 0 or not linear > 0:
        raise ValueError("base and linear: positive numbers required")
    f = torch.tensor(float(base), dtype=torch.float64) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    f = f / float(linear)
    if bands is not None:
        factor, low, high, length = (float(x) for x in bands)
        if not (factor > 0 and 0 <= low < high and length > 0):
            raise ValueError("bands: (factor > 0, 0 <= low < high, length > 0) required")
        share = ((length * f / (2.0 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        f = f * (share + (1.0 - share) / factor)
    return f


def rotation_table(rows, rot, *, freq=None, base=10000.0, magnitude=1.0, device="cuda", stream=None):
    """float32 [rows, rot]: of each position the cosines, then the sines of
    position * freq, times magnitude.  freq: float64 [rot / 2], by default
    rotary_frequencies(rot, base).  See spec_rotation_table."""
    freq = rotary_frequencies(rot, base) if freq is None else freq
    if freq.dtype != torch.float64 or tuple(freq.shape) != (rot // 2,) or rot % 2:
        raise ValueError(f"freq: expected float64 [{rot // 2}]")
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"rotation_table: a CUDA device required, got {device}")
    with _work_on(stream, [freq]), torch.cuda.device(device):
        freq = freq.contiguous().to(device)
        table = torch.empty((rows, rot), dtype=torch.float32, device=device)
        _check(L.lib().spec_rotation_table(rows, rot, _ptr(freq), float(magnitude), _ptr(table),
                                           _stream_handle(None)), "rotation_table")
    return table


class _CachePlan(_DevicePlan):
    """A plan that runs on its tensors' device, whichever is current."""

    _cleared = None  # the event behind which the error words are zero, and the streams that are behind it
    _behind = frozenset()
    _kept = True

    @classmethod
    def _once(cls, *args, **kw):
        """One run, where it is made, of a plan that nobody keeps."""
        plan = cls.__new__(cls)
        plan._kept = False
        plan.__init__(*args, **kw)
        return plan.run()

    def run(self, stream=None):
        """Launch on `stream` (None: the device's current one); returns the
        outputs.  A run comes behind the making of the plan and clear_errors(),
        whatever streams they were on; in a graph's capture, which cannot wait for
        another stream, they have to be complete (torch.cuda.graph sees to it)
        or on the captured stream."""
        if stream is None:
            stream = torch.cuda.current_stream(self._dev)
        elif stream.device != self._dev:
            raise ValueError(f"stream: on {stream.device}, expected {self._dev}")
        if self._cleared is not None and stream.cuda_stream not in self._behind:
            self._wait(stream)
        if torch.cuda.current_device() == self._dev.index:
            return super().run(stream)
        with torch.cuda.device(self._dev):
            return super().run(stream)

    def clear_errors(self, stream=None):
        """Zero seq_error and error_word, on `stream` (None: the current one)."""
        with torch.cuda.stream(stream):
            self._words.zero_()
            if self._dev.type == "cuda":
                self._mark(torch.cuda.current_stream(self._dev))

    def _errors(self, a, B, dev):
        self._words = torch.zeros(B + 1, dtype=torch.int32, device=dev)
        self.out["seq_error"], self.out["error_word"] = self._words[:B], self._words[B:]
        a.seq_error, a.error_word = _ptr(self.out["seq_error"]), _ptr(self.out["error_word"])
        if self._kept and dev.type == "cuda":
            self._mark(torch.cuda.current_stream(dev))

    def _mark(self, stream):
        """`stream`, its device's current one, has zeroed the error words (and
        holds the work that used the plan's memory before)."""
        if torch.cuda.current_device() == stream.device_index:
            captured = torch.cuda.is_current_stream_capturing()
        else:
            with torch.cuda.stream(stream):
                captured = torch.cuda.is_current_stream_capturing()
        if not captured:  # (a captured clearing is the graph's)
            self._cleared, self._behind = stream.record_event(), {stream.cuda_stream}

    def _wait(self, stream):
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return
        stream.wait_event(self._cleared)
        self._behind.add(stream.cuda_stream)


def _heads(t, name, dtypes=None):
    """The (sequence, row, head) strides of a [B, n, H, D] tensor with contiguous heads."""
    if t.dim() != 4 or 0 in t.shape:
        raise ValueError(f"{name}: expected [B, n, H, D], got {list(t.shape)}")
    if t.dtype not in (dtypes or _DTYPES):
        raise TypeError(f"{name}: {t.dtype} is not supported")
    if t.stride(3) != 1:
        raise ValueError(f"{name}: heads must have unit element stride")
    return list(t.stride()[:3])


def _own_rows(t, name):
    """A tensor that is written: no two of its elements in one place."""
    axes = sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1)
    extent = 1  # of the axes so far: from the first of their places to the last
    for s, n in axes:
        if s < extent:
            break
        extent += (n - 1) * s
    else:
        return  # (each axis steps over all that the smaller ones reach)

    def meets(i, at, moved):
        """Whether steps along axes 0 .. i, not all of no length, lead from `at` to 0."""
        if i < 0:
            return moved and at == 0
        s, n = axes[i]
        reach = sum((m - 1) * r for r, m in axes[:i])
        if s == 0:
            return True
        first, last = max(1 - n, -((at + reach) // s)), min(n - 1, (reach - at) // s)
        return any(meets(i - 1, at + d * s, moved or d != 0) for d in range(first, last + 1))

    if meets(len(axes) - 1, 0, False):
        raise ValueError(f"{name}: elements overlap")


def _table_of(table, D, name="table"):
    _f32(table, name)
    if table.dim() != 2 or table.shape[0] < 1 or table.shape[1] % 2 or not 2 <= table.shape[1] <= D:
        raise ValueError(f"{name}: expected [rows, rot], rot even and at most {D}, got {list(table.shape)}")
    return table


class RotateHeadsPlan(_CachePlan):
    """Rotary positions bound to fixed buffers.  See spec_rotate_heads.

    x [B, n, H, D] float32 or bfloat16 (any strides with contiguous heads).
    table: rotation_table(rows, rot); the first rot elements of every head are
    rotated, by halves (element i with i + rot / 2) or with ``pairs=True`` by
    neighbours (2 i with 2 i + 1).  The row's position: positions int32 [B, n],
    or prefix_len int32 [B] (None: 0) plus its place.  transpose=True: the
    inverse rotation, and the gradient of a forward one.  out: a tensor like x,
    ``x`` itself, or None: allocated contiguous.

    ``run()`` returns out, seq_error int32 [B] and error_word."""

    def __init__(self, x, table, *, positions=None, prefix_len=None, pairs=False, transpose=False, out=None):
        x_ld = _heads(x, "x")
        B, n, H, D = x.shape
        _table_of(table, D)
        if positions is not None and prefix_len is not None:
            raise ValueError("positions and prefix_len exclude each other")
        _shape(positions, (B, n), "positions")
        _shape(prefix_len, (B,), "prefix_len")
        if out is None:
            out = torch.empty((B, n, H, D), dtype=x.dtype, device=x.device)
        _shape(out, (B, n, H, D), "out")
        if out.dtype != x.dtype:
            raise TypeError("out: the type of x required")
        out_ld = _heads(out, "out")
        _own_rows(out, "out")
        if out.data_ptr() == x.data_ptr() and out_ld != x_ld:
            raise ValueError("out: in place needs the strides of x")
        _on(x.device, table=table, positions=positions, prefix_len=prefix_len, out=out)
        self.keep = [x, table, positions, prefix_len]
        self.out = dict(out=out)
        a = L.RotateArgs()
        a.B, a.n, a.H, a.D, a.rot = B, n, H, D, table.shape[1]
        a.pairs, a.transpose, a.dtype = int(bool(pairs)), int(bool(transpose)), _DTYPES[x.dtype]
        a.x_ld[:], a.out_ld[:] = x_ld, out_ld
        a.x, a.out, a.table, a.table_rows = _ptr(x), _ptr(out), _ptr(table), table.shape[0]
        a.positions, a.prefix_len = _ptr(_i32(positions, "positions")), _ptr(_i32(prefix_len, "prefix_len"))
        self._errors(a, B, x.device)
        self.args = a
        self._bind(L.lib().spec_rotate_heads, x.device)


class AppendCachePlan(_CachePlan):
    """Appending keys and values to a paged cache bound to fixed buffers.  See
    spec_append_cache.

    k, v [B, n, H, D] float32 or bfloat16 (any strides with contiguous heads),
    cache a PagedCache, block_table int32 [B, P]: each sequence's pages in the
    order of its tokens (no page twice among those that get rows).  Row i goes
    to token prefix_len[b] + i (int32 [B]; None: 0).  count int32 [B]: the rows of each sequence (None: n).
    path_nodes int32 [B, depth + 1] and path_len int32 [B], as a tree
    verification returns them: instead, the rows of the kept path.  table: keys
    are rotated (RotateHeadsPlan), each by positions int32 [B, n] or by the
    token that it goes to.

    ``run()`` changes the cache and returns seq_error int32 [B] and error_word."""

    def __init__(self, k, v, cache, block_table, prefix_len=None, *, table=None, pairs=False, positions=None,
                 count=None, path_nodes=None, path_len=None):
        k_ld = _heads(k, "k")
        B, n, H, D = k.shape
        if v.dtype != k.dtype:
            raise TypeError("v: the type of k required")
        _shape(v, (B, n, H, D), "v")
        v_ld = _heads(v, "v")
        pages, heads, page, dim = cache.k_codes.shape
        if (heads, dim) != (H, D):
            raise ValueError(f"k: {H} heads of {D}, the cache has {heads} of {dim}")
        if block_table.dim() != 2 or block_table.shape[0] != B or block_table.shape[1] < 1:
            raise ValueError(f"block_table: expected [{B}, pages], got {list(block_table.shape)}")
        if table is not None:
            _table_of(table, D)
        elif positions is not None:
            raise ValueError("positions: without a table")
        if (path_nodes is None) != (path_len is None):
            raise ValueError("path_nodes and path_len go together")
        if path_nodes is not None and count is not None:
            raise ValueError("count and a path exclude each other")
        if path_nodes is not None and (path_nodes.dim() != 2 or path_nodes.shape[0] != B or path_nodes.shape[1] < 1):
            raise ValueError(f"path_nodes: expected [{B}, depth + 1], got {list(path_nodes.shape)}")
        _shape(positions, (B, n), "positions")
        for name, t in (("prefix_len", prefix_len), ("count", count), ("path_len", path_len)):
            _shape(t, (B,), name)
        dev = cache.device
        _on(dev, k=k, v=v, block_table=block_table, prefix_len=prefix_len, table=table, positions=positions,
            count=count, path_nodes=path_nodes, path_len=path_len)
        self.keep = [k, v, cache, block_table, prefix_len, table, positions, count, path_nodes, path_len]
        self.out = {}
        a = L.AppendArgs()
        a.B, a.n, a.H, a.D, a.page, a.pages, a.table_pages = B, n, H, D, page, pages, block_table.shape[1]
        if table is not None:
            a.rot, a.table, a.table_rows = table.shape[1], _ptr(table), table.shape[0]
        a.pairs, a.dtype = int(bool(pairs)), _DTYPES[k.dtype]
        a.k_ld[:], a.v_ld[:] = k_ld, v_ld
        a.k, a.v = _ptr(k), _ptr(v)
        a.positions, a.prefix_len = _ptr(_i32(positions, "positions")), _ptr(_i32(prefix_len, "prefix_len"))
        a.count, a.block_table = _ptr(_i32(count, "count")), _ptr(_i32(block_table, "block_table"))
        a.path_nodes, a.path_len = _ptr(_i32(path_nodes, "path_nodes")), _ptr(_i32(path_len, "path_len"))
        a.max_depth = 0 if path_nodes is None else path_nodes.shape[1] - 1
        a.k_codes, a.v_codes = _ptr(cache.k_codes), _ptr(cache.v_codes)
        a.k_exps, a.v_exps = _ptr(cache.k_exps), _ptr(cache.v_exps)
        self._errors(a, B, dev)
        self.args = a
        self._bind(L.lib().spec_append_cache, dev)


class AttendCachePlan(_CachePlan):
    """Attention of drafted rows over a paged cache bound to fixed buffers.  See
    spec_attend_cache.

    q bfloat16 [B, n, Hq, D] (strides multiples of 8 elements, contiguous
    heads), Hq a multiple of the cache's heads.  Sequence b's tokens are
    prefix_len[b] (int32 [B]; None: 0) committed ones and count[b] (int32 [B];
    None: n) drafted ones behind them, in the pages that block_table int32
    [B, P] names.  parent None: a chain, row i sees the drafted tokens up to its
    own; parent int32 [B, n]: a tree, row i sees its own token and its
    ancestors'.  scale: of the scores, by default 1 / sqrt(D).  out: a bfloat16
    tensor like q, or None: allocated contiguous.

    ``run()`` returns out (rows from count[b] on are zeros), seq_error int32 [B]
    and error_word."""

    def __init__(self, q, cache, block_table, prefix_len=None, *, count=None, parent=None, scale=None, out=None,
                 workspace=None):
        q_ld = _heads(q, "q", (torch.bfloat16,))
        B, n, Hq, D = q.shape
        pages, H, page, dim = cache.k_codes.shape
        if D != dim or Hq % H:
            raise ValueError(f"q: {Hq} heads of {D}, the cache has {H} of {dim}")
        if block_table.dim() != 2 or block_table.shape[0] != B or block_table.shape[1] < 1:
            raise ValueError(f"block_table: expected [{B}, pages], got {list(block_table.shape)}")
        for name, t in (("prefix_len", prefix_len), ("count", count)):
            _shape(t, (B,), name)
        _shape(parent, (B, n), "parent")
        if out is None:
            out = torch.empty((B, n, Hq, D), dtype=q.dtype, device=q.device)
        _shape(out, (B, n, Hq, D), "out")
        out_ld = _heads(out, "out", (torch.bfloat16,))
        _own_rows(out, "out")
        dev = cache.device
        _on(dev, q=q, block_table=block_table, prefix_len=prefix_len, count=count, parent=parent, out=out)
        lib = L.lib()
        need = int(lib.spec_attend_workspace_size(B, n, Hq, H, D))
        if need == 0:
            raise ValueError(f"attend_cache: sizes out of range: B={B} n={n} Hq={Hq} H={H} D={D}")
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        self.workspace = workspace
        self.keep = [q, cache, block_table, prefix_len, count, parent]
        self.out = dict(out=out)
        a = L.AttendArgs()
        a.B, a.n, a.Hq, a.H, a.D, a.page, a.pages, a.table_pages = B, n, Hq, H, D, page, pages, block_table.shape[1]
        a.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
        # (the stride of an axis of one entry is nobody's)
        a.q_ld[:] = [s if m > 1 else 0 for s, m in zip(q_ld, q.shape)]
        a.out_ld[:] = out_ld
        a.q, a.out = _ptr(q), _ptr(out)
        a.prefix_len, a.count = _ptr(_i32(prefix_len, "prefix_len")), _ptr(_i32(count, "count"))
        a.parent, a.block_table = _ptr(_i32(parent, "parent")), _ptr(_i32(block_table, "block_table"))
        a.k_codes, a.v_codes = _ptr(cache.k_codes), _ptr(cache.v_codes)
        a.k_exps, a.v_exps = _ptr(cache.k_exps), _ptr(cache.v_exps)
        a.workspace, a.workspace_bytes = _ptr(workspace), _workspace(workspace, dev)
        self._errors(a, B, dev)
        self.args = a
        self._bind(lib.spec_attend_cache, dev)


def rotate_heads(x, table, *, positions=None, prefix_len=None, pairs=False, transpose=False, out=None, stream=None):
    """Rotate heads by their positions; returns out, seq_error, error_word.  See
    RotateHeadsPlan (tensors on the CPU beside a table on the GPU: results on the CPU)."""
    host = x.device.type == "cpu"
    if host and out is not None:
        raise ValueError("out: device tensors only")
    with _work_on(stream, [x, table, positions, prefix_len, out]):
        if host:
            x, positions, prefix_len = _to_device([x, positions, prefix_len], table.device)
        return _results(RotateHeadsPlan._once(x, table, positions=positions, prefix_len=prefix_len, pairs=pairs,
                                              transpose=transpose, out=out), host)


def append_cache(k, v, cache, block_table, prefix_len=None, *, table=None, pairs=False, positions=None, count=None,
                 path_nodes=None, path_len=None, stream=None):
    """Append keys and values to a paged cache; returns seq_error, error_word.
    See AppendCachePlan (the cache and the table are on the GPU)."""
    host = k.device.type == "cpu"
    given = [k, v, block_table, prefix_len, positions, count, path_nodes, path_len]
    with _work_on(stream, [*given, table, cache.k_codes, cache.v_codes, cache.k_exps, cache.v_exps]):
        if host:
            given = _to_device(given, cache.device)
        k, v, block_table, prefix_len, positions, count, path_nodes, path_len = given
        return _results(AppendCachePlan._once(k, v, cache, block_table, prefix_len, table=table, pairs=pairs,
                                              positions=positions, count=count, path_nodes=path_nodes,
                                              path_len=path_len), host)


def attend_cache(q, cache, block_table, prefix_len=None, *, count=None, parent=None, scale=None, out=None,
                 stream=None):
    """Attention of drafted rows over a paged cache; returns out, seq_error,
    error_word.  See AttendCachePlan (the cache is on the GPU)."""
    host = q.device.type == "cpu"
    if host and out is not None:
        raise ValueError("out: device tensors only")
    given = [q, block_table, prefix_len, count, parent]
    with _work_on(stream, [*given, out, cache.k_codes, cache.v_codes, cache.k_exps, cache.v_exps]):
        if host:
            given = _to_device(given, cache.device)
        q, block_table, prefix_len, count, parent = given
        return _results(AttendCachePlan._once(q, cache, block_table, prefix_len, count=count, parent=parent, scale=scale,
                                              out=out), host)
