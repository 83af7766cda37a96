"""Torch-facing binding of the logit-side operators (argument marshalling
only; include/spec_logits.h): what stands between a model's hidden states and
the logits that a verification reads.

  * ``quantize_int4 / QuantizeInt4Plan``: an LM head in 4 bits with group scales;
  * ``int4_product / Int4ProductPlan``: the logits of a few rows from such a head;
  * ``process_logits / ProcessLogitsPlan``: penalties, biases and grammar masks,
    each row with the tokens before its own position.

As for the verifications, a plan binds its buffers once and ``run()`` launches
without Python-side allocation (what a plan clears, it clears on the stream that
is current where it is made: run it there, or behind it); the functions take one
call's tensors (device tensors stay on the device; CPU tensors are copied there
and the results back, complete on return).  With ``stream`` all of a function's
work goes to that stream, behind what the current one holds; the results belong
to it.
"""

from __future__ import annotations

import contextlib

import torch

from . import _lib as L
from .api import _DTYPES, _Plan, _f32, _finish, _i32, _ptr, _to_device


COUNTER_BYTES = 1024  # of a product's workspace: what has to be zero before a run


def _logit_rows(t: torch.Tensor, name: str) -> int:
    """Row stride (elements) of a [B, n, V] view whose rows are evenly strided."""
    if t.dim() != 3:
        raise ValueError(f"{name}: expected [B, n, V], got {tuple(t.shape)}")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name}: logits must be float32 or bfloat16")
    B, n, V = t.shape
    if V > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: logits must have unit element stride")
    if n == 1:
        return t.stride(0) if B > 1 else V
    if B > 1 and t.stride(0) != n * t.stride(1):
        raise ValueError(f"{name}: rows must be evenly strided")
    return t.stride(1)


def _on(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name}: on {t.device}, expected {dev}")


def _shape(t, shape, name):
    if t is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name}: expected {list(shape)}, got {list(t.shape)}")
    return t


def _matrix_ld(t: torch.Tensor, name: str) -> int:
    """Row stride of a 2-D tensor with contiguous rows."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected a 2-D tensor with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


class _DevicePlan(_Plan):
    """A plan that runs on the GPU's tensors only (a host address never reaches a kernel)."""

    def _bind(self, call, dev):
        self._call, self._dev = call, dev
        if dev.type != "cuda":
            self.run = self._refuse

    def _refuse(self, stream=None):
        raise ValueError(f"{type(self).__name__}: bound to tensors on {self._dev}, CUDA tensors required")


def _workspace(t, dev):
    """A caller's workspace, and its bytes."""
    _on(dev, workspace=t)
    if not t.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    return t.numel() * t.element_size()


class ProcessLogitsPlan(_DevicePlan):
    """Per-request processing of logits bound to fixed buffers.  See
    spec_process_logits.

    logits [B, n, V] (float32 or bfloat16).  tokens int32 [B, T]: the drafted
    tokens of a chain (T >= n - 1), or with parent int32 [B, n] the node
    tokens of a tree (T >= n).  history int32 [B, H] with history_len and
    prompt_len int32 [B] (or None: H and 0).  repetition, frequency, presence
    float32 [B] or None (1, 0, 0).  bias_tokens int32 and bias_values float32
    [B, K] with bias_len int32 [B] (or None: K).  mask int32 [M, words]: bit
    v % 32 of word v // 32 set where token v is allowed, mask_index int32
    [B, n] (-1: not masked; None: row (b, i) uses mask row b * n + i).  out:
    a [B, n, V] tensor of the same type, ``logits`` itself to work in place,
    or None: allocated with logits' row stride, or where that is twice a row or
    more, with the least one of the same remainder by 16 bytes.

    ``run()`` returns logits (out), seq_error int32 [B] and error_word."""

    def __init__(self, logits, tokens=None, *, parent=None, history=None, history_len=None, prompt_len=None,
                 repetition=None, frequency=None, presence=None, bias_tokens=None, bias_values=None, bias_len=None,
                 mask=None, mask_index=None, out=None, workspace=None):
        ld = _logit_rows(logits, "logits")
        B, n, V = logits.shape
        dev = logits.device
        if out is None:
            # (rows of one position of many, or of a wider matrix: not the memory between them as well, but a
            # stride after which rows start at the same place of a 16-byte vector, so that whole vectors are stored)
            width = ld if ld < 2 * V else V + (ld - V) % (16 // logits.element_size())
            out = torch.empty((B, n, width), dtype=logits.dtype, device=dev)[:, :, :V]
        if out.dtype != logits.dtype:
            raise TypeError("out: the type of logits required")
        _shape(out, (B, n, V), "out")
        out_ld = _logit_rows(out, "out")
        if out.data_ptr() == logits.data_ptr() and out_ld != ld:
            raise ValueError("out: in place needs the row stride of logits")
        if parent is not None and tokens is None:
            raise ValueError("parent: a tree needs its node tokens")
        if tokens is not None and (tokens.dim() != 2 or tokens.shape[0] != B
                                   or tokens.shape[1] < (n if parent is not None else n - 1)):
            raise ValueError(f"tokens: expected [{B}, at least {n if parent is not None else n - 1}], "
                             f"got {list(tokens.shape)}")
        if history is not None and (history.dim() != 2 or history.shape[0] != B):
            raise ValueError(f"history: expected [{B}, H], got {list(history.shape)}")
        if history is None and (history_len is not None or prompt_len is not None):
            raise ValueError("history_len, prompt_len: without a history")
        if (bias_tokens is None) != (bias_values is None) or (bias_tokens is None and bias_len is not None):
            raise ValueError("bias_tokens and bias_values go together")
        if bias_tokens is not None and (bias_tokens.dim() != 2 or bias_tokens.shape[0] != B):
            raise ValueError(f"bias_tokens: expected [{B}, K], got {list(bias_tokens.shape)}")
        if mask is None and mask_index is not None:
            raise ValueError("mask_index: without a mask")
        words = (V + 31) // 32
        if mask is not None:
            if mask.dtype != torch.int32:
                raise TypeError("mask: expected int32 words")
            mask_ld = _matrix_ld(mask, "mask")
            if mask.shape[0] < 1 or mask.shape[1] < words:
                raise ValueError(f"mask: expected [rows, at least {words}], got {list(mask.shape)}")
            if mask_index is None and mask.shape[0] < B * n:
                raise ValueError(f"mask: {B * n} rows required without mask_index")
        for name, t in (("parent", parent), ("mask_index", mask_index)):
            _shape(t, (B, n), name)
        for name, t in (("history_len", history_len), ("prompt_len", prompt_len), ("bias_len", bias_len),
                        ("repetition", repetition), ("frequency", frequency), ("presence", presence)):
            _shape(t, (B,), name)
        if bias_values is not None:
            _shape(bias_values, tuple(bias_tokens.shape), "bias_values")
        _on(dev, out=out, tokens=tokens, parent=parent, history=history, history_len=history_len,
            prompt_len=prompt_len, repetition=repetition, frequency=frequency, presence=presence,
            bias_tokens=bias_tokens, bias_values=bias_values, bias_len=bias_len, mask=mask, mask_index=mask_index)
        lib = L.lib()
        self.keep = [logits, tokens, parent, history, history_len, prompt_len, repetition, frequency, presence,
                     bias_tokens, bias_values, bias_len, mask, mask_index]
        self.out = dict(logits=out, seq_error=torch.empty(B, dtype=torch.int32, device=dev),
                        error_word=torch.zeros(1, dtype=torch.int32, device=dev))
        need = int(lib.spec_process_workspace_size(B, n, V, 0 if history is None else history.shape[1],
                                                   0 if bias_tokens is None else bias_tokens.shape[1]))
        if need == 0:
            raise ValueError(f"process_logits: sizes out of range: B={B} n={n} V={V}")
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        self.workspace = workspace
        a = L.ProcessArgs()
        a.B, a.n, a.V, a.dtype = B, n, V, _DTYPES[logits.dtype]
        a.ld, a.out_ld = ld, out_ld
        a.logits, a.out = _ptr(logits), _ptr(out)
        a.tokens, a.parent = _ptr(_i32(tokens, "tokens")), _ptr(_i32(parent, "parent"))
        a.tokens_ld = 0 if tokens is None else tokens.shape[1]
        a.history, a.history_ld = _ptr(_i32(history, "history")), 0 if history is None else history.shape[1]
        a.history_len, a.prompt_len = _ptr(_i32(history_len, "history_len")), _ptr(_i32(prompt_len, "prompt_len"))
        a.repetition, a.frequency = _ptr(_f32(repetition, "repetition")), _ptr(_f32(frequency, "frequency"))
        a.presence = _ptr(_f32(presence, "presence"))
        a.bias_tokens, a.bias_values = _ptr(_i32(bias_tokens, "bias_tokens")), _ptr(_f32(bias_values, "bias_values"))
        a.bias_len = _ptr(_i32(bias_len, "bias_len"))
        a.bias_ld = 0 if bias_tokens is None else bias_tokens.shape[1]
        a.mask, a.mask_index = _ptr(mask), _ptr(_i32(mask_index, "mask_index"))
        a.mask_rows, a.mask_ld = (0, 0) if mask is None else (mask.shape[0], mask_ld)
        a.seq_error, a.error_word = _ptr(self.out["seq_error"]), _ptr(self.out["error_word"])
        a.workspace, a.workspace_bytes = _ptr(workspace), _workspace(workspace, dev)
        self.args = a
        self._bind(lib.spec_process_logits, dev)


class QuantizeInt4Plan(_DevicePlan):
    """4-bit quantisation with group scales bound to fixed buffers.  See
    spec_quantize_int4.

    weights [V, d] float32 or bfloat16, group 32, 64 or 128 (a divisor of d).
    ``run()`` returns codes uint8 [V, d / 2] (two codes to a byte, the even
    column in the low nibble), scales bfloat16 [d / group, V] and, with
    ``zeros=True``, zeros uint8 [d / group, V]."""

    def __init__(self, weights, *, group=128, zeros=False):
        if weights.dtype not in _DTYPES:
            raise TypeError("weights: float32 or bfloat16 required")
        ld = _matrix_ld(weights, "weights")
        V, d = weights.shape
        if group not in (32, 64, 128) or d % group or not 32 <= d <= 65536 or not 1 <= V <= 2097152:
            raise ValueError(f"quantize_int4: sizes out of range: V={V} d={d} group={group}")
        lib = L.lib()
        dev = weights.device
        self.keep = [weights]
        self.out = dict(codes=torch.empty((V, d // 2), dtype=torch.uint8, device=dev),
                        scales=torch.empty((d // group, V), dtype=torch.bfloat16, device=dev))
        if zeros:
            self.out["zeros"] = torch.empty((d // group, V), dtype=torch.uint8, device=dev)
        a = L.QuantizeInt4Args()
        a.V, a.d, a.group, a.dtype = V, d, group, _DTYPES[weights.dtype]
        a.ld, a.codes_ld, a.scales_ld, a.zeros_ld = ld, d // 2, V, V
        a.weights, a.codes, a.scales = _ptr(weights), _ptr(self.out["codes"]), _ptr(self.out["scales"])
        a.zeros = _ptr(self.out.get("zeros"))
        self.args = a
        self._bind(lib.spec_quantize_int4, dev)


class Int4ProductPlan(_DevicePlan):
    """Products of a few rows with a 4-bit matrix bound to fixed buffers.  See
    spec_int4_product.

    x bfloat16 [R, d] (or [B, n, d]), codes, scales and zeros as
    quantize_int4 returns them (rows of codes and x may be padded).  A workspace
    that the caller passes must hold zeros before its first use.  ``run()``
    returns logits [R, V] (or [B, n, V]) of out_dtype and error_word.  After a
    run that set ERR_INTERNAL in error_word (a bounded wait gave up), call
    ``reset()`` before the next: the run may have left counts of half-summed
    tiles in the workspace."""

    def __init__(self, x, codes, scales, zeros=None, *, group=128, out_dtype=torch.bfloat16, out=None,
                 workspace=None):
        lead = tuple(x.shape[:-1])
        if x.dtype != torch.bfloat16 or x.dim() not in (2, 3):
            raise TypeError("x: bfloat16 [R, d] or [B, n, d] required")
        if x.dim() == 3:
            if not x.is_contiguous():
                raise ValueError("x: [B, n, d] must be contiguous")
            x = x.view(-1, x.shape[2])
        x_ld = _matrix_ld(x, "x")
        R, d = x.shape
        if codes.dtype != torch.uint8 or scales.dtype != torch.bfloat16:
            raise TypeError("codes: uint8 and scales: bfloat16 required")
        if zeros is not None and zeros.dtype != torch.uint8:
            raise TypeError("zeros: uint8 required")
        if out_dtype not in _DTYPES:
            raise TypeError("out_dtype: float32 or bfloat16 required")
        codes_ld, V = _matrix_ld(codes, "codes"), codes.shape[0]
        lib = L.lib()
        need = int(lib.spec_int4_product_workspace_size(R, V, d, group))
        if need == 0:
            raise ValueError(f"int4_product: sizes out of range: R={R} V={V} d={d} group={group}")
        _shape(codes, (V, d // 2), "codes")
        _shape(scales, (d // group, V), "scales")
        _shape(zeros, (d // group, V), "zeros")
        scales_ld = _matrix_ld(scales, "scales")
        zeros_ld = 0 if zeros is None else _matrix_ld(zeros, "zeros")
        dev = x.device
        if out is None:
            out = torch.empty((*lead, V), dtype=out_dtype, device=dev)
        elif tuple(out.shape) != (*lead, V) or out.dtype != out_dtype:
            raise ValueError(f"out: expected {[*lead, V]} of {out_dtype}")
        out_ld = _logit_rows(out, "out") if out.dim() == 3 else _matrix_ld(out, "out")
        _on(dev, codes=codes, scales=scales, zeros=zeros, out=out)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
            workspace[:COUNTER_BYTES].zero_()
        self.workspace = workspace
        self.keep = [x, codes, scales, zeros]
        self.out = dict(logits=out, error_word=torch.zeros(1, dtype=torch.int32, device=dev))
        a = L.Int4ProductArgs()
        a.R, a.V, a.d, a.group, a.out_dtype = R, V, d, group, _DTYPES[out_dtype]
        a.x_ld, a.codes_ld, a.scales_ld, a.zeros_ld, a.out_ld = x_ld, codes_ld, scales_ld, zeros_ld, out_ld
        a.x, a.codes, a.scales, a.zeros, a.out = _ptr(x), _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(out)
        a.error_word = _ptr(self.out["error_word"])
        a.workspace, a.workspace_bytes = _ptr(workspace), _workspace(workspace, dev)
        self.args = a
        self._bind(lib.spec_int4_product, dev)

    def reset(self, stream=None):
        """Clear the workspace's counters and error_word, on the run's stream
        (None: the current one)."""
        with torch.cuda.stream(stream):
            self.workspace.view(torch.uint8)[:COUNTER_BYTES].zero_()
            self.out["error_word"].zero_()


@contextlib.contextmanager
def _work_on(stream, tensors):
    """What a call allocates, clears, copies and launches inside goes to `stream`,
    behind the work that the current one holds.  `tensors`: the call's inputs,
    whose memory stays theirs until `stream` is done with them."""
    if stream is None or stream == torch.cuda.current_stream():
        yield
        return
    stream.wait_stream(torch.cuda.current_stream())
    for t in tensors:
        if t is not None and t.device.type == "cuda":
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        yield


def _results(out, host):
    """A call's results: the device's tensors, or complete copies on the host."""
    out = _finish(out, host)
    if host:
        torch.cuda.current_stream().synchronize()
    return out


def process_logits(logits, tokens=None, *, parent=None, history=None, history_len=None, prompt_len=None,
                   repetition=None, frequency=None, presence=None, bias_tokens=None, bias_values=None,
                   bias_len=None, mask=None, mask_index=None, out=None, device="cuda", stream=None):
    """Process B sequences' logit rows; returns logits, seq_error, error_word.
    See ProcessLogitsPlan (host tensors in, host tensors out)."""
    host = logits.device.type == "cpu"
    given = dict(parent=parent, history=history, history_len=history_len, prompt_len=prompt_len,
                 repetition=repetition, frequency=frequency, presence=presence, bias_tokens=bias_tokens,
                 bias_values=bias_values, bias_len=bias_len, mask=mask, mask_index=mask_index)
    if host and out is not None:
        raise ValueError("out: device tensors only")
    with _work_on(stream, [logits, tokens, out, *given.values()]):
        if host:
            logits, tokens = _to_device([logits, tokens], device)
            given = dict(zip(given, _to_device(list(given.values()), device)))
        return _results(ProcessLogitsPlan(logits, tokens, out=out, **given).run(), host)


def quantize_int4(weights, *, group=128, zeros=False, device="cuda", stream=None):
    """Quantise a matrix to 4 bits; returns codes, scales and, with
    ``zeros=True``, zeros.  See QuantizeInt4Plan."""
    host = weights.device.type == "cpu"
    with _work_on(stream, [weights]):
        if host:
            (weights,) = _to_device([weights], device)
        return _results(QuantizeInt4Plan(weights, group=group, zeros=zeros).run(), host)


def int4_product(x, codes, scales, zeros=None, *, group=128, out_dtype=torch.bfloat16, device="cuda", stream=None):
    """Products of x's rows with a 4-bit matrix; returns logits, error_word.
    See Int4ProductPlan."""
    host = x.device.type == "cpu"
    with _work_on(stream, [x, codes, scales, zeros]):
        if host:
            x, codes, scales, zeros = _to_device([x, codes, scales, zeros], device)
        return _results(Int4ProductPlan(x, codes, scales, zeros, group=group, out_dtype=out_dtype).run(), host)
