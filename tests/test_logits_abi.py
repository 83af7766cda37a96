"""The logit-side operators without a GPU: include/spec_logits.h against the
binding, the refusals of the C entry points and of the plans."""

import ctypes as C
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "spec_logits.h")


@pytest.fixture(scope="module")
def lib():
    from draft_verification_gb300 import _lib, build
    if shutil.which("nvcc") is None and not os.path.exists(build.lib_path()):
        pytest.skip("neither nvcc nor a built library is available")
    build.build()
    return _lib.lib()


def test_every_declared_symbol_is_exported(lib):
    from draft_verification_gb300 import _lib
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(spec_\w+)\s*\(", text, re.M)))
    assert sorted(_lib.LOGITS_SIGNATURES) == names
    for n in names:
        assert hasattr(lib, n), n


def test_struct_layout_matches_header(tmp_path):
    from draft_verification_gb300 import _lib
    cuda_inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if shutil.which("gcc") is None or not os.path.exists(os.path.join(cuda_inc, "cuda_runtime_api.h")):
        pytest.skip("gcc or CUDA headers missing")
    structs = {"spec_process_args": _lib.ProcessArgs, "spec_quantize_int4_args": _lib.QuantizeInt4Args,
               "spec_int4_product_args": _lib.Int4ProductArgs}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "spec_logits.h"', "int main(void){"]
    for cname, py in structs.items():
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        for f, _ in py._fields_:
            lines.append(f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));')
    lines.append("return 0;}")
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", cuda_inc, str(src), "-o", str(exe)],
                   check=True)
    got = {}
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n"):
        if line:
            s, f, v = line.split()
            got[(s, f)] = int(v)
    for cname, py in structs.items():
        assert got[(cname, "size")] == C.sizeof(py), cname
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset, (cname, f)


FAKE = 0x10000  # never dereferenced: validation fails first


def _fill(a, pointers, kw):
    for f in pointers:
        setattr(a, f, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _process(**kw):
    from draft_verification_gb300 import _lib
    a = _lib.ProcessArgs()
    a.B, a.n, a.V, a.dtype, a.ld, a.out_ld = 2, 4, 100, _lib.SPEC_BF16, 100, 100
    a.tokens_ld, a.history_ld, a.bias_ld, a.mask_rows, a.mask_ld = 4, 7, 3, 8, 4
    a.workspace_bytes = 1 << 30
    return _fill(a, ("logits", "tokens", "history", "bias_tokens", "bias_values", "mask", "workspace"),
                 {"out": 0x20000, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), -1), (dict(B=65536), -1), (dict(n=0), -1), (dict(n=1025), -1), (dict(V=0), -1),
    (dict(V=2097153, ld=2097153, out_ld=2097153), -1), (dict(ld=99), -1), (dict(out_ld=99), -1),
    (dict(logits=None), -1), (dict(out=None), -1), (dict(dtype=7), -2), (dict(logits=FAKE + 8), -3),
    (dict(out=FAKE + 2), -3), (dict(out=FAKE, out_ld=104), -1), (dict(tokens_ld=2), -1),
    (dict(parent=FAKE, tokens_ld=3), -1), (dict(parent=FAKE, tokens=None), -1), (dict(history_ld=-1), -1),
    (dict(bias_values=None), -1), (dict(bias_ld=-1), -1), (dict(mask_rows=0), -1), (dict(mask_rows=7), -1),
    (dict(mask_ld=3), -1), (dict(workspace=None), -4), (dict(workspace_bytes=64), -4), (dict(workspace=FAKE + 16), -4),
])
def test_process_refusals(lib, kw, code):
    assert lib.spec_process_logits(C.byref(_process(**kw)), None) == code
    assert lib.spec_process_logits(None, None) == -1


def _quantize(**kw):
    from draft_verification_gb300 import _lib
    a = _lib.QuantizeInt4Args()
    a.V, a.d, a.group, a.dtype, a.ld, a.codes_ld, a.scales_ld, a.zeros_ld = 10, 256, 64, _lib.SPEC_BF16, 256, 128, 10, 10
    return _fill(a, ("weights", "codes", "scales", "zeros"), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(V=0), -1), (dict(V=2097153), -1), (dict(d=0), -1), (dict(d=65600), -1), (dict(d=96), -1),
    (dict(group=16), -1), (dict(group=256), -1), (dict(ld=255), -1), (dict(codes_ld=112), -1),
    (dict(codes_ld=136), -1), (dict(scales_ld=9), -1), (dict(zeros_ld=9), -1), (dict(weights=None), -1),
    (dict(codes=None), -1), (dict(scales=None), -1), (dict(dtype=3), -2), (dict(weights=FAKE + 1), -3),
    (dict(codes=FAKE + 8), -3), (dict(scales=FAKE + 1), -3),
])
def test_quantize_refusals(lib, kw, code):
    assert lib.spec_quantize_int4(C.byref(_quantize(**kw)), None) == code
    assert lib.spec_quantize_int4(None, None) == -1


def _product(**kw):
    from draft_verification_gb300 import _lib
    a = _lib.Int4ProductArgs()
    a.R, a.V, a.d, a.group, a.out_dtype = 3, 10, 256, 64, _lib.SPEC_F32
    a.x_ld, a.codes_ld, a.scales_ld, a.zeros_ld, a.out_ld = 256, 128, 10, 10, 10
    a.workspace_bytes = 1 << 30
    return _fill(a, ("x", "codes", "scales", "zeros", "out", "workspace"), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), -1), (dict(R=65536), -1), (dict(V=0), -1), (dict(d=96), -1), (dict(group=48), -1),
    (dict(x_ld=255), -1), (dict(x_ld=260), -1), (dict(codes_ld=112), -1), (dict(codes_ld=136), -1),
    (dict(scales_ld=9), -1), (dict(zeros_ld=9), -1), (dict(out_ld=9), -1), (dict(x=None), -1),
    (dict(codes=None), -1), (dict(scales=None), -1), (dict(out=None), -1), (dict(out_dtype=4), -2),
    (dict(x=FAKE + 8), -3), (dict(codes=FAKE + 8), -3), (dict(scales=FAKE + 1), -3), (dict(out=FAKE + 2), -3),
    (dict(workspace=None), -4), (dict(workspace_bytes=0), -4), (dict(workspace=FAKE + 16), -4),
])
def test_product_refusals(lib, kw, code):
    assert lib.spec_int4_product(C.byref(_product(**kw)), None) == code
    assert lib.spec_int4_product(None, None) == -1


def test_product_workspace_size_is_zero_outside_the_limits(lib):
    size = lib.spec_int4_product_workspace_size
    assert size(1, 1000, 256, 128) > 0
    for bad in [(0, 10, 256, 64), (65536, 10, 256, 64), (1, 0, 256, 64), (1, 2097153, 256, 64), (1, 10, 96, 64),
                (1, 10, 256, 16), (1, 10, 65664, 128)]:
        assert size(*bad) == 0, bad


def test_process_workspace_size_is_zero_outside_the_limits(lib):
    size = lib.spec_process_workspace_size
    assert size(1, 1, 10, 0, 0) > 0
    for bad in [(0, 1, 10, 0, 0), (65536, 1, 10, 0, 0), (1, 0, 10, 0, 0), (1, 1025, 10, 0, 0), (1, 1, 0, 0, 0),
                (1, 1, 2097153, 0, 0), (1, 1, 10, -1, 0), (1, 1, 10, 0, -1)]:
        assert size(*bad) == 0, bad


def test_process_plan_refusals():
    from draft_verification_gb300 import ProcessLogitsPlan
    x = torch.zeros(2, 3, 50)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    tok = i32(2, 3)
    with pytest.raises(TypeError):
        ProcessLogitsPlan(x.double())
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x[0])
    with pytest.raises(ValueError):
        ProcessLogitsPlan(torch.zeros(2, 3, 100)[:, :, ::2])
    with pytest.raises(ValueError):
        ProcessLogitsPlan(torch.zeros(2, 5, 50)[:, :3])            # rows not evenly strided
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x, tok[:, :1])                           # a chain needs n - 1 drafted tokens
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x, tok[:, :2].contiguous(), parent=tok)  # a tree needs n
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x, parent=tok)
    with pytest.raises(TypeError):
        ProcessLogitsPlan(x, tok.long())
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x, tok, history_len=i32(2))
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x, tok, history=i32(3, 4))
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x, tok, history=i32(2, 4), history_len=i32(3))
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x, tok, bias_tokens=i32(2, 4))
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x, tok, bias_tokens=i32(2, 4), bias_values=torch.zeros(2, 5))
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x, tok, mask_index=i32(2, 3))
    with pytest.raises(TypeError):
        ProcessLogitsPlan(x, tok, mask=torch.ones(6, 50, dtype=torch.bool))
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x, tok, mask=i32(6, 1))                  # 50 tokens are two words
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x, tok, mask=i32(5, 2))                  # one row each without an index
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x, tok, repetition=torch.ones(3))
    with pytest.raises(TypeError):
        ProcessLogitsPlan(x, tok, out=x.bfloat16())
    with pytest.raises(ValueError):
        ProcessLogitsPlan(x, tok, out=torch.zeros(2, 3, 51))


def test_int4_plan_refusals():
    from draft_verification_gb300 import Int4ProductPlan, QuantizeInt4Plan
    with pytest.raises(TypeError):
        QuantizeInt4Plan(torch.zeros(4, 64, dtype=torch.float64))
    with pytest.raises(ValueError):
        QuantizeInt4Plan(torch.zeros(4, 96), group=64)
    with pytest.raises(ValueError):
        QuantizeInt4Plan(torch.zeros(4, 128).t(), group=32)
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    codes = torch.zeros(10, 32, dtype=torch.uint8)
    scales = torch.zeros(2, 10, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        Int4ProductPlan(x.float(), codes, scales, group=32)
    with pytest.raises(TypeError):
        Int4ProductPlan(x, codes.int(), scales, group=32)
    with pytest.raises(TypeError):
        Int4ProductPlan(x, codes, scales.float(), group=32)
    with pytest.raises(TypeError):
        Int4ProductPlan(x, codes, scales, group=32, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        Int4ProductPlan(x, codes, scales, group=48)
    with pytest.raises(ValueError):
        Int4ProductPlan(x, codes, scales, group=64)                # one group: one row of scales
    with pytest.raises(ValueError):
        Int4ProductPlan(x, codes[:, :16], scales, group=32)
    with pytest.raises(ValueError):
        Int4ProductPlan(x, codes, scales, scales.to(torch.uint8)[:1], group=32)
