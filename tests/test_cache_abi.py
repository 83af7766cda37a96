"""The cache operators without a GPU: include/spec_cache.h against the binding,
the refusals of the C entry points and of the plans, the frequencies."""

import ctypes as C
import math
import os
import re
import shutil
import subprocess

import pytest
import torch

import draft_verification_gb300 as dv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "spec_cache.h")


@pytest.fixture(scope="module")
def lib():
    from draft_verification_gb300 import _lib, build
    if shutil.which("nvcc") is None and not os.path.exists(build.lib_path()):
        pytest.skip("neither nvcc nor a built library is available")
    build.build()
    return _lib.lib()


def test_every_declared_symbol_is_exported(lib):
    from draft_verification_gb300 import _lib
    names = sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(spec_\w+)\s*\(", open(HEADER).read(), re.M)))
    assert sorted(_lib.CACHE_SIGNATURES) == names
    for n in names:
        assert hasattr(lib, n), n


def test_struct_layout_matches_header(tmp_path):
    from draft_verification_gb300 import _lib
    cuda_inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if shutil.which("gcc") is None or not os.path.exists(os.path.join(cuda_inc, "cuda_runtime_api.h")):
        pytest.skip("gcc or CUDA headers missing")
    structs = {"spec_rotate_args": _lib.RotateArgs, "spec_append_args": _lib.AppendArgs,
               "spec_attend_args": _lib.AttendArgs}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "spec_cache.h"', "int main(void){"]
    for cname, py in structs.items():
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        for f, _ in py._fields_:
            lines.append(f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));')
    lines.append(f'printf("bits %d %d\\n", SPEC_ERR_CACHE, SPEC_ERR_POSITION);')
    lines.append("return 0;}")
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", cuda_inc, str(src), "-o", str(exe)], check=True)
    text = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    got = {tuple(line.split()[:2]): int(line.split()[2]) for line in text.splitlines()}
    for cname, py in structs.items():
        assert got[(cname, "size")] == C.sizeof(py), cname
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset, (cname, f)
    assert got[("bits", str(_lib.ERR_CACHE))] == _lib.ERR_POSITION


FAKE = 0x10000  # never dereferenced: validation fails first


def _fill(a, pointers, kw):
    for f in pointers:
        setattr(a, f, FAKE)
    for k, v in kw.items():
        if k.endswith("_ld"):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


def _rotate(**kw):
    from draft_verification_gb300 import _lib
    a = _lib.RotateArgs()
    a.B, a.n, a.H, a.D, a.rot, a.dtype, a.table_rows = 2, 3, 4, 64, 64, _lib.SPEC_BF16, 10
    a.x_ld[:] = a.out_ld[:] = (768, 256, 64)
    return _fill(a, ("x", "table"), {"out": 0x20000, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), -1), (dict(B=65536), -1), (dict(n=0), -1), (dict(n=2 ** 20 + 1), -1), (dict(H=0), -1),
    (dict(H=1025), -1), (dict(D=0), -1), (dict(D=1026), -1), (dict(D=65, rot=64), -1), (dict(rot=0), -1),
    (dict(rot=66), -1), (dict(rot=3), -1), (dict(table_rows=0), -1), (dict(x=None), -1), (dict(out=None), -1),
    (dict(table=None), -1), (dict(dtype=9), -2), (dict(x=FAKE + 1), -3), (dict(out=FAKE + 1), -3),
    (dict(table=FAKE + 8), -3), (dict(out=FAKE, out_ld=(768, 256, 72)), -1),
])
def test_rotate_refusals(lib, kw, code):
    assert lib.spec_rotate_heads(C.byref(_rotate(**kw)), None) == code
    assert lib.spec_rotate_heads(None, None) == -1


@pytest.mark.parametrize("args,code", [
    ((0, 64, FAKE, 1.0, FAKE), -1), ((2 ** 30 + 1, 64, FAKE, 1.0, FAKE), -1), ((5, 0, FAKE, 1.0, FAKE), -1),
    ((5, 63, FAKE, 1.0, FAKE), -1), ((5, 1026, FAKE, 1.0, FAKE), -1), ((5, 64, None, 1.0, FAKE), -1),
    ((5, 64, FAKE, math.inf, FAKE), -1), ((5, 64, FAKE, 1.0, None), -1), ((5, 64, FAKE + 4, 1.0, FAKE), -3),
    ((5, 64, FAKE, 1.0, FAKE + 2), -3),
])
def test_table_refusals(lib, args, code):
    assert lib.spec_rotation_table(*args, None) == code


def _append(**kw):
    from draft_verification_gb300 import _lib
    a = _lib.AppendArgs()
    a.B, a.n, a.H, a.D, a.page, a.pages, a.table_pages = 2, 3, 4, 64, 16, 20, 5
    a.rot, a.table_rows, a.dtype = 64, 100, _lib.SPEC_BF16
    a.k_ld[:] = a.v_ld[:] = (768, 256, 64)
    return _fill(a, ("k", "v", "table", "block_table", "k_codes", "v_codes", "k_exps", "v_exps"), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), -1), (dict(B=65536), -1), (dict(n=0), -1), (dict(n=2 ** 20 + 1), -1), (dict(H=0), -1),
    (dict(D=8), -1), (dict(D=72, rot=64), -1), (dict(D=272), -1), (dict(page=8), -1), (dict(page=48), -1),
    (dict(pages=0), -1), (dict(pages=2 ** 26), -1), (dict(table_pages=0), -1), (dict(table_pages=2 ** 27), -1),
    (dict(rot=66), -1), (dict(rot=-2), -1), (dict(rot=5), -1), (dict(table_rows=0), -1), (dict(table=None), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(block_table=None), -1), (dict(k_codes=None), -1),
    (dict(v_codes=None), -1), (dict(k_exps=None), -1), (dict(v_exps=None), -1), (dict(path_nodes=FAKE), -1),
    (dict(path_len=FAKE), -1), (dict(path_nodes=FAKE, path_len=FAKE, count=FAKE), -1),
    (dict(path_nodes=FAKE, path_len=FAKE, max_depth=-1), -1),
    (dict(path_nodes=FAKE, path_len=FAKE, max_depth=65535), -1), (dict(dtype=5), -2), (dict(k=FAKE + 1), -3),
    (dict(v=FAKE + 1), -3), (dict(table=FAKE + 4), -3), (dict(k_codes=FAKE + 8), -3), (dict(v_codes=FAKE + 8), -3),
])
def test_append_refusals(lib, kw, code):
    assert lib.spec_append_cache(C.byref(_append(**kw)), None) == code
    assert lib.spec_append_cache(None, None) == -1


def _attend(**kw):
    from draft_verification_gb300 import _lib
    a = _lib.AttendArgs()
    a.B, a.n, a.Hq, a.H, a.D, a.page, a.pages, a.table_pages, a.scale = 2, 3, 8, 4, 64, 16, 20, 5, 0.125
    a.q_ld[:] = a.out_ld[:] = (1536, 512, 64)
    a.workspace_bytes = 1 << 40
    return _fill(a, ("q", "out", "block_table", "k_codes", "v_codes", "k_exps", "v_exps", "workspace"), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), -1), (dict(B=65536), -1), (dict(n=0), -1), (dict(n=1025), -1), (dict(Hq=6), -1), (dict(Hq=2), -1),
    (dict(Hq=1028), -1), (dict(H=0), -1), (dict(D=8), -1), (dict(D=72), -1), (dict(D=272), -1), (dict(page=0), -1),
    (dict(pages=0), -1), (dict(pages=2 ** 26), -1), (dict(table_pages=0), -1), (dict(table_pages=2 ** 27), -1),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=math.nan), -1), (dict(scale=math.inf), -1),
    (dict(q=None), -1), (dict(out=None), -1), (dict(block_table=None), -1), (dict(k_codes=None), -1),
    (dict(v_codes=None), -1), (dict(k_exps=None), -1), (dict(v_exps=None), -1), (dict(q=FAKE + 8), -3),
    (dict(q_ld=(1536, 516, 64)), -3), (dict(out=FAKE + 1), -3), (dict(k_codes=FAKE + 8), -3),
    (dict(v_codes=FAKE + 8), -3), (dict(workspace=None), -4), (dict(workspace_bytes=16), -4),
    (dict(workspace=FAKE + 16), -4),
])
def test_attend_refusals(lib, kw, code):
    assert lib.spec_attend_cache(C.byref(_attend(**kw)), None) == code
    assert lib.spec_attend_cache(None, None) == -1


def test_workspace_sizes(lib):
    assert lib.spec_attend_workspace_size(2, 3, 8, 4, 64) > 0
    for bad in ((0, 3, 8, 4, 64), (2, 0, 8, 4, 64), (2, 3, 7, 4, 64), (2, 3, 8, 4, 60), (2, 1025, 8, 4, 64)):
        assert lib.spec_attend_workspace_size(*bad) == 0


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def cache(pages=4, H=2, page=16, D=64):
    return dv.PagedCache.empty(pages, H, page, D, device="cpu")


@pytest.mark.parametrize("make,error", [
    (lambda: dv.PagedCache.empty(4, 2, 24, 64, device="cpu"), ValueError),
    (lambda: dv.PagedCache.empty(4, 2, 16, 60, device="cpu"), ValueError),
    (lambda: dv.PagedCache.empty(0, 2, 16, 64, device="cpu"), ValueError),
    (lambda: dv.PagedCache(i32(4, 2, 16, 64), i32(4, 2, 16, 64), i32(4, 2), i32(4, 2)), TypeError),
    (lambda: dv.PagedCache(cache().k_codes, cache().v_codes, cache().k_exps, cache(5).v_exps), ValueError),
    (lambda: dv.PagedCache(cache().k_codes.transpose(0, 1), cache().v_codes, cache().k_exps, cache().v_exps), TypeError),
    (lambda: dv.RotateHeadsPlan(bf(2, 3, 64), torch.zeros(5, 64)), ValueError),
    (lambda: dv.RotateHeadsPlan(bf(2, 3, 4, 64).half(), torch.zeros(5, 64)), TypeError),
    (lambda: dv.RotateHeadsPlan(bf(2, 3, 64, 4).transpose(2, 3), torch.zeros(5, 64)), ValueError),
    (lambda: dv.RotateHeadsPlan(bf(2, 3, 4, 64), torch.zeros(5, 66)), ValueError),
    (lambda: dv.RotateHeadsPlan(bf(2, 3, 4, 64), torch.zeros(5, 63)), ValueError),
    (lambda: dv.RotateHeadsPlan(bf(2, 3, 4, 64), bf(5, 64)), TypeError),
    (lambda: dv.RotateHeadsPlan(bf(2, 3, 4, 64), torch.zeros(5, 64), positions=i32(2, 4)), ValueError),
    (lambda: dv.RotateHeadsPlan(bf(2, 3, 4, 64), torch.zeros(5, 64), positions=i32(2, 3).long()), TypeError),
    (lambda: dv.RotateHeadsPlan(bf(2, 3, 4, 64), torch.zeros(5, 64), positions=i32(2, 3), prefix_len=i32(2)), ValueError),
    (lambda: dv.RotateHeadsPlan(bf(2, 3, 4, 64), torch.zeros(5, 64), out=bf(2, 3, 4, 64).float()), TypeError),
    (lambda: dv.RotateHeadsPlan(bf(2, 3, 4, 64), torch.zeros(5, 64), out=bf(2, 3, 1, 64).expand(2, 3, 4, 64)), ValueError),
    (lambda: dv.AppendCachePlan(bf(2, 3, 4, 64), bf(2, 3, 4, 64), cache(), i32(2, 4)), ValueError),
    (lambda: dv.AppendCachePlan(bf(2, 3, 2, 64), bf(2, 3, 2, 64).float(), cache(), i32(2, 4)), TypeError),
    (lambda: dv.AppendCachePlan(bf(2, 3, 2, 64), bf(2, 4, 2, 64), cache(), i32(2, 4)), ValueError),
    (lambda: dv.AppendCachePlan(bf(2, 3, 2, 64), bf(2, 3, 2, 64), cache(), i32(3, 4)), ValueError),
    (lambda: dv.AppendCachePlan(bf(2, 3, 2, 64), bf(2, 3, 2, 64), cache(), i32(2, 4), positions=i32(2, 3)), ValueError),
    (lambda: dv.AppendCachePlan(bf(2, 3, 2, 64), bf(2, 3, 2, 64), cache(), i32(2, 4), path_nodes=i32(2, 3)), ValueError),
    (lambda: dv.AppendCachePlan(bf(2, 3, 2, 64), bf(2, 3, 2, 64), cache(), i32(2, 4), path_nodes=i32(2, 3),
                                path_len=i32(2), count=i32(2)), ValueError),
    (lambda: dv.AppendCachePlan(bf(2, 3, 2, 64), bf(2, 3, 2, 64), cache(), i32(2, 4), i32(3)), ValueError),
    (lambda: dv.AttendCachePlan(bf(2, 3, 3, 64), cache(), i32(2, 4)), ValueError),
    (lambda: dv.AttendCachePlan(bf(2, 3, 4, 32), cache(), i32(2, 4)), ValueError),
    (lambda: dv.AttendCachePlan(bf(2, 3, 4, 64).float(), cache(), i32(2, 4)), TypeError),
    (lambda: dv.AttendCachePlan(bf(2, 3, 4, 64), cache(), i32(2, 4), parent=i32(2, 4)), ValueError),
    (lambda: dv.AttendCachePlan(bf(2, 3, 4, 64), cache(), i32(2, 4), count=i32(3)), ValueError),
    (lambda: dv.AttendCachePlan(bf(2, 3, 4, 64), cache(), i32(2, 4), out=bf(2, 3, 4, 32)), ValueError),
    (lambda: dv.AttendCachePlan(bf(2, 1025, 4, 64), cache(), i32(2, 4)), ValueError),
    (lambda: dv.rotation_table(5, 64, device="cpu"), ValueError),
    (lambda: dv.rotation_table(5, 64, freq=torch.zeros(31, dtype=torch.float64)), ValueError),
    (lambda: dv.rotary_frequencies(7), ValueError),
    (lambda: dv.rotary_frequencies(8, bands=(4.0, 4.0, 1.0, 100)), ValueError),
])
def test_plan_refusals(lib, make, error):
    with pytest.raises(error):
        make()


def test_plans_on_host_tensors_refuse_to_run(lib):
    for plan in (dv.RotateHeadsPlan(bf(2, 3, 4, 64), torch.zeros(5, 64)),
                 dv.AppendCachePlan(bf(2, 3, 2, 64), bf(2, 3, 2, 64), cache(), i32(2, 4)),
                 dv.AttendCachePlan(bf(2, 3, 4, 64), cache(), i32(2, 4))):
        with pytest.raises(ValueError, match="CUDA tensors required"):
            plan.run()


def test_frequencies():
    f = dv.rotary_frequencies(8, 10000.0)
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64))
    assert torch.equal(dv.rotary_frequencies(8, 10000.0, linear=4.0), f / 4)
    # wavelengths 6.3, 63, 628, 6283 of a length of 1000: 159, 15.9, 1.59 and 0.159 turns
    g = dv.rotary_frequencies(8, 10000.0, bands=(8.0, 1.0, 4.0, 1000.0))
    assert torch.equal(g[:2], f[:2]) and math.isclose(g[3], f[3] / 8, rel_tol=1e-12)
    share = (1000 * 0.01 / (2 * math.pi) - 1.0) / 3.0
    assert math.isclose(g[2], 0.01 * (share + (1 - share) / 8), rel_tol=1e-9)


def test_cache_values():
    c = cache()
    c.k_codes[1, 0, 3, 5] = 0x38
    c.k_exps[1, 0] = -3
    k, v = c.values()
    assert k[1, 0, 3, 5] == 0.125 and k.abs().sum() == 0.125 and not v.any()
