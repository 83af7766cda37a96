"""The logit-side operators on the GPU against the float64 oracle.

Tolerances, with u = finfo(type).eps / 2 the half step of a type:
  processing   every float32 step of an element is off by at most u32 of its
               result, so the value before the last rounding is off by at most
               (steps) u32 of the magnitudes the oracle adds up (`scale`); the
               last rounding adds u of the result.  Elements nothing applies
               to keep their bits.
  quantisation the bits are the rule's: equality.
  products     a group's sum and the sum over the groups are float32 sums of
               d terms and d / group scaled sums in an order of the kernel's;
               each addition may truncate (a whole step, 2 u32) and each
               product of a scale rounds once, so the value is off by at most
               2 u32 (group + 2 d / group + 2) times the sum of the terms'
               magnitudes; the last rounding adds u of the result.
"""

import numpy as np
import pytest
import torch

from oracle import logits as O

pytestmark = pytest.mark.gpu

U32 = torch.finfo(torch.float32).eps / 2
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def dev(a, device):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(device)


def values(t):
    return t.double().cpu().numpy()


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).cpu().numpy()


# ---------------------------------------------------------------------------
# processing
# ---------------------------------------------------------------------------

def strided(B, n, V, pad, dtype, device):
    return torch.empty((B, n, V + pad), dtype=dtype, device=device)[:, :, :V]


def make_process(rng, B, n, V, H=20, tree=False, bias=5, density=None, rho=True):
    w = dict(tokens=rng.integers(0, V, (B, n), dtype=np.int32))
    # few distinct tokens: histories and paths repeat them
    few = rng.integers(0, V, 6, dtype=np.int32)
    pick = rng.random((B, n)) < 0.6
    w["tokens"] = np.where(pick, few[rng.integers(0, 6, (B, n))], w["tokens"]).astype(np.int32)
    if tree:
        w["parent"] = np.array([[-1] + [int(rng.integers(max(0, i - 5), i)) for i in range(1, n)] for _ in range(B)],
                               np.int32)
    if H is not None:
        h = rng.integers(0, V, (B, H), dtype=np.int32)
        w["history"] = np.where(rng.random((B, H)) < 0.5, few[rng.integers(0, 6, (B, H))], h).astype(np.int32)
        w["history_len"] = rng.integers(0, H + 1, B, dtype=np.int32)
        w["prompt_len"] = rng.integers(0, H + 1, B, dtype=np.int32)
    if rho:
        w["repetition"] = rng.uniform(0.5, 2.0, B).astype(np.float32)
        w["frequency"] = rng.uniform(-0.5, 1.0, B).astype(np.float32)
        w["presence"] = rng.uniform(-0.5, 1.0, B).astype(np.float32)
    if bias:
        t = rng.integers(0, V, (B, bias), dtype=np.int32)
        w["bias_tokens"] = np.where(rng.random((B, bias)) < 0.5, few[rng.integers(0, 6, (B, bias))], t).astype(np.int32)
        w["bias_values"] = rng.normal(0, 5, (B, bias)).astype(np.float32)
        w["bias_len"] = rng.integers(0, bias + 1, B, dtype=np.int32)
    if density is not None:
        words = (V + 31) // 32
        rows = max(3, B * n // 2)
        p = np.array([density, 1.0, 0.0])[np.minimum(np.arange(rows), 2)] if rows == 3 else rng.random(rows) * density
        on = rng.random((rows, words * 32)) < p[:, None]
        if rows > 3:
            on[0], on[1] = True, False  # one row allows everything, one nothing
        w["mask"] = np.packbits(on, axis=1, bitorder="little").view(np.int32)
        w["mask_index"] = rng.integers(-1, rows, (B, n), dtype=np.int32)
    return w


def run_process(logits, w, device, out=None, stream=None):
    import draft_verification_gb300 as dv
    kw = {k: dev(v, device) for k, v in w.items() if k != "tokens"}
    return dv.ProcessLogitsPlan(logits, dev(w.get("tokens"), device), out=out, **kw).run(stream)


def check_process(x, out, w):
    """x: the logits as they were (a copy); out: run()'s result."""
    dtype = x.dtype
    got = values(out["logits"])
    want, touched, scale, err = O.process_logits(values(x), **w)
    assert np.array_equal(out["seq_error"].cpu().numpy(), err), (out["seq_error"], err)
    assert int(out["error_word"]) == int(np.bitwise_or.reduce(err))
    assert np.array_equal(bits(out["logits"])[~touched], bits(x)[~touched])
    steps = 6 + (0 if "bias_tokens" not in w else w["bias_tokens"].shape[1])
    u = half_step(dtype)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(want), np.isnan(got))
    assert np.array_equal(want[~fin & ~np.isnan(want)], got[~fin & ~np.isnan(want)])
    tol = u * np.abs(want[fin]) + (1 + u) * steps * U32 * scale[fin]
    off = np.abs(got[fin] - want[fin]) - tol
    assert not off.size or off.max() <= 0, off.max()


PROCESS = [
    # B, n, V, pad, dtype, kwargs
    (1, 1, 1, 0, "f32", dict(H=3, bias=2)),
    (1, 1, 1, 0, "bf16", dict(H=0, bias=0, density=0.5)),
    (2, 3, 7, 0, "bf16", dict(density=0.5)),
    (3, 5, 31, 1, "f32", dict(density=0.5)),
    (2, 4, 33, 3, "bf16", dict(density=0.9)),
    (4, 5, 1000, 0, "f32", dict(H=37, density=0.3)),
    (2, 9, 2047, 0, "bf16", dict(H=100)),
    (2, 3, 2048, 0, "bf16", dict(density=0.2)),
    (2, 3, 2049, 7, "bf16", dict(density=0.2)),
    (3, 2, 4099, 0, "f32", dict(H=5000, bias=70)),
    (1, 64, 5003, 0, "bf16", dict(tree=True, density=0.3)),
    (16, 7, 50257, 0, "bf16", dict(tree=True, density=0.1, H=777)),
    (40, 3, 66001, 0, "bf16", dict(H=3000, bias=300, density=0.5)),      # the long slabs, every alignment
    (40, 2, 66000, 8, "bf16", dict(H=300, bias=0)),
    (24, 3, 66003, 2, "f32", dict(H=300, density=0.5)),
    (1, 300, 1200, 0, "f32", dict(H=64, density=0.5)),                    # a long chain, split into parts
    (700, 2, 300, 0, "bf16", dict(H=9, density=0.5)),
    (2, 4, 4000, 0, "f32", dict(H=None, bias=0, rho=False, density=0.5)),  # a mask alone
    (2, 4, 4000, 0, "bf16", dict(H=None, bias=0, rho=True)),               # drafted tokens alone
    (2, 4, 4000, 0, "bf16", dict(H=20, bias=33, rho=False)),               # biases alone
]


@pytest.mark.parametrize("B,n,V,pad,dtype,kw", PROCESS, ids=lambda v: str(v) if not isinstance(v, dict) else None)
def test_process(cuda_device, B, n, V, pad, dtype, kw):
    rng = np.random.default_rng(B * 7919 + n * 104729 + V)
    w = make_process(rng, B, n, V, **kw)
    x = strided(B, n, V, pad, DTYPES[dtype], cuda_device)
    x.copy_(torch.from_numpy(rng.normal(0, 3, (B, n, V)).astype(np.float32)))
    x0 = x.clone()
    out = run_process(x, w, cuda_device)
    assert np.array_equal(bits(x), bits(x0))
    check_process(x0, out, w)
    first = bits(out["logits"]).copy()
    # other output strides (rows that start at other offsets than the input's)
    for other in (pad + 1, pad + 8):
        y = strided(B, n, V, other, DTYPES[dtype], cuda_device)
        assert np.array_equal(bits(run_process(x, w, cuda_device, out=y)["logits"]), first)
    # in place
    assert np.array_equal(bits(run_process(x, w, cuda_device, out=x)["logits"]), first)
    assert np.array_equal(bits(x), first)


@pytest.mark.parametrize("B,n,V,pad,dtype,kw", [
    # more tokens than one bitmap holds
    (3, 3, 300001, 0, "bf16", dict(H=500, bias=40, density=0.5)),
    (3, 2, 300001, 3, "f32", dict(H=501, bias=3)),
    # exactly one bitmap, and one token more
    (6, 2, 262144, 0, "bf16", dict(H=300, tree=True)),
    (6, 2, 262145, 7, "bf16", dict(H=300)),
    # more distinct tokens than one window holds
    (40, 2, 66000, 0, "bf16", dict(H=40000, bias=500)),
    (24, 2, 66001, 0, "f32", dict(H=40001, bias=9)),
    # more entries in a slab than are kept in shared memory, from one slab and from two
    (60, 2, 20000, 0, "bf16", dict(H=40000, bias=10, density=0.8)),
    (60, 2, 20001, 0, "bf16", dict(H=40002, bias=10)),
    # a wide tree
    (2, 257, 33000, 8, "bf16", dict(H=64, tree=True)),
    # the same sizes with histories long enough to be gathered first
    (3, 3, 300001, 0, "bf16", dict(H=60000, bias=40, density=0.5)),
    (3, 2, 300001, 3, "f32", dict(H=30001, bias=3)),
    (6, 2, 262144, 0, "bf16", dict(H=30000, tree=True)),
    (6, 2, 262145, 7, "bf16", dict(H=30000, density=0.3)),
    (40, 5, 66000, 3, "bf16", dict(H=14000, tree=True, bias=0)),
], ids=lambda v: str(v) if not isinstance(v, dict) else None)
def test_process_large(cuda_device, B, n, V, pad, dtype, kw):
    rng = np.random.default_rng(B * 7919 + n * 104729 + V)
    w = make_process(rng, B, n, V, **kw)
    w["history_len"][::2] = kw["H"]
    x = strided(B, n, V, pad, DTYPES[dtype], cuda_device)
    x.copy_(torch.from_numpy(rng.normal(0, 3, (B, n, V)).astype(np.float32)))
    out = run_process(x, w, cuda_device)
    check_process(x, out, w)
    first = bits(out["logits"]).copy()
    assert np.array_equal(bits(run_process(x, w, cuda_device, out=x)["logits"]), first)


def test_process_special_values(cuda_device):
    """Infinities and NaN in masked, penalised and untouched places; a mask
    row of nothing; biases of -inf and of the type's lowest value."""
    B, n, V = 2, 3, 2500
    rng = np.random.default_rng(3)
    for dtype in DTYPES.values():
        w = make_process(rng, B, n, V, H=200, bias=0, density=0.4)
        x = torch.from_numpy(rng.normal(0, 3, (B, n, V)).astype(np.float32)).to(cuda_device, dtype)
        for k, v in enumerate((float("inf"), -float("inf"), float("nan"), -0.0, torch.finfo(dtype).min)):
            x[:, :, k::11] = v
        w["bias_tokens"] = np.tile(np.arange(0, 60, 2, dtype=np.int32), (B, 1))
        w["bias_values"] = np.tile(np.array([-np.inf, np.finfo(np.float32).min, 1.0] * 10, np.float32), (B, 1))
        w["bias_len"] = np.array([30, 17], np.int32)
        out = run_process(x, w, cuda_device)
        got = values(out["logits"])
        want, touched, _, _ = O.process_logits(values(x), **w)
        assert np.array_equal(bits(out["logits"])[~touched], bits(x)[~touched])
        assert np.array_equal(np.isnan(got), np.isnan(want))
        # the lowest value plus more rounds to it or to -inf: compare after rounding to the type
        rounded = values(torch.from_numpy(want).to(dtype))
        big = np.abs(want) > 1e30
        assert np.array_equal(got[big], rounded[big])
        nothing = ~w["mask"].any(axis=1)  # mask rows that allow no token
        masked = (w["mask_index"] >= 0) & nothing[np.maximum(w["mask_index"], 0)]
        assert np.isneginf(got[masked]).all()


def test_process_a_deep_and_a_wide_tree(cuda_device):
    rng = np.random.default_rng(5)
    n, V = 1024, 700
    for parent in (np.arange(-1, n - 1), np.r_[-1, np.zeros(n - 1, int)], np.r_[-1, (np.arange(1, n) - 1) // 2]):
        w = make_process(rng, 1, n, V, H=50, bias=0)
        w["parent"] = parent[None].astype(np.int32)
        x = torch.from_numpy(rng.normal(0, 3, (1, n, V)).astype(np.float32)).to(cuda_device)
        check_process(x, run_process(x, w, cuda_device), w)


@pytest.mark.parametrize("V,H", [(900, 30), (70000, 30), (300000, 30000)])  # the last: gathered first
def test_process_data_errors(cuda_device, V, H):
    rng = np.random.default_rng(6)
    B, n = 9, 4
    for tree in (False, True):
        w = make_process(rng, B, n, V, H=H, tree=tree, density=0.5)
        w["history_len"][:] = H
        w["bias_len"][:] = 5
        w["history"][0, 3], w["history"][1, 29] = -1, V
        w["history_len"][2], w["history_len"][3] = H + 1, -2
        w["tokens"][4, 1] = V + 5
        w["bias_tokens"][5, 2] = -7
        w["bias_len"][6] = 6
        w["mask_index"][7, 3] = w["mask"].shape[0]
        if tree:
            w["parent"][8, 2] = 2
        x = torch.from_numpy(rng.normal(0, 3, (B, n, V)).astype(np.float32)).to(cuda_device)
        out = run_process(x, w, cuda_device)
        check_process(x, out, w)
        want = [1, 1, 1, 1, 1, 1, 1, 64, 2 if tree else 0]
        assert out["seq_error"].tolist() == want


@pytest.mark.parametrize("B,n,V,H", [(20, 5, 30001, 500), (60, 2, 20000, 30000)])  # one kernel, and gathered first
def test_process_deterministic_on_a_side_stream_and_in_a_graph(cuda_device, B, n, V, H):
    rng = np.random.default_rng(7)
    w = make_process(rng, B, n, V, H=H, density=0.5, bias=40)
    x = torch.from_numpy(rng.normal(0, 3, (B, n, V)).astype(np.float32)).to(cuda_device, torch.bfloat16)
    first = bits(run_process(x, w, cuda_device)["logits"]).copy()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = run_process(x, w, cuda_device)
    side.synchronize()
    assert np.array_equal(bits(out["logits"]), first)
    import draft_verification_gb300 as dv
    kw = {k: dev(v, cuda_device) for k, v in w.items() if k != "tokens"}
    plan = dv.ProcessLogitsPlan(x, dev(w["tokens"], cuda_device), **kw)
    plan.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    x.copy_(torch.from_numpy(rng.normal(0, 3, (B, n, V)).astype(np.float32)))
    graph.replay()
    torch.cuda.synchronize()
    check_process(x, plan.out, w)


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------

def check_quantize(w, out, group, zeros):
    codes, scales, z = O.quantize_int4(w.float().cpu().numpy(), group, zeros)
    assert np.array_equal(out["scales"].view(torch.int16).cpu().numpy().view(np.uint16), scales)
    assert np.array_equal(out["codes"].cpu().numpy(), codes)
    assert ("zeros" in out) == zeros
    if zeros:
        assert np.array_equal(out["zeros"].cpu().numpy(), z)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,d,group", [(1, 32, 32), (1, 128, 128), (31, 96, 32), (33, 192, 64), (100, 256, 128),
                                       (257, 1152, 128), (65, 2080, 32), (1000, 512, 64)])
def test_quantize(cuda_device, V, d, group, dtype, zeros):
    import draft_verification_gb300 as dv
    g = torch.Generator().manual_seed(V + d)
    # row magnitudes over the whole range of the type
    w = torch.randn(V, d, generator=g) * torch.exp2(torch.randint(-130, 120, (V, 1), generator=g).float())
    w[:, ::17] = 0.0
    w = w.to(cuda_device, DTYPES[dtype])
    check_quantize(w, dv.quantize_int4(w, group=group, zeros=zeros), group, zeros)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_ties_and_special_groups(cuda_device, dtype, zeros):
    import draft_verification_gb300 as dv
    group, V = 32, 70
    rng = np.random.default_rng(8)
    # small integers over power-of-two and odd scales: quotients that are exactly half way
    w = (rng.integers(-30, 31, (V, 4 * group)) * rng.choice([0.25, 0.5, 0.75, 1.0, 1.25, 3.0], (V, 1))).astype(np.float32)
    w[:, 0::group] = 15.0
    w[:, 1::group] = -14.0
    w[3] = 0.0
    w[4, :group] = -1.0     # one sign
    w[5, :group] = 1.0
    w[6, 2], w[7, 40], w[8, 100] = np.inf, -np.inf, np.nan
    w[9, :group] = 1e-40    # subnormal in float32 and bfloat16
    w[10, :2] = [3e38, -3e38]
    w[11] *= np.float32(2.0 ** -125)
    t = torch.from_numpy(w).to(cuda_device, DTYPES[dtype])
    check_quantize(t, dv.quantize_int4(t, group=group, zeros=zeros), group, zeros)


def test_quantize_strided_and_unaligned(cuda_device):
    import draft_verification_gb300 as dv
    g = torch.Generator().manual_seed(9)
    for dtype in DTYPES.values():
        wide = torch.randn(50, 401, generator=g).to(cuda_device, dtype)
        for first in (0, 1, 8):
            w = wide[:, first:first + 320]
            check_quantize(w, dv.quantize_int4(w, group=64, zeros=True), 64, True)
            one = wide[3:4, first:first + 320]
            check_quantize(one, dv.quantize_int4(one, group=32), 32, False)


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def make_product(R, V, d, group, zeros, seed, device):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (V, d // 2), generator=g, dtype=torch.uint8)
    scales = (torch.rand(d // group, V, generator=g) * 0.02 + 1e-3).bfloat16()
    z = torch.randint(0, 16, (d // group, V), generator=g, dtype=torch.uint8) if zeros else None
    x = (torch.randn(R, d, generator=g) + 0.3).bfloat16()
    return [None if t is None else t.to(device) for t in (x, codes, scales, z)]


def product_tolerance(mag, want, d, group, dtype):
    u = half_step(dtype)
    return u * np.abs(want) + (1 + u) * 2 * U32 * (group + 2 * d // group + 2) * mag


def check_product(got, x, codes, scales, z, group):
    sb = scales.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    want, mag = O.int4_product(values(x), codes.cpu().numpy(), sb, None if z is None else z.cpu().numpy(), group)
    off = np.abs(values(got) - want) - product_tolerance(mag, want, x.shape[1], group, got.dtype)
    assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))


@pytest.mark.parametrize("R,V,d,group,zeros,dtype", [
    (1, 1, 32, 32, False, "f32"),
    (1, 127, 64, 64, True, "bf16"),
    (1, 128, 128, 128, False, "f32"),
    (1, 129, 96, 32, True, "f32"),
    (1, 5003, 4096, 128, False, "bf16"),
    (2, 300, 256, 64, True, "f32"),
    (5, 1000, 256, 32, True, "f32"),
    (8, 2000, 1024, 128, True, "bf16"),
    (9, 500, 320, 64, False, "f32"),
    (16, 777, 512, 128, False, "f32"),
    (17, 777, 544, 32, False, "f32"),
    (31, 1300, 1920, 128, True, "bf16"),
    (33, 2500, 2048, 64, True, "f32"),
    (64, 900, 640, 32, True, "f32"),
    (65, 400, 384, 128, True, "f32"),
    (100, 19500, 512, 64, True, "bf16"),
    (128, 1000, 1024, 128, False, "f32"),
    (128, 1000, 1024, 32, True, "f32"),
    (129, 300, 256, 128, False, "f32"),
    (300, 260, 192, 64, True, "bf16"),
    (3, 100, 65536, 128, True, "f32"),       # the widest: many partial sums per entry
    (40, 100, 16384, 32, False, "f32"),
    (7, 39000, 256, 128, True, "f32"),       # many entries, little width
])
def test_product(cuda_device, R, V, d, group, zeros, dtype):
    import draft_verification_gb300 as dv
    x, codes, scales, z = make_product(R, V, d, group, zeros, R + V + d, cuda_device)
    plan = dv.Int4ProductPlan(x, codes, scales, z, group=group, out_dtype=DTYPES[dtype])
    out = plan.run()
    assert int(out["error_word"]) == 0
    check_product(out["logits"], x, codes, scales, z, group)
    first = bits(out["logits"]).copy()
    out["logits"].fill_(7.0)
    plan.run()  # the same plan and workspace again: the same bits
    assert np.array_equal(bits(out["logits"]), first)


@pytest.mark.parametrize("R,V,d,group,zeros,dtype", [
    (5, 1000, 8192, 128, False, "f32"),     # equal parts of tiles
    (300, 10000, 1024, 32, True, "bf16"),   # whole tiles, more than CTAs
    (70, 9000, 512, 64, True, "f32"),       # whole tiles, fewer
    (9, 9800, 5120, 64, True, "bf16"),      # evenly, fewer tiles than CTAs
    (400, 4990, 4096, 128, False, "f32"),   # evenly, more
])
def test_product_divisions(cuda_device, R, V, d, group, zeros, dtype):
    import draft_verification_gb300 as dv
    x, codes, scales, z = make_product(R, V, d, group, zeros, R + V, cuda_device)
    plan = dv.Int4ProductPlan(x, codes, scales, z, group=group, out_dtype=DTYPES[dtype])
    first = plan.run()["logits"].clone()
    check_product(first, x, codes, scales, z, group)
    for _ in range(5):
        assert torch.equal(plan.run()["logits"], first)
    assert int(plan.out["error_word"]) == 0


@pytest.mark.parametrize("R,V,d,group", [(1, 300, 512, 128), (33, 1000, 1024, 64), (128, 260, 768, 32)])
def test_product_of_small_integers_is_exact(cuda_device, R, V, d, group):
    """Integer hidden states and power-of-two scales: every sum is exact in float32, whatever its order."""
    import draft_verification_gb300 as dv
    g = torch.Generator().manual_seed(10)
    x = torch.randint(-4, 5, (R, d), generator=g).bfloat16().to(cuda_device)
    codes = torch.randint(0, 256, (V, d // 2), generator=g, dtype=torch.uint8).to(cuda_device)
    scales = torch.exp2(torch.randint(-2, 3, (d // group, V), generator=g).float()).bfloat16().to(cuda_device)
    z = torch.randint(0, 16, (d // group, V), generator=g, dtype=torch.uint8).to(cuda_device)
    for zeros in (None, z):
        out = dv.int4_product(x, codes, scales, zeros, group=group, out_dtype=torch.float32)
        sb = scales.view(torch.int16).cpu().numpy().view(np.uint16)
        want, _ = O.int4_product(values(x), codes.cpu().numpy(), sb, None if zeros is None else z.cpu().numpy(), group)
        assert np.array_equal(values(out["logits"]), want)


def test_product_strides_and_shapes(cuda_device):
    """Padded rows of x, codes, scales, zeros and out; [B, n, d] rows."""
    import draft_verification_gb300 as dv
    R, V, d, group = 6, 333, 320, 64
    x, codes, scales, z = make_product(R, V, d, group, True, 11, cuda_device)

    def padded(t, extra):
        p = torch.full((t.shape[0], t.shape[1] + extra), 77, dtype=t.dtype, device=t.device)
        p[:, :t.shape[1]] = t
        return p[:, :t.shape[1]]

    out = torch.full((R, V + 5), 7.0, device=cuda_device)
    px, pc, ps, pz = padded(x, 24), padded(codes, 48), padded(scales, 3), padded(z, 5)
    plan = dv.Int4ProductPlan(px, pc, ps, pz, group=group, out_dtype=torch.float32, out=out[:, :V])
    check_product(plan.run()["logits"], x, codes, scales, z, group)
    assert bool((out[:, V:] == 7.0).all())
    y3 = dv.int4_product(x.view(2, 3, d), codes, scales, z, group=group, out_dtype=torch.float32)["logits"]
    assert y3.shape == (2, 3, V)
    assert np.array_equal(bits(y3.reshape(R, V)), bits(out[:, :V].contiguous()))


def test_product_non_finite_values_stay_in_their_rows(cuda_device):
    import draft_verification_gb300 as dv
    R, V, d, group = 20, 400, 512, 128
    x, codes, scales, z = make_product(R, V, d, group, True, 12, cuda_device)
    clean = dv.int4_product(x, codes, scales, z, group=group, out_dtype=torch.float32)["logits"].clone()
    x[3, 7], x[11, 300] = float("nan"), float("inf")
    scales[1, 5] = float("nan")
    got = dv.int4_product(x, codes, scales, z, group=group, out_dtype=torch.float32)["logits"]
    rows = [r for r in range(R) if r not in (3, 11)]
    cols = [v for v in range(V) if v != 5]
    assert bool(got[3].isnan().all()) and not bool(got[11].isfinite().any()) and bool(got[:, 5].isnan().all())
    assert np.array_equal(bits(got[rows][:, cols]), bits(clean[rows][:, cols]))


def test_product_on_a_side_stream_and_in_a_graph(cuda_device):
    import draft_verification_gb300 as dv
    R, V, d, group = 12, 9000, 1024, 64
    x, codes, scales, z = make_product(R, V, d, group, True, 13, cuda_device)
    plan = dv.Int4ProductPlan(x, codes, scales, z, group=group, out_dtype=torch.float32)
    first = bits(plan.run()["logits"]).copy()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.run(side)
    side.synchronize()
    assert np.array_equal(bits(plan.out["logits"]), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    x.neg_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    check_product(plan.out["logits"], x, codes, scales, z, group)


def test_quantised_head_and_its_products_agree(cuda_device):
    """What quantize_int4 writes is what int4_product reads, host tensors in and out as well."""
    import draft_verification_gb300 as dv
    g = torch.Generator().manual_seed(14)
    w = torch.randn(900, 256, generator=g) * 0.02
    x = torch.randn(4, 256, generator=g).bfloat16()
    for zeros in (False, True):
        q = dv.quantize_int4(w, group=64, zeros=zeros)
        y = dv.int4_product(x, q["codes"], q["scales"], q.get("zeros"), group=64, out_dtype=torch.float32)["logits"]
        torch.cuda.synchronize()
        check_product(y, x, q["codes"], q["scales"], q.get("zeros"), 64)
        # against the matrix itself: a weight is off by at most half a step of its scale, plus what the rounding
        # of the scale (half a step of bfloat16, at most 15 codes away) and of the zero point (half a step) moves it by
        sb = q["scales"].view(torch.int16).numpy().view(np.uint16)
        step = np.repeat(O.bf16_values(sb).T.astype(np.float64), 64, axis=1)
        off = step * (0.5 + 15 * half_step(torch.bfloat16) + (0.5 if zeros else 0.0))
        _, mag = O.int4_product(values(x), q["codes"].numpy(), sb, q["zeros"].numpy() if zeros else None, 64)
        near = values(x) @ w.double().numpy().T
        bound = np.abs(values(x)) @ off.T + product_tolerance(mag, values(y), 256, 64, torch.float32)
        assert (np.abs(values(y) - near) <= bound).all()
