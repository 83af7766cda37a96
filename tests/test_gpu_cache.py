"""The cache operators on the GPU against the oracle.

Rotation and appending are rules of float32 steps, a rounding per operation:
equality.  Attention, with u = finfo(type).eps / 2 the half step of a type
(bfloat16 2^-8, float32 2^-24), against float64 on the codes' exact values:
  scores   a query enters as two e4m3 numbers, off by at most 2^-18 of its
           largest element; D products are summed in float32, each addition
           may truncate (2 u32), and the exponent of a weight takes four more
           float32 steps: a score is off by e = score (2^-18 + (2 D + 16) u32),
           `score` the largest sum of a row's terms' magnitudes;
  weights  off by e from their score, by 2^-8 from two e4m3 numbers after a
           step of float16 (2^-11), or by 2^-18 of the largest weight of their
           one or two tiles (`floor`; both with their pages' value exponents);
           their sum by e, a few u32 per tile, and the floor without the
           exponents, which may lie 2^3 apart (`sums`);
  out      the weighted sum of magnitudes (`mass`) times both, and u16 of
           itself for its own rounding.
"""

import numpy as np
import pytest
import torch

import draft_verification_gb300 as dv
from oracle import cache as O

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def dev(a, device="cuda"):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(device)


def rounded(a, dtype):
    """float32 values of `a` in dtype."""
    return torch.from_numpy(np.asarray(a, np.float32)).to(DTYPES[dtype]).float().numpy()


def like(t, layout):
    """t in another layout: a view with the same values."""
    B, n, H, D = t.shape
    if layout == "fused":  # heads of a wider projection, rows behind one another
        wide = torch.zeros((B, n, H + 3, D), dtype=t.dtype, device=t.device)
        wide[:, :, 2:2 + H] = t
        return wide[:, :, 2:2 + H]
    if layout == "heads":  # [B, H, n, D]
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "odd":  # rows that start anywhere
        wide = torch.zeros(B * n * (H * D + 1) + 1, dtype=t.dtype, device=t.device)
        view = wide.as_strided((B, n, H, D), (n * (H * D + 1), H * D + 1, D, 1), 1)
        view.copy_(t)
        return view
    return t


def same(got, want):
    return np.array_equal(np.asarray(got, np.float64), np.asarray(want, np.float64), equal_nan=True)


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("B,n,H,D,rot,pairs,dtype,layout", [
    (1, 1, 1, 2, 2, False, "f32", "plain"), (1, 1, 32, 128, 128, False, "bf16", "plain"),
    (3, 5, 7, 128, 128, True, "bf16", "fused"), (2, 9, 5, 96, 48, True, "f32", "heads"),
    (2, 3, 4, 80, 40, False, "bf16", "fused"), (2, 17, 3, 64, 64, False, "f32", "odd"),
    (1, 33, 9, 10, 6, True, "bf16", "plain"), (4, 2, 2, 256, 64, False, "bf16", "heads"),
    (2, 3, 3, 128, 128, True, "bf16", "odd"), (1, 2, 5, 1024, 1024, False, "bf16", "plain"),
])
def test_rotate(cuda_device, B, n, H, D, rot, pairs, dtype, layout):
    rng = np.random.default_rng(D + rot)
    x = rounded(rng.normal(0, 2, (B, n, H, D)), dtype)
    table = O.rotation_table(700, rng.random(rot // 2), 1.25)
    at = rng.integers(0, 700, (B, n), dtype=np.int32)
    t = like(dev(x).to(DTYPES[dtype]), layout)
    for given in (dict(positions=dev(at)), dict(prefix_len=dev(at[:, 0] % 600)), {}):
        for transpose in (False, True):
            plan = dv.RotateHeadsPlan(t, dev(table), pairs=pairs, transpose=transpose, **given)
            out = plan.run()
            want, _ = O.rotate_heads(x, table, at if "positions" in given else None,
                                     at[:, 0] % 600 if "prefix_len" in given else None, pairs, transpose)
            assert same(out["out"].float().cpu(), rounded(want, dtype))
            assert not out["seq_error"].any() and not out["error_word"].any()
    # in place, strided
    want, _ = O.rotate_heads(x, table, at, None, pairs)
    dv.RotateHeadsPlan(t, dev(table), positions=dev(at), pairs=pairs, out=t).run()
    assert same(t.float().cpu(), rounded(want, dtype))


def test_rotate_positions_outside_the_table(cuda_device):
    x = torch.ones((3, 4, 2, 32), device=cuda_device)
    table = dv.rotation_table(10, 16)
    at = torch.tensor([[0, 9, 3, 4], [0, 10, 3, 4], [-1, 2, 2 ** 31 - 1, 4]], dtype=torch.int32, device=cuda_device)
    plan = dv.RotateHeadsPlan(x, table, positions=at)
    out = plan.run()
    bad = ((at < 0) | (at >= 10)).cpu().numpy()
    y = out["out"].cpu().numpy()
    assert (np.isnan(y[..., :16]).all((2, 3)) == bad).all() and (y[..., 16:] == 1).all()
    assert out["seq_error"].tolist() == [0, dv.ERR_POSITION, dv.ERR_POSITION]
    assert out["error_word"].tolist() == [dv.ERR_POSITION]
    plan.clear_errors()
    assert not out["seq_error"].any() and not out["error_word"].any()


def test_rotation_table(cuda_device):
    freq = dv.rotary_frequencies(64, 500000.0, bands=(8.0, 1.0, 4.0, 8192))
    table = dv.rotation_table(1 << 18, 64, freq=freq, magnitude=1.125).cpu().numpy()
    at = np.r_[0:100, (1 << 18) - 1000:1 << 18]
    angle = at[:, None] * freq.numpy()
    want = 1.125 * np.concatenate([np.cos(angle), np.sin(angle)], 1)
    # one rounding to float32, a step of the 64-bit functions at angles up to 2^18
    assert (np.abs(table[at] - want) <= U32 * np.abs(want) + 2.0 ** -33).all()


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_gradient(cuda_device, pairs):
    """The transposed rotation is the gradient: against the formula's transpose
    by differences of a linear function, which differences give exactly but for
    rounding: 4 float32 steps of each of the two products per element."""
    rng = np.random.default_rng(5)
    x, g = (torch.from_numpy(rng.normal(0, 1, (2, 3, 2, 32)).astype(np.float32)).to(cuda_device) for _ in range(2))
    table = dv.rotation_table(40, 24, magnitude=1.5)
    at = dev(rng.integers(0, 40, (2, 3), dtype=np.int32))
    dx = dv.rotate_heads(g, table, positions=at, pairs=pairs, transpose=True)["out"].double()

    def loss(x):
        return (dv.rotate_heads(x, table, positions=at, pairs=pairs)["out"].double() * g.double()).sum()

    for _ in range(5):
        step = torch.from_numpy(rng.normal(0, 1, x.shape).astype(np.float32)).to(cuda_device)
        up, down = x + step, x - step
        got = loss(up) - loss(down)
        want = (dx * (up.double() - down.double())).sum()
        size = (g.abs().double() * 1.5 * 2 * (up.abs() + down.abs()).max()).sum()
        assert abs(got - want) <= 8 * U32 * size


# ---------------------------------------------------------------------------
# appending
# ---------------------------------------------------------------------------

def make_cache(rng, pages, H, page, D):
    c = {}
    for m in "kv":
        codes = rng.integers(0, 256, (pages, H, page, D)).astype(np.uint8)
        c[m + "_codes"] = np.where(codes & 127 == 127, 0, codes).astype(np.uint8)
        c[m + "_exps"] = rng.integers(-8, -2, (pages, H)).astype(np.int8)
    return c


def on_gpu(c):
    return dv.PagedCache(*(dev(c[k]) for k in ("k_codes", "v_codes", "k_exps", "v_exps")))


def check_cache(got, want):
    for m in "kv":
        assert np.array_equal(getattr(got, m + "_exps").cpu().numpy(), want[m + "_exps"]), m
        codes = getattr(got, m + "_codes").cpu().numpy()
        assert same(O.VALUES[codes], O.VALUES[want[m + "_codes"]]), m


APPENDS = [
    # B, n, H, D, page, rot, pairs, dtype, layout, prefix
    (1, 1, 1, 16, 16, 0, False, "f32", "plain", (0,)), (1, 1, 8, 128, 16, 128, False, "bf16", "plain", (1001,)),
    (3, 6, 2, 128, 64, 128, False, "bf16", "fused", (0, 63, 64)), (2, 40, 3, 80, 16, 40, True, "f32", "heads", (5, 15)),
    (2, 130, 1, 64, 128, 64, True, "bf16", "odd", (127, 126)), (4, 7, 2, 256, 32, 128, False, "f32", "fused", (0, 31, 32, 26)),
    (2, 33, 2, 48, 32, 2, True, "bf16", "plain", (1, 30)), (1, 300, 2, 96, 64, 96, False, "bf16", "heads", (20,)),
]


@pytest.mark.parametrize("B,n,H,D,page,rot,pairs,dtype,layout,prefix", APPENDS)
def test_append(cuda_device, B, n, H, D, page, rot, pairs, dtype, layout, prefix):
    rng = np.random.default_rng(n * D)
    prefix = np.array(prefix, np.int32)
    width = (prefix.max() + n + page - 1) // page
    table = rng.permutation(B * width + 2)[:B * width].reshape(B, width).astype(np.int32)
    k, v = (rounded(rng.normal(0, 1, (B, n, H, D)) * np.exp(rng.normal(0, 2, (1, 1, H, D))), dtype) for _ in range(2))
    turns = O.rotation_table(prefix.max() + n, rng.random(rot // 2)) if rot else None
    kt, vt = (like(dev(x).to(DTYPES[dtype]), layout) for x in (k, v))
    for extra in ({}, dict(count=rng.integers(0, n + 1, B).astype(np.int32)),
                  dict(positions=rng.integers(0, prefix.max() + n, (B, n)).astype(np.int32)) if rot else {}):
        c = make_cache(rng, B * width + 2, H, page, D)
        want, err = O.append_cache(k, v, c, table, prefix, turns, pairs, **extra)
        got = on_gpu(c)
        plan = dv.AppendCachePlan(kt, vt, got, dev(table), dev(prefix), table=dev(turns), pairs=pairs,
                                  **{a: dev(x) for a, x in extra.items()})
        for _ in range(2):  # appending the same rows once more changes nothing
            out = plan.run()
            check_cache(got, want)
        assert not err.any() and not out["seq_error"].any() and not out["error_word"].any()


def test_append_scales_earlier_tokens(cuda_device):
    """A page whose tokens are far smaller, or larger, than the appended ones; zeros; the ends of the range."""
    rng = np.random.default_rng(3)
    B, n, H, D, page = 7, 3, 2, 32, 16
    size = np.array([1e-30, 1.0, 2.0 ** 20, 1e30, 0.0, 2.0 ** -126, 3e38])
    k = rounded(rng.uniform(-1, 1, (B, n, H, D)) * size[:, None, None, None], "f32")
    v = rounded(rng.uniform(-1, 1, (B, n, H, D)) * size[::-1][:, None, None, None], "f32")
    k[1, 0, 0, 0] = 2.0 ** 7  # a power of two takes no larger exponent
    c = make_cache(rng, B, H, page, D)
    table = np.arange(B, dtype=np.int32).reshape(B, 1)
    for prefix in (0, 13):
        start = np.full(B, prefix, np.int32)
        want, err = O.append_cache(k, v, c, table, start)
        got = on_gpu(c)
        out = dv.AppendCachePlan(dev(k), dev(v), got, dev(table), dev(start)).run()
        check_cache(got, want)
        assert np.array_equal(out["seq_error"].cpu().numpy(), err)


def test_append_path(cuda_device):
    rng = np.random.default_rng(4)
    B, n, H, D, page, depth = 6, 20, 2, 64, 16, 5
    k, v = (rounded(rng.normal(0, 1, (B, n, H, D)), "bf16") for _ in range(2))
    turns = O.rotation_table(100, rng.random(32))
    path = np.full((B, depth + 1), -1, np.int32)
    length = np.array([0, 5, 3, 2, 7, 4], np.int32)
    for b in range(B):
        m = min(length[b], depth)
        path[b, 0] = 0
        path[b, 1:m + 1] = np.sort(rng.choice(np.arange(1, n), m, replace=False))
    path[3] = -1       # the verification's marking of a data error: skipped
    path[5, 2] = n     # no such node
    prefix = np.array([0, 15, 31, 7, 3, 4], np.int32)
    table = rng.permutation(B * 3).reshape(B, 3).astype(np.int32)
    c = make_cache(rng, B * 3, H, page, D)
    want, err = O.append_cache(k, v, c, table, prefix, turns, path_nodes=path, path_len=length)
    assert list(err) == [0, 0, 0, 0, dv.ERR_CACHE, dv.ERR_PARENT]
    got = on_gpu(c)
    out = dv.append_cache(dev(k).bfloat16(), dev(v).bfloat16(), got, dev(table), dev(prefix), table=dev(turns),
                          path_nodes=dev(path), path_len=dev(length))
    check_cache(got, want)
    assert np.array_equal(out["seq_error"].cpu().numpy(), err)


def test_append_data_errors(cuda_device):
    rng = np.random.default_rng(6)
    B, n, H, D, page = 9, 20, 1, 32, 16
    k, v = (rounded(rng.normal(0, 1, (B, n, H, D)), "f32") for _ in range(2))
    k[0, 3, 0, 2], v[1, 4, 0, 5], v[1, 5, 0, 6] = np.nan, np.inf, -np.inf
    turns = O.rotation_table(30, rng.random(8))
    table = np.arange(B * 2, dtype=np.int32).reshape(B, 2)
    table[2, 0], table[3, 1] = -1, 18
    prefix = np.array([0, 2, 1, 0, -1, 13, 5, 2 ** 31 - 1, 11], np.int32)
    count = np.array([20, 20, 20, 20, 1, 20, 21, 5, 20], np.int32)
    c = make_cache(rng, 18, H, page, D)
    want, err = O.append_cache(k, v, c, table, prefix, turns, count=count)
    E = dv
    assert list(err) == [E.ERR_NONFINITE, E.ERR_NONFINITE, E.ERR_CACHE, E.ERR_CACHE, E.ERR_CACHE, E.ERR_CACHE,
                         E.ERR_CACHE, E.ERR_CACHE, E.ERR_POSITION]
    got = on_gpu(c)
    out = dv.append_cache(dev(k), dev(v), got, dev(table), dev(prefix), table=dev(turns), count=dev(count))
    check_cache(got, want)
    assert np.array_equal(out["seq_error"].cpu().numpy(), err)
    assert out["error_word"].tolist() == [E.ERR_NONFINITE | E.ERR_CACHE | E.ERR_POSITION]


@pytest.mark.parametrize("page,D,n,dtype", [
    (16, 32, 20, "bf16"), (64, 128, 100, "bf16"), (128, 256, 140, "bf16"), (64, 64, 70, "f32"), (128, 128, 130, "f32"),
    (128, 256, 128, "f32"), (32, 48, 40, "bf16"),
])
def test_append_non_finite_rows(cuda_device, page, D, n, dtype):
    """NaN and infinities beside finite rows, in pages of every size: the finite ones alone make the exponent."""
    rng = np.random.default_rng(page + D)
    B, H = 3, 2
    k, v = (rounded(rng.normal(0, 1, (B, n, H, D)) * 2.0 ** rng.integers(-20, 20, (B, 1, H, 1)), dtype) for _ in range(2))
    k[0, n // 2, 0, D - 1], k[0, 1, 1, 3], v[1, n - 1, 1, 0], v[1, 0, 0, D // 2] = np.nan, -np.inf, np.inf, np.nan
    prefix = np.array([3, page - 1, 0], np.int32)
    width = (page - 1 + n) // page + 1
    table = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    turns = O.rotation_table(page + n, rng.random(8))
    c = make_cache(rng, B * width, H, page, D)
    want, err = O.append_cache(k, v, c, table, prefix, turns)
    assert list(err) == [dv.ERR_NONFINITE, dv.ERR_NONFINITE, 0]
    got = on_gpu(c)
    out = dv.append_cache(dev(k).to(DTYPES[dtype]), dev(v).to(DTYPES[dtype]), got, dev(table), dev(prefix), table=dev(turns))
    check_cache(got, want)
    assert np.array_equal(out["seq_error"].cpu().numpy(), err)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def make_parents(rng, B, n):
    """Trees of every kind: bushy, a chain, a star."""
    p = np.zeros((B, n), np.int32)
    p[:, 0] = -1
    for i in range(1, n):
        p[:, i] = rng.integers(max(0, i - 1 - i // 2), i, B)
    if B > 1:
        p[1, 1:] = np.arange(n - 1)
    if B > 2:
        p[2, 1:] = 0
    return p


def make_attend(rng, B, n, Hq, H, D, page, prefix, tree, spread=1.0):
    prefix = np.asarray(prefix, np.int32)
    width = max(1, int(prefix.max() + n + page - 1) // page)
    c = {}
    for m in "kv":
        codes = O.to_e4m3(np.clip(rng.normal(0, 40, (B * width + 1, H, page, D)), -300, 300))
        c[m + "_codes"] = codes
        c[m + "_exps"] = rng.integers(-7, -3, (B * width + 1, H)).astype(np.int8)
    table = (1 + rng.permutation(B * width)).reshape(B, width).astype(np.int32)
    q = rounded(rng.normal(0, spread, (B, n, Hq, D)), "bf16")
    return dict(q=q, c=c, table=table, prefix=prefix, parent=make_parents(rng, B, n) if tree else None)


def attend_bound(out, bound, D):
    # Scores: queries to 2^-18, D products and their scaling in float32.  Weights: e4m3 twice is 2^-4 * 2^-4 of
    # themselves, and 2^-11 for the float16 on the way, or 2^-18 of the largest near them (2^-10 of 256: half a step
    # of the least e4m3 codes), once more where float16's own rounding adds to it.  The sum of the weights is made of
    # the same numbers, each divided by its value exponent: up to 2^3 times the floor.
    e = (bound["score"] * (2.0 ** -18 + (2 * D + 16) * U32))[..., None]
    return (bound["mass"] * (2.0 ** -8 + 2.0 ** -11 + 2 * e + 2.0 ** -17) + bound["floor"] * 2.0 ** -17 +
            np.abs(out) * (U16 + bound["sums"][..., None] * 2.0 ** -15))


def check_attend(w, got, rows=None, **kw):
    want, bound, err = O.attend_cache(w["q"], w["c"], w["table"], w["prefix"], parent=w["parent"], **kw)
    y = got["out"].double().cpu().numpy()
    assert np.array_equal(np.isnan(y), np.isnan(want))
    fine = ~np.isnan(want)
    off = np.abs(y - want)[fine] - attend_bound(want, bound, want.shape[3])[fine]
    assert (off <= 0).all(), off.max()
    assert np.array_equal(got["seq_error"].cpu().numpy(), err)
    return want


def run_attend(w, layout="plain", **kw):
    q = like(dev(w["q"]).bfloat16(), layout)
    return dv.AttendCachePlan(q, on_gpu(w["c"]), dev(w["table"]), dev(w["prefix"]), parent=dev(w["parent"]),
                              **{k: dev(x) if isinstance(x, np.ndarray) else x for k, x in kw.items()}).run()


ATTENDS = [
    # B, n, Hq, H, D, page, prefix, tree, layout
    (1, 1, 1, 1, 16, 16, (0,), False, "plain"), (1, 1, 8, 2, 128, 16, (1001,), False, "plain"),
    (3, 6, 8, 2, 128, 64, (0, 63, 500), False, "fused"), (2, 3, 12, 12, 80, 32, (301, 127), False, "heads"),
    (3, 20, 4, 1, 64, 128, (128, 1, 257), True, "plain"), (2, 64, 8, 2, 128, 64, (300, 64), True, "fused"),
    (3, 33, 3, 3, 96, 16, (0, 95, 112), True, "heads"), (2, 5, 14, 2, 256, 32, (130, 250), False, "plain"),
    (2, 17, 6, 2, 144, 16, (17, 383), True, "fused"), (1, 200, 2, 1, 64, 64, (77,), False, "plain"),
    (2, 150, 2, 2, 32, 32, (10, 129), True, "plain"), (1, 2, 64, 1, 128, 64, (255,), False, "plain"),
    (2, 1, 5, 5, 48, 128, (126, 127), False, "plain"), (40, 2, 4, 2, 64, 16, tuple(range(0, 80, 2)), False, "plain"),
    (1, 4, 8, 8, 128, 128, (9000,), False, "plain"),
    (2, 20, 4, 2, 128, 32, (700, 260), True, "plain"), (3, 11, 4, 1, 80, 16, (200, 5, 1333), False, "plain"),
    # many tiles per CTA, over the ends of sequences
    (3, 9, 64, 16, 128, 64, (1500, 777, 2301), False, "plain"),
    (5, 3, 12, 12, 80, 32, (3001, 2500, 2222, 1999, 3000), False, "plain"),
    (9, 2, 48, 48, 64, 16, (700, 1, 64, 900, 333, 511, 513, 127, 128), True, "plain"),
    (6, 20, 32, 32, 128, 128, (1500, 300, 1301, 1, 1000, 640), True, "plain"),
    (4, 2, 64, 16, 256, 64, (1500, 777, 1301, 900), False, "plain"),
    # each size of a block, with rows of its own number and with fewer
    (2, 12, 4, 1, 128, 64, (1030, 257), True, "plain"), (2, 47, 1, 1, 64, 16, (250, 255), True, "fused"),
    (1, 16, 4, 1, 128, 32, (900,), False, "plain"), (2, 3, 7, 1, 128, 16, (515, 260), True, "heads"),
    (2, 5, 3, 1, 112, 128, (1000, 128), False, "plain"), (2, 4, 8, 1, 176, 64, (500, 3), True, "plain"),
    (3, 2, 8, 1, 256, 128, (129, 640, 2), False, "fused"), (2, 1, 8, 1, 96, 64, (2048, 1023), False, "plain"),
    # long trees
    (1, 513, 2, 1, 64, 64, (65,), True, "fused"), (1, 1024, 1, 1, 32, 128, (300,), True, "plain"),
]


@pytest.mark.parametrize("B,n,Hq,H,D,page,prefix,tree,layout", ATTENDS)
def test_attend(cuda_device, B, n, Hq, H, D, page, prefix, tree, layout):
    rng = np.random.default_rng(B * 1000 + D)
    w = make_attend(rng, B, n, Hq, H, D, page, prefix, tree)
    got = run_attend(w, layout)
    check_attend(w, got)
    count = rng.integers(0, n + 1, B).astype(np.int32)
    count[-1] = n
    got = run_attend(w, layout, count=count, scale=0.3)
    check_attend(w, got, count=count, scale=0.3)


@pytest.mark.parametrize("n,G", [(2, 4), (6, 4), (8, 4), (12, 4), (16, 4)])
@pytest.mark.parametrize("tree", [False, True])
def test_attend_counts(cuda_device, n, G, tree):
    """Sequences of every count of rows, some without a token, between long ones."""
    rng = np.random.default_rng(n)
    prefix = (0, 400, 0, 128, 1, 0, 255, 0, 640, 0)
    w = make_attend(rng, len(prefix), n, 2 * G, 2, 128, 64, prefix, tree)
    count = np.array([0, n, 0, 1, n - 1, 0, 0, n, 2, 1], np.int32)
    check_attend(w, run_attend(w, count=count), count=count)


@pytest.mark.parametrize("n,G,D", [(2, 4, 128), (6, 4, 128), (8, 4, 64), (12, 4, 128), (16, 4, 80), (3, 4, 256)])
@pytest.mark.parametrize("apart", [3, 4, 40])
def test_attend_value_exponents_apart(cuda_device, n, G, D, apart):
    """Pages whose value exponents lie near one another, or too far for one sum, over several steps."""
    rng = np.random.default_rng(100 * n + apart)
    w = make_attend(rng, 3, n, 2 * G, 2, D, 32, (1100, 515, 31), True)
    w["c"]["v_exps"] = (rng.integers(0, 2, w["c"]["v_exps"].shape) * apart - apart // 2).astype(np.int8)
    check_attend(w, run_attend(w))


@pytest.mark.parametrize("n,G", [(2, 4), (6, 4), (8, 4), (12, 4), (16, 4)])
def test_attend_nan_of_drafted_tokens(cuda_device, n, G):
    """NaN values of drafted tokens, over the end of a tile, reach the rows that see them and no others."""
    rng = np.random.default_rng(n)
    w = make_attend(rng, 2, n, 2 * G, 2, 128, 16, (255, 510), True)
    for b, past in enumerate((255, 510)):
        for j in (n - 1, n // 2):
            at = past + j
            w["c"]["v_codes"][w["table"][b, at // 16], 1, at % 16, 5] = 0x7F
    got = run_attend(w)
    want, bound, _ = O.attend_cache(w["q"], w["c"], w["table"], w["prefix"], parent=w["parent"])
    y, hit = got["out"].double().cpu().numpy(), np.isnan(want).any(3)
    # (a drafted token's NaN may take all elements of the rows that read it)
    assert np.array_equal(np.isnan(y).any(3), hit) and np.isnan(y[hit][:, 5]).all() and hit.any() and not hit.all()
    assert (np.abs(y - want)[~hit] <= attend_bound(want, bound, 128)[~hit]).all()


@pytest.mark.parametrize("spread", [0.0, 1e-3, 30.0])
def test_attend_flat_and_peaked(cuda_device, spread):
    """Weights that are all alike, and rows where one token has nearly all of it."""
    rng = np.random.default_rng(11)
    w = make_attend(rng, 2, 4, 8, 2, 128, 32, (700, 333), False, spread)
    check_attend(w, run_attend(w))


def test_attend_sink(cuda_device):
    """A first token with most of the weight and hardly any value: what the
    others add is far below its weight, and all of the output."""
    rng = np.random.default_rng(12)
    w = make_attend(rng, 1, 2, 4, 1, 64, 64, (4000,), False, 0.05)
    first = w["table"][0, 0]
    w["c"]["k_codes"][first, 0, 0] = O.to_e4m3(np.full(64, 200.0))
    w["c"]["v_codes"][first, 0, 0] = 0
    w["q"] = rounded(w["q"] + 0.12, "bf16")
    want = check_attend(w, run_attend(w))
    assert np.abs(want).max() < 0.05  # (the sink has it)


def test_attend_scales_of_pages(cuda_device):
    """Pages whose exponents lie far apart, and at the ends of their range."""
    rng = np.random.default_rng(13)
    w = make_attend(rng, 2, 3, 4, 2, 64, 16, (200, 77), False)
    w["c"]["v_exps"][:] = rng.integers(-100, 101, w["c"]["v_exps"].shape)
    w["c"]["k_exps"][:] = rng.integers(-100, -5, w["c"]["k_exps"].shape)
    check_attend(w, run_attend(w))


def test_attend_ignores_what_no_row_sees(cuda_device):
    """NaN codes behind the last token, and in pages of the table behind it."""
    rng = np.random.default_rng(14)
    for tree in (False, True):
        w = make_attend(rng, 3, 5, 4, 2, 128, 32, (100, 0, 27), tree)
        count = np.array([5, 3, 0], np.int32)
        wide = np.full((3, 8), 2 ** 30, np.int32)  # entries that are not pages, behind the last token
        wide[:, :w["table"].shape[1]] = w["table"]
        for b in range(3):
            for t in range(w["prefix"][b] + count[b], w["table"].shape[1] * 32):
                p = w["table"][b, t // 32]
                w["c"]["k_codes"][p, :, t % 32] = 0x7F
                w["c"]["v_codes"][p, :, t % 32] = 0xFF
        for b in range(3):
            wide[b, -(-(w["prefix"][b] + count[b]) // 32):] = -7
        w["table"] = wide
        check_attend(w, run_attend(w, count=count), count=count)


def test_attend_nan_reaches_the_rows_that_see_it(cuda_device):
    rng = np.random.default_rng(15)
    w = make_attend(rng, 2, 6, 4, 2, 128, 32, (40, 127), True)
    w["parent"][:] = [[-1, 0, 0, 1, 1, 2], [-1, 0, 1, 0, 3, 4]]
    at = lambda b, j: (w["table"][b, (w["prefix"][b] + j) // 32], (w["prefix"][b] + j) % 32)  # noqa: E731
    p, r = at(0, 1)
    w["c"]["k_codes"][p, 0, r, 5] = 0x7F   # node 1's key of head 0: rows 1, 3 and 4
    p, r = at(1, 3)
    w["c"]["v_codes"][p, 1, r, :] = 0xFF   # node 3's value of head 1: rows 3, 4 and 5
    want = check_attend(w, run_attend(w))
    hit = np.isnan(want).all(3)
    assert hit.sum() == 2 * 3 * 2 and hit[0, [1, 3, 4], :2].all() and hit[1, [3, 4, 5], 2:].all()
    # queries: the row's own head alone
    w = make_attend(rng, 1, 3, 4, 2, 64, 16, (50,), False)
    w["q"][0, 1, 2, 7], w["q"][0, 2, 0, 0] = np.nan, np.inf
    y = run_attend(w)["out"].isnan().all(3).cpu().numpy()
    assert y.sum() == 2 and y[0, 1, 2] and y[0, 2, 0]


def test_attend_data_errors(cuda_device):
    rng = np.random.default_rng(16)
    w = make_attend(rng, 6, 4, 4, 2, 64, 16, (50, 3, 20, 70, 9, 33), True)
    pages = w["c"]["k_codes"].shape[0]
    w["prefix"][1], w["prefix"][3] = -2, w["table"].shape[1] * 16 - 3
    w["table"][2, 0], w["table"][5, 1] = pages, -1
    w["parent"][4, 2], w["parent"][0, 1] = 3, -1
    count = np.array([4, 4, 4, 4, 4, 3], np.int32)
    got = run_attend(w, count=count)
    want = check_attend(w, got, count=count)
    assert got["seq_error"].tolist() == [dv.ERR_PARENT, dv.ERR_CACHE, dv.ERR_CACHE, dv.ERR_CACHE, dv.ERR_PARENT,
                                         dv.ERR_CACHE]
    assert np.isnan(want[2]).all() and np.isnan(want[5, :3]).all() and not want[5, 3].any() and not want[[1, 3]].any()


def test_attend_strided_out(cuda_device):
    rng = np.random.default_rng(17)
    w = make_attend(rng, 2, 5, 6, 2, 80, 16, (70, 20), False)
    plain = run_attend(w)["out"]
    hold = torch.full((2, 6, 7, 84), 7.0, dtype=torch.bfloat16, device=cuda_device)
    out = hold[:, :, 1:6, 2:82].transpose(1, 2)
    run_attend(w, out=out)
    assert torch.equal(out, plain)
    hold[:, :, 1:6, 2:82] = 7.0
    assert (hold == 7.0).all()  # nothing else was written


# ---------------------------------------------------------------------------
# calls
# ---------------------------------------------------------------------------

def test_far_pages(cuda_device):
    """Codes more than 2^32 bytes from the cache's start."""
    rng = np.random.default_rng(18)
    H, page, D, pages = 8, 128, 128, 36000
    big = dv.PagedCache.empty(pages, H, page, D, device=cuda_device)
    assert big.k_codes.numel() > 2 ** 32
    w = make_attend(rng, 1, 3, 8, H, D, page, (300,), False)
    k, v = (rounded(rng.normal(0, 1, (1, 303, H, D)), "bf16") for _ in range(2))
    far = np.array([[pages - 1, 3, pages - 2]], np.int32)
    dv.append_cache(dev(k).bfloat16(), dev(v).bfloat16(), big, dev(far))
    got = dv.attend_cache(dev(w["q"]).bfloat16(), big, dev(far), dev(w["prefix"]))
    small = {n: t[far[0].tolist()].cpu().numpy() for n, t in (
        ("k_codes", big.k_codes), ("v_codes", big.v_codes), ("k_exps", big.k_exps), ("v_exps", big.v_exps))}
    zero = {n: np.zeros_like(a) for n, a in small.items()}
    want, _ = O.append_cache(k, v, zero, np.array([[0, 1, 2]], np.int32))
    for m in "kv":
        assert np.array_equal(small[m + "_exps"], want[m + "_exps"])
        assert same(O.VALUES[small[m + "_codes"]], O.VALUES[want[m + "_codes"]])
    w["c"], w["table"] = small, np.array([[0, 1, 2]], np.int32)
    check_attend(w, got)


def test_repeats_are_equal_and_streams_apart(cuda_device):
    """The same bits every time; two plans at once on two streams."""
    rng = np.random.default_rng(19)
    ws = [make_attend(rng, 4, 6, 8, 2, 128, 64, (3000, 100, 777, 0), False),
          make_attend(rng, 3, 40, 4, 2, 64, 16, (500, 64, 90), True)]
    plans = [dv.AttendCachePlan(dev(w["q"]).bfloat16(), on_gpu(w["c"]), dev(w["table"]), dev(w["prefix"]),
                                parent=dev(w["parent"])) for w in ws]
    first = [p.run()["out"].clone() for p in plans]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for p, s in zip(plans, streams):
            p.run(s)
    torch.cuda.synchronize()
    for p, f, w in zip(plans, first, ws):
        assert torch.equal(p.out["out"], f)
        check_attend(w, p.out)


def test_graph_with_other_lengths(cuda_device):
    """A step captured once and replayed with other tensors' contents: rotate, append, attend."""
    rng = np.random.default_rng(20)
    B, n, Hq, H, D, page, width = 3, 4, 8, 2, 64, 16, 12
    turns = O.rotation_table(width * page, rng.random(32))
    c = make_cache(rng, B * width, H, page, D)
    table = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    q, k, v = (torch.zeros((B, n, m, D), dtype=torch.bfloat16, device=cuda_device) for m in (Hq, H, H))
    prefix = torch.zeros(B, dtype=torch.int32, device=cuda_device)
    cache, bt, tt = on_gpu(c), dev(table), dev(turns)
    rotate = dv.RotateHeadsPlan(q, tt, prefix_len=prefix)
    append = dv.AppendCachePlan(k, v, cache, bt, prefix, table=tt)
    attend = dv.AttendCachePlan(rotate.out["out"], cache, bt, prefix)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for p in (rotate, append, attend):
            p.run()
    torch.cuda.current_stream().wait_stream(side)
    for name, t in (("k_codes", cache.k_codes), ("v_codes", cache.v_codes), ("k_exps", cache.k_exps), ("v_exps", cache.v_exps)):
        t.copy_(dev(c[name]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for p in (rotate, append, attend):
            p.run()
    for lengths in ((0, 17, 60), (100, 31, 188)):
        w = dict(q=rounded(rng.normal(0, 1, (B, n, Hq, D)), "bf16"), table=table, prefix=np.array(lengths, np.int32),
                 parent=None)
        kv = [rounded(rng.normal(0, 1, (B, n, H, D)), "bf16") for _ in range(2)]
        for t, a in zip((q, k, v), (w["q"], *kv)):
            t.copy_(dev(a))
        prefix.copy_(dev(w["prefix"]))
        c, _ = O.append_cache(*kv, c, table, w["prefix"], turns)
        graph.replay()
        check_cache(cache, c)
        turned, _ = O.rotate_heads(w["q"], turns, prefix_len=w["prefix"])
        w["q"], w["c"] = rounded(turned, "bf16"), c
        check_attend(w, attend.out)


def test_host_tensors_and_a_side_stream(cuda_device):
    rng = np.random.default_rng(21)
    w = make_attend(rng, 2, 3, 4, 2, 64, 16, (30, 11), True)
    cache = on_gpu(w["c"])
    cpu = lambda a: torch.from_numpy(np.ascontiguousarray(a))  # noqa: E731
    got = dv.attend_cache(cpu(w["q"]).bfloat16(), cache, cpu(w["table"]), cpu(w["prefix"]), parent=cpu(w["parent"]))
    assert got["out"].device.type == "cpu"
    check_attend(w, got)
    side = torch.cuda.Stream()
    again = dv.attend_cache(dev(w["q"]).bfloat16(), cache, dev(w["table"]), dev(w["prefix"]), parent=dev(w["parent"]),
                            stream=side)
    side.synchronize()
    assert torch.equal(again["out"].cpu(), got["out"])
    table = dv.rotation_table(64, 64, stream=side)
    side.synchronize()
    turned = dv.rotate_heads(cpu(w["q"]).bfloat16(), table, prefix_len=cpu(w["prefix"]))["out"]
    want, _ = O.rotate_heads(w["q"], table.cpu().numpy(), prefix_len=w["prefix"])
    assert same(turned.float(), rounded(want, "bf16"))
    k = rounded(rng.normal(0, 1, (2, 3, 2, 64)), "f32")
    out = dv.append_cache(cpu(k), cpu(k), cache, cpu(w["table"]), cpu(w["prefix"]), table=table)
    want, _ = O.append_cache(k, k, w["c"], w["table"], w["prefix"], table.cpu().numpy())
    check_cache(cache, want)
    assert out["seq_error"].device.type == "cpu" and not out["seq_error"].any()


def test_a_whole_tree_step(cuda_device):
    """Two steps as a user makes them: rotate and append a tree's rows, attend,
    verify the tree, append the kept path again, and attend a chain behind it."""
    rng = np.random.default_rng(22)
    B, n, Hq, H, D, page, V, width = 4, 12, 4, 2, 64, 32, 500, 6
    parent = make_parents(rng, B, n)
    depth = np.zeros((B, n), np.int32)
    for b in range(B):
        for i in range(1, n):
            depth[b, i] = depth[b, parent[b, i]] + 1
    turns = O.rotation_table(width * page, rng.random(32))
    c = make_cache(rng, B * width, H, page, D)
    table = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    prefix = np.array([5, 31, 60, 90], np.int32)
    q, k, v = (rounded(rng.normal(0, 1, (B, n, m, D)), "bf16") for m in (Hq, H, H))
    at = prefix[:, None] + depth
    cache, bt, tt, pt = on_gpu(c), dev(table), dev(turns), dev(prefix)
    kt, vt = dev(k).bfloat16(), dev(v).bfloat16()

    turned = dv.rotate_heads(dev(q).bfloat16(), tt, positions=dev(at))["out"]
    dv.append_cache(kt, vt, cache, bt, pt, table=tt, positions=dev(at))
    c, _ = O.append_cache(k, v, c, table, prefix, turns, positions=at)
    check_cache(cache, c)
    got = dv.attend_cache(turned, cache, bt, pt, parent=dev(parent))
    check_attend(dict(q=turned.float().cpu().numpy(), c=c, table=table, prefix=prefix, parent=parent), got)

    logits = torch.from_numpy(rng.normal(0, 2, (B, n, V)).astype(np.float32)).to(cuda_device)
    tokens = dev(rng.integers(0, V, (B, n), dtype=np.int32))
    for b in range(B):  # the target's argmax is the last child's token
        for i in range(1, n):
            logits[b, parent[b, i]] = 0.0
        for i in range(1, n):
            logits[b, parent[b, i], tokens[b, i].long()] = 20.0 + i
    kept = dv.verify_tree(dev(parent), tokens, logits, None, prefix_len=pt, max_depth=n - 1, greedy=True)
    nodes, length = kept["path_nodes"].cpu().numpy(), kept["path_len"].cpu().numpy()
    assert (length > 0).all()
    dv.append_cache(kt, vt, cache, bt, pt, table=tt, path_nodes=kept["path_nodes"], path_len=kept["path_len"])
    c, err = O.append_cache(k, v, c, table, prefix, turns, path_nodes=nodes, path_len=length)
    assert not err.any()
    check_cache(cache, c)

    after = prefix + length + 1
    assert np.array_equal(after, kept["rollback_idx"].cpu().numpy() + 1)
    q, k, v = (rounded(rng.normal(0, 1, (B, 2, m, D)), "bf16") for m in (Hq, H, H))
    dv.append_cache(dev(k).bfloat16(), dev(v).bfloat16(), cache, bt, dev(after), table=tt)
    c, _ = O.append_cache(k, v, c, table, after, turns)
    check_cache(cache, c)
    turned = dv.rotate_heads(dev(q).bfloat16(), tt, prefix_len=dev(after))["out"]
    got = dv.attend_cache(turned, cache, bt, dev(after))
    check_attend(dict(q=turned.float().cpu().numpy(), c=c, table=table, prefix=after, parent=None), got)
