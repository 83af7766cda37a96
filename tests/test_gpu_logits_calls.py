"""How the logit-side operators are called: streams, host tensors, workspaces,
buffers that do not begin or end where a copy would like them to, and the
limits of the arguments.  The tolerances are those of test_gpu_logits."""

import numpy as np
import pytest
import torch

from oracle import logits as O

from . import test_gpu_logits as T

pytestmark = pytest.mark.gpu


def later(t, device):
    """A copy of t that the current stream finishes some ten milliseconds from now."""
    r = torch.zeros_like(t, device=device)
    torch.cuda._sleep(20_000_000)
    r.copy_(t)
    return r


def test_functions_do_all_their_work_on_the_given_stream(cuda_device):
    """Inputs that the current stream has yet to write, free memory full of
    ones (a workspace taken from it has to be cleared in order), results read
    after the given stream alone."""
    import draft_verification_gb300 as dv
    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            for n in (1 << 9, 1 << 12, 3 << 20, 3 << 20, 20 << 20):
                torch.full((n,), 0xff, dtype=torch.uint8, device=cuda_device)
    R, V, d, group = 5, 1000, 8192, 128  # every tile is shared by CTAs
    x, codes, scales, z = T.make_product(R, V, d, group, True, 21, cuda_device)
    late = later(x, cuda_device)
    out = dv.int4_product(late, codes, scales, z, group=group, out_dtype=torch.float32, stream=side)
    del late
    torch.full((R, d), 1e9, dtype=torch.bfloat16, device=cuda_device)  # (the freed input's block, used again)
    side.synchronize()
    assert int(out["error_word"]) == 0
    T.check_product(out["logits"], x, codes, scales, z, group)

    w = torch.randn(300, 256, generator=torch.Generator().manual_seed(22)).to(cuda_device)
    out = dv.quantize_int4(later(w, cuda_device), group=64, zeros=True, stream=side)
    side.synchronize()
    T.check_quantize(w, out, 64, True)

    rng = np.random.default_rng(23)
    B, n, V = 3, 4, 5000
    p = T.make_process(rng, B, n, V, H=300, density=0.5)
    x = torch.from_numpy(rng.normal(0, 3, (B, n, V)).astype(np.float32)).to(cuda_device)
    kw = {k: T.dev(v, cuda_device) for k, v in p.items()}
    out = dv.process_logits(later(x, cuda_device), stream=side, **kw)
    side.synchronize()
    T.check_process(x, out, p)


@pytest.mark.parametrize("own_stream", [False, True])
def test_functions_return_complete_host_tensors(cuda_device, own_stream):
    """Host tensors in: the host may read the results as soon as the call returns."""
    import draft_verification_gb300 as dv
    stream = torch.cuda.Stream() if own_stream else None
    rng = np.random.default_rng(24)
    for k in range(3):
        x, codes, scales, z = T.make_product(40, 9000, 1024, 64, True, 25 + k, "cpu")
        out = dv.int4_product(x, codes, scales, z, group=64, stream=stream)
        assert out["logits"].device.type == "cpu"
        T.check_product(out["logits"].clone(), x, codes, scales, z, 64)
        w = torch.from_numpy(rng.normal(0, 1, (2000, 512)).astype(np.float32))
        T.check_quantize(w, {k: v.clone() for k, v in dv.quantize_int4(w, group=32, stream=stream).items()}, 32, False)
        p = T.make_process(rng, 4, 5, 30000, H=300, density=0.5)
        y = torch.from_numpy(rng.normal(0, 3, (4, 5, 30000)).astype(np.float32))
        out = dv.process_logits(y, stream=stream, **{k: torch.from_numpy(v) for k, v in p.items()})
        T.check_process(y, {k: v.clone() for k, v in out.items()}, p)


@pytest.mark.parametrize("V", [1, 7, 15, 16, 17, 100, 128, 129, 143, 144, 257, 400])
@pytest.mark.parametrize("group,d", [(32, 96), (128, 384), (64, 1024)])
def test_product_of_matrices_that_start_and_end_anywhere(cuda_device, V, group, d):
    """Scales and zero points at every byte that their type allows, between bytes that would show: NaN scales,
    zero points beyond 15."""
    import draft_verification_gb300 as dv
    x, codes, scales, z = T.make_product(3, V, d, group, True, V + d, cuda_device)
    rows = d // group
    first = None
    for k, pad in enumerate((0, 1, 3, 8, 0, 5, 16, 0)):
        def within(t, lead, fill):
            flat = torch.full((lead + (rows - 1) * (V + pad) + V + 16,), fill, dtype=t.dtype, device=cuda_device)
            view = flat.as_strided((rows, V), (V + pad, 1), lead)
            view.copy_(t)
            return view
        for zl in (2 * k, 2 * k + 1):
            out = dv.int4_product(x, codes, within(scales, k, float("nan")), within(z, zl, 255), group=group,
                                  out_dtype=torch.float32)
            assert int(out["error_word"]) == 0
            if first is None:
                T.check_product(out["logits"], x, codes, scales, z, group)
                first = out["logits"]
            assert torch.equal(out["logits"], first)


@pytest.mark.parametrize("addressed", [False, True])
def test_process_lengths_beyond_lists_of_width_zero(cuda_device, addressed):
    """A length of a list that holds nothing is out of its range too, whether or not the list has an address."""
    import draft_verification_gb300 as dv
    rng = np.random.default_rng(31)
    B, n, V = 4, 3, 500
    x = torch.from_numpy(rng.normal(0, 3, (B, n, V)).astype(np.float32)).to(cuda_device)
    w = dict(tokens=rng.integers(0, V, (B, n), dtype=np.int32), history=np.zeros((B, 0), np.int32),
             history_len=np.array([0, 1, -1, 0], np.int32), prompt_len=np.zeros(B, np.int32),
             bias_tokens=np.zeros((B, 0), np.int32), bias_values=np.zeros((B, 0), np.float32),
             bias_len=np.array([0, 0, 0, 2], np.int32), frequency=np.full(B, 0.5, np.float32))
    kw = {k: T.dev(v, cuda_device) for k, v in w.items()}
    if addressed:
        for k in ("history", "bias_tokens", "bias_values"):
            kw[k] = torch.ones((B, 4), dtype=kw[k].dtype, device=cuda_device)[:, :0]
    out = dv.ProcessLogitsPlan(x, kw.pop("tokens"), **kw).run()
    T.check_process(x, out, w)
    assert out["seq_error"].tolist() == [0, 1, 1, 1]
    # without the lists at all their lengths do not exist
    out = dv.ProcessLogitsPlan(x, T.dev(w["tokens"], cuda_device), frequency=kw["frequency"]).run()
    assert out["seq_error"].tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("B,n,V,H", [(3, 3, 2000, 60), (128, 2, 66000, 9000)])  # one kernel, and gathered first
def test_process_takes_the_stated_float32_steps(cuda_device, B, n, V, H):
    """Bit by bit."""
    f = np.float32
    rng = np.random.default_rng(32)
    K = 60
    w = dict(tokens=rng.integers(0, V, (B, n), dtype=np.int32), history=rng.integers(0, V, (B, H), dtype=np.int32),
             prompt_len=np.full(B, H // 3, np.int32), repetition=rng.uniform(0.7, 1.6, B).astype(f),
             frequency=np.full(B, 0.5, f), presence=np.full(B, 0.25, f),
             bias_tokens=np.stack([rng.permutation(V)[:K] for _ in range(B)]).astype(np.int32),
             bias_values=(rng.choice([1e-9, 1.0, -3e38, 3e38], (B, K)) * rng.uniform(0.5, 1.0, (B, K))).astype(f))
    # half of the biased tokens occur, some of them drafted
    w["bias_tokens"][:, ::2] = w["history"][:, -(K // 2):]
    w["tokens"][:, 0] = w["bias_tokens"][:, 2]
    x = rng.choice([0.75, 1.25, -0.75, 2.0, 3e38, -3e38], (B, n, V)).astype(f)
    want = np.empty_like(x)
    for b in range(B):
        made0 = np.bincount(w["history"][b, H // 3:], minlength=V)
        seen0 = np.bincount(w["history"][b], minlength=V) > 0
        bias = np.zeros(V, f)
        for t, v in zip(w["bias_tokens"][b], w["bias_values"][b]):
            with np.errstate(over="ignore"):
                bias[t] = f(bias[t] + v)  # in their order
        rho = w["repetition"][b]
        inv = f(1) / rho
        for i in range(n):
            path = np.bincount(w["tokens"][b, :i], minlength=V)
            made, seen = made0 + path, seen0 | (path > 0)
            with np.errstate(over="ignore"):
                x1 = np.where(seen, x[b, i] * np.where(x[b, i] > 0, inv, rho), x[b, i])
                x2 = np.where(made > 0, x1 - (0.5 * made + 0.25).astype(f), x1)  # (exact: small multiples of 1/4)
                want[b, i] = np.where(bias != 0, x2 + bias, x2)
    assert want.dtype == f
    out = T.run_process(T.dev(x, cuda_device), w, cuda_device)
    assert out["seq_error"].abs().sum() == 0
    assert np.array_equal(out["logits"].cpu().numpy(), want)


@pytest.mark.parametrize("B,n,V,H", [(2, 3, 2000, 60), (128, 2, 66000, 9000)])  # one kernel, and gathered first
def test_process_subtracts_the_penalty_before_it_adds_the_bias(cuda_device, B, n, V, H):
    """An element that the penalty cancels keeps a small bias; one that it takes past float32's end stays there."""
    f = np.float32
    history = np.full((B, H), 3, np.int32)
    history[:, 0], history[:, H // 2], history[:, H - 1] = 5, 7, V - 1
    w = dict(tokens=np.full((B, n), 11, np.int32), history=history,
             presence=np.where(np.arange(B) % 2, f(-3e38), f(0.75)).astype(f),
             bias_tokens=np.tile(np.array([5, 7, 11, V - 1], np.int32), (B, 1)),
             bias_values=np.where(np.arange(B)[:, None] % 2, f(-3e38), f(1e-9)).repeat(4, 1).astype(f))
    x = np.where(np.arange(B)[:, None, None] % 2, f(3e38), f(0.75)) * np.ones((B, n, V), f)
    want = x.copy()
    for b in range(B):
        for i in range(n):
            for t in (3, 5, 7, V - 1) + ((11,) if i else ()):
                want[b, i, t] = np.inf if b % 2 else 0.0
            for t in (5, 7, 11, V - 1):
                with np.errstate(over="ignore"):
                    want[b, i, t] = f(want[b, i, t] + w["bias_values"][b, 0])
    out = T.run_process(T.dev(x, cuda_device), w, cuda_device)
    assert np.array_equal(out["logits"].cpu().numpy(), want)


def test_product_reset_clears_what_a_given_up_run_leaves(cuda_device):
    """Counters that a run which gave up would leave (planted: some tiles counted once) are gone after reset(), on
    the stream it is given; so is the error word."""
    import draft_verification_gb300 as dv
    R, V, d, group = 5, 1000, 8192, 128  # every tile is shared by CTAs
    x, codes, scales, z = T.make_product(R, V, d, group, True, 41, cuda_device)
    need = dv.Int4ProductPlan(x, codes, scales, z, group=group).workspace.numel()
    for workspace in (None, torch.zeros(need, dtype=torch.uint8, device=cuda_device)):
        plan = dv.Int4ProductPlan(x, codes, scales, z, group=group, out_dtype=torch.float32, workspace=workspace)
        first = plan.run()["logits"].clone()
        T.check_product(first, x, codes, scales, z, group)
        for stream in (None, torch.cuda.Stream()):
            plan.workspace[:1024].view(torch.int32)[::3] = 1
            plan.out["error_word"].fill_(dv.ERR_INTERNAL)
            plan.out["logits"].fill_(7.0)
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            plan.reset(stream)
            out = plan.run(stream)
            torch.cuda.synchronize()
            assert int(out["error_word"]) == 0
            assert torch.equal(out["logits"], first)
        assert not plan.workspace[:1024].any()


def test_process_one_position_of_many(cuda_device):
    """Rows that lie far apart: the output's are close, and the same."""
    rng = np.random.default_rng(42)
    for V, dtype in ((5000, torch.bfloat16), (5001, torch.float32)):
        B = 6
        w = T.make_process(rng, B, 1, V, H=100, density=0.5)
        x = torch.from_numpy(rng.normal(0, 3, (B, 9, V)).astype(np.float32)).to(cuda_device, dtype)
        rows = x[:, :1]
        out = T.run_process(rows, w, cuda_device)
        assert out["logits"].untyped_storage().nbytes() < 2 * B * V * dtype.itemsize
        T.check_process(rows.contiguous(), out, w)


GATHERED = [  # many sequences with long lists: their entries are gathered first
    # B, n, V, pad, dtype, tokens below, kwargs
    (150, 2, 20000, 0, "bf16", None, dict(H=12000, bias=10, density=0.8)),
    (150, 2, 20001, 0, "bf16", None, dict(H=12002, bias=10)),
    # more distinct tokens than one window holds, and more than 1024 entries in a slab, from one slab and from two
    (150, 2, 66000, 0, "bf16", None, dict(H=20000, bias=500)),
    (150, 2, 66000, 0, "bf16", 5000, dict(H=20000, bias=30, density=0.6)),
    (150, 1, 66001, 3, "f32", 5000, dict(H=20001, bias=9)),
    (150, 3, 66000, 3, "bf16", None, dict(H=14000, tree=True, bias=0)),
    # exactly one bitmap of tokens, one token more, and more than one
    (40, 2, 262144, 0, "bf16", None, dict(H=4000, tree=True)),
    (40, 2, 262145, 7, "f32", None, dict(H=4000, density=0.3)),
    (40, 2, 300001, 0, "bf16", None, dict(H=4000, bias=40, density=0.5)),
    (40, 1, 300001, 7, "bf16", None, dict(H=40000, bias=3)),
]


@pytest.mark.parametrize("B,n,V,pad,dtype,below,kw", GATHERED, ids=lambda v: str(v) if not isinstance(v, dict) else None)
def test_process_gathered(cuda_device, B, n, V, pad, dtype, below, kw):
    import draft_verification_gb300 as dv
    rng = np.random.default_rng(B * 7919 + n * 104729 + V)
    w = T.make_process(rng, B, n, V, **kw)
    w["history_len"][::2] = kw["H"]
    if below:
        w["history"] %= below
    x = T.strided(B, n, V, pad, T.DTYPES[dtype], cuda_device)
    x.copy_(torch.from_numpy(rng.normal(0, 3, (B, n, V)).astype(np.float32)))
    args = {k: T.dev(v, cuda_device) for k, v in w.items()}
    plan = dv.ProcessLogitsPlan(x, args.pop("tokens"), **args)
    plan.workspace.fill_(0xa5)
    out = plan.run()
    assert not bool((plan.workspace == 0xa5).all())  # (it was used: the gathered form)
    T.check_process(x, out, w)
    first = T.bits(out["logits"]).copy()
    assert np.array_equal(T.bits(T.run_process(x, w, cuda_device, out=x)["logits"]), first)


@pytest.mark.parametrize("B,n,V,H", [(1, 9, 128256, 300000), (3, 2, 128256, 131072), (16, 1, 32000, 131072)])
def test_process_few_long_histories_are_read_where_they_apply(cuda_device, B, n, V, H):
    """One CTA per sequence would go through such a history alone, window by window (4 sequences of 131072 tokens
    over 128256: 420 us against 93): the entries are not gathered, the workspace is not used."""
    import draft_verification_gb300 as dv
    rng = np.random.default_rng(51)
    w = T.make_process(rng, B, n, V, H=H)
    x = torch.from_numpy(rng.normal(0, 3, (B, n, V)).astype(np.float32)).to(cuda_device, torch.bfloat16)
    args = {k: T.dev(v, cuda_device) for k, v in w.items()}
    plan = dv.ProcessLogitsPlan(x, args.pop("tokens"), **args)
    plan.workspace.fill_(0xa5)
    out = plan.run()
    assert bool((plan.workspace == 0xa5).all())
    T.check_process(x, out, w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [66000, 66001, 66003, 66004, 66007])
def test_process_gathered_tokens_at_the_slabs_borders(cuda_device, V, dtype):
    """Every token near a slab's border is touched; rows that start within a vector take some from the slab before."""
    rng = np.random.default_rng(52)
    B, n, H = 130, 2, 9000
    slab = 1024 if dtype == "f32" else 2048
    near = (np.arange(0, V, slab)[:, None] + np.arange(-9, 10)).ravel()
    near = near[(near >= 0) & (near < V)].astype(np.int32)
    w = T.make_process(rng, B, n, V, H=H, bias=40)
    w["history"] = near[rng.integers(0, len(near), (B, H))]
    w["history_len"][:] = H
    w["tokens"] = near[rng.integers(0, len(near), (B, n))]
    x = T.strided(B, n, V, 0, T.DTYPES[dtype], cuda_device)
    x.copy_(torch.from_numpy(rng.normal(0, 3, (B, n, V)).astype(np.float32)))
    T.check_process(x, T.run_process(x, w, cuda_device), w)
