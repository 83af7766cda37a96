"""attend_cache where a CTA takes many steps, so that all that it keeps in turn
(scores, weights, sums, maxima) comes round several times.

The NumPy oracle takes minutes at such sizes: ``attend64`` is the same rule and
the same bounds in float64 torch operations, on whatever device its tensors are,
and is itself compared with the oracle on the CPU.  Tolerances are those of
test_gpu_cache.py.
"""

import numpy as np
import pytest
import torch

from oracle import cache as O

from . import test_gpu_cache as T


def attend64(q, c, table, prefix, parent=None, device="cpu", tile=128):
    """oracle.cache.attend_cache of sequences of n rows each, finite codes, pages all there: (out, bound)."""
    B, n, Hq, D = q.shape
    H, page = c["k_codes"].shape[1:3]
    G = Hq // H
    scale = 1.0 / np.sqrt(D)
    values = torch.from_numpy(O.VALUES).to(device)
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
    kc, vc, ke, ve = (put(c[m]) for m in ("k_codes", "v_codes", "k_exps", "v_exps"))
    x = put(np.asarray(q, np.float64))
    out = torch.zeros((B, n, Hq, D), dtype=torch.float64, device=device)
    bound = dict(mass=torch.zeros_like(out), floor=torch.zeros_like(out), score=torch.zeros_like(out[..., 0]),
                 sums=torch.zeros_like(out[..., 0]))
    for b in range(B):
        past, keys = int(prefix[b]), int(prefix[b]) + n
        seen = torch.zeros((n, keys), dtype=torch.bool)
        seen[:, :past] = True
        for i in range(n):
            seen[i, [past + j for j in O.own_rows(None if parent is None else parent[b], i)[0]]] = True
        hidden = ~seen.to(device).repeat_interleave(G, 0)  # [n G, keys], rows in the order token, head
        pages = put(table[b, :-(-keys // page)].astype(np.int64))
        tiles = -(-keys // tile)
        pad = lambda a: torch.cat((a, a.new_zeros((tiles * tile - keys, *a.shape[1:]))))  # noqa: E731
        for h in range(H):
            k = (values[kc[pages, h].long()] * torch.exp2(ke[pages, h].double())[:, None, None]).reshape(-1, D)[:keys]
            v = values[vc[pages, h].long()].reshape(-1, D)[:keys]
            s = torch.exp2(ve[pages, h].double()).repeat_interleave(page)[:keys]
            rows = x[b, :, h * G:(h + 1) * G].reshape(n * G, D)
            y = (rows @ k.T * scale).masked_fill(hidden, -np.inf)
            w = torch.exp(y - y.amax(1, keepdim=True))
            total = w.sum(1, keepdim=True)
            to = lambda a: a.reshape(n, G, -1)  # noqa: E731
            at = (b, slice(None), slice(h * G, (h + 1) * G))
            out[at] = to((w * s) @ v / total)
            bound["mass"][at] = to((w * s) @ v.abs() / total)
            tops = []
            for z in (w * s, w):
                top = pad(z.T).reshape(tiles, tile, -1).amax(1)  # [tiles, n G]
                near = torch.zeros((tiles + 2, top.shape[1]), dtype=top.dtype, device=device)
                near[1:-1] = top
                tops.append(torch.maximum(torch.maximum(near[:-2], near[1:-1]), near[2:]))
            # (of the tokens that a row sees: a tile with unseen ones counts token by token)
            live = (~hidden).double()
            cover = tops[0].repeat_interleave(tile, 0)[:keys].T * live
            bound["floor"][at] = to(cover @ v.abs() / total)
            bound["sums"][at] = to((tops[1].repeat_interleave(tile, 0)[:keys].T * live).sum(1, keepdim=True) / total)[..., 0]
            size = k.abs().sum(1).expand(n * G, keys).masked_fill(hidden, 0.0).amax(1)
            bound["score"][at] = to(scale * rows.abs().amax(1) * size)[..., 0]
    return out.cpu().numpy(), {m: a.cpu().numpy() for m, a in bound.items()}


@pytest.mark.parametrize("tree", [False, True])
def test_the_rule_in_torch_is_the_oracles(tree):
    rng = np.random.default_rng(31)
    w = T.make_attend(rng, 3, 5, 6, 2, 32, 16, (300, 127, 0), tree)
    w["c"]["v_exps"] = rng.integers(-50, 51, w["c"]["v_exps"].shape).astype(np.int8)
    out, bound = attend64(w["q"], w["c"], w["table"], w["prefix"], w["parent"])
    want, wanted, err = O.attend_cache(w["q"], w["c"], w["table"], w["prefix"], parent=w["parent"])
    assert not err.any()
    for a, b in ((out, want), *((bound[m], wanted[m]) for m in wanted)):
        assert np.allclose(a, b, rtol=1e-12, atol=1e-300)


def many_steps(rng, n, G, D, apart, tree):
    """12 tiles and more for each of 304 CTAs, twice as many for each of 152."""
    B, H, page, prefix = 2, 8, 32, np.array((32768 + 5, 30001), np.int32)
    width = int(prefix.max() + n + page - 1) // page
    some = O.to_e4m3(np.clip(rng.normal(0, 40, 4096), -300, 300))
    c = {}
    for m in "kv":
        c[m + "_codes"] = some[rng.integers(0, 4096, (B * width, H, page, D), dtype=np.uint16)]
        c[m + "_exps"] = rng.integers(-7, -3, (B * width, H)).astype(np.int8)
    c["v_exps"] = (rng.integers(0, 2, (B * width, H)) * apart - apart // 2).astype(np.int8)
    if apart == 40:  # pages of zeros, as appending leaves them
        c["v_exps"][::7] = -100
        c["v_codes"][::7] = 0
    return dict(q=T.rounded(rng.normal(0, 1, (B, n, G * H, D)), "bf16"), c=c, prefix=prefix,
                table=rng.permutation(B * width).reshape(B, width).astype(np.int32),
                parent=T.make_parents(rng, B, n) if tree else None)


@pytest.mark.gpu
@pytest.mark.parametrize("n,G,D,tree", [
    (2, 4, 128, False), (1, 8, 64, False), (4, 4, 128, True), (6, 4, 128, False), (8, 4, 128, False),
    (12, 4, 128, True), (16, 4, 128, False), (4, 4, 256, False), (8, 4, 256, True),
])
@pytest.mark.parametrize("apart", [0, 4, 40])
def test_attend_many_steps(cuda_device, n, G, D, tree, apart):
    """Every size of a block, with value exponents that one sum holds and that lie too far apart for it; the same
    bits every time."""
    import draft_verification_gb300 as dv
    w = many_steps(np.random.default_rng(1000 * n + D + apart), n, G, D, apart, tree)
    plan = dv.AttendCachePlan(T.dev(w["q"]).bfloat16(), T.on_gpu(w["c"]), T.dev(w["table"]), T.dev(w["prefix"]),
                              parent=T.dev(w["parent"]))
    first = plan.run()["out"].clone()
    want, bound = attend64(w["q"], w["c"], w["table"], w["prefix"], w["parent"], cuda_device)
    off = np.abs(first.double().cpu().numpy() - want) - T.attend_bound(want, bound, D)
    assert (off <= 0).all(), off.max()
    for _ in range(20):
        assert torch.equal(plan.run()["out"], first)
    assert not plan.out["error_word"].any()


@pytest.mark.gpu
@pytest.mark.parametrize("n,G,D", [(2, 4, 128), (4, 4, 128), (6, 4, 128), (8, 4, 64), (12, 4, 128), (16, 4, 80), (3, 4, 256)])
@pytest.mark.parametrize("exponents", [(100, 98), (60, 60), (-58, -60), (-100, -99)])
def test_attend_tiles_without_all_their_pages(cuda_device, n, G, D, exponents):
    """Tiles that end after one page and more, of values whose exponents are all far from 0."""
    rng = np.random.default_rng(n + 1000 + exponents[0])
    w = T.make_attend(rng, 4, n, G, 1, D, 16, (250, 128, 3, 391), False)
    w["c"]["v_exps"] = rng.choice(np.array(exponents, np.int8), w["c"]["v_exps"].shape)
    T.check_attend(w, T.run_attend(w))
