"""The cache operators, written out plainly: rotary positions, appending to a
paged cache of e4m3 codes, attention of drafted rows over it.

TEST INFRASTRUCTURE ONLY (see the package docstring): only the test suite and
``__graft_entry__.smoke()`` call it.

Rotation and appending are rules of float32 steps, so they are restated in
float32 NumPy (a rounding per operation) and their results are the bits, not an
approximation of them.  Attention is float64 on the codes' exact values; it
follows Staged Speculative Decoding (arXiv 2308.04623), abstract, in that a
tree's row sees the committed tokens and its own root path.
"""

from __future__ import annotations

import numpy as np

ERR_PARENT, ERR_NONFINITE, ERR_CACHE, ERR_POSITION = 2, 4, 128, 256
LOW, HIGH = -100, 100


# ---------------------------------------------------------------------------
# e4m3
# ---------------------------------------------------------------------------

def e4m3_values():
    """The 256 codes' values: sign, 4 exponent bits (bias 7), 3 mantissa bits;
    exponent 0 subnormal, all ones but the sign NaN."""
    out = np.empty(256)
    for code in range(256):
        e, m = code >> 3 & 15, code & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[code] = np.nan if code & 127 == 127 else -v if code & 128 else v
    return out


VALUES = e4m3_values()


def to_e4m3(x):
    """float array -> codes, to nearest, ties to even; beyond 448 and NaN: NaN."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    good = a <= 448.0
    a = np.where(good, a, 0.0)
    _, power = np.frexp(a)  # a = part 2^power, part in [0.5, 1)
    step = 2.0 ** (np.maximum(power - 1, -6) - 3)
    r = np.rint(a / step) * step
    code = np.searchsorted(VALUES[:127], r).astype(np.uint8)
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(good, code, 127).astype(np.uint8)


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------

def rotation_table(rows, freq, magnitude=1.0):
    angle = np.arange(rows, dtype=np.float64)[:, None] * np.asarray(freq, np.float64)
    return (np.concatenate([np.cos(angle), np.sin(angle)], 1) * magnitude).astype(np.float32)


def _turn(x, row, pairs, transpose=False):
    """x float32 [H, D] by a table row [rot] (or None: NaN)."""
    if row is None:
        return None
    half = len(row) // 2
    c, s = row[:half].astype(np.float32), row[half:].astype(np.float32)
    s = -s if transpose else s
    y = x.astype(np.float32).copy()
    ia = np.arange(half) * 2 if pairs else np.arange(half)
    ib = ia + 1 if pairs else ia + half
    a, b = x[:, ia].astype(np.float32), x[:, ib].astype(np.float32)
    y[:, ia] = a * c - b * s
    y[:, ib] = b * c + a * s
    return y


def rotate_heads(x, table, positions=None, prefix_len=None, pairs=False, transpose=False):
    """x [B, n, H, D] (exact values); returns (float32 [B, n, H, D] before the
    last rounding, error bits [B])."""
    B, n, H, D = x.shape
    y = np.asarray(x, np.float32).copy()
    err = np.zeros(B, np.int32)
    rot = table.shape[1]
    for b in range(B):
        for i in range(n):
            t = int(positions[b, i]) if positions is not None else (int(prefix_len[b]) if prefix_len is not None else 0) + i
            if 0 <= t < len(table):
                y[b, i] = _turn(y[b, i], table[t], pairs, transpose)
            else:
                y[b, i, :, :rot] = np.nan
                err[b] |= ERR_POSITION
    return y, err


# ---------------------------------------------------------------------------
# appending
# ---------------------------------------------------------------------------

def exponent_of(x):
    """The least e with |x| <= 2^(e + 7) for all finite x, in range."""
    a = np.abs(np.asarray(x, np.float64))
    a = a[np.isfinite(a)]
    m = a.max() if a.size else 0.0
    if m < 2.0 ** -126:
        return LOW
    part, power = np.frexp(m)
    return int(np.clip(power - (1 if part == 0.5 else 0) - 7, LOW, HIGH))


def append_cache(k, v, cache, block_table, prefix_len=None, table=None, pairs=False, positions=None, count=None,
                 path_nodes=None, path_len=None):
    """cache: dict of k_codes, v_codes uint8 [pages, H, page, D], k_exps, v_exps
    int8 [pages, H]; returns (the cache afterwards, error bits [B])."""
    B, n, H, D = k.shape
    out = {name: a.copy() for name, a in cache.items()}
    pages, _, page, _ = cache["k_codes"].shape
    err = np.zeros(B, np.int32)
    for b in range(B):
        start = 0 if prefix_len is None else int(prefix_len[b])
        if path_nodes is not None:
            if path_nodes[b, 0] == -1:
                continue
            m = int(path_len[b]) + 1
            if not 1 <= m <= path_nodes.shape[1]:
                err[b] |= ERR_CACHE
                m = 0
            rows = [int(r) for r in path_nodes[b, :m]]
            if any(not 0 <= r < n for r in rows):
                err[b] |= ERR_PARENT
        else:
            m = n if count is None else int(count[b])
            if not 0 <= m <= n:
                err[b] |= ERR_CACHE
            rows = list(range(max(m, 0)))
        if start < 0 or start + m > block_table.shape[1] * page:
            err[b] |= ERR_CACHE
        if err[b]:
            continue
        done = 0
        while done < len(rows):
            at = (start + done) % page
            take = min(page - at, len(rows) - done)
            p = int(block_table[b, (start + done) // page])
            mine = rows[done:done + take]
            if not 0 <= p < pages:
                err[b] |= ERR_CACHE
                done += take
                continue
            for name, x in (("k", k), ("v", v)):
                for h in range(H):
                    e = exponent_of(x[b, mine, h])
                    codes = out[name + "_codes"][p, h]
                    if at > 0:
                        old = int(out[name + "_exps"][p, h])
                        e = max(e, old)
                        if e > old:
                            codes[:at] = to_e4m3(VALUES[codes[:at]] * 2.0 ** (old - e))
                    out[name + "_exps"][p, h] = e
                    for r, row in enumerate(mine):
                        y = np.asarray(x[b, row, h], np.float32)
                        lost = np.zeros(D, bool)
                        if name == "k" and table is not None:
                            t = int(positions[b, row]) if positions is not None else start + done + r
                            if 0 <= t < len(table):
                                y = _turn(y[None], table[t], pairs)[0]
                            else:
                                y = y.copy()
                                y[:table.shape[1]] = np.nan
                                lost[:table.shape[1]] = True
                                err[b] |= ERR_POSITION
                        z = y.astype(np.float64) * 2.0 ** -e
                        if (~(np.abs(z) <= 448.0) & ~lost).any():
                            err[b] |= ERR_NONFINITE
                        codes[at + r] = to_e4m3(z)
            done += take
    return out, err


def cache_values(codes, exps):
    return VALUES[codes] * 2.0 ** exps.astype(np.float64)[..., None, None]


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def own_rows(parent, i):
    """The drafted rows that row i sees: itself and, in a chain (parent None),
    those before it, in a tree its ancestors.  (rows, whether a parent was malformed)"""
    if parent is None:
        return set(range(i + 1)), False
    seen, bad = {i, 0}, False
    while i > 0:
        p = int(parent[i])
        if not 0 <= p < i:
            p, bad = 0, True
        seen.add(p)
        i = p
    return seen, bad


def attend_cache(q, cache, block_table, prefix_len=None, count=None, parent=None, scale=None, tile=128):
    """q [B, n, Hq, D] (exact values).  Returns (out float64 [B, n, Hq, D], a
    dict of what an error bound is made of, error bits [B]):

      mass   sum_t w_t |v_t| / sum_t w_t, as out
      floor  sum over tiles of `tile` tokens of the largest w of the tile and
             its two neighbours (weights are rounded relative to the largest of
             one or two tiles next to each other) times the tile's sum of |v|,
             over sum_t w_t, as out.  Weights here carry the value exponent of
             their page in both sums, as the kernel's do
      sums   the same for the sum of the weights: sum over tiles of the largest
             w of the tile and its neighbours, without exponents, times the
             tile's tokens, over sum_t w_t, [B, n, Hq]
      score  the largest |scale * q . k| term sum of a row: scale * max |q| *
             max_t sum |k|, [B, n, Hq]
    """
    B, n, Hq, D = q.shape
    pages, H, page, _ = cache["k_codes"].shape
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out = np.zeros((B, n, Hq, D))
    bound = dict(mass=np.zeros_like(out), floor=np.zeros_like(out), score=np.zeros((B, n, Hq)),
                 sums=np.zeros((B, n, Hq)))
    err = np.zeros(B, np.int32)
    kv, vv = cache_values(cache["k_codes"], cache["k_exps"]), VALUES[cache["v_codes"]]
    ve = 2.0 ** cache["v_exps"].astype(np.float64)
    for b in range(B):
        past = 0 if prefix_len is None else int(prefix_len[b])
        rows = n if count is None else int(count[b])
        if past < 0 or not 0 <= rows <= n or past + rows > block_table.shape[1] * page:
            err[b] |= ERR_CACHE
            continue
        keys = past + rows
        own = []
        for i in range(rows):
            seen, bad = own_rows(None if parent is None else parent[b], i)
            own.append(seen)
            err[b] |= ERR_PARENT if bad else 0
        t = np.arange(keys)
        where = block_table[b, t // page].astype(np.int64)
        lost = (where < 0) | (where >= pages)
        err[b] |= ERR_CACHE if lost.any() else 0
        where = np.where(lost, 0, where)
        for h in range(H):
            k, v, s = kv[where, h, t % page].copy(), vv[where, h, t % page].copy(), ve[where, h]
            k[lost] = np.nan
            for i in range(rows):
                seen = (t < past) | np.isin(t - past, list(own[i]))
                for g in range(h * (Hq // H), (h + 1) * (Hq // H)):
                    with np.errstate(invalid="ignore", over="ignore"):
                        x = k[seen] @ q[b, i, g] * scale
                        top = np.max(x[~np.isnan(x)], initial=-np.inf)
                        w = np.exp(x - (top if np.isfinite(top) else 0.0))
                        ws = w * s[seen]
                        out[b, i, g] = ws @ v[seen] / w.sum()
                        bound["mass"][b, i, g] = ws @ np.abs(v[seen]) / w.sum()
                        mine = t[seen] // tile
                        tops = np.zeros((2, keys // tile + 3))
                        for m, y in enumerate((ws, w)):
                            np.fmax.at(tops[m], mine + 1, y)
                        tops = np.fmax(np.fmax(tops[:, :-2], tops[:, 1:-1]), tops[:, 2:])
                        bound["floor"][b, i, g] = (tops[0][mine] @ np.abs(np.nan_to_num(v[seen]))) / w.sum()
                        bound["sums"][b, i, g] = tops[1][mine].sum() / w.sum()
                    bound["score"][b, i, g] = scale * np.abs(q[b, i, g]).max() * np.abs(k[seen]).sum(1).max()
    return out, bound, err
