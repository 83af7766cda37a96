"""What the operators of the key-value cache are measured on.

Three operators stand between a layer's projections and the attention output
that a verification step needs: the rotation of heads by their positions, the
appending of keys and values to a paged cache of 8-bit codes (keys rotated on
the way), and the attention of drafted rows, a chain's or a tree's, over that
cache.  Where ``own`` is true ``run`` calls the framework's kernels, otherwise
elementary torch operations compute the same results.

A cache holds pages of ``page`` tokens: codes [pages, heads, page, D] in e4m3
and one exponent for each page and head; a code c stands for c * 2^exponent.
A page's exponent is the least e with max |x| <= 2^(e + 7) over what a call
appends to it (of keys before their rotation, which moves a value by a factor
of at most 2.83: codes stay below 448), not below the page's earlier one while
that page holds earlier tokens, which are then scaled along.
"""

import math

import torch

own = False

BF16, F32 = "bfloat16", "float32"
FP8 = torch.float8_e4m3fn
LOW, HIGH = -100, 100  # an exponent's range


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one request, one token, queries of one layer: all latency
        dict(name="rotate_one", op="rotate", B=1, n=1, H=32, D=128, rot=128, pairs=False, tree=False, L=2000, dtype=BF16),
        # the queries of a batch of draft trees, positions by depth
        dict(name="rotate_tree", op="rotate", B=16, n=64, H=32, D=128, rot=128, pairs=False, tree=True, L=4100,
             dtype=BF16),
        # two odd prompts of a float32 model that rotates neighbouring pairs in half of each head, far positions
        dict(name="rotate_prompt_f32", op="rotate", B=2, n=4095, H=20, D=96, rot=48, pairs=True, tree=False, L=100000,
             dtype=F32),
        # one request, one token: all latency
        dict(name="append_one", op="append", B=1, n=1, H=8, D=128, rot=128, pairs=False, page=16, L=1001, path=0,
             dtype=BF16),
        # a batch of draft chains: the last token and five drafts each
        dict(name="append_chain", op="append", B=64, n=6, H=8, D=128, rot=128, pairs=False, page=64, L=1000, path=0,
             dtype=BF16),
        # after a tree verification: the kept paths' rows, float32, heads of an odd size
        dict(name="append_path_f32", op="append", B=16, n=64, H=12, D=80, rot=32, pairs=True, page=32, L=777, path=7,
             dtype=F32),
        # prompts of a batch, odd lengths
        dict(name="append_prompt", op="append", B=4, n=8191, H=8, D=128, rot=128, pairs=False, page=64, L=5, path=0,
             dtype=BF16),
        # one request, one token: all latency
        dict(name="attend_one", op="attend", B=1, n=1, Hq=32, H=8, D=128, page=16, L=1001, tree=False, ragged=False),
        # a small odd batch of a model without shared heads
        dict(name="attend_odd", op="attend", B=5, n=3, Hq=12, H=12, D=80, page=32, L=3001, tree=False, ragged=True),
        # a batch of draft chains over chat histories of different lengths
        dict(name="attend_chain", op="attend", B=64, n=6, Hq=32, H=8, D=128, page=64, L=8192, tree=False, ragged=True),
        # a batch of draft trees: enough rows for the products to bound it
        dict(name="attend_tree", op="attend", B=16, n=64, Hq=32, H=8, D=128, page=64, L=4100, tree=True, ragged=True),
        # two long documents: one sequence has to fill the GPU
        dict(name="attend_long", op="attend", B=2, n=9, Hq=32, H=8, D=128, page=128, L=131072, tree=False,
             ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotate", "append", "append", "attend", "attend", "attend"))
    D = rng.choice((64, 80, 96, 128, 128, 128, 256))
    page = rng.choice((16, 32, 64, 128))
    H = rng.choice((1, 2, 4, 7, 8, 12))
    if op == "attend":
        Hq = H * rng.choice((1, 2, 4, 4, 7, 8))
        tree = rng.random() < 0.4
        n = _log_int(rng, 2, 64) if tree else _log_int(rng, 1, 16)
        L = _log_int(rng, 1, 131072)
        most = min(64, 400_000_000 // (L * H * D), 50_000_000_000 // (L * Hq * n * D * 4))
        return dict(op=op, B=_log_int(rng, 1, max(1, most)), n=n, Hq=Hq, H=H, D=D, page=page, L=L, tree=tree,
                    ragged=rng.random() < 0.7) if most >= 1 else draw(rng)
    rot = rng.choice((D, D, D // 2))
    if op == "rotate":
        H = H * rng.choice((1, 4))
        n = _log_int(rng, 1, 8191)
        most = max(1, min(64, 2 * 4095 * 20 * 96 // (n * H * D)))
        return dict(op=op, B=_log_int(rng, 1, most), n=min(n, 2 * 4095 * 20 * 96 // (H * D)), H=H, D=D, rot=rot,
                    pairs=rng.random() < 0.5, tree=n <= 64 and rng.random() < 0.5, L=_log_int(rng, 1, 100000),
                    dtype=rng.choice((BF16, BF16, F32)))
    path = rng.choice((0, 0, rng.randint(1, 8)))
    n = _log_int(rng, 8, 64) if path else _log_int(rng, 1, 8191)
    most = max(1, min(64, 2 ** 24 // (n * H * D)))
    return dict(op=op, B=_log_int(rng, 1, most), n=min(n, 2 ** 24 // (H * D)), H=H, D=D, rot=rot,
                pairs=rng.random() < 0.5, page=page, L=_log_int(rng, 1, 4000), path=path,
                dtype=rng.choice((BF16, BF16, F32)))


def _lengths(c):
    """Committed tokens of each sequence, known from the case."""
    if not c.get("ragged", True):
        return [c["L"]] * c["B"]
    return [c["L"] - b * (c["L"] // 2) // c["B"] for b in range(c["B"])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _table(rows, rot):
    """cos and sin of position * frequency, frequencies halved four times for a long context."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot) / 4.0
    angle = torch.arange(rows, dtype=torch.float64, device="cuda").unsqueeze(1) * freq
    return torch.cat((angle.cos(), angle.sin()), 1).float()


def _parents(B, n, g):
    at = torch.arange(n, device="cuda", dtype=torch.float32)
    # children follow their parent within a few widths: depths of a handful
    back = 1 + torch.rand((B, n), generator=g, device="cuda") * torch.clamp(at * 0.6, min=1.0)
    parent = torch.clamp(at - back, min=0.0).to(torch.int32)
    parent[:, 0] = -1
    return parent


def _depths(parent):
    B, n = parent.shape
    return _ancestors(parent).sum(2).to(torch.int32) - 1


def _ancestors(parent):
    """[B, n, n]: whether node j is node i or lies on the path from the root to it."""
    B, n = parent.shape
    step = torch.zeros((B, n, n), dtype=torch.float64, device="cuda")
    step.scatter_(2, parent.clamp(min=0).long().unsqueeze(2), 1.0)
    step[:, 0] = 0.0
    eye = torch.eye(n, dtype=torch.float64, device="cuda")
    return torch.linalg.matrix_power(eye + step, n) > 0


def _codes(shape, g):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, 30.0, generator=g)
    return x.clamp_(-128.0, 128.0).to(FP8).view(torch.uint8)


def _pages(c, tokens, g):
    """A block table: each sequence's pages, anywhere in the cache."""
    width = (tokens + c["page"] - 1) // c["page"]
    total = c["B"] * width + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    return order[:c["B"] * width].view(c["B"], width).contiguous(), total


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    B, n, H, D = c["B"], c["n"], c["H"], c["D"]
    s = dict(op=c["op"])
    lengths = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
    if c["op"] == "rotate":
        s["x"] = torch.empty((B, n, H, D), dtype=torch.float32, device="cuda").normal_(generator=g).to(
            getattr(torch, c["dtype"]))
        s["table"], s["pairs"] = _table(c["L"] + n, c["rot"]), c["pairs"]
        within = _depths(_parents(B, n, g)) if c["tree"] else torch.arange(n, dtype=torch.int32, device="cuda")
        s["positions"] = (lengths.unsqueeze(1) + within).contiguous()
        return s
    rows = n if c["op"] == "attend" or not c["path"] else c["path"] + 1
    s["block_table"], total = _pages(c, c["L"] + rows, g)
    s["prefix_len"] = lengths
    for name in ("k", "v"):
        s[name + "_codes"] = _codes((total, H, c["page"], D), g)
        s[name + "_exps"] = torch.randint(-7, -4, (total, H), generator=g, device="cuda", dtype=torch.int8)
    if c["op"] == "append":
        for name in ("k", "v"):
            x = torch.empty((B, n, H, D), dtype=torch.float32, device="cuda").normal_(generator=g)
            # a few channels of every head are much larger than the others
            x *= torch.where(torch.rand((H, D), generator=g, device="cuda") < 0.03, 6.0, 1.0)
            s[name] = x.to(getattr(torch, c["dtype"]))
        s["table"], s["pairs"] = _table(c["L"] + rows, c["rot"]), c["pairs"]
        s["path_nodes"] = s["path_len"] = None
        if c["path"]:
            # an ascending path from the root; nodes past its length are -1, as the verification leaves them
            pick = torch.rand((B, n - 1), generator=g, device="cuda").argsort(1)[:, :c["path"]].sort(1).values + 1
            s["path_len"] = torch.randint(0, c["path"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            pick = torch.where(torch.arange(c["path"], device="cuda") < s["path_len"].unsqueeze(1), pick, -1)
            s["path_nodes"] = torch.cat((torch.zeros_like(pick[:, :1]), pick), 1).to(torch.int32).contiguous()
        return s
    G = c["Hq"] // H
    q = torch.empty((B, n, H, G, D), dtype=torch.float32, device="cuda").normal_(generator=g)
    # the first token draws most of the attention and adds little: queries and its key share a direction
    along = torch.randn((H, D), generator=g, device="cuda").sign()
    q += along.unsqueeze(1)
    first = s["block_table"][:, 0].long()
    s["k_codes"].view(FP8)[first, :, 0] = (along * 28.0).to(FP8)
    s["k_exps"][first] = -5
    s["v_codes"].view(FP8)[first, :, 0] = torch.randn((B, H, D), generator=g, device="cuda").to(FP8)
    s["q"] = q.view(B, n, c["Hq"], D).bfloat16()
    s["parent"] = _parents(B, n, g) if c["tree"] else None
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _turned(x, table, pairs):
    """x [..., D] rotated by table rows [..., rot] (broadcast over the heads)."""
    half = table.shape[-1] // 2
    cos, sin = table[..., :half], table[..., half:]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    if pairs:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        head = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((head, rest), -1)


def _plain_rotate(s):
    rows = s["table"][s["positions"].long()].unsqueeze(2)
    return _turned(s["x"].float(), rows, s["pairs"]).to(s["x"].dtype)


def _plain_append(s, name, slots, row, new, pages, touched):
    codes, exps, x = s[name + "_codes"], s[name + "_exps"], s[name]
    page = codes.shape[2]
    x = x[torch.arange(x.shape[0], device="cuda").view(-1, 1, 1), row].float()  # [B, pages, page, H, D]
    most = torch.where(new[..., None, None], x.abs(), 0.0).amax((2, 4))
    part, power = torch.frexp(most)
    e = torch.where(most > 0, power - (part == 0.5).int() - 7, LOW).clamp(LOW, HIGH)
    before = exps[pages].int()
    earlier = (slots[:, :, :1] < s["prefix_len"].view(-1, 1, 1)) & touched.unsqueeze(2)
    e = torch.where(earlier, torch.maximum(e, before), e)
    if name == "k" and s["table"] is not None:
        x = _turned(x, s["table"][slots.clamp(max=s["table"].shape[0] - 1)].unsqueeze(3), s["pairs"])
    fresh = torch.ldexp(x, -e[:, :, None, :, None]).to(FP8).view(torch.uint8).transpose(2, 3)
    held = codes[pages]
    scaled = torch.ldexp(held.view(FP8).float(), (before - e)[..., None, None]).to(FP8).view(torch.uint8)
    past = (slots < s["prefix_len"].view(-1, 1, 1))[:, :, None, :, None]
    made = torch.where(new[:, :, None, :, None], fresh, torch.where(past, scaled, held))
    at = pages[touched]
    codes[at] = made[touched]
    exps[at] = e[touched].to(torch.int8)


def _plain_append_both(s):
    B, n = s["k"].shape[:2]
    page, width = s["k_codes"].shape[2], s["block_table"].shape[1]
    prefix = s["prefix_len"].long().view(B, 1)
    rows = n if s["path_nodes"] is None else s["path_nodes"].shape[1]
    count = torch.full_like(prefix, n) if s["path_len"] is None else s["path_len"].long().view(B, 1) + 1
    at = prefix // page + torch.arange((rows + page - 2) // page + 1, device="cuda")
    pages = s["block_table"].gather(1, at.clamp(max=width - 1)).long()
    slots = (at * page).unsqueeze(2) + torch.arange(page, device="cuda")
    i = slots - prefix.unsqueeze(2)
    new = (i >= 0) & (i < count.unsqueeze(2))
    row = i.clamp(0, rows - 1)
    if s["path_nodes"] is not None:
        row = s["path_nodes"].long().gather(1, row.flatten(1)).view_as(row).clamp(min=0)
    touched = new.any(2)
    for name in ("k", "v"):
        _plain_append(s, name, slots, row, new, pages, touched)


def _held(codes, exps, table):
    """A sequence's keys or values as float32 [B, H, tokens, D]."""
    index = table.long()
    x = torch.ldexp(codes[index].view(FP8).float(), exps[index].int()[..., None, None])
    B, P, H, page, D = x.shape
    return x.transpose(1, 2).reshape(B, H, P * page, D)


def _plain_attend(s):
    q = s["q"]
    B, n, Hq, D = q.shape
    k = _held(s["k_codes"], s["k_exps"], s["block_table"])
    H, tokens = k.shape[1], k.shape[2]
    G = Hq // H
    x = q.float().view(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    x = (x @ k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    at = torch.arange(tokens, device="cuda") - s["prefix_len"].view(B, 1)  # [B, tokens]
    if s["parent"] is None:
        over = torch.ones((n, n), dtype=torch.bool, device="cuda").tril().expand(B, n, n)
    else:
        over = _ancestors(s["parent"])
    inside = over.gather(2, at.clamp(0, n - 1).unsqueeze(1).expand(B, n, tokens))
    seen = (at < 0).unsqueeze(1) | ((at >= 0) & (at < n)).unsqueeze(1) & inside
    x = x.masked_fill(~seen.repeat_interleave(G, 1).unsqueeze(1), float("-inf"))
    x = torch.exp(x - x.amax(3, keepdim=True))
    total = x.sum(3, keepdim=True)
    y = (x @ _held(s["v_codes"], s["v_exps"], s["block_table"])) / total
    return y.view(B, H, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D).to(q.dtype)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _state(s):
    """The cache after an append: codes as the e4m3 values that they are, and their exponents."""
    return dict(k=s["k_codes"].view(FP8), v=s["v_codes"].view(FP8), k_exps=s["k_exps"], v_exps=s["v_exps"])


def run(state):
    s = state
    if own:
        import draft_verification_gb300 as dv
        plan = s.get("plan")
        if plan is None:  # bound once to the caller's buffers, run every step
            if s["op"] == "rotate":
                plan = dv.RotateHeadsPlan(s["x"], s["table"], positions=s["positions"], pairs=s["pairs"])
            else:
                cache = dv.PagedCache(s["k_codes"], s["v_codes"], s["k_exps"], s["v_exps"])
                if s["op"] == "append":
                    plan = dv.AppendCachePlan(s["k"], s["v"], cache, s["block_table"], s["prefix_len"],
                                              table=s["table"], pairs=s["pairs"], path_nodes=s["path_nodes"],
                                              path_len=s["path_len"])
                else:
                    plan = dv.AttendCachePlan(s["q"], cache, s["block_table"], s["prefix_len"], parent=s["parent"])
            s["plan"] = plan
        out = plan.run()
        return _state(s) if s["op"] == "append" else dict(y=out["out"])
    if s["op"] == "rotate":
        return dict(y=_plain_rotate(s))
    if s["op"] == "append":
        _plain_append_both(s)
        return _state(s)
    return dict(y=_plain_attend(s))


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    B, n, H, D = c["B"], c["n"], c["H"], c["D"]
    if c["op"] == "attend":
        keys = sum(_lengths(c)) + B * n
        return {"bytes": 2 * keys * H * D + 4 * keys // c["page"] + 2 * keys // c["page"] * H
                + 4 * B * n * c["Hq"] * D, "flops": 4 * keys * n * c["Hq"] * D}
    e = 4 if c["dtype"] == F32 else 2
    if c["op"] == "rotate":
        return {"bytes": 2 * B * n * H * D * e + B * n * 4 + min(B * n, c["L"] + n) * c["rot"] * 4,
                "flops": 3 * B * n * H * c["rot"]}
    rows = B * n if not c["path"] else B * (1 + c["path"] // 2)
    return {"bytes": 2 * rows * H * D * (e + 1) + min(rows, c["L"] + n) * c["rot"] * 4, "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_turn(x, angles, pairs):
    """x [rows, H, D] in 64 bits as complex numbers times cos + i sin, [rows, rot]."""
    half = angles.shape[1] // 2
    turn = torch.complex(angles[:, :half].double(), angles[:, half:].double()).unsqueeze(1)
    y = x.clone()
    re = slice(0, 2 * half, 2) if pairs else slice(0, half)
    im = slice(1, 2 * half, 2) if pairs else slice(half, 2 * half)
    z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * turn
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_append(s):
    out = dict(k_exps=None, v_exps=None)
    page = s["k_codes"].shape[2]
    B, n = s["k"].shape[:2]
    for name in ("k", "v"):
        held = s[name + "_codes"].view(FP8).double()
        exps = s[name + "_exps"].tolist()
        for b in range(B):
            start = int(s["prefix_len"][b])
            rows = torch.arange(n, device="cuda")
            if s["path_nodes"] is not None:
                rows = s["path_nodes"][b, :int(s["path_len"][b]) + 1].long()
            x = s[name][b, rows].double()
            y = x
            if name == "k":
                y = _exact_turn(x, s["table"][start:start + len(rows)], s["pairs"])
            done = 0
            while done < len(rows):
                at = (start + done) % page
                take = min(page - at, len(rows) - done)
                p = int(s["block_table"][b, (start + done) // page])
                most = x[done:done + take].abs().amax((0, 2)).tolist()
                for h, m in enumerate(most):
                    e = LOW
                    if m > 0:
                        part, power = math.frexp(m)
                        e = max(LOW, min(HIGH, power - (7 if part > 0.5 else 8)))
                    if at > 0:
                        e = max(e, exps[p][h])
                        held[p, h, :at] *= 2.0 ** (exps[p][h] - e)
                    held[p, h, at:at + take] = y[done:done + take, h] * 2.0 ** -e
                done += take
        out[name] = held
    return out


def _exact_attend(s):
    q = s["q"].double()
    B, n, Hq, D = q.shape
    H, page = s["k_codes"].shape[1:3]
    out = torch.empty_like(q)
    parents = None if s["parent"] is None else s["parent"].tolist()
    for b in range(B):
        past = int(s["prefix_len"][b])
        keys = past + n
        pages = s["block_table"][b, :(keys + page - 1) // page].long()
        allowed = torch.zeros((n, keys), dtype=torch.bool)
        allowed[:, :past] = True
        for i in range(n):
            j = i
            while j >= 0:
                allowed[i, past + j] = True
                j = j - 1 if parents is None else parents[b][j] if j > 0 else -1
        allowed = allowed.cuda()
        for h in range(H):
            k, v = (s[m + "_codes"][pages, h].view(FP8).double()
                    * torch.exp2(s[m + "_exps"][pages, h].double()).view(-1, 1, 1) for m in ("k", "v"))
            k, v = k.reshape(-1, D)[:keys], v.reshape(-1, D)[:keys]
            group = slice(h * (Hq // H), (h + 1) * (Hq // H))
            w = (q[b, :, group] @ k.t() / math.sqrt(D)).masked_fill(~allowed.unsqueeze(1), float("-inf")).softmax(2)
            out[b, :, group] = w @ v
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rotate":
        x = s["x"].double()
        rows = s["table"][s["positions"].long()].flatten(0, 1)
        return dict(y=_exact_turn(x.flatten(0, 1), rows, s["pairs"]).view_as(x))
    if s["op"] == "append":
        return _exact_append(s)
    return dict(y=_exact_attend(s))
