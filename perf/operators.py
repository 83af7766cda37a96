"""What the logit-side operators are measured on.

Three operators stand between a model's hidden states and the logits that a
verification reads: the 4-bit group quantisation of an LM head, the product of
a few rows with such a head, and the per-request processing of logits
(penalties for repeated tokens, biases, grammar masks).  Where ``own`` is true
``run`` calls the framework's kernels, otherwise elementary torch operations
compute the same results.
"""

import math

import torch

own = False

BF16, F32 = "bfloat16", "float32"
GROUPS = (32, 64, 128)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one request drafting one token: all latency
        dict(name="process_draft_step", op="process", B=1, n=1, V=32000, H=200, tree=False, mask=False, bias=8,
             dtype=BF16),
        # a toy vocabulary in float32, constrained by a grammar, with an odd history
        dict(name="process_small_f32", op="process", B=4, n=5, V=1000, H=37, tree=False, mask=True, bias=3, dtype=F32),
        # a batch of chat requests: penalties and long bias lists, no grammar
        dict(name="process_chain_32k", op="process", B=32, n=9, V=32000, H=2048, tree=False, mask=False, bias=300,
             dtype=BF16),
        # draft trees over an odd vocabulary (rows start at every alignment), grammar masks per node
        dict(name="process_tree_50k", op="process", B=16, n=64, V=50257, H=777, tree=True, mask=True, bias=0,
             dtype=BF16),
        # the largest batch: long histories, every row masked or nearly so
        dict(name="process_chain_128k", op="process", B=128, n=9, V=128256, H=8192, tree=False, mask=True, bias=20,
             dtype=BF16),
        # a toy head, float32 weights, the finest groups with zero points
        dict(name="quantize_small_f32", op="quantize", V=1000, d=512, group=32, zeros=True, dtype=F32),
        # a small draft model's head
        dict(name="quantize_50k", op="quantize", V=50257, d=1024, group=64, zeros=True, dtype=BF16),
        # a 128k-vocabulary head, converted once when a model is loaded
        dict(name="quantize_128k", op="quantize", V=128256, d=4096, group=128, zeros=False, dtype=BF16),
        # a toy head: all latency
        dict(name="product_small", op="product", R=5, V=1000, d=256, group=32, zeros=True, dtype=F32),
        # one request drafting one token with a 128k-vocabulary head
        dict(name="product_one_row", op="product", R=1, V=128256, d=4096, group=128, zeros=False, dtype=BF16),
        # an odd batch over an odd vocabulary, zero points, float32 logits
        dict(name="product_odd", op="product", R=33, V=50257, d=2048, group=64, zeros=True, dtype=F32),
        # a full batch drafting one token each
        dict(name="product_batch", op="product", R=128, V=128256, d=4096, group=128, zeros=False, dtype=BF16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("process", "process", "quantize", "product", "product"))
    if op == "process":
        tree = rng.random() < 0.4
        n = _log_int(rng, 2, 64) if tree else _log_int(rng, 1, 16)
        V = _log_int(rng, 1000, 128256)
        most = max(1, min(128, 128 * 9 * 128256 // (n * V)))
        return dict(op=op, B=_log_int(rng, 1, most), n=n, V=V, H=_log_int(rng, 1, 8192) - 1, tree=tree,
                    mask=rng.random() < 0.6, bias=rng.choice((0, 1, _log_int(rng, 2, 300))),
                    dtype=rng.choice((BF16, BF16, F32)) if n * V * most < 64 * 2 ** 20 else BF16)
    group = rng.choice(GROUPS)
    V = _log_int(rng, 100, 128256)
    d = group * max(1, _log_int(rng, 128, 8192) // group)
    d = max(group, min(d, 128256 * 4096 // V // group * group))
    zeros = rng.random() < 0.5
    if op == "quantize":
        return dict(op=op, V=V, d=d, group=group, zeros=zeros,
                    dtype=F32 if V * d < 2 ** 27 and rng.random() < 0.5 else BF16)
    return dict(op=op, R=_log_int(rng, 1, 128), V=V, d=d, group=group, zeros=zeros,
                dtype=rng.choice((BF16, F32)) if V < 64000 else BF16)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _tokens(shape, V, g):
    # frequent tokens have low indices, as in a byte-pair vocabulary
    return (torch.rand(shape, generator=g, device="cuda").pow(4) * V).to(torch.int32).clamp_(0, V - 1)


def _prepare_process(c, g):
    B, n, V, H = c["B"], c["n"], c["V"], c["H"]
    s = dict(op="process", V=V)
    logits = torch.empty((B, n, V), dtype=getattr(torch, c["dtype"]), device="cuda")
    logits.normal_(0.0, 2.5, generator=g)
    s["logits"] = logits
    s["tokens"] = _tokens((B, n), V, g)
    s["parent"] = None
    if c["tree"]:
        at = torch.arange(n, device="cuda", dtype=torch.float32)
        # children follow their parent within a few widths: depths of a handful
        back = 1 + torch.rand((B, n), generator=g, device="cuda") * torch.clamp(at * 0.6, min=1.0)
        s["parent"] = torch.clamp(at - back, min=0.0).to(torch.int32)
        s["parent"][:, 0] = -1
    s["history"] = _tokens((B, max(H, 1)), V, g)
    s["history_len"] = torch.randint(H // 2, H + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    s["prompt_len"] = (s["history_len"] * torch.rand(B, generator=g, device="cuda")).to(torch.int32)
    s["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=g, device="cuda")
    s["frequency"] = 0.5 * torch.rand(B, generator=g, device="cuda")
    s["presence"] = torch.rand(B, generator=g, device="cuda") - 0.25
    K = c["bias"]
    s["bias_tokens"] = _tokens((B, K), V, g) if K else None
    s["bias_values"] = torch.randn((B, K), generator=g, device="cuda") * 4.0 if K else None
    s["bias_len"] = torch.randint(0, K + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if K else None
    s["mask"] = s["mask_index"] = None
    if c["mask"]:
        W = (V + 31) // 32
        # a grammar allows anything from a handful of tokens to nearly all:
        # per row, words without an allowed token, sparse words and full ones
        share = torch.exp(math.log(1e-3) * torch.rand((B * n, 1), generator=g, device="cuda"))
        words = torch.randint(-2 ** 31, 2 ** 31, (B * n, W), generator=g, device="cuda", dtype=torch.int64)
        full = torch.rand((B * n, W), generator=g, device="cuda") < share * 0.7
        words = torch.where(full, torch.full_like(words, -1), words)
        some = torch.rand((B * n, W), generator=g, device="cuda") < share
        s["mask"] = torch.where(some, words, torch.zeros_like(words)).to(torch.int32)
        index = torch.arange(B * n, device="cuda", dtype=torch.int32).view(B, n)
        free = torch.rand((B, n), generator=g, device="cuda") < 0.2
        s["mask_index"] = torch.where(free, torch.full_like(index, -1), index)
    return s


def _weights(c, g):
    w = torch.empty((c["V"], c["d"]), dtype=torch.float32, device="cuda").normal_(0.0, 0.02, generator=g)
    w *= 0.5 + torch.rand((c["V"], 1), generator=g, device="cuda")
    return w


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    if c["op"] == "process":
        return _prepare_process(c, g)
    w = _weights(c, g)
    if c["op"] == "quantize":
        return dict(op="quantize", w=w.to(getattr(torch, c["dtype"])), group=c["group"], zeros=c["zeros"])
    codes, scales, zeros = _plain_quantize(w, c["group"], c["zeros"])
    x = torch.empty((c["R"], c["d"]), dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=g)
    # final-norm outputs: a few channels are much larger than the others
    x *= torch.where(torch.rand(c["d"], generator=g, device="cuda") < 0.01, 8.0, 1.0)
    return dict(op="product", x=x.to(torch.bfloat16), codes=codes, scales=scales, zeros=zeros, group=c["group"],
                dtype=getattr(torch, c["dtype"]))


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_path(s, B, n):
    """[B, n, n]: whether drafted token j lies before row i (on its path, for a tree)."""
    if s["parent"] is None:
        # a chain: row i follows the drafted tokens 0 .. i - 1
        return torch.ones((n, n), device="cuda").tril(-1).expand(B, n, n)
    step = torch.zeros((B, n, n), dtype=torch.float64, device="cuda")
    step.scatter_(2, s["parent"].clamp(min=0).long().unsqueeze(2), 1.0)
    eye = torch.eye(n, dtype=torch.float64, device="cuda")
    on_path = (torch.linalg.matrix_power(step * (1 - eye[0]).view(1, n, 1) + eye, max(n - 1, 1)) > 0).float()
    on_path[:, :, 0] = 0.0  # the root's token is the history's last
    return on_path


def _plain_process(s):
    x = s["logits"].float()
    B, n, V = x.shape
    hist = s["history"].long()
    at = torch.arange(hist.shape[1], device="cuda")
    there = (at < s["history_len"].unsqueeze(1))
    made = there & (at >= s["prompt_len"].unsqueeze(1))
    zero = torch.zeros((B, V), device="cuda")
    count = zero.scatter_add(1, hist, made.float())
    seen = zero.scatter_add(1, hist, there.float())
    path = torch.zeros((B, n, V), device="cuda")
    path.scatter_add_(2, s["tokens"].long().unsqueeze(1).expand(B, n, n), _plain_path(s, B, n))
    seen = (seen.unsqueeze(1) + path) > 0
    count = path.add_(count.unsqueeze(1))
    rho = s["repetition"].view(B, 1, 1)
    x = torch.where(seen, torch.where(x > 0, x / rho, x * rho), x)
    x = x - (s["frequency"].view(B, 1, 1) * count + s["presence"].view(B, 1, 1) * (count > 0).float())
    if s["bias_tokens"] is not None:
        K = s["bias_tokens"].shape[1]
        valid = torch.arange(K, device="cuda") < s["bias_len"].unsqueeze(1)
        bias = zero.scatter_add(1, s["bias_tokens"].long(), torch.where(valid, s["bias_values"], 0.0))
        x = x + bias.unsqueeze(1)
    if s["mask"] is not None:
        bits = (s["mask"].unsqueeze(2) >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        allowed = bits.flatten(1)[:, :V].bool()
        index = s["mask_index"]
        allowed = allowed[index.clamp(min=0).long()] | (index < 0).unsqueeze(2)
        x = torch.where(allowed, x, float("-inf"))
    return x.to(s["logits"].dtype)


def _plain_quantize(w, group, with_zeros):
    V, d = w.shape
    x = w.float().view(V, d // group, group)
    if with_zeros:
        lo, hi = x.amin(2).clamp(max=0.0), x.amax(2).clamp(min=0.0)
        scale = ((hi - lo) / torch.full_like(hi, 15.0)).bfloat16()
        s = scale.float()
        z = torch.where(s > 0, (-lo / s).round().clamp(0, 15), 0.0)
        low, high, zero = 0.0, 15.0, z.unsqueeze(2)
    else:
        amax = x.abs().amax(2)
        scale = (amax / torch.full_like(amax, 7.0)).bfloat16()
        s, z = scale.float(), None
        low, high, zero = 0.0, 15.0, 8.0
    q = torch.where(s.unsqueeze(2) > 0, (x / s.unsqueeze(2)).round(), 0.0)
    q = (q + zero).clamp_(low, high).to(torch.uint8).view(V, d // 2, 2)
    codes = q[:, :, 0] | (q[:, :, 1] << 4)
    return codes, scale.t().contiguous(), None if z is None else z.to(torch.uint8).t().contiguous()


def _plain_product(s):
    codes, group = s["codes"], s["group"]
    V, d = codes.shape[0], codes.shape[1] * 2
    q = torch.stack((codes & 15, codes >> 4), 2).view(V, d // group, group).float()
    z = 8.0 if s["zeros"] is None else s["zeros"].t().float().unsqueeze(2)
    w = ((q - z) * s["scales"].t().float().unsqueeze(2)).view(V, d)
    return (s["x"].float() @ w.t()).to(s["dtype"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        import draft_verification_gb300 as dv
        plan = s.get("plan")
        if plan is None:  # bound once to the caller's buffers, run every step
            if s["op"] == "process":
                plan = dv.ProcessLogitsPlan(
                    s["logits"], s["tokens"], parent=s["parent"], history=s["history"],
                    history_len=s["history_len"], prompt_len=s["prompt_len"], repetition=s["repetition"],
                    frequency=s["frequency"], presence=s["presence"], bias_tokens=s["bias_tokens"],
                    bias_values=s["bias_values"], bias_len=s["bias_len"], mask=s["mask"],
                    mask_index=s["mask_index"])
            elif s["op"] == "quantize":
                plan = dv.QuantizeInt4Plan(s["w"], group=s["group"], zeros=s["zeros"])
            else:
                plan = dv.Int4ProductPlan(s["x"], s["codes"], s["scales"], s["zeros"], group=s["group"],
                                          out_dtype=s["dtype"])
            s["plan"] = plan
        out = plan.run()
        if s["op"] == "quantize":
            return dict(codes=out["codes"], scales=out["scales"], zeros=out.get("zeros"))
        return dict(y=out["logits"])
    if s["op"] == "process":
        return dict(y=_plain_process(s))
    if s["op"] == "quantize":
        codes, scales, zeros = _plain_quantize(s["w"], s["group"], s["zeros"])
        # 4-bit codes, two to a byte, and the whole zero points
        return dict(codes=codes, scales=scales, zeros=zeros)
    return dict(y=_plain_product(s))


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    e = 4 if c["dtype"] == F32 else 2
    if c["op"] == "process":
        rows = c["B"] * c["n"]
        b = 2 * rows * c["V"] * e + 4 * c["B"] * c["H"] + 8 * c["B"] * c["bias"] + 4 * rows
        if c["mask"]:
            b += rows * (c["V"] + 31) // 32 * 4
        return {"bytes": b, "flops": 0}
    groups = c["V"] * (c["d"] // c["group"])
    weights = c["V"] * c["d"] // 2 + groups * (3 if c["zeros"] else 2)
    if c["op"] == "quantize":
        return {"bytes": c["V"] * c["d"] * e + weights, "flops": 0}
    return {"bytes": weights + c["R"] * c["d"] * 2 + c["R"] * c["V"] * e, "flops": 2 * c["R"] * c["V"] * c["d"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_process(s):
    logits, V = s["logits"], s["V"]
    B, n = logits.shape[:2]
    out = torch.empty((B, n, V), dtype=torch.float64, device="cuda")
    tokens = s["tokens"].tolist()
    parent = None if s["parent"] is None else s["parent"].tolist()
    length, prompt = s["history_len"].tolist(), s["prompt_len"].tolist()
    index = None if s["mask"] is None else s["mask_index"].tolist()
    lane = torch.arange(V, device="cuda")
    for b in range(B):
        hist = s["history"][b, :length[b]].long()
        rho, af, ap = (float(s[k][b].double()) for k in ("repetition", "frequency", "presence"))
        base_seen = torch.bincount(hist, minlength=V)
        base_count = torch.bincount(hist[prompt[b]:], minlength=V)
        bias = torch.zeros(V, dtype=torch.float64, device="cuda")
        if s["bias_tokens"] is not None:
            k = int(s["bias_len"][b])
            bias.index_add_(0, s["bias_tokens"][b, :k].long(), s["bias_values"][b, :k].double())
        for i in range(n):
            before = tokens[b][:i]
            if parent is not None:
                before, j = [], i
                while j > 0:
                    before.append(tokens[b][j])
                    j = parent[b][j]
            seen, count = base_seen, base_count
            if before:
                path = torch.bincount(torch.tensor(before, device="cuda"), minlength=V)
                seen, count = seen + path, count + path
            x = logits[b, i].double()
            x = torch.where((seen > 0) & (x > 0), x / rho, torch.where(seen > 0, x * rho, x))
            x = x - af * count.double() - ap * (count > 0).double() + bias
            if index is not None and index[b][i] >= 0:
                word = s["mask"][index[b][i]].long()[lane // 32]
                x = x.masked_fill(((word >> (lane % 32)) & 1) == 0, float("-inf"))
            out[b, i] = x
    return dict(y=out)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "process":
        return _exact_process(s)
    group = s["group"]
    if s["op"] == "quantize":
        w, rows = s["w"], 16384
        parts = []
        for v in range(0, w.shape[0], rows):
            x = w[v:v + rows].double().unflatten(1, (-1, group))
            if s["zeros"]:
                parts.append((x.amax(2).clamp(min=0) - x.amin(2).clamp(max=0)).div(15).t())
            else:
                parts.append(x.abs().amax(2).div(7).t())
        return dict(codes=None, scales=torch.cat(parts, 1), zeros=None)
    V, rows = s["codes"].shape[0], 8192
    y = torch.empty((s["x"].shape[0], V), dtype=torch.float64, device="cuda")
    for v in range(0, V, rows):
        byte = s["codes"][v:v + rows].to(torch.int64)
        w = torch.empty((byte.shape[0], 2 * byte.shape[1]), dtype=torch.float64, device="cuda")
        w[:, 0::2] = (byte % 16).double()
        w[:, 1::2] = (byte // 16).double()
        zero = 8.0 if s["zeros"] is None else s["zeros"][:, v:v + rows].double().t().repeat_interleave(group, 1)
        w = (w - zero) * s["scales"][:, v:v + rows].double().t().repeat_interleave(group, 1)
        y[:, v:v + rows] = s["x"].double() @ w.t()
    return dict(y=y)
