"""The decoder block's operators between its linears, as measured work.

A served model's block runs, between the Q4_0 products: the append of a step's
keys and values to the paged cache (per-head norms and position rotation on
the way), attention over that cache (causal, sliding window, first tokens that
stay visible), and the norms around a block with its gate and residual scale.
Each case is one call of one of them.  Where ``own`` is true ``run`` calls the
framework, elsewhere it computes the same in elementary torch operations.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda:0"
WORKSPACE_BYTES = 134217728     # one buffer that serves every call of the framework
GOLDEN = 0.6180339887498949


# ---- cases ------------------------------------------------------------------
def _append(name, tokens, heads, kv_heads, dim, rot, page, norm, interleaved, half, far):
    return {"name": name, "op": "append", "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "rot": rot, "page": page, "norm": norm, "interleaved": interleaved,
            "half": half, "far": far}


def _attention(name, batch, tokens, kv, spread, heads, kv_heads, dim, page, window, sinks, half):
    return {"name": name, "op": "attention", "batch": batch, "tokens": tokens, "kv": kv,
            "spread": spread, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "window": window, "sinks": sinks, "half": half}


def _residual(name, rows, dim, post, gate, half_in, half_out):
    return {"name": name, "op": "residual", "rows": rows, "dim": dim, "post": post, "gate": gate,
            "half_in": half_in, "half_out": half_out}


def listed():
    return [
        # one conversation draws its next token: a 4B-class block's q, k, v rows, norms of q and
        # k, positions past what 32-bit angles carry
        _append("append_token", 1, 32, 8, 128, 128, 16, True, False, False, 300000),
        # a prefill pass of 512 positions of the same block
        _append("append_pass", 512, 32, 8, 128, 128, 16, True, False, False, 4096),
        # long prompts of a model with wide heads, half of each head rotated, binary16 rows
        _append("append_prompt", 8191, 16, 8, 256, 128, 64, False, True, True, 32768),
        # one conversation, 448 positions of context: latency
        _attention("decode_one", 1, 1, 448, 0.0, 32, 8, 128, 16, 0, 0, False),
        # 64 conversations of every length up to 8192 in one pass
        _attention("decode_batch", 64, 1, 8192, 0.95, 32, 8, 128, 64, 0, 0, True),
        # long conversations under a sliding window, the first four tokens kept, evicted pages
        # given back
        _attention("decode_window", 32, 1, 30001, 0.5, 16, 4, 256, 32, 4096, 4, False),
        # one very long conversation: the key axis has to be split
        _attention("decode_long", 1, 1, 131071, 0.0, 32, 8, 128, 64, 0, 0, True),
        # a prefill pass of 512 positions behind 3600 cached ones, window and first tokens
        _attention("pass_window", 1, 512, 4112, 0.0, 32, 8, 128, 16, 1024, 4, True),
        # two prompts of unequal length from an empty cache
        _attention("prompt_pair", 2, 5001, 5001, 0.6, 32, 8, 128, 64, 0, 0, True),
        # the residual stream of one token
        _residual("norm_token", 1, 2560, True, "none", False, False),
        # a prefill pass, a gate for each channel, binary16 for the next products
        _residual("norm_pass", 512, 2560, True, "channel", False, True),
        # many long prompts, wide stream, a gate for each token, odd row count
        _residual("norm_prompts", 16383, 5120, True, "row", True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _within(case):
    w = work(case)
    if case["op"] != "attention":
        return w["bytes"] <= 8.0e8
    big = (case["batch"] * case["heads"] * case["tokens"] * case["kv"] <= 1.6e9
           and case["batch"] * case["kv_heads"] * case["kv"] * case["dim"] <= 5.3e8)
    return big and w["bytes"] <= 1.1e9 and w["flops"] <= 2.8e11


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "residual"])
    while True:
        if op == "append":
            dim = rng.choice([64, 96, 128, 256])
            kv_heads = rng.choice([1, 2, 4, 8])
            case = _append("", _log(rng, 1, 8191), kv_heads * rng.choice([1, 2, 3, 4, 5, 8]),
                           kv_heads, dim, rng.choice([dim, dim, dim // 2]),
                           rng.choice([16, 32, 64, 128]), rng.random() < 0.5, rng.random() < 0.3,
                           rng.random() < 0.4, _log(rng, 16, 500000))
        elif op == "attention":
            kv_heads = rng.choice([1, 2, 4, 8])
            kv = _log(rng, 1, 131071)
            tokens = rng.choice([1, 1, rng.randint(1, 8), _log(rng, 9, 5001)])
            case = _attention("", _log(rng, 1, 64), min(kv, tokens), kv,
                              rng.choice([0.0, 0.5, 0.95]),
                              kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8]), kv_heads,
                              rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128]),
                              rng.choice([0, 0, _log(rng, 1, 4096)]), rng.randint(0, 8),
                              rng.random() < 0.5)
        else:
            case = _residual("", _log(rng, 1, 16383), _log(rng, 64, 8192), rng.random() < 0.7,
                             rng.choice(["none", "row", "channel", "full"]), rng.random() < 0.4,
                             rng.random() < 0.5)
        if _within(case):
            del case["name"]
            return case


# ---- lengths and work -------------------------------------------------------
def _lengths(case):
    """(new tokens, cached length with them) of every conversation of a batch."""
    out = []
    for i in range(case["batch"]):
        f = 1.0 - case["spread"] * ((i * GOLDEN) % 1.0)
        kv = max(1, int(case["kv"] * f))
        out.append((min(kv, max(1, int(case["tokens"] * f))), kv))
    return out


def _seen(p, window, sinks):
    """Keys that the query at position p sees."""
    if window == 0 or p + 1 <= window:
        return p + 1
    return window + min(sinks, p + 1 - window)


def _first(p, window):
    """First key of the window of the query at position p."""
    return max(0, p - window + 1) if window else 0


def work(case):
    if case["op"] == "append":
        n, d, hq, hk = case["tokens"], case["dim"], case["heads"], case["kv_heads"]
        el = 2 if case["half"] else 4
        values = n * d * (hq + 2 * hk)
        return {"bytes": values * el + n * d * hq * el + 2 * n * d * hk * 2 + 12 * n + 2 * case["rot"],
                "flops": 3 * n * (hq + hk) * case["rot"]
                + (4 * n * (hq + hk) * d if case["norm"] else 0)}
    if case["op"] == "residual":
        n, d = case["rows"], case["dim"]
        gate = {"none": 0, "row": n, "channel": d, "full": n * d}[case["gate"]]
        el = (2 if case["half_in"] else 4) + 8 + (2 if case["half_out"] else 4)
        return {"bytes": n * d * el + 4 * gate + 4 * d * (2 if case["post"] else 1),
                "flops": n * d * (10 if case["post"] else 6)}
    d, w, s = case["dim"], case["window"], case["sinks"]
    keys = pairs = new = 0
    for nq, kv in _lengths(case):
        lo = _first(kv - nq, w)
        keys += kv - lo + min(s, lo)
        pairs += sum(_seen(p, w, s) for p in range(kv - nq, kv))
        new += nq
    return {"bytes": keys * case["kv_heads"] * d * 4
            + 2 * new * case["heads"] * d * (2 if case["half"] else 4),
            "flops": 4 * pairs * case["heads"] * d}


# ---- inputs -----------------------------------------------------------------
def _rand(g, *shape):
    return torch.randn(*shape, device=DEVICE, generator=g)


def _prepare_append(case, g):
    n, d, hq, hk, page = (case[k] for k in ("tokens", "dim", "heads", "kv_heads", "page"))
    dt = torch.float16 if case["half"] else torch.float32
    qkv = _rand(g, n, (hq + 2 * hk) * d).mul_(2.0).to(dt)    # one product's row: q, k, v
    q, k, v = qkv.split([hq * d, hk * d, hk * d], dim=1)
    held = (n + page - 1) // page
    pages = held + held // 2 + 1                             # others' pages among them
    cache = [_rand(g, pages, hk, page, d).to(torch.float16) for _ in range(2)]
    own_pages = torch.randperm(pages, device=DEVICE, generator=g)[:held]
    start = int(torch.randint(0, case["far"], (1,), device=DEVICE, generator=g))
    step = torch.arange(n, device=DEVICE)
    inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEVICE, dtype=torch.float64)
                      / case["rot"])
    state = {"q": q, "k": k, "v": v, "k_cache": cache[0], "v_cache": cache[1],
             "positions": (start + step).to(torch.int32),
             "slots": own_pages[step // page] * page + step % page,
             "inv_freq": inv.to(torch.float32), "interleaved": case["interleaved"],
             "q_out": torch.empty(n, hq, d, dtype=dt, device=DEVICE), "q_norm": None,
             "k_norm": None, "eps": 1e-6}
    if case["norm"]:
        state["q_norm"] = 1.0 + 0.2 * _rand(g, d)
        state["k_norm"] = 1.0 + 0.2 * _rand(g, d)
    return state


def _prepare_attention(case, g):
    d, hq, hk, page, w = (case[k] for k in ("dim", "heads", "kv_heads", "page", "window"))
    dt = torch.float16 if case["half"] else torch.float32
    lengths = _lengths(case)
    n = sum(nq for nq, _ in lengths)
    width = max((kv + page - 1) // page for _, kv in lengths)
    table = torch.full((len(lengths), width), -1, dtype=torch.int64)
    held = 0
    for i, (nq, kv) in enumerate(lengths):                   # pages out of every sight are free
        p = torch.arange((kv + page - 1) // page)
        keep = (p * page + page > _first(kv - nq, w)) | (p * page < case["sinks"])
        count = int(keep.sum())
        table[i, p[keep]] = torch.arange(held, held + count)
        held += count
    pages = held + 3
    order = torch.randperm(pages, device=DEVICE, generator=g)
    table = table.to(DEVICE)
    table = torch.where(table < 0, table, order[table.clamp(min=0)]).to(torch.int32)
    q_start = torch.zeros(len(lengths) + 1, dtype=torch.int64)
    q_start[1:] = torch.tensor([nq for nq, _ in lengths]).cumsum(0)
    return {"q": _rand(g, n, hq, d).mul_(1.5).to(dt),
            "k_cache": _rand(g, pages, hk, page, d).to(torch.float16),
            "v_cache": _rand(g, pages, hk, page, d).to(torch.float16),
            "table": table, "q_start": q_start.to(torch.int32).to(DEVICE),
            "kv_len": torch.tensor([kv for _, kv in lengths], dtype=torch.int32, device=DEVICE),
            "window": w, "sinks": case["sinks"], "scale": d ** -0.5,
            "longest": max(nq for nq, _ in lengths), "lengths": lengths,
            "y": torch.empty(n, hq, d, dtype=dt, device=DEVICE),
            "ws": torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=DEVICE)}


def _prepare_residual(case, g):
    n, d = case["rows"], case["dim"]
    shape = {"none": None, "row": (n, 1), "channel": (1, d), "full": (n, d)}[case["gate"]]
    h = _rand(g, n, d).mul_(3.0)
    return {"b": _rand(g, n, d).mul_(0.7).to(torch.float16 if case["half_in"] else torch.float32),
            "h": h, "post": 1.0 + 0.2 * _rand(g, d) if case["post"] else None,
            "pre": 1.0 + 0.2 * _rand(g, d),
            "gate": None if shape is None else torch.sigmoid(_rand(g, *shape)),
            "alpha": 0.75, "eps": 1e-6, "h_out": torch.empty_like(h),
            "y": torch.empty(n, d, dtype=torch.float16 if case["half_out"] else torch.float32,
                             device=DEVICE)}


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    make = {"append": _prepare_append, "attention": _prepare_attention,
            "residual": _prepare_residual}[case["op"]]
    return {"op": case["op"], **make(case, g)}


# ---- the plain forms --------------------------------------------------------
def _rms(x, weight, eps):
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + eps) * weight


def _rotated(x, cos, sin, interleaved):
    half = cos.shape[-1]
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        out = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = rot[..., :half], rot[..., half:]
        out = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([out, rest], dim=-1)


def _plain_append(s):
    n, hq, d = s["q_out"].shape
    page = s["k_cache"].shape[2]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = s["q"].reshape(n, hq, d).float()
    k = s["k"].reshape(n, -1, d).float()
    if s["q_norm"] is not None:
        q, k = _rms(q, s["q_norm"], s["eps"]), _rms(k, s["k_norm"], s["eps"])
    s["q_out"].copy_(_rotated(q, cos, sin, s["interleaved"]))
    at, off = s["slots"] // page, s["slots"] % page
    s["k_cache"][at, :, off] = _rotated(k, cos, sin, s["interleaved"]).to(torch.float16)
    s["v_cache"][at, :, off] = s["v"].reshape(n, -1, d).to(torch.float16)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    n, hq, d = s["q"].shape
    b, width = s["table"].shape
    _, hk, page, _ = s["k_cache"].shape
    t = s["longest"]
    at = s["table"].clamp(min=0).long()
    k = s["k_cache"][at].transpose(1, 2).reshape(b, hk, width * page, d).float()
    v = s["v_cache"][at].transpose(1, 2).reshape(b, hk, width * page, d).float()
    first, new = s["q_start"][:-1].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    step = torch.arange(t, device=DEVICE)
    rows = (first[:, None] + step).clamp(max=n - 1)                       # [b, t]
    q = s["q"][rows].float().reshape(b, t, hk, hq // hk, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(b, hk, (hq // hk) * t, d)
    key = torch.arange(width * page, device=DEVICE)
    p = (s["kv_len"].long() - new)[:, None, None] + step[:, None]         # [b, t, 1]
    seen = key <= p
    if s["window"]:
        seen &= (key > p - s["window"]) | (key < s["sinks"])
    v = torch.where(seen.any(dim=1)[:, None, :, None], v, 0.0)
    score = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(s["scale"])
    score = score.view(b, hk * (hq // hk), t, width * page)
    score.masked_fill_(~seen[:, None], -math.inf)
    score.sub_(score.amax(dim=-1, keepdim=True)).exp_()
    total = score.sum(dim=-1)                                             # [b, hq, t]
    out = torch.matmul(score.view(b, hk, (hq // hk) * t, width * page), v)
    out = out.view(b, hq, t, d) / total[..., None]
    owner = torch.repeat_interleave(torch.arange(b, device=DEVICE), new, output_size=n)
    s["y"].copy_(out[owner, :, torch.arange(n, device=DEVICE) - first[owner]])
    return s["y"]


def _plain_residual(s):
    b = s["b"].float()
    if s["post"] is not None:
        b = _rms(b, s["post"], s["eps"])
    if s["gate"] is not None:
        b = b * s["gate"]
    torch.add(s["h"], b, alpha=s["alpha"], out=s["h_out"])
    s["y"].copy_(_rms(s["h_out"], s["pre"], s["eps"]))
    return {"h": s["h_out"], "y": s["y"]}


# ---- the framework's calls --------------------------------------------------
def _own_append(s):
    import gemm_q4_amd as q4
    cache = q4.kv_cache(s["k_cache"], s["v_cache"])
    rot = q4.rotary(s["inv_freq"], interleaved=s["interleaved"], q_norm=s["q_norm"],
                    k_norm=s["k_norm"], eps=s["eps"])
    q4.kv_append(cache, rot, s["q"], s["k"], s["v"], s["positions"], s["slots"],
                 q_out=s["q_out"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attention(s):
    import gemm_q4_amd as q4
    cache = q4.kv_cache(s["k_cache"], s["v_cache"])
    return q4.attention(cache, s["q"], s["q_start"], s["kv_len"], s["table"],
                        window=s["window"], sinks=s["sinks"], scale=s["scale"], y=s["y"],
                        ws=s["ws"])


def _own_residual(s):
    import gemm_q4_amd as q4
    h, y = q4.residual_norm(s["h"], s["b"], s["pre"], post=s["post"], gate=s["gate"],
                            alpha=s["alpha"], eps=s["eps"], h_out=s["h_out"], y=s["y"])
    return {"h": h, "y": y}


def run(state):
    op = state["op"]
    if own:
        call = {"append": _own_append, "attention": _own_attention, "residual": _own_residual}[op]
    else:
        call = {"append": _plain_append, "attention": _plain_attention,
                "residual": _plain_residual}[op]
    return call(state)


# ---- the definitions in 64 bits ---------------------------------------------
def _exact_append(s):
    n, hq, d = s["q_out"].shape
    hk, page = s["k_cache"].shape[1:3]
    half = s["inv_freq"].numel()
    # a pair (a, b) as the complex number a + ib, turned by its angle
    angle = s["positions"].to(torch.float64).outer(s["inv_freq"].to(torch.float64))
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)

    def made(x, heads, weight):
        x = x.to(torch.float64).reshape(n, heads, d).clone()
        if weight is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + s["eps"]) * weight.double()
        if s["interleaved"]:
            z = torch.view_as_complex(x[..., :2 * half].reshape(n, heads, half, 2).contiguous())
            x[..., :2 * half] = torch.view_as_real(z * turn).reshape(n, heads, 2 * half)
        else:
            z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
            x[..., :half], x[..., half:2 * half] = z.real, z.imag
        return x

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    flat = [c.transpose(1, 2).reshape(-1, hk, d) for c in (k_cache, v_cache)]
    flat[0][s["slots"]] = made(s["k"], hk, s["k_norm"])
    flat[1][s["slots"]] = s["v"].to(torch.float64).reshape(n, hk, d)
    k_cache, v_cache = (f.reshape(-1, page, hk, d).transpose(1, 2).contiguous() for f in flat)
    return {"q": made(s["q"], hq, s["q_norm"]), "k_cache": k_cache, "v_cache": v_cache}


def _exact_attention(s):
    n, hq, d = s["q"].shape
    hk, page = s["k_cache"].shape[1:3]
    y = torch.empty(n, hq, d, dtype=torch.float64, device=DEVICE)
    row = 0
    for i, (new, kv) in enumerate(s["lengths"]):
        position = torch.arange(kv - new, kv, device=DEVICE).unsqueeze(1)
        key = torch.arange(kv, device=DEVICE)
        hidden = key > position
        if s["window"]:
            hidden = hidden | ((position - key >= s["window"]) & (key >= s["sinks"]))
        used = key[~hidden.all(dim=0)]                 # keys that some row sees
        hidden = hidden[:, used]
        page_of = s["table"][i].long()[used // page]
        for h in range(hq):
            c = h // (hq // hk)
            k = s["k_cache"][page_of, c, used % page].to(torch.float64)
            v = s["v_cache"][page_of, c, used % page].to(torch.float64)
            a = s["q"][row:row + new, h].to(torch.float64) @ k.T.contiguous() * s["scale"]
            a = torch.softmax(a.masked_fill(hidden, -math.inf), dim=-1)
            y[row:row + new, h] = a @ v
        row += new
    return y


def _exact_residual(s):
    def norm(x, weight):
        return weight.double() * x / x.pow(2).mean(-1, keepdim=True).add(s["eps"]).sqrt()

    b = s["b"].to(torch.float64)
    if s["post"] is not None:
        b = norm(b, s["post"])
    if s["gate"] is not None:
        b = s["gate"].double() * b
    h = s["h"].to(torch.float64) + s["alpha"] * b
    return {"h": h, "y": norm(h, s["pre"])}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention,
            "residual": _exact_residual}[s["op"]](s)
