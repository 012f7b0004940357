"""A decode step of drafted tokens over an 8-bit cache, as measured work.

Beside the Q4_0 products such a step runs: the lookup of its tokens' rows in
the Q4_0 table (with the first norm), the append of keys and values to a paged
cache of 8-bit codes with a scale for each row, attention over that cache, the
reading of cache rows, and the verification of the drafted tokens against the
logits from given random numbers.  Each case is one of them.  Where ``own`` is
true ``run`` calls the framework, elsewhere it computes the same in elementary
torch operations.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda:0"
WORKSPACE_BYTES = 134217728     # one buffer that serves every call of the framework
GOLDEN = 0.6180339887498949
TINY = 2.0 ** -126              # the smallest normal float32


# ---- cases ------------------------------------------------------------------
def _cache(name, tokens, heads, kv_heads, dim, rot, page, norm, interleaved, half, far):
    return {"name": name, "op": "cache", "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "rot": rot, "page": page, "norm": norm, "interleaved": interleaved,
            "half": half, "far": far}


def _attention(name, batch, tokens, kv, spread, heads, kv_heads, dim, page, window, sinks, half):
    return {"name": name, "op": "attention", "batch": batch, "tokens": tokens, "kv": kv,
            "spread": spread, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "window": window, "sinks": sinks, "half": half}


def _verify(name, batch, drafts, spread, vocab, modelled, greedy, half):
    return {"name": name, "op": "verify", "batch": batch, "drafts": drafts, "spread": spread,
            "vocab": vocab, "modelled": modelled, "greedy": greedy, "half": half}


def _embed(name, tokens, vocab, dim, norm, half):
    return {"name": name, "op": "embed", "tokens": tokens, "vocab": vocab, "dim": dim,
            "norm": norm, "half": half}


def listed():
    return [
        # one conversation's next token of a 4B-class block, written in 8 bits; its page and two
        # neighbours read back
        _cache("cache_token", 1, 32, 8, 128, 128, 16, True, False, False, 300000),
        # a prefill pass of 512 positions of the same block
        _cache("cache_pass", 512, 32, 8, 128, 128, 16, True, False, False, 4096),
        # long prompts of a model with wide heads, half of each head rotated, binary16 rows
        _cache("cache_prompt", 8191, 16, 8, 256, 128, 64, False, True, True, 32768),
        # one conversation, 448 positions of context: latency
        _attention("attend_one", 1, 1, 448, 0.0, 32, 8, 128, 16, 0, 0, False),
        # 64 conversations of every length up to 8192, each verifying up to four drafted tokens
        _attention("attend_drafts", 64, 5, 8192, 0.95, 32, 8, 128, 64, 0, 0, True),
        # one very long conversation: the key axis has to be split
        _attention("attend_long", 1, 1, 131071, 0.0, 32, 8, 128, 64, 0, 0, True),
        # two prompts of unequal length from an empty cache
        _attention("attend_prompts", 2, 5001, 5001, 0.6, 32, 8, 128, 64, 0, 0, True),
        # one conversation that drafts for itself (the drafts are picks, not draws): latency
        _verify("verify_one", 1, 4, 0.0, 151936, False, 0.0, False),
        # a small vocabulary of odd size, a few conversations, binary16 logits
        _verify("verify_odd", 12, 3, 0.7, 32003, True, 0.0, True),
        # 64 conversations with up to six tokens each from a draft model, some of them greedy
        _verify("verify_batch", 64, 6, 0.8, 151936, True, 0.2, False),
        # the tokens of one conversation's next step, one drawn and four drafted
        _embed("embed_step", 5, 151936, 2560, True, False),
        # prompts, binary16 for the first products
        _embed("embed_prompt", 8191, 151936, 2560, True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _within(case):
    w = work(case)
    if case["op"] == "attention":
        big = (case["batch"] * case["heads"] * case["tokens"] * case["kv"] <= 1.6e9
               and case["batch"] * case["kv_heads"] * case["kv"] * case["dim"] <= 5.3e8)
        return big and w["bytes"] <= 6.0e8 and w["flops"] <= 2.8e11
    return w["bytes"] <= {"cache": 2.9e8, "verify": 3.8e8, "embed": 1.5e8}[case["op"]]


def draw(rng):
    op = rng.choice(["cache", "attention", "attention", "verify", "verify", "embed"])
    while True:
        if op == "cache":
            dim = rng.choice([64, 96, 128, 256])
            kv_heads = rng.choice([1, 2, 4, 8])
            case = _cache("", _log(rng, 1, 8191), kv_heads * rng.choice([1, 2, 3, 4, 5, 8]),
                          kv_heads, dim, rng.choice([dim, dim, dim // 2]),
                          rng.choice([16, 32, 64, 128]), rng.random() < 0.5, rng.random() < 0.3,
                          rng.random() < 0.4, _log(rng, 16, 500000))
        elif op == "attention":
            kv_heads = rng.choice([1, 2, 4, 8])
            kv = _log(rng, 1, 131071)
            tokens = rng.choice([1, rng.randint(1, 8), rng.randint(1, 8), _log(rng, 9, 5001)])
            case = _attention("", _log(rng, 1, 64), min(kv, tokens), kv,
                              rng.choice([0.0, 0.5, 0.95]),
                              kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8]), kv_heads,
                              rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128]),
                              rng.choice([0, 0, _log(rng, 1, 4096)]), rng.randint(0, 8),
                              rng.random() < 0.5)
        elif op == "verify":
            case = _verify("", _log(rng, 1, 64), rng.randint(0, 8), rng.choice([0.0, 0.5, 0.9]),
                           _log(rng, 100, 200000), rng.random() < 0.6,
                           rng.choice([0.0, 0.0, 0.3, 1.0]), rng.random() < 0.3)
        else:
            case = _embed("", _log(rng, 1, 8191), _log(rng, 500, 200000),
                          32 * _log(rng, 2, 256), rng.random() < 0.7, rng.random() < 0.5)
        if _within(case):
            del case["name"]
            return case


# ---- lengths and work -------------------------------------------------------
def _share(case, i):
    return 1.0 - case["spread"] * ((i * GOLDEN) % 1.0)


def _lengths(case):
    """(new tokens, cached length with them) of every conversation of a batch."""
    out = []
    for i in range(case["batch"]):
        kv = max(1, int(case["kv"] * _share(case, i)))
        out.append((min(kv, max(1, int(case["tokens"] * _share(case, 7 * i + 3)))), kv))
    return out


def _rows(case):
    """Logit rows of every conversation: one more than it has drafts."""
    return [1 + int(round(case["drafts"] * _share(case, i))) for i in range(case["batch"])]


def _seen(p, window, sinks):
    """Keys that the query at position p sees."""
    if window == 0 or p + 1 <= window:
        return p + 1
    return window + min(sinks, p + 1 - window)


def _first(p, window):
    """First key of the window of the query at position p."""
    return max(0, p - window + 1) if window else 0


def _pages(tokens, page):
    """(pages of the tokens, pages of the cache): a few of others beside them."""
    held = (tokens + page - 1) // page
    return held, held + 2


def _groups(dim):
    """Groups of four blocks that a table's row is padded to."""
    return (dim // 32 + 3) // 4


def work(case):
    if case["op"] == "cache":
        n, d, hq, hk = case["tokens"], case["dim"], case["heads"], case["kv_heads"]
        el = 2 if case["half"] else 4
        rows = 2 * hk * _pages(n, case["page"])[1] * case["page"]         # read back
        return {"bytes": n * d * (hq + 2 * hk) * el + n * d * hq * el + 2 * n * hk * (d + 4)
                + rows * (3 * d + 4) + 12 * n + 2 * case["rot"],
                "flops": 3 * n * (hq + hk) * case["rot"] + 4 * n * hk * d + rows * d
                + (4 * n * (hq + hk) * d if case["norm"] else 0)}
    if case["op"] == "verify":
        rows, el = _rows(case), 2 if case["half"] else 4
        read = sum(rows) + (sum(rows) - len(rows) if case["modelled"] else 0)
        return {"bytes": read * case["vocab"] * el + 12 * sum(rows) + 16 * len(rows),
                "flops": 4 * read * case["vocab"]}
    if case["op"] == "embed":
        n, d = case["tokens"], case["dim"]
        return {"bytes": n * d // 32 * 18 + 4 * n + 4 * n * d
                + (n * d * (2 if case["half"] else 4) + 4 * d if case["norm"] else 0),
                "flops": n * d * (6 if case["norm"] else 2)}
    d, w, s = case["dim"], case["window"], case["sinks"]
    keys = pairs = new = 0
    for nq, kv in _lengths(case):
        lo = _first(kv - nq, w)
        keys += kv - lo + min(s, lo)
        pairs += sum(_seen(p, w, s) for p in range(kv - nq, kv))
        new += nq
    return {"bytes": keys * case["kv_heads"] * (d + 4) * 2
            + 2 * new * case["heads"] * d * (2 if case["half"] else 4),
            "flops": 4 * pairs * case["heads"] * d}


# ---- inputs -----------------------------------------------------------------
def _rand(g, *shape):
    return torch.randn(*shape, device=DEVICE, generator=g)


def _quantised(x):
    """Codes and scales of rows of x."""
    s = x.abs().amax(dim=-1) / 127.0
    s = torch.where(s < TINY, 0.0, s)
    c = torch.where((s > 0)[..., None], torch.round(x / s[..., None]), 0.0)
    return c.clamp_(-127, 127).to(torch.int8), s


def _filled(g, pages, heads, page, dim):
    """A cache of rows of several magnitudes."""
    codes = torch.empty(pages, heads, page, dim, dtype=torch.int8, device=DEVICE)
    scales = torch.empty(pages, heads, page, device=DEVICE)
    for i in range(0, pages, 256):                           # less memory on the way
        part = _rand(g, min(256, pages - i), heads, page, dim)
        part *= torch.exp(0.4 * _rand(g, *part.shape[:3], 1))
        codes[i:i + 256], scales[i:i + 256] = _quantised(part)
    return codes, scales


def _prepare_cache(case, g):
    n, d, hq, hk, page = (case[k] for k in ("tokens", "dim", "heads", "kv_heads", "page"))
    dt = torch.float16 if case["half"] else torch.float32
    qkv = _rand(g, n, (hq + 2 * hk) * d).mul_(2.0).to(dt)    # one product's row: q, k, v
    q, k, v = qkv.split([hq * d, hk * d, hk * d], dim=1)
    held, pages = _pages(n, page)
    kc, ks = _filled(g, pages, hk, page, d)
    vc, vs = _filled(g, pages, hk, page, d)
    own_pages = torch.randperm(pages, device=DEVICE, generator=g)[:held]
    start = int(torch.randint(0, case["far"], (1,), device=DEVICE, generator=g))
    step = torch.arange(n, device=DEVICE)
    inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEVICE, dtype=torch.float64)
                      / case["rot"])
    out = (pages * page, hk, d)
    state = {"q": q, "k": k, "v": v, "kc": kc, "ks": ks, "vc": vc, "vs": vs,
             "positions": (start + step).to(torch.int32),
             "slots": own_pages[step // page] * page + step % page,
             "all": torch.arange(pages * page, device=DEVICE),
             "inv_freq": inv.to(torch.float32), "interleaved": case["interleaved"],
             "q_out": torch.empty(n, hq, d, dtype=dt, device=DEVICE), "q_norm": None,
             "k_norm": None, "eps": 1e-6,
             "k_out": torch.empty(out, dtype=torch.float16, device=DEVICE),
             "v_out": torch.empty(out, dtype=torch.float16, device=DEVICE)}
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
    kc, ks = _filled(g, pages, hk, page, d)
    vc, vs = _filled(g, pages, hk, page, d)
    return {"q": _rand(g, n, hq, d).mul_(1.5).to(dt), "kc": kc, "ks": ks, "vc": vc, "vs": vs,
            "table": table, "q_start": q_start.to(torch.int32).to(DEVICE),
            "kv_len": torch.tensor([kv for _, kv in lengths], dtype=torch.int32, device=DEVICE),
            "window": w, "sinks": case["sinks"], "scale": d ** -0.5,
            "longest": max(nq for nq, _ in lengths), "lengths": lengths,
            "y": torch.empty(n, hq, d, dtype=dt, device=DEVICE),
            "ws": torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=DEVICE)}


def _prepare_verify(case, g):
    rows, vocab, batch = _rows(case), case["vocab"], case["batch"]
    n, dt = sum(rows), torch.float16 if case["half"] else torch.float32
    start = torch.zeros(batch + 1, dtype=torch.int64)
    start[1:] = torch.tensor(rows).cumsum(0)
    owner = torch.repeat_interleave(torch.arange(batch), torch.tensor(rows)).to(DEVICE)
    heat = 0.5 + 0.7 * torch.rand(batch, device=DEVICE, generator=g)
    heat = torch.where(torch.arange(batch, device=DEVICE) < case["greedy"] * batch, 0.0, heat)
    # the likely tokens of every row stand out, and the draft model knows most of them
    logits = 2.0 * _rand(g, n, vocab)
    for _ in range(3):
        at = torch.randint(0, vocab, (n, 8), device=DEVICE, generator=g)
        logits.scatter_add_(1, at, 8.0 + 2.0 * _rand(g, n, 8))
    drafted = logits + 0.7 * _rand(g, n, vocab) if case["modelled"] else logits
    logits, drafted = logits.to(dt), drafted.to(dt)
    noise = -torch.log(-torch.log(torch.rand(n, vocab, device=DEVICE, generator=g).clamp_(
        1e-9, 1.0 - 1e-7)))
    if case["modelled"]:                                     # drawn from the draft's own
        picks = (drafted.float() + noise * heat[owner][:, None]).argmax(dim=-1)
    else:                                                    # its best guess, sometimes wrong
        picks = (logits.float() + 0.3 * noise).argmax(dim=-1)
    tokens = torch.empty(n, dtype=torch.int32, device=DEVICE)
    tokens[0] = int(torch.randint(0, vocab, (1,), device=DEVICE, generator=g))
    tokens[1:] = picks[:-1]
    return {"logits": logits, "drafted": drafted if case["modelled"] else None, "tokens": tokens,
            "start": start.to(torch.int32).to(DEVICE), "heat": heat,
            "uniform": torch.rand(n, 2, device=DEVICE, generator=g), "owner": owner,
            "accepted": torch.empty(batch, dtype=torch.int32, device=DEVICE),
            "next": torch.empty(batch, dtype=torch.int32, device=DEVICE), "rows": rows,
            "ws": torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=DEVICE)}


def _prepare_embed(case, g):
    n, vocab, dim = case["tokens"], case["vocab"], case["dim"]
    tiles, groups = (vocab + 15) // 16, _groups(dim)
    # the repacked table: [tile][group][row][block] scales, [tile][group][quarter][row][block] codes
    scales = 0.001 + 0.009 * torch.rand(tiles * groups * 64, device=DEVICE, generator=g)
    codes = torch.randint(0, 256, (tiles * groups * 1024,), device=DEVICE, generator=g,
                          dtype=torch.uint8)
    packed = torch.cat([scales.to(torch.float16).view(torch.uint8), codes])
    # some tokens are far more frequent than others
    u = torch.rand(n, device=DEVICE, generator=g, dtype=torch.float64)
    tokens = torch.randperm(vocab, device=DEVICE, generator=g)[
        (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp(0, vocab - 1)]
    return {"packed": packed, "tokens": tokens.to(torch.int32), "vocab": vocab, "dim": dim,
            "scale": math.sqrt(dim), "pre": 1.0 + 0.2 * _rand(g, dim) if case["norm"] else None,
            "eps": 1e-6, "h": torch.empty(n, dim, device=DEVICE),
            "y": torch.empty(n, dim, dtype=torch.float16 if case["half"] else torch.float32,
                             device=DEVICE) if case["norm"] else None}


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    make = {"cache": _prepare_cache, "attention": _prepare_attention, "verify": _prepare_verify,
            "embed": _prepare_embed}[case["op"]]
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


def _plain_cache(s):
    n, hq, d = s["q_out"].shape
    page = s["kc"].shape[2]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = s["q"].reshape(n, hq, d).float()
    k = s["k"].reshape(n, -1, d).float()
    if s["q_norm"] is not None:
        q, k = _rms(q, s["q_norm"], s["eps"]), _rms(k, s["k_norm"], s["eps"])
    s["q_out"].copy_(_rotated(q, cos, sin, s["interleaved"]))
    at, off = s["slots"] // page, s["slots"] % page
    s["kc"][at, :, off], s["ks"][at, :, off] = _quantised(
        _rotated(k, cos, sin, s["interleaved"]))
    s["vc"][at, :, off], s["vs"][at, :, off] = _quantised(s["v"].reshape(n, -1, d).float())
    at, off = s["all"] // page, s["all"] % page
    s["k_out"].copy_(s["kc"][at, :, off].float() * s["ks"][at, :, off][..., None])
    s["v_out"].copy_(s["vc"][at, :, off].float() * s["vs"][at, :, off][..., None])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"], "k_scale": s["ks"],
            "v_scale": s["vs"]}


def _plain_attention(s):
    n, hq, d = s["q"].shape
    b, width = s["table"].shape
    _, hk, page, _ = s["kc"].shape
    t = s["longest"]
    at = s["table"].clamp(min=0).long()
    k = (s["kc"][at].float() * s["ks"][at][..., None]).transpose(1, 2)
    v = (s["vc"][at].float() * s["vs"][at][..., None]).transpose(1, 2)
    k, v = k.reshape(b, hk, width * page, d), v.reshape(b, hk, width * page, d)
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


def _lowest(mask):
    """Index of each row's first true value (the row's length without one)."""
    at = torch.arange(mask.shape[-1], device=DEVICE)
    return torch.where(mask, at, mask.shape[-1]).amin(dim=-1)


def _plain_verify(s):
    # in 64 bits: a draw lies next to a border of one of 10^5 tokens' shares
    n, vocab = s["logits"].shape
    start = s["start"].long()
    first, last = start[:-1], start[1:] - 1
    heat = s["heat"][s["owner"]].double()[:, None]
    cold = heat <= 0
    rows = torch.arange(n, device=DEVICE)
    draft = s["tokens"].long()[(rows + 1).clamp(max=n - 1)]               # judged by row t

    def weights(x):
        x = x.double()
        top = x.amax(dim=-1, keepdim=True)
        best = _lowest(x == top)
        w = torch.exp((x - top) / torch.where(cold, 1.0, heat))
        one = torch.arange(vocab, device=DEVICE) == best[:, None]
        return torch.where(cold, one.double(), w)

    p = weights(s["logits"])
    p = p / p.sum(dim=-1, keepdim=True)
    one = (torch.arange(vocab, device=DEVICE) == draft[:, None]).double()
    if s["drafted"] is None:
        q = one
    else:
        q = weights(s["drafted"])
        q = torch.where(cold, one, q / q.sum(dim=-1, keepdim=True))
    u = s["uniform"].double()
    taken = u[:, 0] * q[rows, draft] < p[rows, draft]
    taken[last] = False
    refused = torch.where(taken, n, rows)                                 # first one from t on
    after = refused.flip(0).cummin(dim=0).values.flip(0)
    row = after[first]
    p, left = p[row], (p[row] - q[row]).clamp(min=0)
    whole = (row == last)[:, None] | (left.sum(dim=-1, keepdim=True) <= 0)
    left = torch.where(whole, p, left)
    below = left.cumsum(dim=-1)
    found = (below <= u[row, 1][:, None] * below[:, -1:]).sum(dim=-1)
    s["accepted"].copy_(row - first)
    s["next"].copy_(found.clamp(max=vocab - 1))
    return {"accepted": s["accepted"], "next": s["next"]}


def _plain_embed(s):
    n, dim = s["h"].shape
    tiles, groups = (s["vocab"] + 15) // 16, _groups(dim)
    cut = tiles * groups * 128
    scales = s["packed"][:cut].view(torch.float16).view(tiles, groups, 16, 4)
    codes = s["packed"][cut:].view(tiles, groups, 4, 16, 4, 4)
    tile, row = s["tokens"].long() // 16, s["tokens"].long() % 16
    d = scales[tile, :, row].float()                                      # [n, group, block]
    c = codes[tile, :, :, row].permute(0, 1, 3, 2, 4)                     # .., quarter, byte
    c = c.reshape(n, groups, 4, 16)
    w = torch.cat([c & 15, c >> 4], dim=-1).float() - 8.0                 # [n, group, block, 32]
    w = (w * d[..., None]).reshape(n, -1)[:, :dim]
    s["h"].copy_(w * s["scale"])
    if s["pre"] is None:
        return {"h": s["h"]}
    s["y"].copy_(_rms(s["h"], s["pre"], s["eps"]))
    return {"h": s["h"], "y": s["y"]}


# ---- the framework's calls --------------------------------------------------
def _own_cache(s):
    import gemm_q4_amd as q4
    cache = q4.kv_cache8(s["kc"], s["vc"], s["ks"], s["vs"])
    rot = q4.rotary(s["inv_freq"], interleaved=s["interleaved"], q_norm=s["q_norm"],
                    k_norm=s["k_norm"], eps=s["eps"])
    q4.kv_append(cache, rot, s["q"], s["k"], s["v"], s["positions"], s["slots"],
                 q_out=s["q_out"])
    q4.kv_read(cache, s["all"], k=s["k_out"], v=s["v_out"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"], "k_scale": s["ks"],
            "v_scale": s["vs"]}


def _own_attention(s):
    import gemm_q4_amd as q4
    cache = q4.kv_cache8(s["kc"], s["vc"], s["ks"], s["vs"])
    return q4.attention(cache, s["q"], s["q_start"], s["kv_len"], s["table"],
                        window=s["window"], sinks=s["sinks"], scale=s["scale"], y=s["y"],
                        ws=s["ws"])


def _own_verify(s):
    import gemm_q4_amd as q4
    accepted, following = q4.verify(s["logits"], s["tokens"], s["start"], s["uniform"],
                                    draft_logits=s["drafted"], temperature=s["heat"],
                                    accepted=s["accepted"], following=s["next"], ws=s["ws"])
    return {"accepted": accepted, "next": following}


def _own_embed(s):
    import gemm_q4_amd as q4
    h, y = q4.embed(s["packed"], s["tokens"], s["vocab"], s["dim"], scale=s["scale"],
                    pre=s["pre"], eps=s["eps"], h=s["h"], y=s["y"])
    return {"h": h} if s["pre"] is None else {"h": h, "y": y}


def run(state):
    op = state["op"]
    if own:
        call = {"cache": _own_cache, "attention": _own_attention, "verify": _own_verify,
                "embed": _own_embed}[op]
    else:
        call = {"cache": _plain_cache, "attention": _plain_attention, "verify": _plain_verify,
                "embed": _plain_embed}[op]
    return call(state)


# ---- the definitions in 64 bits ---------------------------------------------
def _exact_cache(s):
    n, hq, d = s["q_out"].shape
    hk, page = s["kc"].shape[1:3]
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

    def held(x, codes, scales):
        """Scales and values of the whole cache, by slot, with x's rows in their places."""
        s64 = scales.double().transpose(1, 2).reshape(-1, hk)
        v64 = codes.double().transpose(1, 2).reshape(-1, hk, d) * s64[..., None]
        step = x.abs().max(dim=-1).values / 127
        s64[s["slots"]] = step
        v64[s["slots"]] = torch.round(x / step[..., None]) * step[..., None]
        return s64.reshape(-1, page, hk).transpose(1, 2).contiguous(), v64

    ks, k = held(made(s["k"], hk, s["k_norm"]), s["kc"], s["ks"])
    vs, v = held(s["v"].to(torch.float64).reshape(n, hk, d), s["vc"], s["vs"])
    return {"q": made(s["q"], hq, s["q_norm"]), "k": k, "v": v, "k_scale": ks, "v_scale": vs}


def _exact_attention(s):
    n, hq, d = s["q"].shape
    hk, page = s["kc"].shape[1:3]
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
        page_of, off = s["table"][i].long()[used // page], used % page
        for h in range(hq):
            c = h // (hq // hk)
            k = s["kc"][page_of, c, off].to(torch.float64) * s["ks"][page_of, c, off, None]
            v = s["vc"][page_of, c, off].to(torch.float64) * s["vs"][page_of, c, off, None]
            a = s["q"][row:row + new, h].to(torch.float64) @ k.T.contiguous() * s["scale"]
            a = torch.softmax(a.masked_fill(hidden, -math.inf), dim=-1)
            y[row:row + new, h] = a @ v
        row += new
    return y


def _exact_verify(s):
    accepted, following, at = [], [], 0
    vocab = s["logits"].shape[1]
    tokens, heat, u = s["tokens"].tolist(), s["heat"].tolist(), s["uniform"].double().tolist()

    def share(x, t):
        x = x.to(torch.float64)
        if t > 0:
            return torch.softmax(x / t, dim=-1)
        out = torch.zeros_like(x)
        out[int((x == x.max()).nonzero()[0, 0])] = 1.0
        return out

    for i, rows in enumerate(s["rows"]):
        count = 0
        while True:
            row = at + count
            p = share(s["logits"][row], heat[i])
            if count == rows - 1:
                break
            d = tokens[row + 1]
            q = torch.zeros(vocab, dtype=torch.float64, device=DEVICE)
            if s["drafted"] is None or not heat[i] > 0:
                q[d] = 1.0
            else:
                q = share(s["drafted"][row], heat[i])
            if u[row][0] * float(q[d]) < float(p[d]):
                count += 1
                continue
            rest = torch.relu(p - q)
            p = rest if float(rest.sum()) > 0 else p
            break
        below = torch.cumsum(p, dim=0)
        following.append(min(vocab - 1, int(torch.searchsorted(
            below, (u[row][1] * below[-1]).reshape(1), right=True))))
        accepted.append(count)
        at += rows
    return {"accepted": torch.tensor(accepted, dtype=torch.int32, device=DEVICE),
            "next": torch.tensor(following, dtype=torch.int32, device=DEVICE)}


def _exact_embed(s):
    n, dim = s["h"].shape
    tiles, groups = (s["vocab"] + 15) // 16, _groups(dim)
    i = torch.arange(dim, device=DEVICE)
    block, k = i // 32, i % 32
    tile, row = (s["tokens"].long() // 16)[:, None], (s["tokens"].long() % 16)[:, None]
    half = s["packed"][:tiles * groups * 128].view(torch.float16)
    d = half[((tile * groups + block // 4) * 16 + row) * 4 + block % 4].double()
    byte = (tiles * groups * 128 + (tile * groups + block // 4) * 1024
            + (k % 16 // 4 * 16 + row) * 16 + block % 4 * 4 + k % 4)
    code = torch.where(k < 16, s["packed"][byte] & 15, s["packed"][byte] >> 4)
    h = s["scale"] * d * (code.double() - 8.0)
    if s["pre"] is None:
        return {"h": h}
    return {"h": h, "y": s["pre"].double() * h / h.pow(2).mean(-1, keepdim=True).add(
        s["eps"]).sqrt()}


def exact(case, seed):
    s = prepare(case, seed)
    return {"cache": _exact_cache, "attention": _exact_attention, "verify": _exact_verify,
            "embed": _exact_embed}[s["op"]](s)
