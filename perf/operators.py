"""Measured cases of the serving attention operators: page and slot maps, the paged key/value
cache's writer, attention over whole prompts and attention of new tokens over the paged cache.

`run` computes a case either with the library's operators (`own` true) or in plain form: elementary
torch operations in binary32, rounded once at the end.  `exact` evaluates the definitions in
binary64.

Definitions.  A request's rows are its new tokens; row i of m rows over L cached keys sits at
position L - m + i and sees the keys j <= its position, with a window W > 0 only those with
j > position - W, and no key at or past L.  With s_j = scale * q.k_j over the visible keys,
out = sum_j exp(s_j) v_j / sum_j exp(s_j) and lse = log sum_j exp(s_j); a row that sees nothing
has out = 0 and lse = -inf.  Query head h reads key/value head h // (q_heads / kv_heads).
"""
import math
import random

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a handful of short questions arriving together (one of a single token): latency counts
        {"name": "prompt short", "op": "prompt", "type": "fp16", "seqs": 4, "tokens": 210, "longest": 128,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "window": 0, "mix": 1},
        # a prefill batch of a busy server: ragged prompts packed up to the token budget
        {"name": "prompt packed", "op": "prompt", "type": "bf16", "seqs": 16, "tokens": 8192, "longest": 1537,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "window": 0, "mix": 2},
        # one long document: matrix products dominate
        {"name": "prompt long", "op": "prompt", "type": "fp16", "seqs": 1, "tokens": 8192, "longest": 8192,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "window": 0, "mix": 3},
        # a small model with one key/value head for each query head and a sliding window, odd lengths
        {"name": "prompt window", "op": "prompt", "type": "bf16", "seqs": 3, "tokens": 9001, "longest": 4099,
         "q_heads": 16, "kv_heads": 16, "dim": 64, "window": 1024, "mix": 4},
        # one user's next token: the smallest decode step
        {"name": "decode one", "op": "paged", "type": "fp16", "seqs": 1, "longest": 1000, "shortest": 1000, "news": 1,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "mix": 5},
        # the decode step of a busy server: 64 requests of very different lengths
        {"name": "decode batch", "op": "paged", "type": "bf16", "seqs": 64, "longest": 8192, "shortest": 100, "news": 1,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "mix": 6},
        # a few users of long documents: the cache's bytes are everything
        {"name": "decode long", "op": "paged", "type": "fp16", "seqs": 4, "longest": 131072, "shortest": 100000,
         "news": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "mix": 7},
        # chunked prefill: two requests' next pieces of a long prompt over what is cached already
        {"name": "chunk", "op": "paged", "type": "bf16", "seqs": 2, "longest": 16411, "shortest": 9001, "news": 1000,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 32, "window": 0, "mix": 8},
        # the bookkeeping of a decode step: one token for each of 256 requests
        {"name": "maps decode", "op": "maps", "seqs": 256, "longest": 8192, "news": 1, "page": 16, "spare": 64, "mix": 9},
        # the bookkeeping of a large prefill: long ragged prompts, a quarter of a million tokens
        {"name": "maps prefill", "op": "maps", "seqs": 333, "longest": 3000, "news": 1600, "page": 16, "spare": 100,
         "mix": 10},
        # a decode step's new keys and values into the cache
        {"name": "write decode", "op": "write", "type": "bf16", "tokens": 256, "kv_heads": 8, "dim": 128, "page": 16,
         "pages": 8192, "padding": 0},
        # a prefill's keys and values into the cache, the batch padded to a captured size
        {"name": "write prefill", "op": "write", "type": "fp16", "tokens": 16384, "kv_heads": 8, "dim": 128, "page": 16,
         "pages": 4096, "padding": 100},
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


HEADS = [(32, 8), (32, 32), (16, 16), (64, 8), (28, 4), (40, 8), (8, 1), (12, 4)]


def draw(rng):
    op = rng.choice(["prompt", "prompt", "paged", "paged", "paged", "maps", "write"])
    mix = rng.randrange(1 << 30)
    kind = rng.choice(["fp16", "bf16"])
    q_heads, kv_heads = rng.choice(HEADS)
    dim = rng.choice([64, 128, 128, 128, 80, 96])
    if op == "prompt":
        longest = _between(rng, 1, 4000)
        seqs = _between(rng, 1, max(1, min(64, 8192 // longest)))
        tokens = max(longest, rng.randint(longest, longest * seqs))
        return {"op": op, "type": kind, "seqs": seqs, "tokens": tokens, "longest": longest, "q_heads": q_heads,
                "kv_heads": kv_heads, "dim": dim, "window": rng.choice([0, 0, _between(rng, 1, 2048)]), "mix": mix}
    if op == "paged":
        longest = _between(rng, 1, 131072)
        longest = min(longest, int(4.8e8 / (kv_heads * dim)))
        pairs = 1.3e11 / (q_heads * dim)   # (row, key) pairs of the padded batch that the largest case has
        news = rng.choice([1, 1, _between(rng, 2, 8), _between(rng, 9, 1024)])
        news = min(news, longest, max(1, int(pairs / longest)))
        most = min(256, pairs / (longest * news), 4.8e8 / (longest * kv_heads * dim))
        seqs = _between(rng, 1, max(1, int(most)))
        return {"op": op, "type": kind, "seqs": seqs, "longest": longest, "shortest": rng.randint(news, longest),
                "news": news, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
                "page": rng.choice([8, 16, 16, 32, 64, 128, 24]),
                "window": rng.choice([0, 0, 0, _between(rng, 1, 4096)]), "mix": mix}
    if op == "maps":
        return {"op": op, "seqs": _between(rng, 1, 1024), "longest": _between(rng, 1, 16384),
                "news": rng.choice([1, _between(rng, 2, 400)]), "page": rng.choice([8, 16, 32, 64, 24]),
                "spare": rng.randint(0, 200), "mix": mix}
    tokens = _between(rng, 1, 16384)
    page = rng.choice([8, 16, 32, 64, 24])
    return {"op": op, "type": kind, "tokens": tokens, "kv_heads": kv_heads, "dim": dim, "page": page,
            "pages": -(-tokens // page) + rng.randint(1, 500), "padding": rng.randint(0, tokens - 1)}


# ---------------------------------------------------------------- lengths of a case

def _prompt_lens(case):
    """Lengths of the packed prompts: one has the longest, the others share the rest unevenly."""
    rng = random.Random(case["mix"])
    n, rest = case["seqs"], case["tokens"] - case["longest"]
    weights = [rng.uniform(0.05, 1.0) for _ in range(n - 1)]
    lens = [min(case["longest"], int(rest * w / sum(weights))) for w in weights]
    for i in range(n - 1):   # what the rounding and the cap left over
        add = min(case["longest"] - lens[i], rest - sum(lens))
        lens[i] += add
    lens.insert(rng.randrange(n), case["longest"])
    return lens


def _paged_lens(case):
    """(new tokens, cached keys with them) of each request; some requests of a chunk have one token."""
    rng = random.Random(case["mix"])
    news, keys = [], []
    for i in range(case["seqs"]):
        m = case["news"] if i == 0 or rng.random() < 0.5 else rng.randint(max(1, case["news"] // 2), case["news"])
        if case["news"] > 8 and case["seqs"] > 2 and i > 0 and rng.random() < 0.5:
            m = 1
        length = case["longest"] if i == 0 else _between(rng, case["shortest"], case["longest"])
        news.append(m)
        keys.append(max(m, length))
    return news, keys


def _map_lens(case):
    """(cached tokens, new tokens) of each request."""
    rng = random.Random(case["mix"])
    cached, news = [], []
    for i in range(case["seqs"]):
        cached.append(rng.choice([0, rng.randint(0, case["longest"])]))
        news.append(1 if case["news"] == 1 else rng.randint(0, case["news"]))
    news[0] = max(1, news[0])
    return cached, news


def _seen(m, length, window):
    """(row, key) pairs that m new rows over `length` keys see."""
    pos = torch.arange(length - m, length, dtype=torch.float64)
    seen = pos + 1
    return float((seen if window <= 0 else seen.clamp(max=window)).sum())


def work(case):
    if case["op"] == "maps":
        cached, news = _map_lens(case)
        t, n = sum(news), case["seqs"]
        return {"bytes": 8.0 * n + 8.0 * n + 4 + 12.0 * t + 8.0 * t / case["page"], "flops": 0.0}
    row = case["kv_heads"] * case["dim"]
    if case["op"] == "write":
        used = case["tokens"] - case["padding"]
        return {"bytes": 8.0 * case["tokens"] + 8.0 * used * row, "flops": 0.0}
    if case["op"] == "prompt":
        lens = _prompt_lens(case)
        pairs = sum(_seen(m, m, case["window"]) for m in lens)
        keys, rows = sum(lens), sum(lens)
    else:
        news, lens = _paged_lens(case)
        pairs = sum(_seen(m, c, case["window"]) for m, c in zip(news, lens))
        w = case["window"]
        keys = sum(c if w <= 0 else min(c, w + m - 1) for m, c in zip(news, lens))
        rows = sum(news)
    heads = rows * case["q_heads"]
    return {"bytes": 4.0 * heads * case["dim"] + 4.0 * keys * row + 4.0 * heads,
            "flops": 4.0 * pairs * case["q_heads"] * case["dim"]}


# ---------------------------------------------------------------- inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lens):
    at = [0]
    for m in lens:
        at.append(at[-1] + m)
    return _ints(at)


def _keys_like(x):
    """Keys have a few channels that are much larger than the others."""
    x[..., 3::29] *= 4
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": dict(case)}

    def normal(*shape):
        return torch.empty(shape, dtype=TYPES[case["type"]], device="cuda").normal_(generator=gen)

    def shuffled(n):
        return torch.randperm(n, device="cuda", generator=gen).to(torch.int32)

    if case["op"] == "prompt":
        lens = _prompt_lens(case)
        t, hq, hk, d = sum(lens), case["q_heads"], case["kv_heads"], case["dim"]
        qkv = normal(t, hq + 2 * hk, d)          # the output of one fused projection, used in place
        _keys_like(qkv[:, hq:hq + hk])
        state.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], cu=_starts(lens), longest=max(lens),
                     scale=d ** -0.5, out=normal(t, hq, d), lse=torch.zeros((t, hq), device="cuda"))
    elif case["op"] == "paged":
        news, keys = _paged_lens(case)
        t, hq, hk, d, page = sum(news), case["q_heads"], case["kv_heads"], case["dim"], case["page"]
        each = [-(-c // page) for c in keys]
        used, width = sum(each), max(each)
        order = shuffled(used + 7)
        table = torch.full((len(keys), width), -1, dtype=torch.int32)
        where, at = [], 0
        for i, e in enumerate(each):
            table[i, :e] = torch.arange(at, at + e, dtype=torch.int32)
            at += e
        table = table.cuda()
        table = torch.where(table < 0, table, order[table.clamp(min=0).long()])
        state.update(q=normal(t, hq + 2 * hk, d)[:, :hq], k_cache=_keys_like(normal(used + 7, hk, page, d)),
                     v_cache=normal(used + 7, hk, page, d), table=table, cu=_starts(news), lens=_ints(keys),
                     longest=max(news), scale=d ** -0.5, out=normal(t, hq, d), lse=torch.zeros((t, hq), device="cuda"))
    elif case["op"] == "maps":
        cached, news = _map_lens(case)
        page, t = case["page"], sum(news)
        held = [-(-c // page) for c in cached]
        width = max(-(-(c + m) // page) for c, m in zip(cached, news))
        table = torch.full((len(cached), width), -1, dtype=torch.int32)
        at = 0
        for i, e in enumerate(held):
            table[i, :e] = torch.arange(at, at + e, dtype=torch.int32)
            at += e
        need = sum(-(-(c + m) // page) for c, m in zip(cached, news)) - at
        order = shuffled(at + need + case["spare"])
        table = table.cuda()
        table = torch.where(table < 0, table, order[table.clamp(min=0).long()])
        state.update(cached=_ints(cached), news=_ints(news), table=table, free=order[at:].contiguous(), tokens=t,
                     out={"cu_new": _ints([0] * (len(news) + 1)), "kv_lens": _ints([0] * len(news)),
                          "slot_map": torch.zeros(t, dtype=torch.int64, device="cuda"), "positions": _ints([0] * t),
                          "taken": _ints([0])})
    else:
        t, hk, d = case["tokens"], case["kv_heads"], case["dim"]
        kv = normal(t, 3 * hk, d)
        slots = torch.randperm(case["pages"] * case["page"], device="cuda", generator=gen)[:t]
        slots = torch.where(torch.arange(t, device="cuda") < t - case["padding"], slots, -1)
        state.update(k=kv[:, hk:2 * hk], v=kv[:, 2 * hk:], slots=slots.contiguous(),
                     k_cache=normal(case["pages"], hk, case["page"], d), v_cache=normal(case["pages"], hk, case["page"], d))
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "prompt":
        return _plain_prompt(case, state)
    if case["op"] == "paged":
        return _plain_paged(case, state)
    if case["op"] == "maps":
        return _plain_maps(case, state)
    return _plain_write(state)


def _run_own(case, s):
    import nvfp4_block_scaled_quantize_amd as nv
    if case["op"] == "prompt":
        out, lse = nv.prompt_attn(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"], window=case["window"],
                                  out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    if case["op"] == "paged":
        out, lse = nv.paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["lens"], scale=s["scale"],
                                 window=case["window"], out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    if case["op"] == "maps":
        maps = nv.page_maps(s["cached"], s["news"], s["table"], s["free"], case["page"], s["tokens"], out=s["out"])
        return {"table": s["table"], **maps}
    nv.kv_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _rows(cu, longest, tokens):
    """Token index of each (request, row) of the padded batch, and whether the row exists."""
    row = torch.arange(longest, device=cu.device)
    there = row < (cu[1:] - cu[:-1])[:, None]
    return (cu[:-1, None] + row).clamp(max=tokens - 1).long(), there


def _request_of(cu, tokens):
    """(request, row) of each token."""
    token = torch.arange(tokens, device=cu.device)
    request = torch.searchsorted(cu[1:].long(), token, right=True)
    return request, token - cu.long()[request]


def _attend(q, k, v, seen, scale):
    """q [n, m, q_heads, d], k and v [n, keys, kv_heads, d], seen [n, m, keys] -> out, lse in binary32."""
    n, m, hq, d = q.shape
    keys, hk = k.shape[1], k.shape[2]
    rows = q.float().view(n, m, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
    score = torch.matmul(rows, k.float().permute(0, 2, 3, 1).contiguous()).mul_(scale)
    score = score.view(n, hk, hq // hk, m, keys).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight.view(n, hk, -1, keys), v.float().permute(0, 2, 1, 3).contiguous())
    out = out.view(n, hk, hq // hk, m, d) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    return out.permute(0, 3, 1, 2, 4).reshape(n, m, hq, d), lse.permute(0, 3, 1, 2).reshape(n, m, hq)


def _seen_keys(pos, there, lens, keys, window):
    """[n, m, keys]: whether the row at position pos [n, m] sees each key."""
    key = torch.arange(keys, device=pos.device)
    seen = (key <= pos[..., None]) & (key < lens[:, None, None]) & there[..., None]
    return seen & (key > pos[..., None] - window) if window > 0 else seen


def _plain_prompt(case, s):
    tokens = s["q"].shape[0]
    at, there = _rows(s["cu"], s["longest"], tokens)
    lens = s["cu"][1:] - s["cu"][:-1]
    pos = torch.arange(s["longest"], device=at.device).expand(at.shape)
    seen = _seen_keys(pos, there, lens, s["longest"], case["window"])
    out, lse = _attend(s["q"][at], s["k"][at], s["v"][at], seen, s["scale"])
    request, row = _request_of(s["cu"], tokens)
    return {"out": out[request, row].to(s["q"].dtype), "lse": lse[request, row]}


def _plain_paged(case, s):
    tokens, page = s["q"].shape[0], case["page"]
    at, there = _rows(s["cu"], s["longest"], tokens)
    pos = (s["lens"] - (s["cu"][1:] - s["cu"][:-1]))[:, None] + torch.arange(s["longest"], device=at.device)
    n, width = s["table"].shape
    held = s["table"].clamp(min=0).long()
    k = s["k_cache"][held].transpose(2, 3).reshape(n, width * page, *s["k_cache"].shape[1::2])
    v = s["v_cache"][held].transpose(2, 3).reshape(n, width * page, *s["v_cache"].shape[1::2])
    v = torch.where((torch.arange(width * page, device=at.device) < s["lens"][:, None])[..., None, None], v, 0)
    seen = _seen_keys(pos, there, s["lens"], width * page, case["window"])
    out, lse = _attend(s["q"][at], k, v, seen, s["scale"])
    request, row = _request_of(s["cu"], tokens)
    return {"out": out[request, row].to(s["q"].dtype), "lse": lse[request, row]}


def _plain_maps(case, s):
    page, free, table = case["page"], s["free"], s["table"]
    width = table.shape[1]
    kv = s["cached"] + s["news"]
    held = ((s["cached"] + page - 1) // page).clamp(max=width)
    need = ((kv + page - 1) // page).clamp(max=width) - held
    cu = torch.nn.functional.pad(s["news"].cumsum(0), (1, 0)).to(torch.int32)
    first = need.cumsum(0) - need
    request, row = _request_of(cu, s["tokens"])
    pos = s["cached"][request] + row
    col = pos // page
    fresh = first[request] + col - held[request]
    taken = torch.where(fresh < len(free), free[fresh.clamp(0, len(free) - 1)], -1)
    inside = col.clamp(max=width - 1)
    got = torch.where(col < held[request], table[request, inside], torch.where(col < width, taken, -1))
    # every token of a page writes the same number
    table[request, inside] = torch.where(col < width, got, table[request, inside]).to(torch.int32)
    slot = torch.where(got >= 0, got.long() * page + pos % page, -1)
    return {"table": table, "cu_new": cu, "kv_lens": kv, "slot_map": slot, "positions": pos.to(torch.int32),
            "taken": need.sum(dtype=torch.int32)[None]}


def _plain_write(s):
    page = s["k_cache"].shape[2]
    # tokens without a slot follow those that have one: they repeat token 0
    source = torch.where(s["slots"] >= 0, torch.arange(len(s["slots"]), device="cuda"), 0)
    slot = s["slots"][source]
    s["k_cache"][slot // page, :, slot % page] = s["k"][source]
    s["v_cache"][slot // page, :, slot % page] = s["v"][source]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ---------------------------------------------------------------- binary64

def exact(case, seed):
    """Attention by its definition in binary64, one request and one key/value head at a time; the
    writer's caches through their rows (page, head, place in the page); the maps are whole numbers."""
    if case["op"] == "maps":
        return None
    s = prepare(case, seed)
    if case["op"] == "write":
        used, heads, page = case["tokens"] - case["padding"], case["kv_heads"], case["page"]
        slot = s["slots"][:used, None]
        row = (slot // page * heads + torch.arange(heads, device="cuda")) * page + slot % page
        caches = {}
        for name, new in (("k_cache", s["k"]), ("v_cache", s["v"])):
            rows = s[name].double().view(-1, case["dim"])
            rows[row.reshape(-1)] = new[:used].double().reshape(-1, case["dim"])
            caches[name] = rows.view(s[name].shape)
        return caches
    group = case["q_heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    starts = s["cu"].tolist()
    for i, (a, b) in enumerate(zip(starts, starts[1:])):
        if b == a:
            continue
        for h in range(case["kv_heads"]):
            if case["op"] == "prompt":
                k, v = s["k"][a:b, h].double(), s["v"][a:b, h].double()
            else:
                length = int(s["lens"][i])
                pages = s["table"][i, :-(-length // case["page"])].long()
                k = s["k_cache"][pages, h].reshape(-1, case["dim"])[:length].double()
                v = s["v_cache"][pages, h].reshape(-1, case["dim"])[:length].double()
            length = k.shape[0]
            back = torch.arange(length - (b - a), length, device="cuda")[:, None] - torch.arange(length, device="cuda")
            hidden = (back < 0) | (back >= case["window"]) if case["window"] > 0 else back < 0
            for g in range(h * group, (h + 1) * group):
                x = (s["q"][a:b, g].double() @ k.t()) * s["scale"]
                x[hidden] = -math.inf
                lse[a:b, g] = torch.logsumexp(x, 1)
                out[a:b, g] = torch.exp(x - lse[a:b, g, None]) @ v
    return {"out": out, "lse": lse}
