"""Cases that measure the 8-bit key/value cache operators: writing tokens, reading them back, attention over the cache.

A cache holds keys and values of several sequences in pages of `page` tokens.  A page holds, for each key/value head,
page x d codes (float8 e4m3 or int8) and one fp32 scale for the keys and one for the values; the value of a code is
code * scale.  A table names the pages of each sequence in order; pages of one sequence lie anywhere in the pool.

Writing `count` new tokens of a sequence behind the `start` tokens that it holds, for each page and head they reach:
    a = max |x| over the new tokens of the page
    f = a / 448 (e4m3) or a / 127 (int8); 0 where that is below 2^-126; NaN where the page's new tokens hold a NaN or infinity
    s = f where the page holds no earlier token, else max(old scale, f)
    new codes      round(x * (1 / s)), to nearest even and at most the largest code; 0 where s is 0
    earlier codes  round(code * (old scale * (1 / s))) where the scale grew, else as they are
Reading gives code * scale, rounded to the output's type, for the tokens that a sequence holds; other rows stay as they were.
Attention is softmax(scale q k^T) v of each sequence's tokens, the queries its last positions (query i of n sees the keys up
to length - n + i), with query head h on key/value head h // group; a row that sees no key gives 0 and a log-sum-exp of -inf.
"""
import math

import torch

own = False

_CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_LARGEST = {"e4m3": 448.0, "int8": 127.0}
_TYPE = {"bf16": torch.bfloat16, "fp16": torch.float16}

# No case costs more than these (bytes of the cache's codes for attention, values written or read, and products).
_MOST_CACHE_BYTES = 805_306_368
_MOST_VALUES = 402_653_184
_MOST_PRODUCTS = 2 * 32 * 512 * 12289 * 128


def listed():
    return [
        # one new token of one short chat: the smallest call, all latency
        dict(name="attend one token, short", op="attend", B=1, kv=12, group=1, n=1, len=130, ragged=False, d=64, page=16, code="e4m3", type="fp16"),
        # the long-context decoding workload (8 sequences of 32k tokens, 12 heads of 128) with its cache in 8 bits
        dict(name="attend one token, 32k", op="attend", B=8, kv=12, group=1, n=1, len=32768, ragged=False, d=128, page=64, code="e4m3", type="bf16"),
        # a server's decoding step: 64 sequences of very different lengths, eight query heads on a key/value head, small pages
        dict(name="attend one token, ragged, shared", op="attend", B=64, kv=8, group=8, n=1, len=8191, ragged=True, d=128, page=16, code="int8", type="bf16"),
        # checking five drafted tokens at once
        dict(name="attend five tokens, ragged", op="attend", B=32, kv=4, group=4, n=5, len=4001, ragged=True, d=64, page=32, code="int8", type="fp16"),
        # the chunked workload: 64 queries a sequence over 16k cached tokens, 16 heads of 64
        dict(name="attend 64 tokens, 16k", op="attend", B=4, kv=16, group=1, n=64, len=16384, ragged=False, d=64, page=128, code="e4m3", type="fp16"),
        # a chunk of a long prompt over the part before it: the largest products
        dict(name="attend 512 tokens, shared, 12k", op="attend", B=2, kv=8, group=4, n=512, len=12289, ragged=False, d=128, page=64, code="e4m3", type="bf16"),
        # the write of a decoding step: one token of each of 64 sequences, in the middle of a page
        dict(name="write one token", op="write", B=64, kv=8, n=1, start=1000, ragged=True, d=128, page=64, code="e4m3", type="bf16"),
        # chunks of uneven length behind uneven prefixes
        dict(name="write chunks, ragged", op="write", B=16, kv=16, n=1537, start=700, ragged=True, d=64, page=32, code="int8", type="fp16"),
        # four whole prompts of 8k tokens on 12 heads of 128
        dict(name="write prompts, 8k", op="write", B=4, kv=12, n=8192, start=0, ragged=False, d=128, page=64, code="e4m3", type="bf16"),
        # a short prefix read back
        dict(name="read short prefix", op="read", B=1, kv=8, n=333, ragged=False, d=64, page=16, code="int8", type="fp16"),
        # uneven prefixes read back into padded rows
        dict(name="read prefixes, ragged", op="read", B=16, kv=8, n=4097, ragged=True, d=128, page=128, code="int8", type="bf16"),
        # long sequences read back, as before a pass with 16-bit keys and values
        dict(name="read 32k", op="read", B=4, kv=12, n=32768, ragged=False, d=128, page=64, code="e4m3", type="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "write", "read"])
    c = dict(op=op, B=_log_int(rng, 1, 64), kv=_log_int(rng, 1, 16))
    if op == "attend":
        c.update(group=rng.choice([1, 1, 2, 3, 4, 7, 8]), n=rng.choice([1, 1, _log_int(rng, 2, 8), _log_int(rng, 9, 64), _log_int(rng, 65, 512)]))
    c.update(d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), code=rng.choice(["e4m3", "int8"]),
             type=rng.choice(["bf16", "fp16"]), ragged=rng.random() < 0.5)
    row = c["B"] * c["kv"] * c["d"]
    if op == "attend":
        most = min(32768, _MOST_CACHE_BYTES // (2 * row), _MOST_PRODUCTS // (row * c["group"] * c["n"]))
        c["len"] = _log_int(rng, 1, max(1, most))
    else:
        c["n"] = _log_int(rng, 1, max(1, min(32768, _MOST_VALUES // (2 * row))))
        if op == "write":
            c["n"] = min(c["n"], 8192)
            c["start"] = rng.choice([0, _log_int(rng, 1, 1024)])
    return c


def _spread(count, most, ragged):
    """`count` whole numbers up to `most`: all equal, or spread evenly over the range, one of them 0 where there are four or more."""
    if not ragged:
        return [most] * count
    golden = (math.sqrt(5) - 1) / 2
    return [0 if count >= 4 and b == 1 else max(1, int(most * ((b + 1) * golden % 1.0) + 0.5)) for b in range(count)]


def _starts_counts(c):
    """Tokens that each sequence of a write or read case holds before it, and that it adds or gives."""
    counts = _spread(c["B"], c["n"], c["ragged"])
    starts = [0] * c["B"]
    if c["op"] == "write":
        counts = [c["n"]] * c["B"] if c["n"] == 1 else counts
        starts = _spread(c["B"], c["start"], c["ragged"])
    return starts, counts


def _lengths(c):
    if c["op"] == "attend":
        return _spread(c["B"], c["len"], c["ragged"])
    return [s + n for s, n in zip(*_starts_counts(c))]


def _normal(gen, shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _quantised(x, code):
    """Codes and scales of whole pages x [pages, heads, page, d] in fp32."""
    s = x.abs().amax((2, 3)) / _LARGEST[code]
    y = x * (1.0 / s)[..., None, None]
    y = y.clamp_(-_LARGEST[code], _LARGEST[code])
    return (y if code == "e4m3" else y.round_()).to(_CODE[code]), s


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, kv, d, page = c["B"], c["kv"], c["d"], c["page"]
    lens = _lengths(c)
    held = [-(-n // page) for n in lens]
    width = max(1, max(held), -(-c["n"] // page) if c["op"] == "read" else 0)
    pages = sum(held) + 3
    state = {"case": c}
    # pages of all sequences in one random order; table entries behind a sequence's last page are not read
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    at = torch.tensor([[sum(held[:b]) + j if j < held[b] else -1 for j in range(width)] for b in range(B)], device="cuda")
    table = torch.where(at >= 0, order[at.clamp(min=0)], table).contiguous()
    # keys with a few strong channels, as learnt keys have; values without
    strong = torch.ones(d, device="cuda")
    strong[:: d // 4] = 3.0
    k, ks = _quantised(_normal(gen, (pages, kv, page, d)) * strong, c["code"])
    v, vs = _quantised(_normal(gen, (pages, kv, page, d)), c["code"])
    state.update(k=k, v=v, k_scale=ks, v_scale=vs, table=table)
    t = _TYPE[c["type"]]
    if c["op"] == "attend":
        state["q"] = _normal(gen, (B, kv * c["group"], c["n"], d)).to(t)
        state["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    else:
        starts, counts = _starts_counts(c)
        if c["op"] == "write":
            # new keys and values as a projection leaves them: [B, n, heads, d] seen as [B, heads, n, d]
            state["new_k"] = (_normal(gen, (B, c["n"], kv, d)) * strong).to(t).transpose(1, 2)
            state["new_v"] = _normal(gen, (B, c["n"], kv, d)).to(t).transpose(1, 2)
            state["start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
            state["count"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
        else:
            state["lens"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
            state["out_k"] = torch.zeros(B, kv, c["n"], d, dtype=t, device="cuda")
            state["out_v"] = torch.zeros(B, kv, c["n"], d, dtype=t, device="cuda")
    return state


def run(state):
    if own:
        return _run_own(state)
    return {"attend": _plain_attend, "write": _plain_write, "read": _plain_read}[state["case"]["op"]](state)


def _run_own(s):
    from exact_head_attention_gb300 import exattn
    op = s["case"]["op"]
    cache = exattn.QuantCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"])
    if op == "attend":
        o, lse = exattn.forward_cache(s["q"], cache, s["lens"], causal="bottom_right")
        return {"o": o, "lse": lse}
    if op == "write":
        exattn.cache_write(cache, s["new_k"], s["new_v"], s["start"], s["count"])
        return {n: s[n] for n in ("k", "v", "k_scale", "v_scale")}
    exattn.cache_read(cache, s["lens"], out=(s["out_k"], s["out_v"]))
    return {"k": s["out_k"], "v": s["out_v"]}


def _gathered(codes, scales, table, rows):
    """Values [B, heads, rows, d] in fp32 of the first `rows` tokens in the table's pages."""
    B, W = table.shape
    _, kv, page, d = codes.shape
    x = codes[table.long()].float() * scales[table.long()][..., None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(B, kv, W * page, d)[:, :, :rows]


def _plain_attend(s):
    q, c = s["q"], s["case"]
    B, H, n, d = q.shape
    rows = s["table"].shape[1] * c["page"]
    k = _gathered(s["k"], s["k_scale"], s["table"], rows)
    v = _gathered(s["v"], s["v_scale"], s["table"], rows)
    qf = q.float().reshape(B, c["kv"], c["group"] * n, d) * (1.0 / math.sqrt(d))
    scores = (qf @ k.transpose(2, 3)).reshape(B, c["kv"], c["group"], n, rows)
    last = s["lens"].long()[:, None] - n + torch.arange(n, device=q.device)  # the last key that each query sees
    hidden = torch.arange(rows, device=q.device) > last[..., None]
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, c["kv"], c["group"] * n, rows) @ v).reshape(B, c["kv"], c["group"], n, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = top + total.log()
    return {"o": o.reshape(B, H, n, d).to(q.dtype), "lse": lse.reshape(B, H, n)}


def _plain_write(s):
    _plain_write_one(s, "k")
    _plain_write_one(s, "v")
    return {n: s[n] for n in ("k", "v", "k_scale", "v_scale")}


def _plain_write_one(s, name):
    c, x, codes, scales = s["case"], s["new_" + name], s[name], s[name + "_scale"]
    B, kv, n, d = x.shape
    page, most = c["page"], _LARGEST[c["code"]]
    start, count = s["start"].long(), s["count"].long()
    first = start // page
    span = (n + page - 2) // page + 1  # pages that n tokens can reach
    j = first[:, None] + torch.arange(span, device=x.device)
    reached = (j * page < (start + count)[:, None]) & (count > 0)[:, None]
    pages = s["table"].long().gather(1, j.clamp(max=s["table"].shape[1] - 1))
    token = j[:, :, None] * page + torch.arange(page, device=x.device)  # [B, span, page]
    row = token - start[:, None, None]
    new = (row >= 0) & (row < count[:, None, None]) & reached[..., None]
    old = (row < 0) & reached[..., None]
    xf = x.float().gather(2, row.clamp(0, n - 1).reshape(B, 1, span * page, 1).expand(B, kv, span * page, d))
    xf = xf.reshape(B, kv, span, page, d) * 1.0
    xf = torch.where(new[:, None, ..., None], xf, torch.zeros_like(xf))
    f = xf.abs().amax((3, 4)) / most
    f = torch.where(f < 2.0 ** -126, torch.zeros_like(f), f)
    f = torch.where(f == math.inf, torch.full_like(f, math.nan), f)
    before = scales[pages].permute(0, 2, 1)  # [B, kv, span]
    scale = torch.where(old.any(-1)[:, None], torch.maximum(before, f), f)
    inverse = torch.where(scale == 0, torch.zeros_like(scale), 1.0 / scale)
    grew = (scale > before) & old.any(-1)[:, None]
    held = codes[pages].permute(0, 2, 1, 3, 4)
    y = torch.where(new[:, None, ..., None], xf * inverse[..., None, None],
                    held.float() * torch.where(grew, before * inverse, torch.ones_like(before))[..., None, None])
    y = y.clamp(-most, most)
    y = (y if c["code"] == "e4m3" else y.round()).to(codes.dtype)
    as_is = ~(new[:, None, ..., None] | (old[:, None, ..., None] & grew[..., None, None]))
    y = torch.where(as_is, held.view(torch.uint8), y.view(torch.uint8))
    codes.view(torch.uint8)[pages[reached]] = y.permute(0, 2, 1, 3, 4)[reached]
    scales[pages[reached]] = scale.permute(0, 2, 1)[reached]


def _plain_read(s):
    t = s["out_k"].dtype
    n = s["out_k"].shape[2]
    held = (torch.arange(n, device=s["out_k"].device) < s["lens"][:, None])[:, None, :, None]
    for_k = _gathered(s["k"], s["k_scale"], s["table"], n).to(t)
    torch.where(held, for_k, s["out_k"], out=s["out_k"])
    for_v = _gathered(s["v"], s["v_scale"], s["table"], n).to(t)
    torch.where(held, for_v, s["out_v"], out=s["out_v"])
    return {"k": s["out_k"], "v": s["out_v"]}


def work(case):
    c = case
    size = 2  # bytes of an input's or output's value
    if c["op"] == "attend":
        H, tokens = c["kv"] * c["group"], sum(_lengths(c))
        pages = sum(-(-n // c["page"]) for n in _lengths(c))
        seen = sum(sum(max(0, n - c["n"] + i + 1) for i in range(c["n"])) for n in _lengths(c))
        rows = c["B"] * H * c["n"]
        return {"bytes": 2 * tokens * c["kv"] * c["d"] + 8 * pages * c["kv"] + 4 * pages + 2 * rows * c["d"] * size + 4 * rows + 4 * c["B"],
                "flops": 4 * seen * H * c["d"]}
    starts, counts = _starts_counts(c)
    tokens = sum(counts)
    pages = sum(-(-(s + n) // c["page"]) - s // c["page"] for s, n in zip(starts, counts))
    return {"bytes": 2 * tokens * c["kv"] * c["d"] * (size + 1) + 8 * pages * c["kv"] + 4 * pages + 8 * c["B"], "flops": 4 * tokens * c["kv"] * c["d"]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "write": _exact_write, "read": _exact_read}[case["op"]](s)


def _tokens_of(s, name, b, count):
    """Values of the first `count` tokens of sequence b in 64 bits, [heads, count, d]."""
    page, d = s["case"]["page"], s["case"]["d"]
    ids = s["table"][b, : -(-count // page)].long()
    x = s[name][ids].float().double() * s[name + "_scale"][ids].double()[:, :, None, None]
    return x.transpose(0, 1).reshape(s["case"]["kv"], -1, d)[:, :count]


def _exact_attend(s):
    c, q = s["case"], s["q"]
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    n, g = c["n"], c["group"]
    for b, length in enumerate(s["lens"].tolist()):
        blind = max(0, n - length)  # queries before the first token
        if blind >= n:
            continue
        k, v = _tokens_of(s, "k", b, length), _tokens_of(s, "v", b, length)
        ahead = torch.ones(n - blind, length, dtype=torch.bool, device="cuda").triu(length - (n - blind) + 1)
        for h in range(c["kv"]):
            x = torch.einsum("gnd,td->gnt", q[b, h * g : (h + 1) * g, blind:].double(), k[h]) / math.sqrt(c["d"])
            x = x.masked_fill(ahead, -math.inf)
            z = torch.logsumexp(x, -1)
            lse[b, h * g : (h + 1) * g, blind:] = z
            o[b, h * g : (h + 1) * g, blind:] = torch.exp(x - z[..., None]) @ v[h]
    return {"o": o, "lse": lse}


def _nearest_e4m3(y):
    """y rounded to three bits behind the leading one (to nearest even), exponents from -6, at most 448, in 64 bits."""
    m, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (e - 4).clamp(min=-9))
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _exact_write(s):
    c = s["case"]
    out = {}
    for name in ("k", "v"):
        codes, scales = s[name].float().double(), s[name + "_scale"].double()
        for b, (start, count) in enumerate(zip(s["start"].tolist(), s["count"].tolist())):
            t = start
            while t < start + count:
                j, inside = divmod(t, c["page"])
                take = min(c["page"] - inside, start + count - t)
                p = int(s["table"][b, j])
                x = s["new_" + name][b, :, t - start : t - start + take].double()
                f = x.abs().amax((1, 2)) / _LARGEST[c["code"]]
                if inside:
                    was = scales[p].clone()
                    f = torch.maximum(was, f)
                    again = _nearest_e4m3(codes[p, :, :inside] * (was / f)[:, None, None])
                    codes[p, :, :inside] = torch.where((f > was)[:, None, None], again, codes[p, :, :inside])
                scales[p] = f
                codes[p, :, inside : inside + take] = _nearest_e4m3(x / f[:, None, None])
                t += take
        # whole codes have one right value each in 32 bits: there is nothing nearer to say
        out[name] = codes if c["code"] == "e4m3" else None
        out[name + "_scale"] = scales
    return out


def _exact_read(s):
    c = s["case"]
    out = {name: torch.zeros(s["out_k"].shape, dtype=torch.float64, device="cuda") for name in ("k", "v")}
    for b, length in enumerate(s["lens"].tolist()):
        if length:
            for name in ("k", "v"):
                out[name][b, :, :length] = _tokens_of(s, name, b, length)
    return out
