"""Cases that measure the operators between the projections and the attention: rotary positions with norms of queries and
keys for each head, their gradients, the same on the way into the 8-bit cache, and attention for a tree of drafted tokens.

Norm (where weights w are given) and rotation of one head's vector x at position p, for rotary_dim <= d:
    y = x w / sqrt(mean(x^2) + eps)
    (y_a, y_b) -> (c y_a - s y_b, s y_a + c y_b),  c = amplitude cos(p freq_i), s = amplitude sin(p freq_i)
for the pairs (a, b) = (i, i + rotary_dim / 2) in the "half" layout and (2 i, 2 i + 1) in the "interleaved" one; the
components from rotary_dim on stay y. Row n of sequence b has the position start[b] + offsets[b, n] (or start[b] + n).
Gradients: with g the gradient of y (the rotation transposed) and r = 1 / sqrt(mean(x^2) + eps),
    dw = sum g x r,   dx = r (g w - x r^2 mean(g w x)).

Appending to the cache quantises such keys, and values as they are, from 32 bits: a page holds for each key/value head
page x d e4m3 or int8 codes and one scale for the keys and one for the values, and for each page and head that new tokens reach
    a = max |x| over the new tokens of the page,  f = a / 448 (e4m3) or a / 127 (int8)
    s = f where the page holds no earlier token, else max(old scale, f)
    new codes      round(x * (1 / s)), nearest even, at most the largest code
    earlier codes  round(code * (old scale * (1 / s))) where the scale grew, else as they are

A tree of n drafted tokens stands behind a sequence's prefix: token i sees the prefix, and of the drafted ones itself and
its ancestors (its parent, that one's parent, ...; parent -1 is the prefix's last token). Its mask is bits in 32-bit words,
[n, ceil(n / 32)], its depth the number of drafted ancestors, so that a token's position is that of the first plus its depth.
"""
import math

import torch

own = False

_CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_LARGEST = {"e4m3": 448.0, "int8": 127.0}
_TYPE = {"bf16": torch.bfloat16, "fp16": torch.float16}
_EPS = 1e-6

# No case costs more than these (values of queries and keys, values written, bytes of codes, products of the attention).
_MOST_VALUES = 4 * 24 * 8192 * 128
_MOST_WRITTEN = 4 * 36 * 8192 * 128
_MOST_CACHE_BYTES = 805_306_368
_MOST_PRODUCTS = 32 * 32 * 64 * 4065 * 128


def listed():
    return [
        # a decoding step of one sequence, 12 heads of 128: the smallest call, all latency
        dict(name="rotate one token", op="rope", B=1, kv=12, group=1, n=1, d=128, rot=128, layout="half", norm=False, wide=True,
             scaling="none", start=1000, offsets=False, rows="bnhd", type="bf16"),
        # part of the head, neighbours paired, positions far beyond the trained ones; odd length
        dict(name="rotate part, far", op="rope", B=3, kv=4, group=7, n=1537, d=64, rot=32, layout="interleaved", norm=False, wide=True,
             scaling="yarn", start=900_000, offsets=True, rows="bhnd", type="fp16"),
        # the training workload's 12 heads of 128 and 8k tokens, four sequences, from the projections' layout
        dict(name="norm and rotate, 8k", op="rope", B=4, kv=12, group=1, n=8192, d=128, rot=128, layout="half", norm=True, wide=False,
             scaling="none", start=0, offsets=False, rows="bnhd", type="bf16"),
        # gradients at a short odd length under shared heads, weights in 32 bits
        dict(name="gradients, short", op="grad", B=2, kv=4, group=4, n=333, d=64, rot=64, layout="interleaved", norm=True, wide=True,
             scaling="linear", start=0, offsets=False, rows="bnhd", type="fp16"),
        # the backward of the training workload
        dict(name="gradients, 8k", op="grad", B=4, kv=12, group=1, n=8192, d=128, rot=128, layout="half", norm=True, wide=False,
             scaling="none", start=0, offsets=False, rows="bnhd", type="bf16"),
        # a server's decoding step: one token of each of 64 sequences, queries rotated on the way
        dict(name="append one token", op="append", B=64, kv=8, group=4, n=1, start=1000, ragged=True, d=128, page=64, code="e4m3",
             rot=128, layout="half", norm=True, wide=False, scaling="none", type="bf16"),
        # chunks of uneven length behind uneven prefixes, read back for their own attention in 16 bits
        dict(name="append chunks, ragged, read back", op="append", B=16, kv=16, group=0, n=1537, start=700, ragged=True, d=64, page=32,
             code="int8", rot=32, layout="interleaved", norm=False, wide=True, scaling="linear", type="fp16"),
        # four whole prompts of 8k tokens on 12 heads of 128, with their queries
        dict(name="append prompts, 8k", op="append", B=4, kv=12, group=1, n=8192, start=0, ragged=False, d=128, page=64, code="e4m3",
             rot=128, layout="half", norm=True, wide=False, scaling="none", type="bf16"),
        # a small tree behind a short chat
        dict(name="tree of 13, short", op="tree", B=1, kv=12, group=1, n=13, len=130, ragged=False, d=64, page=16, code="e4m3", type="fp16"),
        # the long-context decoding workload (8 sequences of 32k tokens, 12 heads of 128) with drafts
        dict(name="tree of 16, 32k", op="tree", B=8, kv=12, group=1, n=16, len=32768, ragged=False, d=128, page=64, code="e4m3", type="bf16"),
        # wide trees under shared heads, sequences of very different lengths
        dict(name="tree of 64, ragged, shared", op="tree", B=32, kv=8, group=4, n=64, len=4001, ragged=True, d=128, page=32, code="int8",
             type="bf16"),
        # a whole step: tree, drafted tokens into the cache, attention
        dict(name="verify 24 drafts", op="verify", B=16, kv=8, group=4, n=24, len=4096, ragged=True, d=128, page=64, code="e4m3", rot=128,
             layout="half", norm=True, wide=False, scaling="none", type="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "grad", "append", "tree", "tree", "verify"])
    c = dict(op=op, B=_log_int(rng, 1, 64), kv=_log_int(rng, 1, 16), group=rng.choice([1, 1, 2, 3, 4, 7, 8]), d=rng.choice([64, 128]),
             type=rng.choice(["bf16", "fp16"]))
    if op != "tree":
        c.update(rot=rng.choice([c["d"], c["d"], c["d"] // 2, 16, 48]), layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.5,
                 wide=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "yarn"]))
    if op in ("rope", "grad"):
        row = c["B"] * c["kv"] * (c["group"] + 1) * c["d"]
        c["n"] = _log_int(rng, 1, max(1, min(32768, _MOST_VALUES // row)))
        c.update(start=rng.choice([0, _log_int(rng, 1, 1_000_000)]), offsets=rng.random() < 0.3, rows=rng.choice(["bnhd", "bhnd"]))
        return c
    c.update(page=rng.choice([16, 32, 64, 128]), code=rng.choice(["e4m3", "int8"]) if op != "verify" else "e4m3", ragged=rng.random() < 0.5)
    if op == "append":
        c["group"] = rng.choice([0, c["group"]])
        row = c["B"] * c["kv"] * (c["group"] + 2) * c["d"]
        c["n"] = _log_int(rng, 1, max(1, min(8192, _MOST_WRITTEN // row)))
        c["start"] = rng.choice([0, _log_int(rng, 1, 1024)])
        return c
    c["n"] = rng.choice([_log_int(rng, 1, 24), _log_int(rng, 1, 64), _log_int(rng, 64, 512)])
    row, least = c["B"] * c["kv"] * c["d"], 1 if op == "tree" else 1000
    while row * c["group"] * c["n"] * (c["n"] + least) > _MOST_PRODUCTS:
        c["n"] //= 2
    most = min(32768, _MOST_CACHE_BYTES // (2 * row), _MOST_PRODUCTS // (row * c["group"] * c["n"]))
    c["len"] = _log_int(rng, least, max(least, most - c["n"]))
    return c


def _spread(count, most, ragged):
    """`count` whole numbers up to `most`: all equal, or spread evenly over the range, one of them 0 where there are four or more."""
    if not ragged:
        return [most] * count
    golden = (math.sqrt(5) - 1) / 2
    return [0 if count >= 4 and b == 1 else max(1, int(most * ((b + 1) * golden % 1.0) + 0.5)) for b in range(count)]


def _starts_counts(c):
    """Tokens that each sequence holds before the call, and that it adds."""
    if c["op"] == "append":
        ragged = c["ragged"] and c["n"] > 1
        return _spread(c["B"], c["start"], c["ragged"]), _spread(c["B"], c["n"], ragged)
    # a step that drafts and verifies follows a prompt
    return [max(s, 256 if c["op"] == "verify" else 0) for s in _spread(c["B"], c["len"], c["ragged"])], [c["n"]] * c["B"]


def _frequencies(c):
    """(freq, amplitude): radians for each position and pair, and the factor of the rotated components."""
    i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
    base = 10000.0 if c["scaling"] == "none" else 500000.0
    freq = base ** (-2.0 * i / c["rot"])
    if c["scaling"] == "linear":
        return freq / 4.0, 1.0
    if c["scaling"] == "yarn":  # factor 16 over 8192 trained positions; fast pairs as they are, slow ones interpolated
        turns = 8192 * freq / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return freq * keep + freq / 16.0 * (1.0 - keep), 0.1 * math.log(16.0) + 1.0
    return freq, 1.0


def _normal(gen, shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _quantised(x, code):
    """Codes and scales of whole pages x [pages, heads, page, d] in fp32."""
    s = x.abs().amax((2, 3)) / _LARGEST[code]
    y = (x * (1.0 / s)[..., None, None]).clamp_(-_LARGEST[code], _LARGEST[code])
    return (y if code == "e4m3" else y.round_()).to(_CODE[code]), s


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, kv, n, d, t = c["B"], c["kv"], c["n"], c["d"], _TYPE[c["type"]]
    H = kv * c["group"]
    state = {"case": c}
    # keys with a few strong channels, as learnt keys have
    strong = torch.ones(d, device="cuda")
    strong[:: d // 4] = 3.0

    def rows(heads, by=1.0):
        """[B, heads, n, d], as a projection leaves it ([B, n, heads, d] seen that way) or head by head."""
        if c.get("rows", "bnhd") == "bhnd":
            return (_normal(gen, (B, heads, n, d)) * by).to(t)
        return (_normal(gen, (B, n, heads, d)) * by).to(t).transpose(1, 2)

    if c["op"] != "tree":
        state["freq"], state["amplitude"] = _frequencies(c)
        w = torch.float32 if c["wide"] else t
        state["q_weight"] = (1.0 + 0.2 * _normal(gen, (d,))).to(w) if c["norm"] else None
        state["k_weight"] = (1.0 + 0.2 * _normal(gen, (d,))).to(w) if c["norm"] else None
    if H:
        state["q"] = rows(H)
    if c["op"] in ("rope", "grad"):
        state["k"] = rows(kv, strong)
        if c["op"] == "grad":
            state["dq"], state["dk"] = rows(H), rows(kv)
        starts = _spread(B, c["start"], True) if c["start"] else None
        state["start"] = torch.tensor(starts, dtype=torch.int32, device="cuda") if starts else None
        state["offsets"] = None
        if c["offsets"]:  # sequences packed into a row: positions begin anew now and then
            state["offsets"] = torch.randint(0, max(1, n), (B, n), generator=gen, device="cuda").sort(-1).values.to(torch.int32)
        return state

    page = c["page"]
    starts, counts = _starts_counts(c)
    lens = [s + k for s, k in zip(starts, counts)]
    held = [-(-x // page) for x in lens]
    width, pages = max(1, max(held)), sum(held) + 3
    # pages of all sequences in one random order; table entries behind a sequence's last page are not read
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.tensor([[sum(held[:b]) + j if j < held[b] else -1 for j in range(width)] for b in range(B)], device="cuda")
    state["table"] = torch.where(at >= 0, order[at.clamp(min=0)], torch.zeros_like(order[0])).contiguous()
    state["k"], state["k_scale"] = _quantised(_normal(gen, (pages, kv, page, d)) * strong, c["code"])
    state["v"], state["v_scale"] = _quantised(_normal(gen, (pages, kv, page, d)), c["code"])
    state["start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    state["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if c["op"] == "append":
        state["count"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
        if c["code"] == "int8":
            state["back"] = tuple(torch.zeros(B, kv, n, d, dtype=t, device="cuda") for _ in range(2))
    if c["op"] != "tree":
        state["new_k"], state["new_v"] = rows(kv, strong), rows(kv)
    if c["op"] != "append":
        # each drafted token behind any earlier one, or behind the prefix
        i = torch.arange(n, device="cuda")
        state["parents"] = (torch.rand((B, n), generator=gen, device="cuda") * (i + 1)).long().clamp(max=i).sub(1).to(torch.int32)
    if c["op"] == "tree":
        state["tree"], _ = _plain_tree(state["parents"])  # one for all layers of a step
    return state


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "grad": _own_grad, "append": _own_append, "tree": _own_tree, "verify": _own_verify}[op](state)
    return {"rope": _plain_rope, "grad": _plain_grad, "append": _plain_append, "tree": _plain_attend, "verify": _plain_verify}[op](state)


def _own_rope(s):
    from exact_head_attention_gb300 import exattn
    q, k = exattn.rope_forward(s["q"], s["k"], s["freq"], start=s["start"], offsets=s["offsets"], layout=s["case"]["layout"],
                               amplitude=s["amplitude"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=_EPS)
    return {"q": q, "k": k}


def _own_grad(s):
    from exact_head_attention_gb300 import exattn
    dq, dk, dqw, dkw = exattn.rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["freq"], start=s["start"], offsets=s["offsets"],
                                            layout=s["case"]["layout"], amplitude=s["amplitude"], q_weight=s["q_weight"],
                                            k_weight=s["k_weight"], eps=_EPS)
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _own_append(s, offsets=None):
    from exact_head_attention_gb300 import exattn
    cache = exattn.QuantCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"])
    q = exattn.cache_append(cache, s["new_k"], s["new_v"], s["freq"], s["start"], s.get("count"), offsets=offsets, q=s.get("q"),
                            layout=s["case"]["layout"], amplitude=s["amplitude"], q_weight=s["q_weight"] if "q" in s else None,
                            k_weight=s["k_weight"], eps=_EPS)
    if "back" in s:  # the values that the codes stand for
        exattn.cache_read(cache, s["lens"], start=s["start"], out=s["back"])
        return {"k": s["back"][0], "v": s["back"][1], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "q": q}
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "q": q}


def _own_tree(s):
    from exact_head_attention_gb300 import exattn
    cache = exattn.QuantCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"])
    o, lse = exattn.forward_cache_tree(s["q"], cache, s["lens"], s["tree"])
    return {"o": o, "lse": lse}


def _own_verify(s):
    from exact_head_attention_gb300 import exattn
    tree, depth = exattn.draft_tree(s["parents"])
    out = _own_append(s, offsets=depth)
    cache = exattn.QuantCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"])
    o, lse = exattn.forward_cache_tree(out.pop("q"), cache, s["lens"], tree)
    return dict(out, o=o, lse=lse, tree=tree, depth=depth)


def _plain_angles(s, n, offsets):
    """Cosines and sines [B or 1, 1, n, rot / 2] in 32 bits of angles in 64."""
    p = torch.arange(n, device=s["freq"].device)[None] if offsets is None else offsets.long()
    p = p if s["start"] is None else p + s["start"].long()[:, None]
    t = (p.double()[..., None] * s["freq"])[:, None]
    return (t.cos() * s["amplitude"]).float(), (t.sin() * s["amplitude"]).float()


def _plain_pairs(y, c):
    if c["layout"] == "half":
        return y[..., : c["rot"] // 2], y[..., c["rot"] // 2 : c["rot"]]
    return y[..., 0 : c["rot"] : 2], y[..., 1 : c["rot"] : 2]


def _plain_joined(a, b, y, c):
    both = torch.cat((a, b), -1) if c["layout"] == "half" else torch.stack((a, b), -1).flatten(-2)
    return both if c["rot"] == c["d"] else torch.cat((both, y[..., c["rot"] :]), -1)


def _plain_rotated(x, weight, s, cos, sin):
    """Norm and rotation in 32 bits."""
    y = x.float()
    if weight is not None:
        y = y * (y.square().mean(-1, keepdim=True) + _EPS).rsqrt() * weight.float()
    a, b = _plain_pairs(y, s["case"])
    return _plain_joined(a * cos - b * sin, a * sin + b * cos, y, s["case"])


def _plain_rope(s):
    cos, sin = _plain_angles(s, s["case"]["n"], s["offsets"])
    return {x: _plain_rotated(s[x], s[x + "_weight"], s, cos, sin).to(s[x].dtype) for x in ("q", "k")}


def _plain_grad(s):
    cos, sin = _plain_angles(s, s["case"]["n"], s["offsets"])
    dq, dqw = _plain_grad_one(s, "q", cos, sin)
    dk, dkw = _plain_grad_one(s, "k", cos, sin)
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _plain_grad_one(s, name, cos, sin):
    w, g = s[name + "_weight"], s["d" + name].float()
    a, b = _plain_pairs(g, s["case"])
    g = _plain_joined(a * cos + b * sin, b * cos - a * sin, g, s["case"])
    if w is None:
        return g.to(s[name].dtype), None
    x = s[name].float()
    r = (x.square().mean(-1, keepdim=True) + _EPS).rsqrt()
    dw = (g * (x * r)).sum((0, 1, 2))
    g = g * w.float()
    dx = r * (g - x * (r.square() * (g * x).mean(-1, keepdim=True)))
    return dx.to(s[name].dtype), dw.to(w.dtype)


def _gathered(codes, scales, table, rows):
    """Values [B, heads, rows, d] in fp32 of the first `rows` tokens in the table's pages."""
    B, W = table.shape
    _, kv, page, d = codes.shape
    x = codes[table.long()].float() * scales[table.long()][..., None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(B, kv, W * page, d)[:, :, :rows]


def _plain_append(s, offsets=None):
    c = s["case"]
    cos, sin = _plain_angles(s, c["n"], offsets)
    _plain_write(s, "k", _plain_rotated(s["new_k"], s["k_weight"], s, cos, sin))
    _plain_write(s, "v", s["new_v"].float())
    q = _plain_rotated(s["q"], s["q_weight"], s, cos, sin).to(s["q"].dtype) if "q" in s else None
    if "back" in s:
        rows = s["start"].long()[:, None] + torch.arange(c["n"], device=s["k"].device)
        new = (rows < s["lens"][:, None])[:, None, :, None]
        rows = rows.clamp(max=s["table"].shape[1] * c["page"] - 1)[:, None, :, None].expand(-1, c["kv"], -1, c["d"])
        k = _gathered(s["k"], s["k_scale"], s["table"], s["table"].shape[1] * c["page"]).gather(2, rows).to(_TYPE[c["type"]])
        v = _gathered(s["v"], s["v_scale"], s["table"], s["table"].shape[1] * c["page"]).gather(2, rows).to(_TYPE[c["type"]])
        torch.where(new, k, s["back"][0], out=s["back"][0])
        torch.where(new, v, s["back"][1], out=s["back"][1])
        return {"k": s["back"][0], "v": s["back"][1], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "q": q}
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "q": q}


def _plain_write(s, name, x):
    """Rows x [B, kv, n, d] in fp32 into the cache."""
    c, codes, scales = s["case"], s[name], s[name + "_scale"]
    B, kv, n, d = x.shape
    page, most = c["page"], _LARGEST[c["code"]]
    start = s["start"].long()
    count = s["lens"].long() - start
    first = start // page
    span = (n + page - 2) // page + 1  # pages that n tokens can reach
    j = first[:, None] + torch.arange(span, device=x.device)
    reached = (j * page < (start + count)[:, None]) & (count > 0)[:, None]
    pages = s["table"].long().gather(1, j.clamp(max=s["table"].shape[1] - 1))
    row = j[:, :, None] * page + torch.arange(page, device=x.device) - start[:, None, None]  # [B, span, page]
    new = ((row >= 0) & (row < count[:, None, None]) & reached[..., None])[:, None]
    old = ((row < 0) & reached[..., None])[:, None]
    x = x.gather(2, row.clamp(0, n - 1).reshape(B, 1, span * page, 1).expand(B, kv, span * page, d)).reshape(B, kv, span, page, d)
    x = torch.where(new[..., None], x, torch.zeros_like(x))
    f = x.abs().amax((3, 4)) * (1.0 / most)
    f = torch.where(f < 2.0 ** -126, torch.zeros_like(f), f)
    before = scales[pages].permute(0, 2, 1)  # [B, kv, span]
    scale = torch.where(old.any(-1), torch.maximum(before, f), f)
    inverse = torch.where(scale == 0, torch.zeros_like(scale), 1.0 / scale)
    grew = (scale > before) & old.any(-1)
    held = codes[pages].permute(0, 2, 1, 3, 4)
    y = torch.where(new[..., None], x * inverse[..., None, None],
                    held.float() * torch.where(grew, before * inverse, torch.ones_like(before))[..., None, None]).clamp(-most, most)
    y = (y if c["code"] == "e4m3" else y.round()).to(codes.dtype)
    as_is = ~(new[..., None] | (old & grew[..., None])[..., None])
    y = torch.where(as_is, held.view(torch.uint8), y.view(torch.uint8))
    codes.view(torch.uint8)[pages[reached]] = y.permute(0, 2, 1, 3, 4)[reached]
    scales[pages[reached]] = scale.permute(0, 2, 1)[reached]


def _plain_sees(parents):
    """Truth values [B, n, n]: token i sees drafted token j."""
    B, n = parents.shape
    j = torch.arange(n, device=parents.device)
    sees = ((parents[..., None] == j) | (j[:, None] == j)).float()
    for _ in range((n - 1).bit_length()):  # paths of twice the length
        sees = (sees @ sees).clamp(max=1.0)
    return sees > 0.5


def _plain_tree(parents):
    """The mask's words [B, n, ceil(n / 32)] and the depths [B, n]."""
    sees = _plain_sees(parents)
    B, n, _ = sees.shape
    depth = sees.sum(-1).sub(1).to(torch.int32)
    bits = torch.nn.functional.pad(sees, (0, -n % 32)).reshape(B, n, -1, 32).long()
    words = (bits << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32), depth


def _plain_attend(s):
    n = s["case"]["n"]
    sees = (s["tree"][..., None] >> torch.arange(32, device=s["tree"].device)) & 1
    return _plain_attention(s, s["q"], sees.flatten(-2)[..., :n] != 0)


def _plain_attention(s, q, sees):
    c = s["case"]
    B, H, n, d = q.shape
    rows = s["table"].shape[1] * c["page"]
    k = _gathered(s["k"], s["k_scale"], s["table"], rows)
    v = _gathered(s["v"], s["v_scale"], s["table"], rows)
    qf = q.float().reshape(B, c["kv"], c["group"] * n, d) * (1.0 / math.sqrt(d))
    scores = (qf @ k.transpose(2, 3)).reshape(B, c["kv"], c["group"], n, rows)
    j = torch.arange(rows, device=q.device) - s["start"].long()[:, None]  # drafted token of each row of the cache
    drafted = sees.gather(2, j.clamp(0, n - 1)[:, None].expand(B, n, rows)) & (j < n)[:, None]
    hidden = ~((j < 0)[:, None] | drafted)
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, c["kv"], c["group"] * n, rows) @ v).reshape(B, c["kv"], c["group"], n, d) / total
    return {"o": o.reshape(B, H, n, d).to(q.dtype), "lse": (top + total.log()).reshape(B, H, n)}


def _plain_verify(s):
    tree, depth = _plain_tree(s["parents"])
    out = _plain_append(s, depth)
    return dict(out, **_plain_attention(s, out.pop("q"), _plain_sees(s["parents"])), tree=tree, depth=depth)


def work(case):
    c = case
    B, kv, n, d = c["B"], c["kv"], c["n"], c["d"]
    H = kv * c["group"]
    size = 2  # bytes of an input's or output's value
    turning = 6 if c.get("norm") else 3  # operations a value, norm and rotation
    if c["op"] in ("rope", "grad"):
        values = B * n * (H + kv) * d
        passes = (2 if c["op"] == "rope" else 3) if c["norm"] else 2
        extra = 4 * c["rot"] + (4 * B * n if c["offsets"] else 0) + (8 * d * (4 if c["wide"] else 2) if c["norm"] else 0)
        return {"bytes": passes * values * size + extra, "flops": turning * values * (2 if c["op"] == "grad" else 1)}
    starts, counts = _starts_counts(c)
    tokens = sum(counts)
    pages = sum(-(-(s + k) // c["page"]) - s // c["page"] for s, k in zip(starts, counts) if k)
    written = 2 * tokens * kv * d * (size + 1) + 8 * pages * kv + 4 * pages + 2 * B * n * H * d * size + 12 * B
    if c["op"] == "append":
        back = 2 * tokens * kv * d * (size + 1) if c["code"] == "int8" else 0
        return {"bytes": written + back, "flops": (turning + 4) * tokens * kv * d + turning * B * n * H * d}
    lens = [s + k for s, k in zip(starts, counts)]
    held = sum(-(-x // c["page"]) for x in lens)
    # what each row sees depends on the tree: the prefix, and about the logarithm of n drafted tokens
    seen = sum(n * s + n * (1 + math.log(n)) for s in starts)
    words = 4 * B * n * -(-n // 32)
    read = 2 * sum(lens) * kv * d + 8 * held * kv + 4 * held + 2 * B * H * n * d * size + 4 * B * H * n + words + 4 * B
    if c["op"] == "tree":
        return {"bytes": read, "flops": 4 * seen * H * d}
    return {"bytes": read + written + words + 8 * B * n, "flops": 4 * seen * H * d + turning * tokens * (H + kv) * d}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "grad": _exact_grad, "append": _exact_append, "tree": _exact_tree, "verify": _exact_verify}[case["op"]](s)


def _exact_turn(s, b, n, offsets, back=False):
    """The rotation of sequence b's rows as complex numbers [n, rot / 2], conjugated for `back`."""
    first = 0 if s["start"] is None else int(s["start"][b])
    p = torch.arange(n, device="cuda") if offsets is None else offsets[b].long()
    t = (p + first).double()[:, None] * s["freq"]
    return torch.polar(torch.full_like(t, s["amplitude"]), -t if back else t)


def _exact_rotated(y, turn, c):
    """y [heads, n, d] in 64 bits."""
    y = y.clone()
    a, b = (slice(0, c["rot"] // 2), slice(c["rot"] // 2, c["rot"])) if c["layout"] == "half" else (slice(0, c["rot"], 2), slice(1, c["rot"], 2))
    z = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * turn
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_normed(x, w):
    return x if w is None else x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + _EPS) * w.double()


def _exact_one(s, name, weight, offsets):
    x = s[name]
    out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for b in range(x.shape[0]):
        turn = _exact_turn(s, b, x.shape[2], offsets)
        for h in range(x.shape[1]):
            out[b, h] = _exact_rotated(_exact_normed(x[b, h].double(), s[weight]), turn, s["case"])
    return out


def _exact_rope(s):
    return {x: _exact_one(s, x, x + "_weight", s["offsets"]) for x in ("q", "k")}


def _exact_grad(s):
    out = {}
    for name in ("q", "k"):
        x, w = s[name], s[name + "_weight"]
        dx = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(x.shape[-1], dtype=torch.float64, device="cuda")
        for b in range(x.shape[0]):
            turn = _exact_turn(s, b, x.shape[2], s["offsets"], back=True)
            for h in range(x.shape[1]):
                g = _exact_rotated(s["d" + name][b, h].double(), turn, s["case"])
                if w is not None:
                    v = x[b, h].double()
                    root = torch.sqrt((v * v).mean(-1, keepdim=True) + _EPS)
                    unit = v / root
                    dw += (g * unit).sum(0)
                    g = g * w.double()
                    g = (g - unit * (g * unit).mean(-1, keepdim=True)) / root
                dx[b, h] = g
        out["d" + name] = dx
        out["d" + name + "_weight"] = None if w is None else dw
    return out


def _nearest_e4m3(y):
    """y rounded to three bits behind the leading one (to nearest even), exponents from -6, at most 448, in 64 bits."""
    m, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (e - 4).clamp(min=-9))
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _exact_write(s, name, x):
    """Codes and scales in 64 bits after rows x [B, kv, n, d] went in."""
    c = s["case"]
    most = _LARGEST[c["code"]]
    nearest = _nearest_e4m3 if c["code"] == "e4m3" else lambda y: torch.round(y).clamp(-most, most)
    codes, scales, table = s[name].float().double(), s[name + "_scale"].double(), s["table"].tolist()
    for b, (start, count) in enumerate(zip(*_starts_counts(c))):
        t = start
        while t < start + count:
            j, inside = divmod(t, c["page"])
            take = min(c["page"] - inside, start + count - t)
            p = table[b][j]
            rows = x[b, :, t - start : t - start + take]
            f = rows.abs().amax((1, 2)) / most
            if inside:
                was = scales[p].clone()
                f = torch.maximum(was, f)
                again = nearest(codes[p, :, :inside] * (was / f)[:, None, None])
                codes[p, :, :inside] = torch.where((f > was)[:, None, None], again, codes[p, :, :inside])
            scales[p] = f
            codes[p, :, inside : inside + take] = nearest(rows / f[:, None, None])
            t += take
    return codes, scales


def _exact_append(s, offsets=None):
    c = s["case"]
    out = {"q": _exact_one(s, "q", "q_weight", offsets) if "q" in s else None}
    for name, x in (("k", _exact_one(s, "new_k", "k_weight", offsets)), ("v", s["new_v"].double())):
        codes, out[name + "_scale"] = _exact_write(s, name, x)
        if "back" in s:
            values = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
            for b, (start, count) in enumerate(zip(*_starts_counts(c))):
                if count:
                    values[b, :, :count] = _values(codes, out[name + "_scale"], s["table"], b, start + count)[:, start:]
            codes = values
        out[name] = codes
    return out


def _values(codes, scales, table, b, count):
    """The first `count` tokens of sequence b in 64 bits, [heads, count, d]."""
    ids = table[b, : -(-count // codes.shape[2])].long()
    x = codes[ids].double() * scales[ids].double()[:, :, None, None]
    return x.transpose(0, 1).reshape(codes.shape[1], -1, codes.shape[3])[:, :count]


def _exact_ancestors(parents):
    """Truth values [B, n, n] on the CPU."""
    B, n = parents.shape
    sees = torch.zeros(B, n, n, dtype=torch.bool)
    up = parents.tolist()
    for b in range(B):
        for i in range(n):
            if up[b][i] >= 0:
                sees[b, i] = sees[b, up[b][i]]
            sees[b, i, i] = True
    return sees


def _exact_attention(s, q, codes):
    c = s["case"]
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    sees = _exact_ancestors(s["parents"]).cuda()
    n, g = c["n"], c["group"]
    for b, (start, length) in enumerate(zip(s["start"].tolist(), s["lens"].tolist())):
        k = _values(codes["k"].float() if "k" in codes else s["k"].float(), codes.get("k_scale", s["k_scale"]), s["table"], b, length)
        v = _values(codes["v"].float() if "v" in codes else s["v"].float(), codes.get("v_scale", s["v_scale"]), s["table"], b, length)
        hidden = torch.cat((torch.zeros(n, start, dtype=torch.bool, device="cuda"), ~sees[b]), 1)
        for h in range(c["kv"]):
            x = torch.einsum("gnd,td->gnt", q[b, h * g : (h + 1) * g].double(), k[h]) / math.sqrt(c["d"])
            x = x.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(x, -1)
            lse[b, h * g : (h + 1) * g] = z
            o[b, h * g : (h + 1) * g] = torch.exp(x - z[..., None]) @ v[h]
    return {"o": o, "lse": lse}


def _exact_tree(s):
    return _exact_attention(s, s["q"], {})


def _exact_verify(s):
    sees = _exact_ancestors(s["parents"])
    depth = (sees.sum(-1) - 1).to(torch.int32).cuda()
    out = _exact_append(s, depth)
    return dict(out, **_exact_attention(s, out.pop("q").to(_TYPE[s["case"]["type"]]), out), tree=None, depth=None)
