"""Appending to the 8-bit cache with norms and rotary positions on the way, on the GPU.

Keys are compared with the definition in 64 bits (plain_rope), values with the write's own rule, which must be followed to
the bit; queries must be rope_forward's bits, and without norm and rotation the whole must be cache_write's.  Tolerances:
  rotated keys  the norm's error as in test_gpu_rope.py, 1.04e-6; angles of rows in order are the product of two, each sine
                and cosine within 1e-7 and its angle within 2^-25.3, and three roundings: 4.2e-7, and 2.4e-7 for the
                amplitude, the products and the sum: together under 2^-19 of the size that plain_rope gives, in fp32
  scale         that of the largest key, over the largest code, and two roundings: 2^-19 of the largest size and 2^-23 of it
  codes         half a code's step: relative 2^-4 for e4m3 from 2^-6 of a scale on, 2^-10 of a scale below; half a scale for
                int8; to the key's own error and that of the scale (2^-22 of the value for the reciprocal and the product)
"""
import math

import pytest
import torch

import plain_rope
from exact_head_attention_gb300 import exattn
from test_gpu_cache import DEV, LARGEST, TYPES, make_cache, plain_write, tokens
from test_gpu_rope import LARGE

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


def _on(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def code_step(y, s, code):
    """Half a step of the code nearest y at scale s."""
    if code == "int8":
        return 0.5 * s.expand_as(y)
    return torch.maximum(y.abs() * 2.0 ** -4, 2.0 ** -10 * s)


def check_keys(cache, before, table, y, size, starts, counts, code):
    """The cache's keys after rows y [B, heads, N, d] (64 bits, their errors counted in `size`) were appended to `before`."""
    page, B = cache.k.shape[2], y.shape[0]
    after = {"k": cache.k.cpu(), "k_scale": cache.k_scale.cpu()}
    touched = torch.zeros(cache.k.shape[0], dtype=torch.bool)
    for b in range(B):
        start, count = starts[b], counts[b]
        for j in range(start // page, -(-(start + count) // page) if count else 0):
            p = int(table[b, j])
            touched[p] = True
            lo, hi = max(start, j * page), min(start + count, (j + 1) * page)
            rows, sizes = y[b, :, lo - start : hi - start], size[b, :, lo - start : hi - start]
            inside = lo - j * page
            was, s = before["k_scale"][p].double(), after["k_scale"][p].double()
            a = rows.abs().amax((1, 2)) / LARGEST[code]
            want = torch.maximum(was, a) if inside else a
            err = (2.0 ** -19 + 2.0 ** -22) * sizes.amax((1, 2)) / LARGEST[code]
            assert torch.all((s - want).abs() <= err), ((s - want) / err).abs().max()
            codes = after["k"][p].view(cache.k.dtype).float().double()
            got = codes[:, inside : inside + hi - lo] * s[:, None, None]
            tol = code_step(rows, s[:, None, None], code) * (1 + 2.0 ** -18) + 2.0 ** -18 * sizes
            assert torch.all((got - rows).abs() <= tol), ((got - rows).abs() / tol).max()
            # the scale is the new tokens' largest value: rounding may not saturate by more than its own error
            held, old = codes[:, :inside], before["k"][p].float().double()[:, :inside]
            grew = s > was
            assert torch.equal(held[~grew], old[~grew])
            if inside and grew.any():
                value = old[grew] * was[grew, None, None]
                tol = code_step(value, s[grew, None, None], code) * (1 + 2.0 ** -20)
                assert torch.all((held[grew] * s[grew, None, None] - value).abs() <= tol)
            rest = slice(inside + hi - lo, page)
            assert torch.equal(after["k"].view(torch.uint8)[p, :, rest], before["k"].view(torch.uint8)[p, :, rest])
    assert torch.equal(after["k"].view(torch.uint8)[~touched], before["k"].view(torch.uint8)[~touched])
    assert torch.equal(after["k_scale"][~touched], before["k_scale"][~touched])


def run_append(B, heads, H, N, page, d, code, dtype, starts, counts, rot, layout, norm, wide, seed=0, amplitude=1.0, offsets=None, width=None,
               position_start=None):
    t = TYPES[dtype]
    width = width or -(-(max(starts) + N) // page) + 1
    cache, host, table = make_cache(B, heads, page, d, width, code, seed=seed + 20)
    g = torch.Generator().manual_seed(seed + 21)
    k = (torch.randn((B, N, heads, d), generator=g) * torch.rand((B, N, 1, 1), generator=g) * 8).to(t).transpose(1, 2)
    v = (torch.randn((B, N, heads, d), generator=g) * 0.01).to(t).transpose(1, 2)
    q = torch.randn((B, N, H, d), generator=g).to(t).transpose(1, 2) if H else None
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(torch.float32 if wide else t) if norm else None for _ in range(2))
    wq = wq if H else None
    freq = exattn.rope_frequencies(rot, device="cpu")[0] if rot else None
    before = {n: host[n].clone() for n in ("k", "k_scale")}
    st, ct = _i32(starts), _i32(counts)
    kw = dict(layout=layout, amplitude=amplitude)
    gq, gk, gv, gf, gst, gct, gof, gwq, gwk, gps = _on(q, k, v, freq, st, ct, offsets, wq, wk, position_start)
    out = exattn.cache_append(cache, gk, gv, gf, gst, gct, gof, q=gq, q_weight=gwq, k_weight=gwk, position_start=gps, **kw)
    assert exattn.check_device_error() == 0
    begin = st if position_start is None else position_start
    y, size = plain_rope.norm_rotate(k, freq, plain_rope.positions(B, N, begin, offsets), layout, amplitude, wk)
    check_keys(cache, before, table, y, size, starts, counts, code)
    plain_write(host, table, "v", v, starts, counts, code)
    assert torch.equal(cache.v.view(torch.uint8).cpu(), host["v"].view(torch.uint8))
    assert torch.equal(cache.v_scale.cpu(), host["v_scale"])
    if H:
        want, _ = exattn.rope_forward(gq, None, gf, gst if gps is None else gps, gof, q_weight=gwq, **kw)
        assert torch.equal(out, want)
    else:
        assert out is None


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_pages(d, page, code, dtype):
    """Starts and ends inside pages and on them, single tokens, nothing at all."""
    run_append(7, 2, 3, 150, page, d, code, dtype, [0, 5, page, page + 1, 2 * page - 1, 3, 0], [150, 1, page, 2, 1, 0, 1], d, "half",
               True, page == 32)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (64, 64), (128, 48), (128, 128)])
def test_layouts(d, rot, norm, layout):
    offsets = torch.randint(0, 9000, (3, 40), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    run_append(3, 3, 5, 40, 32, d, "e4m3", "bf16", [0, 31, 70], [40, 40, 7], rot, layout, norm, True, seed=3, amplitude=1.2, offsets=offsets)


@pytest.mark.parametrize("B,heads,H,N", [(1, 1, 0, 1), (1, 1, 1, 1), (64, 8, 32, 1), (2, 5, 0, 777), (1, 2, 70, 300), (300, 1, 2, 5)], ids=str)
def test_sizes(B, heads, H, N):
    starts = [(37 * b) % 130 for b in range(B)]
    run_append(B, heads, H, N, 64, 128, "int8", "bf16", starts, [N] * B, 128, "half", True, False, seed=5)


def test_positions_apart_from_places():
    run_append(3, 2, 2, 20, 16, 64, "int8", "fp16", [4, 0, 17], [20, 20, 20], 64, "half", False, False, seed=6,
               position_start=_i32([100_000, -5, 0]), offsets=_i32([(7 * i) % 11 for i in range(20)]))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_without_norm_and_rotation_it_is_the_write(code):
    starts, counts = [0, 9, 33, 16], [50, 3, 50, 0]
    a, host, table = make_cache(4, 2, 32, 64, 4, code, seed=31)
    b, _, _ = make_cache(4, 2, 32, 64, 4, code, seed=31)
    k, v = (torch.randn((4, 2, 50, 64), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).to(DEV) for i in (1, 2))
    assert exattn.cache_append(a, k, v, None, *_on(_i32(starts), _i32(counts))) is None
    exattn.cache_write(b, k, v, *_on(_i32(starts), _i32(counts)))
    for n in ("k", "v"):
        assert torch.equal(getattr(a, n).view(torch.uint8), getattr(b, n).view(torch.uint8))
        assert torch.equal(getattr(a, n + "_scale"), getattr(b, n + "_scale"))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_one_by_one(code):
    """Growing tokens, each rounding the earlier codes of its page again."""
    cache, host, table = make_cache(2, 1, 16, 64, 3, code, seed=32)
    g = torch.Generator().manual_seed(33)
    freq = exattn.rope_frequencies(64, device="cpu")[0]
    for t in range(20):
        before = {"k": cache.k.cpu(), "k_scale": cache.k_scale.cpu()}
        k = torch.randn((2, 1, 1, 64), generator=g).mul(1.3 ** t).to(torch.float16)
        starts = [t, t + 20]
        exattn.cache_append(cache, *_on(k, k, freq, _i32(starts)))
        y, size = plain_rope.norm_rotate(k, freq, _i32(starts)[:, None].long())
        check_keys(cache, before, table, y, size, starts, [1, 1], code)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_special_values(code):
    """A NaN or infinity makes the page's scale NaN, values too small for a scale make it zero; values stay apart from keys."""
    rows = [0.0, 1e-38, 3e38, math.nan, math.inf, -math.inf]
    B = len(rows)
    cache, host, table = make_cache(B, 1, 16, 64, 2, code, seed=34)
    k = torch.zeros((B, 1, 3, 64))
    k[:, 0, 1, 7] = torch.tensor(rows)
    k = k.to(torch.bfloat16)
    freq = exattn.rope_frequencies(64)[0]
    v = torch.ones_like(k)
    exattn.cache_append(cache, k.to(DEV), v.to(DEV), freq)
    s = cache.k_scale[table[:, 0].long().to(DEV), 0].cpu()
    assert s[0] == 0 and s[1] == 0 and torch.isfinite(s[2]) and s[2] > 0 and torch.isnan(s[3:]).all()
    codes = cache.k.view(torch.uint8)[table[:, 0].long().to(DEV), 0, :3].cpu()
    assert torch.all(codes[[0, 1, 3, 4, 5]] == 0)
    plain_write(host, table, "v", v, [0] * B, [3] * B, code)
    assert torch.equal(cache.v.view(torch.uint8).cpu(), host["v"].view(torch.uint8)) and torch.equal(cache.v_scale.cpu(), host["v_scale"])


def test_what_is_out_of_range():
    """A negative start, one past the table, a page that is none, counts past N: reported, and only what is in range written."""
    cache, host, table = make_cache(4, 2, 16, 64, 3, "int8", seed=35)
    broken = cache.page_table.clone()
    broken[3, 1] = cache.k.shape[0]
    bad = exattn.QuantCache(cache.k, cache.v, cache.k_scale, cache.v_scale, broken)
    before = {"k": cache.k.cpu(), "k_scale": cache.k_scale.cpu()}
    k = torch.randn((4, 2, 20, 64), generator=torch.Generator().manual_seed(1)).to(torch.float16)
    freq = exattn.rope_frequencies(64, device="cpu")[0]
    q = torch.randn((4, 3, 20, 64), generator=torch.Generator().manual_seed(2)).to(torch.float16)
    starts = _i32([-1, 40, 0, 10])
    out = exattn.cache_append(bad, *_on(k, k, freq, starts, _i32([20, 20, 21, 20])), q=q.to(DEV))
    assert exattn.check_device_error() == 8
    y, size = plain_rope.norm_rotate(k, freq, plain_rope.positions(4, 20, starts))
    check_keys(cache, before, table, y, size, [0, 40, 0, 10], [0, 8, 20, 6], "int8")
    assert torch.equal(out, exattn.rope_forward(*_on(q, None, freq, starts))[0])


def test_queries_in_place_and_joint_views():
    """Queries, keys and values of one joint projection, the queries turned where they are."""
    B, N, heads, H, d = 3, 9, 2, 4, 64
    cache, host, table = make_cache(B, heads, 16, d, 2, "e4m3", seed=36)
    other, _, _ = make_cache(B, heads, 16, d, 2, "e4m3", seed=36)
    joint = torch.randn((B, N, H + 2 * heads, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    freq, start = exattn.rope_frequencies(d)[0], _i32([0, 3, 7]).to(DEV)
    w = torch.linspace(0.5, 1.5, d, device=DEV)
    q, k, v = (joint[:, :, a:b].transpose(1, 2) for a, b in ((0, H), (H, H + heads), (H + heads, H + 2 * heads)))
    want = exattn.cache_append(other, k.contiguous(), v.contiguous(), freq, start, q=q.contiguous(), q_weight=w, k_weight=w)
    rest = joint[:, :, H:].clone()
    got = exattn.cache_append(cache, k, v, freq, start, q=q, q_weight=w, k_weight=w, out=q)
    assert got is q and torch.equal(q, want) and torch.equal(joint[:, :, H:], rest)
    for n in ("k", "v"):
        assert torch.equal(getattr(cache, n).view(torch.uint8), getattr(other, n).view(torch.uint8))


def test_append_and_attend_in_a_graph():
    """Decoding steps replayed: append at a start that moves on, attend over all that is there."""
    B, heads, H, d, page = 2, 2, 4, 64, 16
    cache, host, table = make_cache(B, heads, page, d, 4, "e4m3", seed=37)
    eager, _, _ = make_cache(B, heads, page, d, 4, "e4m3", seed=37)
    g = torch.Generator().manual_seed(4)
    steps = [[torch.randn((B, h, 1, d), generator=g).to(torch.bfloat16).to(DEV) for h in (H, heads, heads)] for _ in range(5)]
    freq = exattn.rope_frequencies(d)[0]
    q, k, v = (torch.zeros_like(x) for x in steps[0])
    start, lens = _i32([14, 30]).to(DEV), _i32([15, 31]).to(DEV)
    ws = torch.empty(exattn.cache_workspace_size(cache, H, 1), dtype=torch.uint8, device=DEV)

    def step(cache, q, k, v, start, lens, workspace=None):
        r = exattn.cache_append(cache, k, v, freq, start, q=q)
        return exattn.forward_cache(r, cache, lens, workspace=workspace)

    keep = [t.clone() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)]
    step(cache, q, k, v, start, lens, ws)
    torch.cuda.synchronize()
    for t, x in zip((cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale), keep):
        t.copy_(x)
    ws.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step(cache, q, k, v, start, lens, ws)
    es, el = _i32([14, 30]).to(DEV), _i32([15, 31]).to(DEV)
    for x in steps:
        for a, b in zip((q, k, v), x):
            a.copy_(b)
        graph.replay()
        wo, wl = step(eager, *x, es, el)
        assert torch.equal(o, wo) and torch.equal(lse, wl)
        for t in (start, lens, es, el):
            t.add_(1)
    assert exattn.check_device_error() == 0


def test_refused_tensors():
    cache, _, _ = make_cache(2, 2, 16, 64, 3, "int8", seed=38)
    k = torch.zeros((2, 2, 4, 64), dtype=torch.bfloat16, device=DEV)
    freq, w = exattn.rope_frequencies(64)[0], torch.ones(64, device=DEV)
    start = torch.zeros(2, dtype=torch.int32, device=DEV)
    for args, kw in [((k[:, :1], k, freq), {}), ((k, k[:, :, :2], freq), {}), ((k, k, freq.float()), {}), ((k, k, freq.cpu()), {}),
                     ((k, k, freq, start.long()), {}), ((k, k, freq, start, start[:1]), {}), ((k, k, freq, start, None, start), {}),
                     ((k, k, freq), dict(q=k[:1])), ((k, k, freq), dict(q=k[:, :, :2])), ((k, k, freq), dict(q=k.half())),
                     ((k, k, freq), dict(q_weight=w)), ((k, k, freq), dict(out=k)), ((k, k, freq), dict(q=k, out=k[:, :1])),
                     ((k, k, freq), dict(layout="x")), ((k, k, freq), dict(k_weight=w[:8]))]:
        with pytest.raises(ValueError):
            exattn.cache_append(cache, *args, **kw)
    for kw in [dict(k_weight=w, eps=0.0), dict(amplitude=math.nan)]:
        with pytest.raises(exattn.AttnError):
            exattn.cache_append(cache, k, k, freq, **kw)
    assert exattn.check_device_error() == 0


def test_onto_pages_of_nan():
    """A page whose scale is NaN stays so, its earlier codes as they were, and the other pages and heads are not touched by it."""
    cache, host, table = make_cache(2, 2, 16, 64, 3, "e4m3", seed=39)
    bad = int(table[0, 1])
    cache.k_scale[bad, 0] = math.nan
    before = cache.k.view(torch.uint8).clone()
    k = torch.randn((2, 2, 20, 64), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    freq, starts = exattn.rope_frequencies(64, device="cpu")[0], [20, 3]
    exattn.cache_append(cache, *_on(k, k, freq, _i32(starts)))
    assert exattn.check_device_error() == 0
    assert torch.isnan(cache.k_scale[bad, 0]) and torch.isfinite(cache.k_scale[bad, 1])
    codes = cache.k.view(torch.uint8)[bad, 0]
    assert torch.equal(codes[:4], before[bad, 0, :4]) and torch.all(codes[4:] == 0)
    y, _ = plain_rope.norm_rotate(k, freq, plain_rope.positions(2, 20, _i32(starts)))
    s = cache.k_scale[int(table[0, 2]), 0].double().cpu()
    got = cache.k[int(table[0, 2]), 0, :8].float().double().cpu() * s
    assert torch.all((got - y[0, 0, 12:]).abs() <= code_step(y[0, 0, 12:], s, "e4m3") * 1.001)


def test_pool_beyond_32_bits():
    """Pages whose codes lie past 4 GB of the pool."""
    pages, heads, page, d = 70_000, 8, 128, 64
    codes = [torch.empty((pages, heads, page, d), dtype=torch.int8, device=DEV) for _ in range(2)]
    scales = [torch.zeros((pages, heads), device=DEV) for _ in range(2)]
    table = torch.tensor([[pages - 1, 3], [pages - 2, 69_000]], dtype=torch.int32, device=DEV)
    for t in codes:
        t[table.reshape(-1).long()] = 0
    cache = exattn.QuantCache(*codes, *scales, table)
    k = torch.randn((2, heads, 200, d), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    freq, starts = exattn.rope_frequencies(d, device="cpu")[0], [0, 50]
    exattn.cache_append(cache, *_on(k, k, freq, _i32(starts)))
    assert exattn.check_device_error() == 0
    y, size = plain_rope.norm_rotate(k, freq, plain_rope.positions(2, 200, _i32(starts)))
    at = table.cpu()
    for b in range(2):
        for n in (0, 77, 78, 127, 128, 199):
            t = starts[b] + n
            p = int(at[b, t // page])
            s = scales[0][p].double().cpu()[:, None]
            got = codes[0][p, :, t % page].double().cpu() * s
            assert torch.all((got - y[b, :, n]).abs() <= 0.5 * s * 1.001 + 2.0 ** -18 * size[b, :, n])


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("eps", [1e-6, 1e-12])
def test_very_small_keys_with_norms(code, layout, d, page, eps):
    """Keys whose norm eps makes, with zeros among their values, and zero keys behind a page of a tiny scale.  Values below
    2^-126 are whole multiples of 2^-149 in bf16 as well, so that the norm's product with them is off by its own rounding only."""
    sizes = [1e-36, 1e-37, 3e-38, 1e-39]
    B = len(sizes) + 1
    cache, host, table = make_cache(B, 2, page, d, 2, code, seed=40)
    g = torch.Generator().manual_seed(41)
    k = torch.randn((B, 2, 3, d), generator=g) * torch.tensor([*sizes, 0.0])[:, None, None, None]
    k[:, :, :, ::7] = 0
    k = k.to(torch.bfloat16)
    w = 1 + 0.3 * torch.randn(d, generator=g)
    freq, starts = exattn.rope_frequencies(16, device="cpu")[0], [0] * len(sizes) + [5]
    cache.k_scale[int(table[-1, 0])] = 1e-37
    before = {"k": cache.k.cpu(), "k_scale": cache.k_scale.cpu()}
    exattn.cache_append(cache, *_on(k, k, freq, _i32(starts)), layout=layout, k_weight=w.to(DEV), eps=eps)
    assert exattn.check_device_error() == 0
    y, size = plain_rope.norm_rotate(k, freq, plain_rope.positions(B, 3, _i32(starts)), layout, weight=w, eps=eps)
    y[(y.abs().amax((2, 3)) / LARGEST[code] < 2.0 ** -126) & (torch.arange(B) < B - 1)[:, None]] = 0  # a scale that is held as zero
    check_keys(cache, before, table, y, size, starts, [3] * B, code)
    codes = cache.k.view(torch.uint8)[table[:, 0].long().to(DEV)].cpu()
    assert torch.all(codes[-1, :, 5:8] & 0x7F == 0)  # of either sign
    lone = [i for i in range(16, d) if i % 7 == 0]  # behind the rotated part
    assert torch.all(codes[:-1, :, :3][..., lone] & 0x7F == 0)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("given", [False, True])
def test_large_frequencies_at_far_positions(layout, given):
    """Rows in order, whose angles are turned on from one another, and positions of their own."""
    B, N, d = 3, 70, 64
    cache, host, table = make_cache(B, 2, 64, d, 3, "e4m3", seed=42)
    g = torch.Generator().manual_seed(43)
    k = torch.randn((B, 2, N, d), generator=g).to(torch.bfloat16)
    freq = torch.tensor(LARGE + [0.1] * 16, dtype=torch.float64)
    begin = _i32([2 ** 31 - 1, -(2 ** 31), 1_000_003])
    offsets = torch.randint(0, 2 ** 31 - 1, (B, N), generator=g).to(torch.int32) if given else None
    before, starts = {"k": cache.k.cpu(), "k_scale": cache.k_scale.cpu()}, [0, 60, 3]
    exattn.cache_append(cache, *_on(k, k, freq, _i32(starts)), offsets=None if offsets is None else offsets.to(DEV), layout=layout, position_start=begin.to(DEV))
    assert exattn.check_device_error() == 0
    y, size = plain_rope.norm_rotate(k, freq, plain_rope.positions(B, N, begin, offsets), layout)
    check_keys(cache, before, table, y, size, starts, [N] * B, "e4m3")
