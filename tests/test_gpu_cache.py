"""The 8-bit key/value cache on the GPU: its store, its reader and the attention over it.

Every result is compared with a plain implementation of the definition in 64 bits on the CPU.

Tolerances, from the roundings that the operators make and nothing else:
  write    the fp32 steps of the definition are followed exactly: codes and scales must be equal
  read     one rounding of code * scale, a product of a 24-bit by an 8-bit number: at most half a step of the
           output's type and half an fp32 step, relative to the value
  O        the probabilities are rounded to fp16 (2^-11 of each; those below 2^-14 of 2^7 by at most 2^-25 of
           it, that is 2^-32 of the largest and with the lazy maximum 2^-24), O to its type (half a step).  An
           error of relative size e in every probability moves O by at most e * sum p |v| / l <= e max |v|.
           Scores: fp32 sums of d products and the exponential's argument, d * 2^-24 * sum |q k| in the worst
           case; for the inputs here (|s| <= 40 in base 2) an error of 40 * 2^-24 * 8 in the exponent, under
           2^-15 in p.  Together under 2^-10 max |v| + half a step of O.
  LSE      the scores' error above and fp32 sums: under 1e-4 absolute
"""
import math

import pytest
import torch

from exact_head_attention_gb300 import exattn

pytestmark = pytest.mark.gpu

DEV = "cuda"
LARGEST = {"e4m3": 448.0, "int8": 127.0}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _table(B, width, pages, seed=0):
    """Page tables whose rows share no page, in random order."""
    g = torch.Generator().manual_seed(seed)
    assert B * width <= pages
    return torch.randperm(pages, generator=g)[: B * width].reshape(B, width).to(torch.int32)


def make_cache(B, heads, page, d, width, code, seed=0, spread=1.0):
    """A cache full of random codes and scales on the CPU in 64-bit values, and on the GPU."""
    g = torch.Generator().manual_seed(seed)
    pages = B * width + 3
    table = _table(B, width, pages, seed)
    out = {}
    for n in ("k", "v"):
        x = torch.randn((pages, heads, page, d), generator=g)
        s = (torch.rand((pages, heads), generator=g) * spread + 0.5) * (4.0 / LARGEST[code])
        y = (x * (LARGEST[code] / 4)).clamp(-LARGEST[code], LARGEST[code])
        out[n] = (y if code == "e4m3" else y.round()).to(CODES[code])
        out[n + "_scale"] = s
    cache = exattn.QuantCache(out["k"].to(DEV), out["v"].to(DEV), out["k_scale"].to(DEV), out["v_scale"].to(DEV), table.to(DEV))
    return cache, out, table


def tokens(host, name, table, b, n):
    """Values of the first n tokens of sequence b, [heads, n, d] in 64 bits."""
    page = host[name].shape[2]
    ids = table[b, : -(-n // page)].long()
    x = host[name].view(torch.uint8)[ids].view(host[name].dtype).float().double() * host[name + "_scale"][ids].double()[:, :, None, None]
    heads, d = x.shape[1], x.shape[3]
    return x.transpose(0, 1).reshape(heads, -1, d)[:, :n]


def plain_attention(q, host, table, lens, mask, scale):
    """O and LSE in 64 bits, and the largest |v| that each sequence and head holds."""
    B, H, n, d = q.shape
    heads = host["k"].shape[1]
    group = H // heads
    o = torch.zeros((B, H, n, d), dtype=torch.float64)
    lse = torch.full((B, H, n), -math.inf, dtype=torch.float64)
    vmax = torch.zeros((B, H, 1, 1), dtype=torch.float64)
    for b, length in enumerate(lens):
        if length == 0:
            continue
        k, v = tokens(host, "k", table, b, length), tokens(host, "v", table, b, length)
        i, t = torch.arange(n)[:, None], torch.arange(length)[None]
        hidden = {"bottom_right": t > i + length - n, True: t > i, False: t < 0}[mask]
        for h in range(H):
            s = (q[b, h].double() @ k[h // group].T) * scale
            s = s.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(s, -1)
            lse[b, h] = z
            some = z > -math.inf
            o[b, h, some] = torch.exp(s[some] - z[some, None]) @ v[h // group]
            vmax[b, h] = v[h // group].abs().max()
    return o, lse, vmax


def check_attention(q, cache, host, table, lens, mask="bottom_right", scale=None, o=None, lse=None):
    scale = 1 / math.sqrt(q.shape[3]) if scale is None else scale
    if o is None:
        o, lse = exattn.forward_cache(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV), mask, scale)
        torch.cuda.synchronize()
        assert exattn.check_device_error() == 0
    ro, rlse, vmax = plain_attention(q, host, table, lens, mask, scale)
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.equal(lse == -math.inf, rlse == -math.inf)
    seen = rlse > -math.inf
    assert torch.all((lse - rlse)[seen].abs() <= 1e-4), (lse - rlse)[seen].abs().max()
    assert torch.all(o[~seen] == 0)
    tol = 2.0 ** -10 * vmax + torch.finfo(q.dtype).eps / 2 * ro.abs()
    assert torch.all((o - ro).abs() <= tol), ((o - ro).abs() / tol).max()


def _q(B, H, n, d, dtype, seed=1):
    return torch.randn((B, H, n, d), generator=torch.Generator().manual_seed(seed)).to(TYPES[dtype])


# ------------------------------------------------------------------ attention

# lengths of zero and one, ends inside a page, on a page and on a tile, and long enough to be divided
SHORT = [0, 1, 15, 16, 17, 33, 64, 130]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_one_token(d, page, code, dtype):
    cache, host, table = make_cache(len(SHORT), 2, page, d, -(-130 // page) + 1, code)
    check_attention(_q(len(SHORT), 2, 1, d, dtype), cache, host, table, SHORT)


@pytest.mark.parametrize("mask", ["bottom_right", True, False], ids=str)
@pytest.mark.parametrize("group,n", [(1, 1), (3, 1), (8, 1), (16, 1), (17, 1), (1, 5), (4, 5), (5, 8), (2, 33), (1, 130), (3, 65)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_and_masks(group, n, mask, d):
    lens = [0, 1, 31, 129, 300, 77]
    cache, host, table = make_cache(len(lens), 2, 32, d, 10, "e4m3", seed=3)
    check_attention(_q(len(lens), 2 * group, n, d, "bf16"), cache, host, table, lens, mask)


@pytest.mark.parametrize("lens", [[9000], [5000, 0, 3, 4097], [2048] * 3, [257, 4000, 1, 900, 31, 640, 0, 5]], ids=str)
@pytest.mark.parametrize("group,n", [(1, 1), (6, 3), (4, 40)])
@pytest.mark.parametrize("d,page,code", [(128, 64, "int8"), (64, 16, "e4m3")])
def test_divided_keys(lens, group, n, d, page, code):
    cache, host, table = make_cache(len(lens), 3, page, d, -(-max(lens) // page), code, seed=5)
    check_attention(_q(len(lens), 3 * group, n, d, "fp16"), cache, host, table, lens)


def test_many_short_sequences():
    lens = [(7 * b) % 90 for b in range(700)]
    cache, host, table = make_cache(len(lens), 1, 32, 64, 3, "int8", seed=6)
    check_attention(_q(len(lens), 2, 1, 64, "bf16"), cache, host, table, lens)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_uneven_scales(code):
    """Pages whose scales differ by orders of magnitude, pages of zeros, and scores far apart."""
    lens = [400, 33]
    cache, host, table = make_cache(2, 2, 16, 64, 25, code, seed=7)
    for n in ("k_scale", "v_scale"):
        f = torch.tensor([1.0, 1e-3, 30.0 if n == "v_scale" else 3.0, 0.0])[torch.arange(host[n].shape[0]) % 4]
        host[n] = host[n] * f[:, None]
    cache = exattn.QuantCache(cache.k, cache.v, host["k_scale"].to(DEV), host["v_scale"].to(DEV), cache.page_table)
    check_attention(_q(2, 4, 3, 64, "bf16"), cache, host, table, lens)


def test_large_and_small_queries():
    """bf16 queries beyond fp16's range, and tiny ones; the scale brings the scores back."""
    lens = [200]
    cache, host, table = make_cache(1, 1, 64, 128, 4, "e4m3", seed=8)
    for size in (1e8, 1e-12):
        q = (_q(1, 1, 4, 128, "bf16").float() * size).to(torch.bfloat16)
        check_attention(q, cache, host, table, lens, scale=1 / math.sqrt(128) / size)


def test_strided_and_offset_views():
    lens = [100, 257]
    cache, host, table = make_cache(2, 2, 32, 64, 9, "e4m3", seed=9)
    big = torch.randn((2, 3, 6, 80), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    q = big.transpose(1, 2)[:, 1:5, :, 8:72]  # [B, H, n, d] of a wider [B, n, H, .] buffer
    check_attention(q.cpu(), cache, host, table, lens,
                    o=exattn.forward_cache(q, cache, torch.tensor(lens, dtype=torch.int32, device=DEV))[0],
                    lse=exattn.forward_cache(q, cache, torch.tensor(lens, dtype=torch.int32, device=DEV))[1])


def test_nan_token_reaches_only_rows_that_see_it():
    lens = [64, 64]
    cache, host, table = make_cache(2, 2, 16, 64, 4, "e4m3", seed=10)
    cache.v_scale[table[0, 3].item(), 1] = math.nan  # tokens 48..63 of sequence 0, head 1
    q = _q(2, 2, 30, 64, "bf16")
    o, lse = exattn.forward_cache(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV))
    ro, rlse, vmax = plain_attention(q, host, table, lens, "bottom_right", 0.125)
    bad = torch.zeros((2, 2, 30), dtype=torch.bool)
    bad[0, 1, 14:] = True  # query i sees the keys up to 34 + i
    assert torch.isnan(o.cpu()[bad]).all() and not torch.isnan(o.cpu()[~bad]).any()
    err = (o.double().cpu() - ro).abs()[~bad]
    assert torch.all(err <= (2.0 ** -10 * vmax + 2.0 ** -8 * ro.abs())[~bad])
    cache.k_scale[table[0, 3].item(), 1] = math.nan
    o, lse = exattn.forward_cache(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV))
    assert torch.equal(torch.isnan(lse.cpu()), bad) and torch.isnan(o.cpu()[bad]).all()


def test_nan_codes_behind_the_length_are_not_met():
    lens = [37, 5, 48]
    for page in (16, 64):
        cache, host, table = make_cache(3, 2, page, 128, 64 // page, "e4m3", seed=11)
        for n in ("k", "v"):
            codes = getattr(cache, n).view(torch.uint8)
            for b, length in enumerate(lens):
                for t in range(length, 64):
                    codes[table[b, t // page].item(), :, t % page] = 0x7F
        check_attention(_q(3, 4, 2, 128, "bf16"), cache, host, table, lens)


def _plain_rows(q, cache, lens, mask):
    o, lse = exattn.forward_cache(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV), mask)
    assert exattn.check_device_error() == 0
    return o.cpu(), lse.cpu()


ROWS = [(1, 5), (2, 8), (3, 10), (1, 40), (2, 32), (1, 65), (1, 128), (1, 200), (2, 150)]


@pytest.mark.parametrize("mask", ["bottom_right", True], ids=str)
@pytest.mark.parametrize("group,n", ROWS)
@pytest.mark.parametrize("d", [64, 128])
def test_nan_codes_hidden_from_some_rows(group, n, mask, d):
    """A NaN among the codes of a token that only a sequence's last queries see."""
    lens = [n + 37, 300, n]
    cache, host, table = make_cache(3, 2, 16, d, 20, "e4m3", seed=21)
    q = _q(3, 2 * group, n, d, "bf16", seed=5)
    want, want_lse = _plain_rows(q, cache, lens, mask)
    for b, head, at, col in ((0, 1, (lens[0] if mask == "bottom_right" else n) - 2, 5), (2, 0, n // 2, d - 1)):
        cache.v.view(torch.uint8)[table[b, at // 16].item(), head, at % 16, col] = 0xFF
        o, lse = _plain_rows(q, cache, lens, mask)
        first = at - (lens[b] - n if mask == "bottom_right" else 0)  # the first query that sees it
        sees = torch.zeros(want.shape[:3], dtype=torch.bool)
        sees[b, head * group : (head + 1) * group, first:] = True
        assert torch.isnan(o[..., col][sees]).all()
        assert torch.equal(o[~sees], want[~sees]) and torch.equal(lse[~sees], want_lse[~sees])
        cache.v.view(torch.uint8)[table[b, at // 16].item(), head, at % 16, col] = 0
        want, want_lse = _plain_rows(q, cache, lens, mask)
        # in a key: the scores of the rows that see it are NaN, the others' are as they were
        was = cache.k.view(torch.uint8)[table[b, at // 16].item(), head, at % 16, col].item()
        cache.k.view(torch.uint8)[table[b, at // 16].item(), head, at % 16, col] = 0x7F
        o, lse = _plain_rows(q, cache, lens, mask)
        assert torch.equal(torch.isnan(lse), sees) and torch.equal(torch.isnan(o).all(-1), sees)
        assert not torch.isnan(o[~sees]).any()
        cache.k.view(torch.uint8)[table[b, at // 16].item(), head, at % 16, col] = was


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("group,n", ROWS)
def test_infinite_scale_hidden_from_some_rows(group, n, code):
    lens = [(n + 47) // 16 * 16 + 3, n]
    cache, host, table = make_cache(2, 2, 16, 128, 20, code, seed=22)
    q = _q(2, 2 * group, n, 128, "fp16", seed=6)
    ro, rlse, vmax = plain_attention(q, host, table, lens, "bottom_right", 1 / math.sqrt(128))
    page = (lens[0] - 1) // 16  # the last page: queries before its first token do not see it
    sees = torch.zeros(ro.shape[:3], dtype=torch.bool)
    sees[0, group:, max(0, page * 16 - (lens[0] - n)) :] = True
    for value in (math.inf, math.nan):
        cache.v_scale[table[0, page].item(), 1] = value
        o, lse = _plain_rows(q, cache, lens, "bottom_right")
        assert torch.isnan(o[sees]).all() and not torch.isnan(o[~sees]).any()
        assert torch.all((o.double() - ro).abs()[~sees] <= (2.0 ** -10 * vmax + 2.0 ** -11 * ro.abs())[~sees])
        assert torch.all((lse.double() - rlse).abs()[~sees] <= 1e-4)


def test_pages_shared_by_sequences():
    """A common prefix in one set of pages."""
    lens = [200, 170, 130, 128]
    cache, host, table = make_cache(4, 2, 32, 64, 7, "int8", seed=23)
    table[1:, :4] = table[0, :4]
    shared = exattn.QuantCache(cache.k, cache.v, cache.k_scale, cache.v_scale, table.to(DEV))
    for n in (1, 12, 50):
        check_attention(_q(4, 4, n, 64, "bf16"), shared, host, table, lens)
    k, v = exattn.cache_read(shared, torch.tensor(lens, dtype=torch.int32, device=DEV), rows=200)
    for b in range(4):
        assert torch.equal(k[b, :, :128], k[0, :, :128]) and torch.equal(v[b, :, :128], v[0, :, :128])


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 24, 25, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 384, 385])
def test_row_counts_at_the_variants_edges(rows):
    lens = [rows + 130, max(1, rows - 3), 2]
    cache, host, table = make_cache(3, 1, 16, 64, 36, "int8", seed=24)
    check_attention(_q(3, 1, rows, 64, "fp16"), cache, host, table, lens)


@pytest.mark.parametrize("group,n", [(3, 128), (1, 300), (2, 150), (1, 257), (5, 90)])
@pytest.mark.parametrize("d", [64, 128])
def test_items_of_one_and_of_two_row_tiles_in_turn(group, n, d):
    """More items than blocks, every second one with 128 rows or fewer of the 256 that the others have."""
    lens = [700, 1, 513, 650, 129, 400, 0, 1000, 333, 90, 870, 256] * 2
    cache, host, table = make_cache(len(lens), 6, 128, d, 8, "int8", seed=25)
    q = _q(len(lens), 6 * group, n, d, "bf16")
    first = exattn.forward_cache(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV))
    check_attention(q, cache, host, table, lens, o=first[0], lse=first[1])
    for _ in range(20):
        again = exattn.forward_cache(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV))
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert exattn.check_device_error() == 0


@pytest.mark.parametrize("rows,d", [(40, 128), (100, 128), (40, 64), (200, 128), (20, 128)])
def test_long_runs_of_copies(rows, d):
    """The same bits from many calls over long sequences, the copies of keys and values always under way."""
    cache, host, table = make_cache(4, 12, 64, d, 256, "e4m3", seed=26)
    lens = torch.tensor([16384] * 4, dtype=torch.int32, device=DEV)
    q = _q(4, 12, rows, d, "bf16").to(DEV)
    first = exattn.forward_cache(q, cache, lens)
    for _ in range(60):
        again = exattn.forward_cache(q, cache, lens)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert exattn.check_device_error() == 0
    few = exattn.forward_cache(q[:, :, -3:].contiguous(), cache, lens)  # another kernel's result
    # each within 2^-10 of the largest |v|, 6 here, and half a step of bf16
    assert torch.all((few[0].float() - first[0][:, :, -3:].float()).abs() <= 2 * (6 * 2.0 ** -10 + 2.0 ** -8 * first[0][:, :, -3:].float().abs()))
    assert torch.all((few[1] - first[1][:, :, -3:]).abs() <= 2e-4)


def test_pool_beyond_32_bits():
    """Pages whose codes lie past 2^32 bytes."""
    pages, page, d = 270_000, 128, 128
    k, v = (torch.zeros((pages, 1, page, d), dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((pages, 1), device=DEV) for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 7, 262_143, 262_144]], dtype=torch.int32)
    cache = exattn.QuantCache(k, v, ks, vs, table.to(DEV))
    g = torch.Generator().manual_seed(3)
    new = [torch.randn((1, 1, 500, d), generator=g).to(torch.bfloat16) for _ in range(2)]
    exattn.cache_write(cache, new[0].to(DEV), new[1].to(DEV))
    ids = table[0].to(DEV).long()
    host = {"k": k[ids].cpu(), "v": v[ids].cpu(), "k_scale": ks[ids].cpu(), "v_scale": vs[ids].cpu()}
    near = torch.arange(4, dtype=torch.int32)[None]
    assert (host["k"].float() * host["k_scale"][..., None, None]).reshape(-1, d)[:500].sub(new[0][0, 0].float()).abs().max() < 0.05
    for n in (1, 20, 60, 100, 300):
        check_attention(_q(1, 1, n, d, "bf16"), cache, host, near, [500])
    got = exattn.cache_read(cache, torch.tensor([500], dtype=torch.int32, device=DEV), rows=500)
    for t, name in zip(got, "kv"):
        want = tokens(host, name, near, 0, 500)
        assert torch.all((t[0].double().cpu() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -23))


def test_bad_page_numbers_and_lengths():
    lens = [64, 64, 64]
    cache, host, table = make_cache(3, 2, 16, 64, 4, "int8", seed=12)
    for number in (-1, cache.k.shape[0], 2 ** 31 - 1):
        bad = cache.page_table.clone()
        bad[1, 2] = number
        broken = exattn.QuantCache(cache.k, cache.v, cache.k_scale, cache.v_scale, bad)
        for n in (1, 40):
            q = _q(3, 2, n, 64, "bf16")
            o, lse = exattn.forward_cache(q.to(DEV), broken, torch.tensor(lens, dtype=torch.int32, device=DEV))
            assert exattn.check_device_error() == 8
            ro, rlse, vmax = plain_attention(q, host, table, lens, "bottom_right", 0.125)
            fine = torch.tensor([0, 2])
            assert torch.all((o.double().cpu() - ro).abs()[fine] <= (2.0 ** -10 * vmax + 2.0 ** -8 * ro.abs())[fine])
            assert torch.isnan(o[1, :, -1]).all()
    q = _q(3, 2, 1, 64, "bf16")
    # a negative length is none, one past the table is the table's
    o, lse = exattn.forward_cache(q.to(DEV), cache, torch.tensor([-5, 65, 64], dtype=torch.int32, device=DEV))
    assert exattn.check_device_error() == 8
    check_attention(q, cache, host, table, [0, 64, 64], o=o, lse=lse)


def test_same_bits_and_a_dirty_workspace():
    lens = [5000, 123]
    cache, host, table = make_cache(2, 2, 64, 128, 79, "e4m3", seed=13)
    q = _q(2, 8, 3, 128, "bf16").to(DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = exattn.forward_cache(q, cache, n)
    ws = torch.full((exattn.cache_workspace_size(cache, 8, 3),), 255, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        got = exattn.forward_cache(q, cache, n, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ scores and scales that rise along the keys

# Rows a key/value head: both sides of every choice between kernels and row tiles, and items whose last row tile has
# 128 rows or fewer of 256.
RISING_ROWS = [1, 8, 12, 24, 25, 40, 64, 65, 100, 128, 129, 200, 256, 257, 300, 384, 385, 513, 520]


def _copies(host, table, B):
    """B sequences over the pages of one."""
    return exattn.QuantCache(*(host[n].to(DEV) for n in ("k", "v", "k_scale", "v_scale")), table.expand(B, -1).contiguous().to(DEV))


def check_copies(q, host, table, lens, check, **kw):
    """Attention of equal queries over equal tokens: alone, where its keys are cut into the smallest pieces, and 64 times in
    one call, where pieces are long.  `check` compares the results for one sequence; and the same bits each time."""
    cache = _copies(host, table, 64 * len(lens))
    for copies in (1, 64):
        part = _copies(host, table, copies * len(lens)) if copies == 1 else cache
        n = torch.tensor(lens * copies, dtype=torch.int32, device=DEV)
        o, lse = exattn.forward_cache(q.repeat(copies, 1, 1, 1).to(DEV), part, n)
        for _ in range(2):
            again = exattn.forward_cache(q.repeat(copies, 1, 1, 1).to(DEV), part, n)
            assert torch.equal(again[0], o) and torch.equal(again[1], lse)
        assert exattn.check_device_error() == 0
        for c in range(0, copies, 21):
            at = slice(c * len(lens), (c + 1) * len(lens))
            check(q, None, host, table.expand(len(lens), -1), lens, o=o[at], lse=lse[at], **kw)


def rising_scores(rows, d, code, level, tokens_, seed):
    """Queries and a cache in which the scores of token t lie about level(t) in base 2, for all of a row's keys times that
    row's 1, 0 or 1/2: the first component of each is given to it.  |level| <= 30, and the other components add a deviation
    of 1 to 2, so that |s| <= 40 as the tolerances count."""
    page = 32 if d == 64 else 64
    cache, host, table = make_cache(1, 2, page, d, -(-tokens_ // page), code, seed=seed)
    lv = torch.tensor([float(level(t)) for t in range(table.shape[1] * page)]).reshape(-1, 1, page)
    ids = table[0].long()
    codes = host["k"].float()
    codes[ids, :, :, 0] = lv / 15 / host["k_scale"][ids][:, :, None]  # at most 2, which the smallest scale can hold
    codes = codes.clamp(-LARGEST[code], LARGEST[code])
    host["k"] = (codes if code == "e4m3" else codes.round()).to(CODES[code])
    q = torch.randn((2, 2, rows, d), generator=torch.Generator().manual_seed(seed + 1))
    q[:, :, :, 0] = 15 * math.sqrt(d) / math.log2(math.e) * torch.tensor([1.0, 0.0, 0.5])[torch.arange(rows) % 3]
    q[1] = q[0]
    return q, host, table


@pytest.mark.parametrize("rows", RISING_ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_scores_that_rise_from_tile_to_tile(rows, d, code):
    """The running maximum is passed by more than the factor that it may lag by, so that the accumulator is rescaled."""
    lens = [1192, 700]
    for by in (10, 20, 40):
        q, host, table = rising_scores(rows, d, code, lambda t: min(30, t // 128 * by - 30), lens[0], seed=60)
        check_copies(q.to(torch.bfloat16), host, table, lens, check_attention)


@pytest.mark.parametrize("rows", RISING_ROWS)
@pytest.mark.parametrize("d", [64, 128])
def test_one_large_score(rows, d):
    lens = [1192, 700]
    for at in (128 + 77, 2 * 128 + 3, 1191):
        q, host, table = rising_scores(rows, d, "e4m3", lambda t: 30 if t == at else -10, lens[0], seed=61)
        check_copies(q.to(torch.float16), host, table, lens, check_attention)


@pytest.mark.parametrize("rows", RISING_ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_value_scales_that_rise_from_page_to_page(rows, d, code):
    lens = [1192, 700]
    for page, ratio, span in ((128, 20, 6), (128, 1000, 4), (16, 20, 6)):
        cache, host, table = make_cache(1, 2, page, d, -(-lens[0] // page), code, seed=62)
        f = torch.tensor([float(ratio) ** (j % span - span + 1) for j in range(table.shape[1])])
        host["v_scale"][table[0].long()] *= f[:, None]
        q = _q(1, 2, rows, d, "fp16", seed=63).repeat(2, 1, 1, 1)
        check_copies(q, host, table, lens, check_attention)


# ------------------------------------------------------------------ value scales far apart


@pytest.mark.parametrize("group,n", [(1, 1), (1, 12), (2, 12), (1, 60), (1, 100), (1, 300)])
@pytest.mark.parametrize("d", [64, 128])
def test_value_scales_below_the_smallest_normal_number(group, n, d):
    """Their reciprocals are beyond fp32.  O is off by no more than elsewhere, where the smallest bf16 numbers allow that:
    2^-10 of the largest |v|, and with a reference of at least 2^-126 for P * vs, whose rounding to fp16 is 2^-28 of the
    largest, 448 * 2^-154 for each of 700 keys, together with half a bf16 step of 2^-133 under 2^-133."""
    lens = [700, 130]
    for powers in ([-127], [-130], [-149], [-128, -126, -140], [-149, 0, -130, -129]):
        cache, host, table = make_cache(2, 2, 32, d, 22, "e4m3", seed=68)
        f = torch.tensor([2.0 ** powers[j % len(powers)] for j in range(table.shape[1])])
        for b in range(2):
            host["v_scale"][table[b].long()] = f[:, None].expand(-1, 2)
        cache = exattn.QuantCache(*(host[x].to(DEV) for x in ("k", "v", "k_scale", "v_scale")), cache.page_table)
        q = _q(2, 2 * group, n, d, "bf16", seed=69)
        o, lse = exattn.forward_cache(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV))
        ro, rlse, vmax = plain_attention(q, host, table, lens, "bottom_right", 1 / math.sqrt(d))
        some = rlse > -math.inf
        assert torch.all((lse.double().cpu() - rlse)[some].abs() <= 1e-4)
        tol = 2.0 ** -10 * vmax + 2.0 ** -8 * ro.abs() + 2.0 ** -133
        assert torch.all((o.double().cpu() - ro).abs() <= tol), (powers, ((o.double().cpu() - ro).abs() / tol).max())



def check_weighted(q, cache, host, table, lens, o, lse, mask="bottom_right", scale=None):
    """As check_attention, by what each row itself sees and how much it weighs.

    With the reference that P * vs is scaled by within 2^12 of the row's largest P * vs and never above it, the rounding of
    P * vs to fp16 is 2^-11 of each, or 2^-25 where 2^3 stands for no more than the largest: LARGEST * 2^-28 of it in O for
    each key.  The other errors that the tolerances above count are relative to each P: with the first 2^-10 of sum P |v|.
    A reference is held to 2^-126 of the row's largest weight, and a type's smallest numbers are rounded by half of one."""
    scale = 1 / math.sqrt(q.shape[3]) if scale is None else scale
    ro, rlse, _ = plain_attention(q, host, table, lens, mask, scale)
    B, H, n, d = q.shape
    group = H // host["k"].shape[1]
    page = host["k"].shape[2]
    most = LARGEST["e4m3" if host["k"].dtype == CODES["e4m3"] else "int8"]
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.equal(lse == -math.inf, rlse == -math.inf)
    seen = rlse > -math.inf
    assert torch.all((lse - rlse)[seen].abs() <= 1e-4)
    assert torch.all(o[~seen] == 0)
    for b, length in enumerate(lens):
        if length == 0:
            continue
        k, v = tokens(host, "k", table, b, length), tokens(host, "v", table, b, length)
        vs = host["v_scale"][table[b, : -(-length // page)].long()].double().T.repeat_interleave(page, 1)[:, :length]
        i, t = torch.arange(n)[:, None], torch.arange(length)[None]
        hidden = {"bottom_right": t > i + length - n, True: t > i, False: t < 0}[mask]
        for h in range(H):
            s = ((q[b, h].double() @ k[h // group].T) * scale).masked_fill(hidden, -math.inf)
            P = torch.exp(s - rlse[b, h][:, None].clamp(min=-1e300))
            largest = (P * vs[h // group]).amax(1, keepdim=True)
            tol = 2.0 ** -10 * (P @ v[h // group].abs()) + length * most * 2.0 ** -28 * largest
            tol = tol + torch.finfo(q.dtype).eps / 2 * ro[b, h].abs() + length * most * 2.0 ** -154
            tol = tol + (2.0 ** -134 if q.dtype == torch.bfloat16 else 2.0 ** -25)
            assert torch.all((o[b, h] - ro[b, h]).abs() <= tol), (b, h, ((o[b, h] - ro[b, h]).abs() / tol).max())


SCALE_ROWS = [(1, 1), (1, 5), (3, 10), (4, 6), (1, 25), (2, 32), (1, 65), (1, 128), (3, 60), (1, 256), (2, 150), (1, 385)]


@pytest.mark.parametrize("group,n", SCALE_ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mask", ["bottom_right", True], ids=str)
def test_large_value_scales_of_hidden_pages(group, n, d, mask):
    """A page that a sequence's last queries see alone, with values far above the others': the other rows do not notice."""
    lens = [n + 300, n + 3, 500]
    for f in (1e3, 1e6, 1e9, 1e30):
        cache, host, table = make_cache(3, 2, 16, d, -(-(n + 500) // 16), "e4m3", seed=64)
        for b, length in enumerate(lens):
            last = length if mask == "bottom_right" else min(n, length)  # the last key that any row sees is before it
            host["v_scale"][table[b, (last - 1) // 16].item()] *= f
        cache = exattn.QuantCache(*(host[x].to(DEV) for x in ("k", "v", "k_scale", "v_scale")), cache.page_table)
        q = _q(3, 2 * group, n, d, "bf16", seed=65)
        o, lse = exattn.forward_cache(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV), mask)
        check_weighted(q, cache, host, table, lens, o, lse, mask)


@pytest.mark.parametrize("rows", RISING_ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_large_value_scales_of_little_weight(rows, d, code):
    """Tokens that all rows see, of next to no weight for some of them, with values far above the others'."""
    lens = [1192, 700]
    for level, f in ((-25, 1e6), (-25, 1e12), (-30, 1e20), (20, 1e-9)):
        for at in (0, 2, 4):  # 128 tokens each
            q, host, table = rising_scores(rows, d, code, lambda t: level if t // 128 == at else 0, lens[0], seed=66)
            page = host["v"].shape[2]
            host["v_scale"][table[0, at * 128 // page : (at + 1) * 128 // page].long()] *= f
            check_copies(q.to(torch.bfloat16), host, table, lens, check_weighted)


@pytest.mark.parametrize("rows", RISING_ROWS)
@pytest.mark.parametrize("d", [64, 128])
def test_scores_and_value_scales_that_rise_and_fall(rows, d):
    lens = [1192, 700]
    for by, ratio in ((10, 30), (10, 1 / 30), (-10, 1000), (-10, 1 / 1000), (0, 1e4), (0, 1e-4)):
        q, host, table = rising_scores(rows, d, "e4m3", lambda t: max(-30, min(30, (t // 128 - 4) * by)), lens[0], seed=67)
        page = host["v"].shape[2]
        f = torch.tensor([float(ratio) ** (j * page // 128 - 4) for j in range(table.shape[1])])
        host["v_scale"][table[0].long()] *= f[:, None]
        check_copies(q.to(torch.bfloat16), host, table, lens, check_weighted)


# ------------------------------------------------------------------ write and read


def round_code(y, code):
    """fp32 values to codes: nearest even, clamped."""
    y = y.clamp(-LARGEST[code], LARGEST[code])
    return (y if code == "e4m3" else y.round()).to(CODES[code])


def plain_write(host, table, name, x, starts, counts, code):
    """The definition, page by page, with its fp32 steps."""
    page = host[name].shape[2]
    for b, (start, count) in enumerate(zip(starts, counts)):
        t = start
        while t < start + count:
            j, inside = divmod(t, page)
            take = min(page - inside, start + count - t)
            p = int(table[b, j])
            for h in range(x.shape[1]):
                new = x[b, h, t - start : t - start + take].float()
                f = new.abs().max() * (torch.tensor(1.0) / LARGEST[code])
                if not torch.isfinite(new).all():
                    f = torch.tensor(math.nan)
                elif f < 2.0 ** -126:
                    f = torch.tensor(0.0)
                was, s = host[name + "_scale"][p, h].clone(), f
                if inside:
                    s = torch.maximum(was, f)
                inv = 1.0 / s if s > 0 else torch.tensor(0.0)
                held = host[name].view(torch.uint8)[p, h]
                if inside and s > was:
                    again = held[:inside].view(CODES[code]).float() * (was * inv)
                    held[:inside] = round_code(again, code).view(torch.uint8)
                put = round_code(new * inv, code) if s > 0 else torch.zeros_like(new).to(CODES[code])
                held[inside : inside + take] = put.view(torch.uint8)
                host[name + "_scale"][p, h] = s
            t += take


def assert_cache_equal(cache, host):
    for n in ("k", "v"):
        assert torch.equal(getattr(cache, n).view(torch.uint8).cpu(), host[n].view(torch.uint8)), n
        got, want = getattr(cache, n + "_scale").cpu(), host[n + "_scale"]
        assert torch.equal(got.view(torch.int32)[~torch.isnan(want)], want.view(torch.int32)[~torch.isnan(want)])
        assert torch.equal(torch.isnan(got), torch.isnan(want))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_write(d, page, code, dtype):
    starts, counts = [0, 5, page, page + 1, 2 * page - 1, 3, 0], [150, 1, page, 2, 1, 0, 1]
    B, N = len(starts), 150
    cache, host, table = make_cache(B, 2, page, d, -(-160 // page) + 2, code, seed=20)
    g = torch.Generator().manual_seed(21)
    k = torch.randn((B, N, 2, d), generator=g) * torch.rand((B, N, 1, 1), generator=g) * 8
    v = torch.randn((B, N, 2, d), generator=g) * 0.01
    k, v = k.to(TYPES[dtype]).transpose(1, 2), v.to(TYPES[dtype]).transpose(1, 2)
    exattn.cache_write(cache, k.to(DEV), v.to(DEV), torch.tensor(starts, dtype=torch.int32, device=DEV),
                       torch.tensor(counts, dtype=torch.int32, device=DEV))
    assert exattn.check_device_error() == 0
    plain_write(host, table, "k", k, starts, counts, code)
    plain_write(host, table, "v", v, starts, counts, code)
    assert_cache_equal(cache, host)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_write_one_by_one(code):
    """Tokens that grow: the earlier codes of a page are rounded again, as the definition says."""
    cache, host, table = make_cache(2, 1, 16, 64, 3, code, seed=22)
    g = torch.Generator().manual_seed(23)
    for t in range(20):
        k, v = (torch.randn((2, 1, 1, 64), generator=g).mul(1.3 ** t).to(torch.float16) for _ in range(2))
        starts = [t, t + 20]
        exattn.cache_write(cache, k.to(DEV), v.to(DEV), torch.tensor(starts, dtype=torch.int32, device=DEV))
        plain_write(host, table, "k", k, starts, [1, 1], code)
        plain_write(host, table, "v", v, starts, [1, 1], code)
        assert_cache_equal(cache, host)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_write_special_values(code):
    """Zeros, values too small for a scale, the largest ones, NaN and infinities; and tokens after each of them."""
    rows = [0.0, 1e-38, 3e38, math.nan, math.inf, -math.inf, 1.0]
    B = len(rows)
    cache, host, table = make_cache(B, 1, 16, 64, 2, code, seed=24)
    k = torch.full((B, 1, 3, 64), 0.5)
    k[:, 0, 1, 7] = torch.tensor(rows)
    k[0] = 0.0
    k[1] = 1e-38
    k = k.to(torch.bfloat16)
    starts, counts = [0] * B, [3] * B
    exattn.cache_write(cache, k.to(DEV), k.to(DEV))
    for n in ("k", "v"):
        plain_write(host, table, n, k, starts, counts, code)
    assert_cache_equal(cache, host)
    one = torch.ones((B, 1, 1, 64), dtype=torch.bfloat16)
    starts, counts = [3] * B, [1] * B
    exattn.cache_write(cache, one.to(DEV), one.to(DEV), torch.tensor(starts, dtype=torch.int32, device=DEV))
    for n in ("k", "v"):
        plain_write(host, table, n, one, starts, counts, code)
    assert_cache_equal(cache, host)


def test_write_refuses_what_is_out_of_range():
    cache, host, table = make_cache(4, 2, 16, 64, 3, "int8", seed=25)
    bad = cache.page_table.clone()
    bad[3, 1] = cache.k.shape[0]
    broken = exattn.QuantCache(cache.k, cache.v, cache.k_scale, cache.v_scale, bad)
    x = torch.randn((4, 2, 20, 64), generator=torch.Generator().manual_seed(1)).to(torch.float16)
    starts = [-1, 40, 0, 10]  # before the start, past the table's 48 tokens, fine, through a page that is none
    exattn.cache_write(broken, x.to(DEV), x.to(DEV), torch.tensor(starts, dtype=torch.int32, device=DEV))
    assert exattn.check_device_error() == 8
    # what is in range is written, and nothing else
    for n in ("k", "v"):
        plain_write(host, table, n, x, [0, 40, 0, 10], [0, 8, 20, 6], "int8")
    assert_cache_equal(cache, host)
    # a count past N is N, a negative one none
    cache, host, table = make_cache(2, 2, 16, 64, 3, "int8", seed=26)
    exattn.cache_write(cache, x[:2].to(DEV), x[:2].to(DEV), None, torch.tensor([25, -3], dtype=torch.int32, device=DEV))
    assert exattn.check_device_error() == 8
    for n in ("k", "v"):
        plain_write(host, table, n, x, [0, 0], [20, 0], "int8")
    assert_cache_equal(cache, host)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_write_behind_a_scale_below_the_smallest_normal_number(code):
    """The reciprocal of such a scale is beyond fp32 and taken as the largest number: zeros stay zeros."""
    for power in (-127, -130, -149):
        cache, host, table = make_cache(2, 2, 16, 64, 2, code, seed=70)
        ids = table[:, 0].long()
        host["k_scale"][ids] = host["v_scale"][ids] = 2.0 ** power
        cache = exattn.QuantCache(*(host[x].to(DEV) for x in ("k", "v", "k_scale", "v_scale")), cache.page_table)
        x = torch.zeros((2, 2, 3, 64))
        x[1, :, :, ::5] = 2.0 ** -128
        x[1, :, 1, 1] = -2.0 ** -120
        x = x.to(torch.bfloat16)
        exattn.cache_write(cache, x.to(DEV), x.to(DEV), torch.tensor([4, 5], dtype=torch.int32, device=DEV))
        assert exattn.check_device_error() == 0
        inverse = torch.tensor(2.0 ** -power).clamp(max=torch.finfo(torch.float32).max)
        for n in ("k", "v"):
            for b, start in ((0, 4), (1, 5)):
                host[n].view(torch.uint8)[ids[b], :, start : start + 3] = round_code(x[b].float() * inverse, code).view(torch.uint8)
        assert_cache_equal(cache, host)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_read(d, page, code, dtype):
    lens, starts, N = [0, 1, 300, 290, 17], [0, 0, 0, 289, 20], 301
    cache, host, table = make_cache(5, 2, page, d, -(-300 // page), code, seed=30)
    t = TYPES[dtype]
    k = torch.full((5, N, 2, d), 7.0, dtype=t, device=DEV).transpose(1, 2)
    v = torch.full((5, 2, N, d), 9.0, dtype=t, device=DEV)
    exattn.cache_read(cache, torch.tensor(lens, dtype=torch.int32, device=DEV),
                      start=torch.tensor(starts, dtype=torch.int32, device=DEV), out=(k, v))
    assert exattn.check_device_error() == 0
    for n, got, fill in (("k", k, 7.0), ("v", v, 9.0)):
        got = got.double().cpu()
        for b, (s, length) in enumerate(zip(starts, lens)):
            rows = max(0, length - s)
            want = tokens(host, n, table, b, length)[:, s:] if rows else None
            if rows:
                tol = (torch.finfo(t).eps / 2 + 2.0 ** -24) * want.abs() + (2.0 ** -25 if dtype == "fp16" else 0)
                assert torch.all((got[b, :, :rows] - want).abs() <= tol)
            assert torch.all(got[b, :, rows:] == fill)  # rows behind the last token stay


def test_read_bad_pages():
    cache, host, table = make_cache(2, 1, 16, 64, 3, "e4m3", seed=31)
    bad = cache.page_table.clone()
    bad[0, 1] = -7
    broken = exattn.QuantCache(cache.k, cache.v, cache.k_scale, cache.v_scale, bad)
    k, v = exattn.cache_read(broken, torch.tensor([40, 48], dtype=torch.int32, device=DEV), rows=48)
    assert exattn.check_device_error() == 8
    nan = torch.isnan(k.cpu())
    assert nan[0, :, 16:32].all() and nan.sum() == 16 * 64
    k, v = exattn.cache_read(cache, torch.tensor([49, -1], dtype=torch.int32, device=DEV), rows=50)
    assert exattn.check_device_error() == 8
    assert torch.all(k[0, :, 48:] == 0) and torch.all(k[1] == 0) and torch.any(k[0, :, :48] != 0)


# ------------------------------------------------------------------ together


def test_write_attend_read_in_a_graph():
    """Decoding steps as a server captures them: write a token, attend, with lengths that move on the device."""
    B, heads, group, d, page = 3, 2, 4, 128, 16
    table = _table(B, 4, 20).to(DEV)
    cache = exattn.QuantCache.empty(20, heads, page, d, table)
    g = torch.Generator().manual_seed(40)
    prompt = [torch.randn((B, heads, 21, d), generator=g).to(torch.bfloat16) for _ in range(2)]
    counts = [21, 0, 13]
    start = torch.zeros(B, dtype=torch.int32, device=DEV)
    count = torch.tensor(counts, dtype=torch.int32, device=DEV)
    exattn.cache_write(cache, prompt[0].to(DEV), prompt[1].to(DEV), start, count)
    lens = count.clone()
    k1, v1 = (torch.empty((B, heads, 1, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q1 = torch.empty((B, heads * group, 1, d), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(exattn.cache_workspace_size(cache, heads * group, 1), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()

    def step():
        exattn.cache_write(cache, k1, v1, lens)
        lens.add_(1)
        return exattn.forward_cache(q1, cache, lens, workspace=ws)

    with torch.cuda.graph(graph, stream=side):
        o, lse = step()
    for i in range(8):
        new = [torch.randn(x.shape, generator=g).to(torch.bfloat16) for x in (k1, v1, q1)]
        for dst, src in zip((k1, v1, q1), new):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert exattn.check_device_error() == 0
        now = [c + i + 1 for c in counts]
        assert lens.tolist() == now
        host = {n: getattr(cache, n).cpu() for n in ("k", "v", "k_scale", "v_scale")}
        check_attention(new[2], cache, host, table.cpu(), now, o=o, lse=lse)
    # the cache holds the tokens up to the rounding of its codes: half a step of e4m3 (2^-4 of the value, or of
    # the smallest step 2^-9 * scale), once more for each time a page's scale grew (at most 16 tokens a page)
    k, v = exattn.cache_read(cache, lens, rows=24)
    got = k[2, :, :13].float().cpu()
    err = (got - prompt[0][2, :, :13].float()).abs()
    assert (err.norm() / got.norm()) < 2 * 2.0 ** -4


def test_two_streams_with_a_workspace_each():
    cache, host, table = make_cache(4, 2, 64, 64, 40, "e4m3", seed=41)
    lens = [2500, 100, 2000, 1]
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = [_q(4, 4, 2, 64, "fp16", seed=s) for s in (1, 2)]
    dev = [q.to(DEV) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        out = [exattn.forward_cache(q, cache, n, stream=s) for q, s in zip(dev, streams)]
    torch.cuda.synchronize()
    for q, (o, lse) in zip(qs, out):
        check_attention(q, cache, host, table, lens, o=o, lse=lse)


def test_two_graphs_replayed_side_by_side():
    """Two captured calls, each with its workspace, whose replays overlap on two streams."""
    cache, host, table = make_cache(2, 2, 64, 128, 90, "e4m3", seed=42)
    lens = [5600, 3000]
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = [_q(2, 4, rows, 128, "bf16", seed=rows) for rows in (3, 40)]
    calls = []
    for q in qs:
        dev, graph, side = q.to(DEV), torch.cuda.CUDAGraph(), torch.cuda.Stream()
        ws = torch.empty(exattn.cache_workspace_size(cache, 4, q.shape[2]), dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = exattn.forward_cache(dev, cache, n, workspace=ws)
        calls.append((dev, graph, side, ws, out))
    for _ in range(6):
        for _, graph, side, _, _ in calls:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for q, (_, _, _, _, (o, lse)) in zip(qs, calls):
        check_attention(q, cache, host, table, lens, o=o, lse=lse)


def test_one_workspace_for_calls_in_turn():
    """Calls of different shapes one behind the other in one workspace, captured in one graph."""
    cache, host, table = make_cache(2, 2, 64, 64, 80, "int8", seed=43)
    lens = [5000, 4200]
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = [_q(2, 2, rows, 64, "fp16", seed=rows) for rows in (1, 20, 64, 200, 2)]
    dev = [q.to(DEV) for q in qs]
    ws = torch.empty(max(exattn.cache_workspace_size(cache, 2, q.shape[2]) for q in qs), dtype=torch.uint8, device=DEV)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        out = [exattn.forward_cache(q, cache, n, workspace=ws) for q in dev]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for q, (o, lse) in zip(qs, out):
        check_attention(q, cache, host, table, lens, o=o, lse=lse)


def test_refused_workspaces():
    cache, host, table = make_cache(1, 2, 16, 64, 4, "e4m3", seed=44)
    q = _q(1, 2, 1, 64, "bf16").to(DEV)
    n = torch.tensor([50], dtype=torch.int32, device=DEV)
    size = exattn.cache_workspace_size(cache, 2, 1)
    room = torch.empty(size + 256, dtype=torch.uint8, device=DEV)
    assert room.data_ptr() % 256 == 0
    for ws, status in ((room[: size - 1], "ATTN_ERR_WORKSPACE"), (room[16 : size + 16], "ATTN_ERR_MISALIGNED")):
        with pytest.raises(exattn.AttnError) as e:
            exattn.forward_cache(q, cache, n, workspace=ws)
        assert exattn.STATUS_NAMES[e.value.status] == status
    check_attention(q.cpu(), cache, host, table, [50], o=(r := exattn.forward_cache(q, cache, n, workspace=room))[0], lse=r[1])


def test_refused_tensors():
    """What the binding refuses before anything is launched."""
    cache, host, table = make_cache(2, 2, 16, 64, 4, "e4m3", seed=45)
    q = _q(2, 4, 3, 64, "bf16").to(DEV)
    n = torch.tensor([50, 20], dtype=torch.int32, device=DEV)
    size = exattn.cache_workspace_size(cache, 4, 3)
    new = torch.zeros((2, 2, 5, 64), dtype=torch.bfloat16, device=DEV)
    refused = [
        lambda: exattn.forward_cache(q, cache, n, workspace=torch.empty(size, dtype=torch.uint8)),
        lambda: exattn.forward_cache(q, cache, n, workspace=torch.empty((size, 2), dtype=torch.uint8, device=DEV)[:, 0]),
        lambda: exattn.forward_cache(q.cpu(), cache, n),
        lambda: exattn.forward_cache(q, cache, n.cpu()),
        lambda: exattn.forward_cache(q, cache, n.long()),
        lambda: exattn.forward_cache(q, cache, n[:1]),
        lambda: exattn.forward_cache(q[:1], cache, n),
        lambda: exattn.forward_cache(q.transpose(2, 3), cache, n),
        lambda: exattn.cache_write(cache, new, new[:, :1], n),
        lambda: exattn.cache_write(cache, new, new.half(), n),
        lambda: exattn.cache_write(cache, new.cpu(), new.cpu(), n),
        lambda: exattn.cache_write(cache, new, new, n.cpu()),
        lambda: exattn.cache_read(cache, n),
        lambda: exattn.cache_read(cache, n, out=(new, new[:, :, :4])),
        lambda: exattn.cache_read(cache, n.float(), rows=4),
        lambda: exattn.QuantCache(cache.k, cache.v, cache.k_scale, cache.v_scale.cpu(), cache.page_table),
        lambda: exattn.QuantCache(cache.k, cache.v, cache.k_scale[:-1], cache.v_scale[:-1], cache.page_table),
        lambda: exattn.QuantCache(cache.k, cache.v[:-1], cache.k_scale, cache.v_scale, cache.page_table),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(exattn.AttnError):  # five query heads on two key/value heads
        exattn.forward_cache(torch.zeros((2, 5, 1, 64), dtype=torch.bfloat16, device=DEV), cache, n)
    torch.cuda.synchronize()
    assert exattn.check_device_error() == 0
