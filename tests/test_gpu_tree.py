"""Trees of drafted tokens on the GPU: their masks and depths, and the attention over the cache that follows them.

The attention is compared with the definition in 64 bits on the CPU, with the tolerances of test_gpu_cache.py, which hold for
any mask (the roundings are the same).  Masks and depths are whole numbers and equal.
"""
import math

import pytest
import torch

import plain_rope
from exact_head_attention_gb300 import exattn
from test_gpu_cache import DEV, TYPES, _q, make_cache, tokens

pytestmark = pytest.mark.gpu


def random_parents(B, n, seed=0, reach=None):
    g = torch.Generator().manual_seed(seed)
    i = torch.arange(n)
    back = i if reach is None else i.clamp(max=reach)
    return (i - 1 - (torch.rand((B, n), generator=g) * (back + 1)).long().clamp(max=back)).to(torch.int32)


def plain_tree(parents):
    """(sees [B, n, n], depth [B, n]) by walking up."""
    B, n = parents.shape
    sees = torch.zeros((B, n, n), dtype=torch.bool)
    for b in range(B):
        for i in range(n):
            j = i
            while j >= 0:
                sees[b, i, j] = True
                j = int(parents[b, j])
    return sees, sees.sum(-1).to(torch.int32) - 1


def words(sees):
    B, n, _ = sees.shape
    bits = torch.nn.functional.pad(sees, (0, -n % 32)).reshape(B, n, -1, 32).long()
    w = (bits << torch.arange(32)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def plain_attention(q, host, table, lens, sees, scale):
    """O and LSE in 64 bits, and the largest |v| of each sequence and head.  sees [B or 1, n, n]."""
    B, H, n, d = q.shape
    group = H // host["k"].shape[1]
    o = torch.zeros((B, H, n, d), dtype=torch.float64)
    lse = torch.full((B, H, n), -math.inf, dtype=torch.float64)
    vmax = torch.zeros((B, H, 1, 1), dtype=torch.float64)
    for b, length in enumerate(lens):
        if length == 0:
            continue
        k, v = tokens(host, "k", table, b, length), tokens(host, "v", table, b, length)
        hidden = torch.zeros((n, length), dtype=torch.bool)
        last = min(n, length)
        tree = sees[b % sees.shape[0]] & torch.ones((n, n), dtype=torch.bool).tril()
        hidden[:, length - last :] = ~tree[:, n - last :]
        for h in range(H):
            s = (q[b, h].double() @ k[h // group].T) * scale
            s = s.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(s, -1)
            lse[b, h] = z
            some = ~(z == -math.inf)
            o[b, h, some] = torch.exp(s[some] - z[some, None]) @ v[h // group].nan_to_num(0.0)
            vmax[b, h] = v[h // group].nan_to_num(0.0).abs().max()
    return o, lse, vmax


def check(q, cache, host, table, lens, sees, scale=None, got=None):
    scale = 1 / math.sqrt(q.shape[3]) if scale is None else scale
    if got is None:
        got = exattn.forward_cache_tree(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV), words(sees).to(DEV), scale)
        assert exattn.check_device_error() == 0
    ro, rlse, vmax = plain_attention(q, host, table, lens, sees, scale)
    o, lse = (x.double().cpu() for x in got)
    assert torch.equal(lse == -math.inf, rlse == -math.inf)
    seen = rlse > -math.inf
    assert torch.all((lse - rlse)[seen].abs() <= 1e-4), (lse - rlse)[seen].abs().max()
    assert torch.all(o[~seen] == 0)
    tol = 2.0 ** -10 * vmax + torch.finfo(q.dtype).eps / 2 * ro.abs()
    assert torch.all((o - ro).abs() <= tol), ((o - ro).abs() / tol).max()


# ------------------------------------------------------------------ masks and depths

@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 65, 200, 511, 512])
def test_trees(n):
    chain, star = torch.arange(-1, n - 1, dtype=torch.int32), torch.full((n,), -1, dtype=torch.int32)
    two = torch.where(torch.arange(n) < 2, -1, torch.arange(n) - 2).to(torch.int32)
    parents = torch.cat((torch.stack((chain, star, two, (torch.arange(n) - 1).to(torch.int32) // 2)), random_parents(3, n, n), random_parents(2, n, n, 3)))
    parents[3, 0] = -1
    mask, depth = exattn.draft_tree(parents.to(DEV))
    assert exattn.check_device_error() == 0
    sees, want = plain_tree(parents)
    assert torch.equal(depth.cpu(), want) and torch.equal(mask.cpu(), words(sees))
    one, d1 = exattn.draft_tree(parents[4].to(DEV))
    assert one.shape == (1, n, (n + 31) // 32) and torch.equal(one[0], mask[4]) and torch.equal(d1[0], depth[4])


def test_parents_that_are_no_earlier_token():
    parents = torch.tensor([[-1, 0, 2, 7, -2, 3, 2 ** 31 - 1, -(2 ** 31)]], dtype=torch.int32)
    mask, depth = exattn.draft_tree(parents.to(DEV))
    assert exattn.check_device_error() == 9 and "parent" in exattn.last_error()
    sees, want = plain_tree(torch.tensor([[-1, 0, -1, -1, -1, 3, -1, -1]], dtype=torch.int32))
    assert torch.equal(depth.cpu(), want) and torch.equal(mask.cpu(), words(sees))
    assert exattn.check_device_error() == 0


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("group,n", [(1, 1), (1, 2), (8, 1), (1, 8), (3, 5), (1, 16), (1, 17), (2, 12), (1, 24), (1, 25), (1, 64), (1, 65), (5, 13),
                                     (1, 128), (2, 64), (1, 129), (3, 65), (1, 300), (1, 512), (2, 400)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_rows(group, n, d, code):
    """Sequences that end before, at and after the drafted tokens, on a tile and off it."""
    lens = [0, 1, n - 1, n, n + 1, n + 128 - n % 128, 300 + n, 77]
    cache, host, table = make_cache(len(lens), 2, 32, d, -(-max(lens) // 32), code, seed=40)
    check(_q(len(lens), 2 * group, n, d, "bf16"), cache, host, table, lens, plain_tree(random_parents(len(lens), n, n))[0])


@pytest.mark.parametrize("lens", [[9000], [5000, 40, 3, 4097], [2048] * 3], ids=str)
@pytest.mark.parametrize("group,n", [(1, 20), (6, 3), (4, 40), (3, 200)])
@pytest.mark.parametrize("d,page,code", [(128, 64, "int8"), (64, 16, "e4m3")])
def test_divided_keys(lens, group, n, d, page, code):
    cache, host, table = make_cache(len(lens), 3, page, d, -(-max(lens) // page), code, seed=41)
    check(_q(len(lens), 3 * group, n, d, "fp16"), cache, host, table, lens, plain_tree(random_parents(len(lens), n, 5))[0])


@pytest.mark.parametrize("group,n", [(1, 7), (2, 12), (1, 40), (3, 100), (1, 500)])
@pytest.mark.parametrize("d", [64, 128])
def test_masks_that_are_no_trees(group, n, d):
    """Any bits: rows that see no drafted token (nothing at all without a prefix), first tiles hidden, bits behind the row."""
    lens = [n, n + 5, 700 + n, n // 2]
    cache, host, table = make_cache(4, 2, 64, d, -(-max(lens) // 64), "e4m3", seed=42)
    sees = torch.rand((4, n, n), generator=torch.Generator().manual_seed(6)) < 0.3
    sees[:, ::5] = False
    sees[1, :, : n // 2] = False  # only late tokens
    check(_q(4, 2 * group, n, d, "bf16"), cache, host, table, lens, sees)


@pytest.mark.parametrize("group,n", [(1, 9), (2, 10), (1, 24), (1, 60), (4, 130), (1, 512)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_full_masks_are_causal(group, n, d, code):
    """Every drafted token sees all before it; one mask for all sequences and one for each give the same bits."""
    lens = [n, 3, 1000 + n, 0, 640 + n]
    cache, host, table = make_cache(len(lens), 2, 32, d, -(-max(lens) // 32), code, seed=43)
    q, at = _q(len(lens), 2 * group, n, d, "fp16"), torch.tensor(lens, dtype=torch.int32, device=DEV)
    full = torch.full((1, n, (n + 31) // 32), -1, dtype=torch.int32, device=DEV)
    one, each = (exattn.forward_cache_tree(q.to(DEV), cache, at, t) for t in (full, full.expand(len(lens), -1, -1).contiguous()))
    check(q, cache, host, table, lens, torch.ones((1, n, n), dtype=torch.bool), got=one)
    assert torch.equal(one[0], each[0]) and torch.equal(one[1], each[1])


@pytest.mark.parametrize("B,heads,group,n,lens", [(5, 3, 2, 40, [2000, 0, 17, 900, 2100]), (128, 1, 1, 30, None), (129, 1, 1, 30, None), (90, 2, 9, 29, None),
                                                  (3, 40, 1, 300, [310, 5, 1290]), (1, 1, 1, 33, [33]), (40, 4, 1, 64, None), (2, 8, 1, 200, [20000, 300])], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_items_whole_and_divided(B, heads, group, n, lens, d):
    """Batches on both sides of the rule that keeps items whole: equal and spread lengths, more items than blocks and fewer."""
    lens = lens or [n + (977 * b) % 1500 if b % 7 else 0 for b in range(B)]
    cache, host, table = make_cache(B, heads, 64, d, -(-max(lens) // 64), "e4m3", seed=49)
    check(_q(B, heads * group, n, d, "bf16"), cache, host, table, lens, plain_tree(random_parents(1, n, 7, 6))[0])


@pytest.mark.parametrize("group,n", [(1, 1), (4, 2), (1, 16), (3, 8)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("wide", [False, True])
def test_few_rows_are_as_exact_as_their_output(group, n, d, code, wide):
    """fp16, where few keys count: no rounding but the output's shows.  Over thousands of values that rounding's size is the
    64-bit result's own within a tenth; scores are off by some 25 steps of fp32 at sizes up to 20, below 2^-15 in the exponent."""
    lens = [40 + n, n, 700, 333]
    _, host, table = make_cache(len(lens), 3, 16, d, 48, code, seed=47)
    if wide:
        host["v_scale"][::3] *= 64
    cache = exattn.QuantCache(*(host[x].to(DEV) for x in ("k", "v", "k_scale", "v_scale")), table.to(DEV))
    q, (sees, _) = _q(len(lens), 3 * group, n, d, "fp16"), plain_tree(random_parents(len(lens), n, 48))
    scale = 4 / math.sqrt(d)
    o, _ = exattn.forward_cache_tree(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV), words(sees).to(DEV), scale)
    assert exattn.check_device_error() == 0
    want = plain_attention(q, host, table, lens, sees, scale)[0]
    off, own = (torch.linalg.norm(x.double().cpu() - want) / torch.linalg.norm(want) for x in (o, want.half()))
    assert off <= 1.1 * own + 2.0 ** -15, (off, own)


@pytest.mark.parametrize("group,n", [(1, 6), (1, 30), (2, 100)])
def test_one_tree_for_all(group, n):
    lens = [n, 200, 300 + n]
    cache, host, table = make_cache(3, 2, 16, 64, -(-max(lens) // 16), "int8", seed=44)
    check(_q(3, 2 * group, n, 64, "bf16"), cache, host, table, lens, plain_tree(random_parents(1, n, 3))[0])


@pytest.mark.parametrize("group,n", [(1, 8), (3, 8), (1, 40), (3, 64), (1, 512)])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_of_a_branch_stays_there(group, n, d):
    """NaN codes of a drafted token, and a page of a NaN scale, reach the rows that see them and no other."""
    lens = [n, 150 + n]
    cache, host, table = make_cache(2, 2, 16, d, -(-max(lens) // 16), "e4m3", seed=45)
    sees = plain_tree(random_parents(2, n, 8, 4))[0]
    q = _q(2, 2 * group, n, d, "bf16")
    token = [n // 2, n // 3]
    for b in range(2):
        t = lens[b] - n + token[b]
        p = int(table[b, t // 16])
        cache.v.view(torch.uint8)[p, 1, t % 16, 5] = 0x7F
        cache.k.view(torch.uint8)[p, 0, t % 16, 9] = 0xFF
    o, lse = (x.cpu() for x in exattn.forward_cache_tree(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV), words(sees).to(DEV)))
    ro, rlse, vmax = plain_attention(q, host, table, lens, sees, 1 / math.sqrt(d))
    for b in range(2):
        bad = sees[b, :, token[b]] & (torch.arange(n) >= token[b])
        for h in range(2 * group):
            assert torch.isnan(o[b, h][bad]).any(-1).all()
            assert not torch.isnan(o[b, h][~bad]).any() and not torch.isnan(lse[b, h][~bad]).any()
            if h < group:
                assert torch.isnan(lse[b, h][bad]).all()
            err = (o[b, h].double() - ro[b, h]).abs()[~bad]
            assert torch.all(err <= (2.0 ** -10 * vmax[b, h] + 2.0 ** -8 * ro[b, h].abs())[~bad])
    # a scale of NaN or infinity covers the page's tokens
    cache, host, table = make_cache(2, 2, 16, d, -(-max(lens) // 16), "e4m3", seed=46)
    pages = [int(table[b, (lens[b] - n + token[b]) // 16]) for b in range(2)]
    cache.k_scale[pages[0]] = math.nan
    cache.v_scale[pages[1]] = math.inf
    o, lse = (x.cpu() for x in exattn.forward_cache_tree(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV), words(sees).to(DEV)))
    ro, rlse, vmax = plain_attention(q, host, table, lens, sees, 1 / math.sqrt(d))
    for b in range(2):
        first = (lens[b] - n + token[b]) // 16 * 16 - (lens[b] - n)  # drafted tokens first .. first + 15 are bad
        tril = torch.ones((n, n), dtype=torch.bool).tril()
        bad = (sees[b] & tril)[:, max(0, first) : first + 16].any(-1) | (first < 0)
        assert torch.isnan(o[b][:, bad]).all() and not torch.isnan(o[b][:, ~bad]).any()
        err = (o[b].double() - ro[b]).abs()[:, ~bad]
        assert torch.all(err <= (2.0 ** -10 * vmax[b] + 2.0 ** -8 * ro[b].abs())[:, ~bad])


@pytest.mark.parametrize("group,n", [(2, 5), (2, 50)])
def test_views_streams_and_graphs(group, n):
    lens = [90 + n, 400]
    cache, host, table = make_cache(2, 2, 32, 64, -(-(400 + n) // 32), "e4m3", seed=47)
    sees = plain_tree(random_parents(2, n, 9))[0]
    tree, at = words(sees).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    big = torch.randn((2, n, 2 * group + 3, 80), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    q = big.transpose(1, 2)[:, 1 : 1 + 2 * group, :, 8:72]
    want = exattn.forward_cache_tree(q, cache, at, tree)
    check(q.cpu(), cache, host, table, lens, sees, got=want)
    size = exattn.cache_workspace_size(cache, 2 * group, n)
    side, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for s in side:
        got.append(exattn.forward_cache_tree(q, cache, at, tree, workspace=torch.empty(size, dtype=torch.uint8, device=DEV), stream=s))
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    other = torch.zeros_like(tree)
    for t in (tree, other):  # one graph, the tree written anew between replays
        t.copy_(tree)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = exattn.forward_cache_tree(q, cache, at, other, workspace=ws)
    for _ in range(3):
        graph.replay()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    other.fill_(-1)
    graph.replay()
    check(q.cpu(), cache, host, table, lens, torch.ones((1, n, n), dtype=torch.bool), got=(o, lse))


def test_a_step_of_drafting():
    """Tree, append and attention together: each drafted token's output is that of its own path alone behind the prompt."""
    B, heads, group, n, d, page = 2, 2, 3, 11, 64, 16
    start = torch.tensor([37, 128], dtype=torch.int32)
    g = torch.Generator().manual_seed(50)
    parents = random_parents(B, n, 51)
    sees, depth = plain_tree(parents)
    prompt = torch.randn((B, heads, 128, d), generator=g).to(torch.bfloat16)
    q, k, v = (torch.randn((B, h, n, d), generator=g).to(torch.bfloat16) for h in (heads * group, heads, heads))
    freq, w = exattn.rope_frequencies(d)[0], torch.linspace(0.5, 1.5, d)
    table = torch.randperm(B * 9, generator=g).reshape(B, 9).to(torch.int32)

    def fresh():
        c = exattn.QuantCache.empty(B * 9, heads, page, d, table.to(DEV))
        exattn.cache_append(c, prompt.to(DEV), prompt.to(DEV), freq, None, start.to(DEV), k_weight=w.to(DEV))
        return c

    cache = fresh()
    mask, dep = exattn.draft_tree(parents.to(DEV))
    assert torch.equal(dep.cpu(), depth)
    r = exattn.cache_append(cache, k.to(DEV), v.to(DEV), freq, start.to(DEV), offsets=dep, q=q.to(DEV), q_weight=w.to(DEV), k_weight=w.to(DEV))
    o, lse = exattn.forward_cache_tree(r, cache, (start + n).to(DEV), mask)
    assert exattn.check_device_error() == 0
    host = {x: getattr(cache, x).cpu() for x in ("k", "v", "k_scale", "v_scale")}
    ro, rlse, vmax = plain_attention(r.cpu(), host, table, (start + n).tolist(), sees, 1 / math.sqrt(d))
    assert torch.all((o.double().cpu() - ro).abs() <= 2.0 ** -10 * vmax + 2.0 ** -8 * ro.abs())
    # the path's keys in fp64, positions from the depth: 8-bit keys are within half a code of them
    y, _ = plain_rope.norm_rotate(k, freq.cpu(), start[:, None].long() + depth, weight=w)
    for b in range(B):
        at = tokens(host, "k", table, b, int(start[b]) + n)[:, int(start[b]) :]
        scales = torch.stack([host["k_scale"][int(table[b, (int(start[b]) + i) // page])] for i in range(n)], 1).double()
        assert torch.all((at - y[b]).abs() <= torch.maximum(y[b].abs() * 2.0 ** -4, scales[..., None] * 2.0 ** -10) * 1.001)
    # the accepted path goes into the cache for good: written over the drafts, the next step sees a plain sequence
    path = [i for i in range(n) if sees[0, n - 1, i]]
    again = exattn.cache_append(cache, k[:, :, path].to(DEV), v[:, :, path].to(DEV), freq, start.to(DEV), q=q[:, :, path].to(DEV),
                                q_weight=w.to(DEV), k_weight=w.to(DEV))
    o2, lse2 = exattn.forward_cache(again, cache, (start + len(path)).to(DEV))
    assert torch.all((o2[0].cpu().float() - o[0, :, path].cpu().float()).abs() <= 0.2) and torch.all((lse2[0] - lse[0, :, path]).abs().cpu() <= 0.2)


def test_refused():
    cache, _, _ = make_cache(2, 2, 16, 64, 40, "int8", seed=48)
    q = torch.zeros((2, 4, 33, 64), dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([40, 50], dtype=torch.int32, device=DEV)
    tree = torch.zeros((2, 33, 2), dtype=torch.int32, device=DEV)
    for bad in (tree.long(), tree.cpu(), tree[:, :, :1], tree[:, :32].contiguous(), tree[0], tree.expand(4, 2, 33, 2)[0], torch.cat((tree, tree)),
                tree.transpose(1, 2).contiguous().transpose(1, 2)):
        if bad.shape == tree.shape and bad.dtype == tree.dtype and bad.is_cuda and bad.is_contiguous():
            continue
        with pytest.raises(ValueError):
            exattn.forward_cache_tree(q, cache, at, bad)
    big = torch.zeros((2, 2, 513, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(exattn.AttnError):
        exattn.forward_cache_tree(big, cache, at, torch.zeros((1, 513, 17), dtype=torch.int32, device=DEV))
    with pytest.raises(exattn.AttnError):
        exattn.draft_tree(torch.full((1, 513), -1, dtype=torch.int32, device=DEV))
    for bad in (torch.zeros((1, 4), dtype=torch.int64, device=DEV), torch.zeros((1, 4), dtype=torch.int32), torch.zeros((1, 1, 4), dtype=torch.int32, device=DEV)):
        with pytest.raises(ValueError):
            exattn.draft_tree(bad)
    mask, depth = exattn.draft_tree(torch.zeros((0, 4), dtype=torch.int32, device=DEV))
    assert mask.shape == (0, 4, 1) and depth.shape == (0, 4)
    assert exattn.check_device_error() == 0


def test_two_graphs_side_by_side():
    """Two captured steps, a workspace each, replayed on two streams at the same time."""
    sets = []
    for seed, (group, n) in ((60, (1, 18)), (61, (3, 40))):
        lens = [700 + n, n, 90]
        cache, host, table = make_cache(3, 2, 16, 64, -(-max(lens) // 16), "int8", seed=seed)
        sees = plain_tree(random_parents(3, n, seed))[0]
        q, at, tree = _q(3, 2 * group, n, 64, "fp16").to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), words(sees).to(DEV)
        ws = torch.zeros(exattn.cache_workspace_size(cache, 2 * group, n), dtype=torch.uint8, device=DEV)
        exattn.forward_cache_tree(q, cache, at, tree, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = exattn.forward_cache_tree(q, cache, at, tree, workspace=ws)
        sets.append((graph, got, (q.cpu(), cache, host, table, lens, sees), (q, at, tree, ws)))  # what a graph reads is kept
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for s, (graph, _, _, _) in zip(streams, sets):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, got, args, _ in sets:
        check(*args, got=got)
    assert exattn.check_device_error() == 0


@pytest.mark.parametrize("B,heads", [(39, 4), (51, 3)])
def test_a_few_items_more_than_blocks_are_divided(B, heads):
    """One to four items more than blocks, all of one length: kept whole, the blocks with two would take twice as long as the
    others.  A sequence less keeps an item a block, in 1.02 of which the work would go; half as much again is allowed."""
    blocks = torch.cuda.get_device_properties(0).multi_processor_count
    if not blocks < B * heads <= blocks + 4 or (B - 1) * heads > blocks:
        pytest.skip("sized for 152 blocks")
    d, n, lens = 64, 64, 8192
    took = []
    for b in (B, B - 1):
        cache = exattn.QuantCache.empty(b * lens // 64, heads, 64, d, torch.arange(b * lens // 64, dtype=torch.int32, device=DEV).view(b, -1))
        q, at = torch.zeros((b, heads, n, d), dtype=torch.bfloat16, device=DEV), torch.full((b,), lens, dtype=torch.int32, device=DEV)
        tree, _ = exattn.draft_tree(torch.arange(-1, n - 1, dtype=torch.int32, device=DEV))
        ws = torch.empty(exattn.cache_workspace_size(cache, heads, n), dtype=torch.uint8, device=DEV)
        events = [torch.cuda.Event(enable_timing=True) for _ in range(12)]
        for e in events:
            exattn.forward_cache_tree(q, cache, at, tree, workspace=ws)
            e.record()
        torch.cuda.synchronize()
        took.append(min(x.elapsed_time(y) for x, y in zip(events[2:], events[3:])))
    assert took[0] <= 1.5 * took[1], took


@pytest.mark.parametrize("group,n", [(1, 25), (2, 32), (1, 100), (4, 32), (1, 129), (4, 64), (1, 512)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("wide", [False, True])
def test_many_rows_are_about_as_exact_as_their_output(group, n, d, code, wide):
    """fp16 where many keys count alike.  Probabilities of fp16 are off by errors of their own, uniform within half a step, and so
    are outputs; relative to a number of mantissa m in [1, 2) that is e / m, in the mean of squares 0.54 e^2 over evenly spread
    logarithms and e^2 at most.  Values of no common sign make O^2 the sum of p^2 v^2, so that the probabilities' errors add up
    to e^2 O^2 at most beside the rounding's 0.54: sqrt(1 + 1 / 0.54) = 1.69 times the rounding alone; the scores' 2^-15 as above."""
    lens = [40 + n, n, 700 + n, 100 + n // 2]
    _, host, table = make_cache(len(lens), 3, 16, d, -(-max(lens) // 16), code, seed=52)
    if wide:
        host["v_scale"][::3] *= 64
    cache = exattn.QuantCache(*(host[x].to(DEV) for x in ("k", "v", "k_scale", "v_scale")), table.to(DEV))
    q, (sees, _) = _q(len(lens), 3 * group, n, d, "fp16"), plain_tree(random_parents(len(lens), n, 53))
    scale = 1 / math.sqrt(d)
    o, _ = exattn.forward_cache_tree(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV), words(sees).to(DEV), scale)
    assert exattn.check_device_error() == 0
    want = plain_attention(q, host, table, lens, sees, scale)[0]
    off, own = (torch.linalg.norm(x.double().cpu() - want) / torch.linalg.norm(want) for x in (o, want.half()))
    assert off <= 1.69 * own + 2.0 ** -15, (off, own)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_the_accepted_path_of_every_sequence(code):
    """What a server does after a step of drafting: each sequence's accepted path is appended over its drafts, as many tokens as it
    has (the rest of the rows are padding), and the next queries see a plain sequence.  The cache's new keys are compared with the
    definition, and the attention over it with that over the cache as it then is."""
    B, heads, group, n, d, page = 2, 2, 3, 11, 64, 16
    start = torch.tensor([37, 128], dtype=torch.int32)
    g = torch.Generator().manual_seed(54)
    parents = random_parents(B, n, 55)
    sees, depth = plain_tree(parents)
    prompt = torch.randn((B, heads, 128, d), generator=g).to(torch.bfloat16)
    q, k, v = (torch.randn((B, h, n, d), generator=g).to(torch.bfloat16) for h in (heads * group, heads, heads))
    freq, w = exattn.rope_frequencies(d)[0], torch.linspace(0.5, 1.5, d)
    table = torch.randperm(B * 9, generator=g).reshape(B, 9).to(torch.int32)
    cache = exattn.QuantCache.empty(B * 9, heads, page, d, table.to(DEV), code)
    exattn.cache_append(cache, prompt.to(DEV), prompt.to(DEV), freq, None, start.to(DEV), k_weight=w.to(DEV))
    _, dep = exattn.draft_tree(parents.to(DEV))
    exattn.cache_append(cache, k.to(DEV), v.to(DEV), freq, start.to(DEV), offsets=dep, k_weight=w.to(DEV))
    paths = [torch.nonzero(sees[b, int(depth[b].argmax())])[:, 0] for b in range(B)]
    counts = [len(p) for p in paths]
    most = max(counts)
    at = torch.stack([torch.nn.functional.pad(p, (0, most - len(p))) for p in paths])[:, None, :, None]
    pq, pk, pv = (x.gather(2, at.expand(-1, x.shape[1], -1, d)) for x in (q, k, v))
    lens = [int(s) + c for s, c in zip(start, counts)]
    r = exattn.cache_append(cache, *(x.to(DEV) for x in (pk, pv)), freq, start.to(DEV), torch.tensor(counts, dtype=torch.int32, device=DEV),
                            q=pq.to(DEV), q_weight=w.to(DEV), k_weight=w.to(DEV))
    assert exattn.check_device_error() == 0
    host = {x: getattr(cache, x).cpu() for x in ("k", "v", "k_scale", "v_scale")}
    y, size = plain_rope.norm_rotate(pk, freq.cpu(), start[:, None].long() + torch.arange(most), weight=w)
    want, _ = plain_rope.norm_rotate(pq, freq.cpu(), start[:, None].long() + torch.arange(most), weight=w)
    assert torch.all((r.double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * want.abs().amax(-1, keepdim=True))
    for b in range(B):
        c, s0 = counts[b], int(start[b])
        scales = torch.stack([host["k_scale"][int(table[b, (s0 + i) // page])] for i in range(c)], 1).double()[..., None]
        got = tokens(host, "k", table, b, lens[b])[:, s0:]
        step = 0.5 * scales.expand_as(got) if code == "int8" else torch.maximum(y[b, :, :c].abs() * 2.0 ** -4, scales * 2.0 ** -10)
        assert torch.all((got - y[b, :, :c]).abs() <= step * (1 + 2.0 ** -18) + 2.0 ** -18 * size[b, :, :c])
        # this sequence's path alone, as the last tokens of a plain sequence
        own = exattn.QuantCache(cache.k, cache.v, cache.k_scale, cache.v_scale, table[b : b + 1].to(DEV))
        o, lse = exattn.forward_cache(r[b : b + 1, :, :c].contiguous(), own, torch.tensor(lens[b : b + 1], dtype=torch.int32, device=DEV))
        check(r[b : b + 1, :, :c].cpu(), own, host, table[b : b + 1], lens[b : b + 1], torch.ones((1, c, c), dtype=torch.bool), got=(o, lse))
    assert counts[0] != counts[1]
