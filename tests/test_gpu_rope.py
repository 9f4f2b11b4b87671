"""Rotary positions with norms per head, and their gradients, on the GPU.

Every result is compared with the definition in 64 bits on the CPU (plain_rope).  Tolerances, from the roundings that the
operators make; e = 2^-24 is half an fp32 step, relative:
  norm      the sum of d squares, none negative, 16 products and up to 4 joins deep: 21 e, half of it through the root; the
            reciprocal root 2 steps (4 e), eps and the mean 2 e, halved too, two products 2 e: 17.5 e, under 2^-19.8 of y
  angle     2^-32 turns cut off (2^-29.3), half an fp32 step at up to an eighth of a turn (2^-25.3), sine and cosine within
            1e-7, the amplitude and the pair's two products and sum 4 e: 3.7e-7, under 2^-21.3 of |a| + |b|
  together  under 2^-19 of the size that plain_rope gives, and half a step of the output
  gradients the turned gradient as above, r as above (twice), and the mean of d products, 21 e of their absolute sum:
            under 2^-17.5 of the size, and half a step
  dw        the terms as above, and a sum of `rows` of them in fp32, no more than rows additions deep: under
            (2^-17.5 + rows e) of the sum of absolute terms, and half a step of the weights' type
Half a step of fp16 below 2^-14 is 2^-25.
"""
import math

import pytest
import torch

import plain_rope
from exact_head_attention_gb300 import exattn

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _normal(shape, seed, dtype):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _gpu(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def half_step(ref, dtype):
    small = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134
    return (ref.abs() * torch.finfo(dtype).eps / 2).clamp(min=small)


def check(got, ref, size, factor):
    tol = half_step(ref, got.dtype) + factor * size
    err = (got.double().cpu() - ref).abs()
    assert torch.all(err <= tol), (err / tol).max()


def make(B, H, Hk, N, d, rot, dtype, norm, wide, seed=0, start=True, offsets=False):
    t = TYPES[dtype]
    q, k = (_normal((B, h, N, d), seed + i, t) if h else None for i, h in enumerate((H, Hk)))
    w = [1 + 0.3 * _normal((d,), seed + 2 + i, torch.float32) if norm else None for i in range(2)]
    w = [x if x is None or wide else x.to(t) for x in w]
    freq = exattn.rope_frequencies(rot, device="cpu")[0] if rot else None
    g = torch.Generator().manual_seed(seed + 9)
    st = torch.randint(0, 5000, (B,), generator=g).to(torch.int32) if start else None
    of = torch.randint(0, 300, (B, N), generator=g).to(torch.int32) if offsets else None
    return q, k, w[0], w[1], freq, st, of


def check_forward(q, k, wq, wk, freq, start, offsets, layout="half", amplitude=1.0, out=None, **kw):
    x = k if q is None else q
    gq, gk = out if out is not None else exattn.rope_forward(*_gpu(q, k, freq, start, offsets), layout, amplitude, *_gpu(wq, wk), **kw)
    pos = plain_rope.positions(x.shape[0], x.shape[2], start, offsets)
    for x, w, got in ((q, wq, gq), (k, wk, gk)):
        if x is not None:
            check(got, *plain_rope.norm_rotate(x, freq, pos, layout, amplitude, w), 2.0 ** -19)
        else:
            assert got is None


def check_backward(q, k, wq, wk, freq, start, offsets, layout="half", amplitude=1.0, seed=50):
    x = k if q is None else q
    dq, dk = (None if t is None else _normal(t.shape, seed + i, t.dtype) for i, t in enumerate((q, k)))
    got = exattn.rope_backward(*_gpu(dq, dk, q if wq is not None else None, k if wk is not None else None, freq, start, offsets), layout, amplitude, *_gpu(wq, wk))
    pos = plain_rope.positions(x.shape[0], x.shape[2], start, offsets)
    for x, dy, w, gx, gw in ((q, dq, wq, got[0], got[2]), (k, dk, wk, got[1], got[3])):
        if x is None:
            assert gx is None
            continue
        dx, dw, sx, sw = plain_rope.gradients(dy, x, freq, pos, layout, amplitude, w)
        check(gx, dx, sx, 2.0 ** -17.5)
        if w is None:
            assert gw is None
        else:
            rows = x.shape[0] * x.shape[1] * x.shape[2]
            check(gw, dw, sw, 2.0 ** -17.5 + rows * 2.0 ** -24)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm,wide", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (64, 0), (128, 128), (128, 64), (128, 16), (128, 112), (128, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_layouts(d, rot, norm, wide, layout, dtype):
    x = make(2, 5, 2, 37, d, rot, dtype, norm, wide)
    check_forward(*x, layout, 1.25)
    check_backward(*x, layout, 1.25)


@pytest.mark.parametrize("B,H,Hk,N", [(1, 1, 1, 1), (1, 1, 0, 1), (1, 0, 3, 2), (64, 8, 1, 1), (3, 7, 5, 31), (1, 33, 2, 33), (2, 1, 1, 1000),
                                      (1, 12, 12, 2049), (5, 64, 8, 129), (600, 3, 1, 3)], ids=str)
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_sizes(B, H, Hk, N, norm, d):
    x = make(B, H, Hk, N, d, d // 2, "bf16", norm, True, seed=3, offsets=B * N > 60)
    check_forward(*x)
    check_backward(*x)


@pytest.mark.parametrize("which", ["q", "k"])
def test_norm_of_one_tensor(which):
    q, k, wq, wk, *rest = make(2, 6, 3, 50, 128, 128, "bf16", True, False, seed=4)
    x = (q, k, wq if which == "q" else None, wk if which == "k" else None, *rest)
    check_forward(*x)
    check_backward(*x)


def test_positions():
    q, k, wq, wk, freq, start, offsets = make(3, 2, 2, 40, 64, 64, "fp16", False, False, seed=5, offsets=True)
    for st in (None, start):
        for of in (None, offsets, offsets[:1], offsets[0]):
            check_forward(q, k, wq, wk, freq, st, of)
    wide = torch.zeros((3, 77), dtype=torch.int32)
    wide[:, 5:45] = offsets
    got = exattn.rope_forward(*_gpu(q, k, freq, start), wide.to(DEV)[:, 5:45])
    check_forward(q, k, wq, wk, freq, start, offsets, out=got)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_and_negative_positions(layout):
    """Up to the largest sums of two 32-bit positions, where an angle in fp32 (or p f in 64 bits) has no digit left."""
    q, k, wq, wk, freq, _, _ = make(4, 2, 1, 8, 64, 64, "bf16", False, False, seed=6)
    freq = torch.cat((freq[:-2], torch.tensor([-0.37, 900.25])))
    start = torch.tensor([2 ** 31 - 1, -(2 ** 31), 1_000_003, -5], dtype=torch.int32)
    offsets = torch.tensor([0, 1, 2, 2 ** 31 - 1, 2 ** 20, -(2 ** 31), 77, 123_456_789], dtype=torch.int32)
    check_forward(q, k, wq, wk, freq.double(), start, offsets, layout)
    check_backward(q, k, wq, wk, freq.double(), start, offsets, layout)


def test_frequencies_of_any_size():
    q, k, wq, wk, _, start, _ = make(2, 1, 1, 9, 64, 64, "fp16", False, False, seed=7)
    freq = torch.tensor([0.0, -0.0, 5e-324, 1e-300, 1e-18, 2.0 ** -40, 1e-3, -1.0, math.pi, 2 * math.pi, 6.5, 1e4, 2.0 ** 30] + [0.1] * 19,
                        dtype=torch.float64)
    check_forward(q, k, wq, wk, freq, start, None)


def test_special_values_stay_in_their_pair():
    """An infinity or NaN reaches its pair only where there is no norm, and its row where there is; a frequency that is not
    finite its pairs."""
    for layout in ("half", "interleaved"):
        q, k, wq, wk, freq, start, _ = make(1, 3, 1, 5, 128, 64, "bf16", True, True, seed=8)
        q[0, 1, 2, 100] = math.nan  # behind the rotated part
        q[0, 2, 3, 3] = math.inf
        plain = exattn.rope_forward(*_gpu(q, k, freq, start), layout=layout)[0].cpu()
        bad = torch.zeros(q.shape, dtype=torch.bool)
        bad[0, 1, 2, 100] = bad[0, 2, 3, 3] = bad[0, 2, 3, 35 if layout == "half" else 2] = True
        assert torch.equal(~torch.isfinite(plain), bad)
        normed = exattn.rope_forward(*_gpu(q, k, freq, start), layout=layout, q_weight=wq.to(DEV))[0].cpu()
        assert torch.isnan(normed[0, 1, 2]).all() and torch.isfinite(normed[0, 0]).all() and torch.isfinite(normed[0, 1, :2]).all()
        freq[4] = math.inf
        got = exattn.rope_forward(*_gpu(None, k, freq, start), layout=layout)[1].cpu()
        pair = [4, 36] if layout == "half" else [8, 9]
        assert torch.isnan(got[..., pair]).all()
        pair = [i for i in range(128) if i not in pair]
        assert torch.isfinite(got[..., pair]).all()


def test_small_and_large_rows():
    """Rows of zeros, rows where eps counts, and rows far from 1."""
    q, k, wq, wk, freq, start, _ = make(1, 6, 1, 4, 64, 64, "bf16", True, True, seed=9)
    q[0, 0] = 0
    for h, f in enumerate((1e-3, 1e-6, 1e10, 1e-20, 30.0)):
        q[0, 1 + h] = (q[0, 1 + h].float() * f).to(q.dtype)
    check_forward(q, k, wq, wk, freq, start, None)
    check_backward(q, k, wq, wk, freq, start, None)
    got = exattn.rope_forward(*_gpu(q, k, freq, start), q_weight=wq.to(DEV))[0].cpu()
    assert torch.all(got[0, 0] == 0)


def test_views_and_in_place():
    """Heads and rows of wider buffers, as a joint projection leaves them; written back in place, the rest left as it was."""
    B, N, d = 2, 21, 64
    for norm in (False, True):
        _, _, wq, wk, freq, start, _ = make(B, 1, 1, N, d, d, "bf16", norm, False, seed=10)
        joint = _normal((B, N, 11, d + 8), 11, torch.bfloat16)
        gpu = joint.to(DEV)
        at = lambda t: (t[:, :, 1:7, :d].transpose(1, 2), t[:, :, 7:9, :d].transpose(1, 2))  # noqa: E731
        q, k = at(joint)
        out = exattn.rope_forward(*at(gpu), freq.to(DEV), start.to(DEV), **dict(zip(("q_weight", "k_weight"), _gpu(wq, wk))))
        check_forward(q, k, wq, wk, freq, start, None, out=out)
        exattn.rope_forward(*at(gpu), freq.to(DEV), start.to(DEV), out=at(gpu), **dict(zip(("q_weight", "k_weight"), _gpu(wq, wk))))
        assert torch.equal(at(gpu)[0], out[0]) and torch.equal(at(gpu)[1], out[1])
        rest = gpu.cpu()
        for t in at(rest):
            t.zero_()
        for t in at(joint):
            t.zero_()
        assert torch.equal(rest, joint)


def test_gradients_in_place_of_the_outputs():
    q, k, wq, wk, freq, start, _ = make(2, 3, 2, 70, 64, 32, "bf16", True, False, seed=12)
    dq, dk = _normal(q.shape, 60, q.dtype), _normal(k.shape, 61, q.dtype)
    want = exattn.rope_backward(*_gpu(dq, dk, q, k, freq, start), q_weight=wq.to(DEV), k_weight=wk.to(DEV))
    lib, gd, st = exattn.load(), _gpu(dq, dk, q, k, freq, start, wq, wk), lambda t: exattn.Strides(*t.stride()[:3])
    rope = exattn.RopeStruct(gd[4].data_ptr(), gd[5].data_ptr(), None, 0, gd[6].data_ptr(), gd[7].data_ptr(), 32, 0, 0, 1.0, 1e-6)
    dw = torch.empty((2, 64), dtype=q.dtype, device=DEV)
    ws = torch.full((exattn.rope_bwd_workspace_size(64),), 255, dtype=torch.uint8, device=DEV)
    views = [x for t in (gd[0], gd[1], gd[2], gd[3], gd[0], gd[1]) for x in (t.data_ptr(), st(t))]
    assert lib.attn_rope_bwd(*views, dw[0].data_ptr(), dw[1].data_ptr(), 2, 3, 2, 70, 64, rope, 0, ws.data_ptr(), ws.numel(),
                             exattn._stream(None)) == 0
    for a, b in zip((gd[0], gd[1], dw[0], dw[1]), want):
        assert torch.equal(a, b)


def test_autograd_and_attention():
    """A training step's path, rope into attention and back, against the gradients of its steps; leaves that need none."""
    B, H, N, d = 2, 4, 130, 64
    q, k, wq, wk, freq, start, _ = make(B, H, H, N, d, d, "bf16", True, True, seed=13)
    leaves = [t.to(DEV).requires_grad_() for t in (q, k, wq, wk)]
    v = _normal((B, H, N, d), 14, torch.bfloat16).to(DEV).requires_grad_()
    rq, rk = exattn.rope(leaves[0], leaves[1], freq.to(DEV), start.to(DEV), q_weight=leaves[2], k_weight=leaves[3])
    o = exattn.attention(rq, rk, v, causal=True, dq_mode="deterministic")
    do = _normal(o.shape, 15, torch.bfloat16).to(DEV)
    got = torch.autograd.grad(o, [*leaves, v], do)
    o2, lse = exattn.forward(rq.detach(), rk.detach(), v.detach(), True)
    dq, dk, dv = exattn.backward(rq.detach(), rk.detach(), v.detach(), o2, do, lse, True, dq_mode="deterministic")
    want = exattn.rope_backward(dq, dk, *_gpu(q, k, freq, start), q_weight=wq.to(DEV), k_weight=wk.to(DEV))
    for a, b in zip(got, [*want, dv]):
        assert torch.equal(a, b)
    pos = plain_rope.positions(B, N, start)
    for x, dy, w, gx, gw in ((q, dq, wq, got[0], got[2]), (k, dk, wk, got[1], got[3])):
        dx, dw, sx, sw = plain_rope.gradients(dy.cpu(), x, freq, pos, weight=w)
        check(gx, dx, sx, 2.0 ** -17.5)
        check(gw, dw, sw, 2.0 ** -17.5 + B * H * N * 2.0 ** -24)
    # an expanded gradient, and one output left unused
    rq, rk = exattn.rope(leaves[0], leaves[1], freq.to(DEV), start.to(DEV))
    g, = torch.autograd.grad(rq.float().sum(), [leaves[0]])
    dx, _, sx, _ = plain_rope.gradients(torch.ones_like(q), q, freq, pos)
    check(g, dx, sx, 2.0 ** -17.5)


def test_same_bits_and_a_dirty_workspace():
    q, k, wq, wk, freq, start, _ = make(3, 9, 3, 700, 128, 128, "bf16", True, True, seed=16)
    args = _gpu(_normal(q.shape, 70, q.dtype), _normal(k.shape, 71, q.dtype), q, k, freq, start)
    kw = dict(q_weight=wq.to(DEV), k_weight=wk.to(DEV))
    first = exattn.rope_backward(*args, **kw)
    for fill in (0, 255):
        ws = torch.full((exattn.rope_bwd_workspace_size(128),), fill, dtype=torch.uint8, device=DEV)
        for a, b in zip(first, exattn.rope_backward(*args, workspace=ws, **kw)):
            assert torch.equal(a, b)


def test_streams_and_graphs():
    """A side stream behind a busy default stream, and a captured training step replayed on new inputs."""
    q, k, wq, wk, freq, start, _ = make(2, 4, 2, 300, 64, 64, "fp16", True, False, seed=17)
    gq, gk, gf, gs, gwq, gwk = _gpu(q, k, freq, start, wq, wk)
    dq, dk = _gpu(_normal(q.shape, 80, q.dtype), _normal(k.shape, 81, k.dtype))
    want = [*exattn.rope_forward(gq, gk, gf, gs, q_weight=gwq, k_weight=gwk),
            *exattn.rope_backward(dq, dk, gq, gk, gf, gs, q_weight=gwq, k_weight=gwk)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [*exattn.rope_forward(gq, gk, gf, gs, q_weight=gwq, k_weight=gwk, stream=side),
           *exattn.rope_backward(dq, dk, gq, gk, gf, gs, q_weight=gwq, k_weight=gwk, stream=side)]
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    xq, xk = torch.zeros_like(gq), torch.zeros_like(gk)
    pos = torch.zeros_like(gs)
    with torch.cuda.graph(graph):
        got = [*exattn.rope_forward(xq, xk, gf, pos, q_weight=gwq, k_weight=gwk),
               *exattn.rope_backward(dq, dk, xq, xk, gf, pos, q_weight=gwq, k_weight=gwk)]
    for _ in range(2):
        xq.copy_(gq)
        xk.copy_(gk)
        pos.copy_(gs)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for t in got:
            t.fill_(math.nan)


def test_empty_batches():
    freq = exattn.rope_frequencies(64)[0]
    w = torch.ones(64, device=DEV)
    for shape in ((0, 2, 3, 64), (2, 2, 0, 64), (2, 0, 3, 64)):
        q = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
        a, b = exattn.rope_forward(q, q, freq, q_weight=w, k_weight=w)
        assert a.shape == shape and b.shape == shape
        a, b, dwq, dwk = exattn.rope_backward(q, q, q, q, freq, q_weight=w, k_weight=w)
        assert a.shape == shape and torch.all(dwq == 0) and torch.all(dwk == 0)


def test_rows_beyond_32_bits():
    """Offsets of the rows of a wide buffer pass 2^31 elements; a few of them are compared."""
    N, d, stride = 70_000, 64, 40_960
    big = torch.empty(N * stride, dtype=torch.bfloat16, device=DEV)
    x = big.as_strided((1, 2, N, d), (0, 128, stride, 1))
    x.copy_(torch.randn((1, 2, N, d), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV))
    freq = exattn.rope_frequencies(64)[0]
    got, _ = exattn.rope_forward(x, None, freq)
    back, _, _, _ = exattn.rope_backward(got, None, None, None, freq)
    rows = torch.tensor([0, 1, 52_428, 52_429, N - 1])
    ref, size = plain_rope.norm_rotate(x[:, :, rows.to(DEV)].cpu(), freq.cpu(), rows[None])
    check(got[:, :, rows.to(DEV)].cpu(), ref, size, 2.0 ** -19)
    # turned back: one rounding of the pair more, at most two half steps of it together
    err = (back.float() - x.float()).abs()
    assert torch.all(err <= 2.0 ** -8 * (x.float().abs() + 2.0 ** 0.5 * (x[..., :32].float().square() + x[..., 32:].float().square()).sqrt().repeat(1, 1, 1, 2)) * 1.01)


def test_refused_tensors():
    q = torch.zeros((2, 4, 8, 64), dtype=torch.bfloat16, device=DEV)
    freq = exattn.rope_frequencies(64)[0]
    start = torch.zeros(2, dtype=torch.int32, device=DEV)
    w = torch.ones(64, device=DEV)
    for args, kw in [((q, q.half(), freq), {}), ((q, q[:1], freq), {}), ((q, q[:, :, :4], freq), {}), ((q.cpu(), None, freq), {}),
                     ((q, q, freq.float()), {}), ((q, q, freq.cpu()), {}), ((q, q, freq[::2]), {}), ((None, None, freq), {}),
                     ((q, q, freq, start.long()), {}), ((q, q, freq, start[:1]), {}), ((q, q, freq, start, start), {}),
                     ((q, q, freq), dict(layout="other")), ((q, q, freq), dict(q_weight=w[:32])), ((q, q, freq), dict(q_weight=w.double())),
                     ((q.transpose(2, 3), None, freq), {}), ((q, q, freq), dict(out=(q, None))), ((q, q, freq), dict(out=(q, q.half())))]:
        with pytest.raises(ValueError):
            exattn.rope_forward(*args, **kw)
    with pytest.raises(TypeError):
        exattn.rope_forward(q.float(), None, freq)
    with pytest.raises(TypeError):
        exattn.rope_forward(q, q, freq, q_weight=w, k_weight=w.to(torch.bfloat16))
    for args, kw in [((q, q, freq[:20].contiguous()), {}), ((q, q, torch.cat((freq, freq))), {}), ((q[..., :8], None, freq[:4].contiguous()), {}),
                     ((q, q, freq), dict(q_weight=w, eps=0.0)), ((q, q, freq), dict(amplitude=math.inf))]:
        with pytest.raises(exattn.AttnError):
            exattn.rope_forward(*args, **kw)
    with pytest.raises(ValueError):
        exattn.rope_backward(q, q, None, q, freq, q_weight=w)
    with pytest.raises(exattn.AttnError):
        exattn.rope_backward(q, q, q, q, freq, q_weight=w, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))


def test_workspaces_of_graphs_in_turn():
    """One workspace for two graphs' calls in turn and an eager one between, its contents overwritten now and then."""
    q, k, wq, wk, freq, start, _ = make(2, 4, 2, 500, 64, 64, "bf16", True, True, seed=18)
    ws = torch.full((exattn.rope_bwd_workspace_size(64),), 255, dtype=torch.uint8, device=DEV)
    sets = []
    for seed in (90, 92):
        args = _gpu(_normal(q.shape, seed, q.dtype), _normal(k.shape, seed + 1, q.dtype), q, k, freq, start)
        kw = dict(q_weight=wq.to(DEV), k_weight=wk.to(DEV), workspace=ws)
        want = exattn.rope_backward(*args, **kw)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = exattn.rope_backward(*args, **kw)
        sets.append((graph, got, want, args, kw))
    for turn in range(3):
        for graph, got, want, args, kw in sets:
            for t in got:
                t.fill_(math.nan)
            graph.replay()
            if turn == 1:
                ws.random_(0, 256)
            again = exattn.rope_backward(*args, **kw)
            for a, b, c in zip(got, want, again):
                assert torch.equal(a, b) and torch.equal(c, b)


@pytest.mark.parametrize("N", [600, 4000])
def test_sums_of_few_and_of_many_blocks(N):
    """The weights' gradients where the last block adds them up and where a launch of its own does, on a dirty workspace."""
    q, k, wq, wk, freq, start, _ = make(4, 4, 4, N, 64, 64, "bf16", True, True, seed=19)
    check_backward(q, k, wq, wk, freq, start, None)
    args = _gpu(_normal(q.shape, 94, q.dtype), _normal(k.shape, 95, q.dtype), q, k, freq, start)
    kw = dict(q_weight=wq.to(DEV), k_weight=wk.to(DEV))
    want = exattn.rope_backward(*args, **kw)
    ws = torch.full((exattn.rope_bwd_workspace_size(64),), 0x5A, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        for a, b in zip(exattn.rope_backward(*args, workspace=ws, **kw), want):
            assert torch.equal(a, b)


def test_captured_training_step():
    """Norms, rotation, attention and all gradients in one graph, replayed on new inputs, against the eager step."""
    B, H, N, d = 1, 3, 200, 64
    q, k, wq, wk, freq, start, _ = make(B, H, H, N, d, d, "bf16", True, True, seed=20)
    v, do = _normal((B, H, N, d), 21, torch.bfloat16), _normal((B, H, N, d), 22, torch.bfloat16)
    gf, gs, gdo = _gpu(freq, start, do)

    def step(q, k, v, wq, wk):
        rq, rk = exattn.rope(q, k, gf, gs, layout="interleaved", q_weight=wq, k_weight=wk)
        o = exattn.attention(rq, rk, v, causal=True, dq_mode="deterministic")
        return (o.detach(), *torch.autograd.grad(o, (q, k, v, wq, wk), gdo))

    leaves = [t.to(DEV).requires_grad_() for t in (q, k, v, wq, wk)]
    held = [torch.zeros_like(t).requires_grad_() for t in leaves]
    want = step(*leaves)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*held)
    for _ in range(2):
        with torch.no_grad():
            for a, b in zip(held, leaves):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for t in got:
            t.fill_(math.nan)


@pytest.mark.parametrize("which", [0, 1, 2, 3])
def test_capture_beside_a_living_graph_is_refused(which):
    """A leaf whose gradients an autograd graph recorded outside the capture adds up; once that graph is gone the call is taken."""
    q, k, wq, wk, freq, start, _ = make(1, 2, 2, 16, 64, 64, "bf16", True, True, seed=24)
    gf, gs = _gpu(freq, start)
    leaves = [t.to(DEV).requires_grad_(i == which) for i, t in enumerate((q, k, wq, wk))]

    def turned():
        return exattn.rope(leaves[0], leaves[1], gf, gs, q_weight=leaves[2], k_weight=leaves[3])

    living = turned()
    want = [t.detach().clone() for t in living]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="outside"):
        with torch.cuda.graph(graph):
            leaves[0].detach().clone()
            turned()
    del living
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [t.detach() for t in turned()]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


LARGE = [1.9999, 2.0, 3.999999, 4.0, 4.0000001, 8.1, 1e4 + 0.1, 1e6 + 0.3, -1e6 - 0.7, 2.0 ** 30 * 1.2346, -(2.0 ** 40) * 1.7, 2.0 ** 52 + 1,
         2.0 ** 53 * 1.1, 2.0 ** 62 * 1.99, -(2.0 ** 63 - 1024), 2.0 ** 60]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_large_frequencies_at_far_positions(layout):
    """A frequency's turns are within two units of 2^-64 whatever its size, so that an angle at the farthest position, 2^32, is off
    by 2^-31 turns of it: under a hundredth of the angle's other errors.  From 2^63 on a frequency makes its pairs NaN."""
    q, k, wq, wk, _, _, _ = make(4, 2, 1, 8, 64, 64, "bf16", False, False, seed=25)
    freq = torch.tensor(LARGE + [0.1] * 16, dtype=torch.float64)
    start = torch.tensor([2 ** 31 - 1, -(2 ** 31), 1_000_003, -5], dtype=torch.int32)
    offsets = torch.tensor([0, 1, 2, 2 ** 31 - 1, 2 ** 20, -(2 ** 31), 77, 123_456_789], dtype=torch.int32)
    check_forward(q, k, wq, wk, freq, start, offsets, layout)
    check_backward(q, k, wq, wk, freq, start, offsets, layout)
    freq[16:20] = torch.tensor([2.0 ** 63, -1e300, math.inf, math.nan], dtype=torch.float64)
    got = exattn.rope_forward(*_gpu(None, k, freq, start, offsets), layout=layout)[1].cpu()
    bad = [*range(16, 20), *range(48, 52)] if layout == "half" else range(32, 40)
    assert torch.isnan(got[..., bad]).all() and torch.isfinite(got[..., [i for i in range(64) if i not in bad]]).all()


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_capture_without_gradients_beside_a_living_graph(off):
    """Weights whose last loss is still held: a capture that records nothing joins nothing."""
    q, k, wq, wk, freq, start, _ = make(1, 2, 2, 16, 64, 64, "bf16", True, True, seed=26)
    gq, gk, gf, gs, gwq, gwk = _gpu(q, k, freq, start, wq, wk)
    for w in (gwq, gwk):
        w.requires_grad_()
    living = exattn.rope(gq, gk, gf, gs, q_weight=gwq, k_weight=gwk)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with off(), torch.cuda.graph(graph):
        got = exattn.rope(gq, gk, gf, gs, q_weight=gwq, k_weight=gwk)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and not a.requires_grad for a, b in zip(got, living))
    assert all(torch.isfinite(g).all() for g in torch.autograd.grad(sum(t.float().sum() for t in living), (gwq, gwk)))


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("squared", [False, True])
def test_second_gradients_raise(norm, squared):
    """A penalty on gradients, beside another term that has its own: raised, not left out.  Where the gradients depend on nothing
    that needs any (no norm, a loss that is linear) there is nothing to leave out."""
    q, k, wq, wk, freq, start, _ = make(1, 2, 2, 16, 64, 64, "bf16", norm, True, seed=27)
    gf, gs = _gpu(freq, start)
    leaves = [t if t is None else t.to(DEV).requires_grad_() for t in (q, k, wq, wk)]
    wanted = [t for t in leaves if t is not None]

    def loss():
        out = exattn.rope(leaves[0], leaves[1], gf, gs, q_weight=leaves[2], k_weight=leaves[3])
        return sum((t.float().square() if squared else t.float()).sum() for t in out)

    first = torch.autograd.grad(loss(), wanted, create_graph=True)
    for a, b in zip(first, torch.autograd.grad(loss(), wanted)):
        assert torch.equal(a, b)
    penalty = sum(g.float().square().sum() for g in first) + wanted[0].float().square().sum()
    if norm or squared:
        with pytest.raises(RuntimeError, match="once"):
            penalty.backward()
    else:
        assert not first[0].requires_grad
        penalty.backward()
        assert torch.equal(wanted[0].grad, 2 * wanted[0].detach())


@pytest.mark.parametrize("norm,needs", [(n, x) for n in (False, True) for x in [(1, 0, 0, 0), (0, 1, 0, 0), (1, 0, 1, 0), (1, 1, 0, 0), (0, 1, 1, 0)]]
                         + [(True, (0, 0, 1, 0)), (True, (0, 0, 0, 1))], ids=str)
def test_gradients_of_some_inputs(norm, needs, monkeypatch):
    """Inputs and weights that need none: the tensor without is neither kept nor computed, the others' gradients stay as they are."""
    q, k, wq, wk, freq, start, _ = make(2, 4, 2, 50, 64, 64, "bf16", norm, True, seed=28)
    gf, gs = _gpu(freq, start)
    leaves = [t if t is None else t.to(DEV) for t in (q, k, wq, wk)]
    dy = _gpu(_normal(q.shape, 90, q.dtype), _normal(k.shape, 91, k.dtype))
    want = exattn.rope_backward(*dy, *leaves[:2], gf, gs, q_weight=leaves[2], k_weight=leaves[3])
    wanted = [i for i in range(4) if needs[i] and leaves[i] is not None]
    for i in wanted:
        leaves[i].requires_grad_()
    calls, plain = [], exattn.rope_backward
    monkeypatch.setattr(exattn, "rope_backward", lambda *a, **kw: calls.append(a) or plain(*a, **kw))
    out = exattn.rope(leaves[0], leaves[1], gf, gs, q_weight=leaves[2], k_weight=leaves[3])
    for i, g in zip(wanted, torch.autograd.grad(out, [leaves[i] for i in wanted], dy)):
        assert torch.equal(g, want[i])
    (args,) = calls
    for side in range(2):
        some = side in wanted or side + 2 in wanted
        assert (args[side] is not None) == some and (args[2 + side] is not None) == (some and norm)


def test_gradients_of_weights_without_their_tensor():
    q, _, wq, wk, freq, start, _ = make(1, 2, 2, 16, 64, 64, "bf16", True, True, seed=29)
    gq, gf, gs, gwq, gwk = _gpu(q, freq, start, wq, wk)
    for w in (gwq, gwk):
        w.requires_grad_()
    out, none = exattn.rope(gq, None, gf, gs, q_weight=gwq, k_weight=gwk)
    assert none is None
    a, b = torch.autograd.grad(out.float().sum(), (gwq, gwk))
    assert torch.any(a != 0) and torch.all(b == 0)
    out, _ = exattn.rope(gq, None, gf, gs, k_weight=gwk)
    assert torch.all(torch.autograd.grad(out.float().sum(), gwk)[0] == 0)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d", [64, 128])
def test_norms_of_very_small_rows_and_very_large_weights(layout, d):
    """Rows below 2^-126, whose norm eps makes: their products with weights and cosines would lose digits before it.  And weights
    that would bring a row of 1e15 beyond fp32 before it."""
    q, k, wq, wk, freq, start, _ = make(2, 3, 2, 21, d, d, "bf16", True, True, seed=30)
    q = (q.float() * torch.tensor([1e-38, 1e-39, 1e-40])[None, :, None, None]).to(q.dtype)
    k = (k.float() * 1e15).to(k.dtype)
    check_forward(q, k, wq, wk * 1e25, freq, start, None, layout, out=exattn.rope_forward(
        *_gpu(q, k, freq, start), layout=layout, q_weight=wq.to(DEV), k_weight=(wk * 1e25).to(DEV)))
    pos = plain_rope.positions(2, 21, start)
    got, _ = exattn.rope_forward(*_gpu(q, None, freq, start), layout=layout, q_weight=wq.to(DEV), eps=1e-12)
    check(got, *plain_rope.norm_rotate(q, freq, pos, layout, weight=wq, eps=1e-12), 2.0 ** -19)
