"""Rotary positions: the tests' plain form against differences, the frequencies, and what the C entry points refuse (no GPU)."""
import ctypes
import math

import pytest
import torch

import plain_rope
from exact_head_attention_gb300 import build, exattn

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation happens first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return exattn.load()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [False, True])
def test_plain_gradients_against_differences(layout, norm):
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn((2, 2, 3, 16), generator=g, dtype=torch.float64) for _ in range(2))
    w = 1 + 0.3 * torch.randn(16, generator=g, dtype=torch.float64) if norm else None
    freq, amplitude = exattn.rope_frequencies(8, device="cpu")[0], 1.3
    pos = plain_rope.positions(2, 3, torch.tensor([5, 70]))
    loss = lambda x, w: (plain_rope.norm_rotate(x, freq, pos, layout, amplitude, w)[0] * dy).sum()  # noqa: E731
    dx, dw, _, _ = plain_rope.gradients(dy, x, freq, pos, layout, amplitude, w)
    for i in (0, 17, 63, 100, 191):
        h = torch.zeros(x.numel(), dtype=torch.float64)
        h[i] = 1e-5
        h = h.reshape(x.shape)
        assert abs((loss(x + h, w) - loss(x - h, w)) / 2e-5 - dx.reshape(-1)[i]) < 1e-8
    if norm:
        for i in range(16):
            h = torch.zeros(16, dtype=torch.float64)
            h[i] = 1e-5
            assert abs((loss(x, w + h) - loss(x, w - h)) / 2e-5 - dw[i]) < 1e-8


def test_plain_angles():
    freq = torch.tensor([1.0, 0.25, -3.5], dtype=torch.float64)
    pos = torch.tensor([[0, 1, 1000]])
    t = pos[..., None] * freq
    got = plain_rope.angles(pos, freq)
    assert torch.all((got.cos() - t.cos()).abs() < 1e-12) and torch.all((got.sin() - t.sin()).abs() < 1e-12)


def test_frequencies():
    freq, amplitude = exattn.rope_frequencies(64, 10000.0, device="cpu")
    assert freq.dtype == torch.float64 and freq.shape == (32,) and amplitude == 1.0
    assert freq[0] == 1.0 and abs(freq[16] - 0.01) < 1e-15
    linear, _ = exattn.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(linear * 4, freq, rtol=1e-15, atol=0)
    ntk, _ = exattn.rope_frequencies(64, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == 1.0 and abs(ntk[-1] * 4 / freq[-1] - 1) < 1e-12
    yarn, a = exattn.rope_frequencies(64, scaling="yarn", factor=16.0, trained=4096, device="cpu")
    assert abs(a - (0.1 * math.log(16) + 1)) < 1e-15
    turns = 4096 * freq / (2 * math.pi)
    assert torch.equal(yarn[turns > 32], freq[turns > 32]) and torch.allclose(yarn[turns < 1] * 16, freq[turns < 1], rtol=1e-15, atol=0)
    between = (turns >= 1) & (turns <= 32)
    assert between.any() and torch.all(yarn[between] <= freq[between]) and torch.all(yarn[between] >= freq[between] / 16)
    for args in [(0,), (-2,), (7,), (64, -1.0)]:
        with pytest.raises(ValueError):
            exattn.rope_frequencies(*args, device="cpu")
    for kw in [dict(scaling="other"), dict(scaling="yarn"), dict(scaling="yarn", trained=10, fast=1.0), dict(factor=0.0)]:
        with pytest.raises(ValueError):
            exattn.rope_frequencies(64, device="cpu", **kw)


def _calls(lib, q=FAKE, k=FAKE, out=FAKE, dw=FAKE, ws=FAKE, ws_bytes=1 << 40, B=2, H=4, Hk=2, N=3, d=64, dtype=0, row=64, null=False, freq=FAKE,
           start=FAKE, offsets=FAKE, stride=3, qw=FAKE, kw=FAKE, rot=64, layout=0, amplitude=1.0, eps=1e-6):
    """Status of the forward and the backward with the given arguments."""
    st = exattn.Strides(8192, 2048, row)
    rope = None if null else ctypes.byref(exattn.RopeStruct(freq, start, offsets, stride, qw, kw, rot, layout, 0, amplitude, eps))
    vp = ctypes.c_void_p
    fwd = lib.attn_rope_fwd(vp(q), st, vp(k), st, vp(out), st, vp(out), st, B, H, Hk, N, d, rope, dtype, None)
    bwd = lib.attn_rope_bwd(vp(out), st, vp(out), st, vp(q), st, vp(k), st, vp(out), st, vp(out), st, vp(dw), vp(dw), B, H, Hk, N, d, rope,
                            dtype, vp(ws), ws_bytes, None)
    return {"fwd": fwd, "bwd": bwd}


@pytest.mark.parametrize("kw,calls,code", [
    (dict(B=0), "fwd bwd", 1), (dict(N=-1), "fwd bwd", 1), (dict(H=-1), "fwd bwd", 1), (dict(H=0, Hk=0), "fwd bwd", 1),
    (dict(H=65536), "fwd bwd", 1), (dict(B=2 ** 20, N=2 ** 11), "fwd bwd", 1), (dict(d=96), "fwd bwd", 2), (dict(dtype=2), "fwd bwd", 1),
    (dict(q=None), "fwd bwd", 1), (dict(k=None), "fwd bwd", 1), (dict(out=None), "fwd bwd", 1), (dict(dw=None), "bwd", 1),
    (dict(ws=None), "bwd", 6), (dict(ws=FAKE + 128), "bwd", 3), (dict(q=FAKE + 8), "fwd bwd", 3), (dict(out=FAKE + 2), "fwd bwd", 3),
    (dict(row=60), "fwd bwd", 1), (dict(row=68), "fwd bwd", 1), (dict(null=True), "fwd bwd", 1), (dict(freq=None), "fwd bwd", 1),
    (dict(freq=FAKE + 4), "fwd bwd", 3), (dict(start=FAKE + 2), "fwd bwd", 3), (dict(offsets=FAKE + 1), "fwd bwd", 3),
    (dict(stride=2), "fwd bwd", 1), (dict(stride=-3), "fwd bwd", 1), (dict(qw=FAKE + 8), "fwd bwd", 3), (dict(kw=FAKE + 4), "fwd bwd", 3),
    (dict(rot=-16), "fwd bwd", 1), (dict(rot=24), "fwd bwd", 1), (dict(rot=80), "fwd bwd", 1), (dict(layout=2), "fwd bwd", 1),
    (dict(amplitude=math.nan), "fwd bwd", 1), (dict(eps=0.0), "fwd bwd", 1), (dict(eps=-1.0), "fwd bwd", 1), (dict(eps=math.inf), "fwd bwd", 1),
], ids=str)
def test_rules(lib, kw, calls, code):
    got = _calls(lib, **kw)
    for name in calls.split():
        assert got[name] == code, (name, got)


@pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls with fake pointers must not reach a GPU")
@pytest.mark.parametrize("kw", [{}, dict(rot=0, freq=None), dict(H=0, q=None), dict(Hk=0, k=None), dict(stride=0), dict(qw=None, kw=None, eps=0.0),
                                dict(start=None, offsets=None)], ids=str)
def test_valid_calls_reach_the_device(lib, kw):
    assert set(_calls(lib, **kw).values()) <= {2, 4}  # no such device, or no driver


def test_workspace_size_of_other_heads(lib):
    assert exattn.rope_bwd_workspace_size(96) == 0


def _append(lib, cache, q=FAKE, out=FAKE, k=FAKE, v=FAKE, start=FAKE, count=None, B=2, H=4, N=3, dtype=0, row=64, null=False, **rope):
    st, vp = exattn.Strides(8192, 2048, row), ctypes.c_void_p
    f = dict(freq=FAKE, start=None, offsets=None, offset_stride=0, q_weight=FAKE, k_weight=FAKE, rotary_dim=64, layout=0, weight_fp32=0,
             amplitude=1.0, eps=1e-6)
    f.update(rope)
    r = None if null else ctypes.byref(exattn.RopeStruct(**f))
    return lib.attn_cache_append(None if cache is None else ctypes.byref(cache), vp(q), st, vp(out), st, vp(k), st, vp(v), st, vp(start),
                                 vp(count), B, H, N, r, dtype, None)


def _cache(**kw):
    f = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, page_table=FAKE, num_pages=10, heads=2, page_size=16, d=64, table_width=4, format=0)
    f.update(kw)
    return exattn.CacheStruct(**f)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(N=0), 1), (dict(H=-1), 1), (dict(H=65536), 1), (dict(dtype=2), 1), (dict(q=None), 1), (dict(out=None), 1),
    (dict(k=None), 1), (dict(v=None), 1), (dict(q=FAKE + 8), 3), (dict(out=FAKE + 4), 3), (dict(k=FAKE + 2), 3), (dict(start=FAKE + 2), 3),
    (dict(count=FAKE + 1), 3), (dict(row=60), 1), (dict(null=True), 1), (dict(freq=None), 1), (dict(rotary_dim=40), 1),
    (dict(rotary_dim=128), 1), (dict(layout=-1), 1), (dict(eps=0.0), 1), (dict(amplitude=math.inf), 1), (dict(k_weight=FAKE + 8), 3),
    (dict(offsets=FAKE, offset_stride=1), 1), (dict(B=2 ** 30), 1),
], ids=str)
def test_append_rules(lib, kw, code):
    assert _append(lib, _cache(), **kw) == code


def test_append_rules_of_the_cache(lib):
    assert _append(lib, None) == 1
    assert _append(lib, _cache(page_size=24)) == 1 and _append(lib, _cache(d=96)) == 2 and _append(lib, _cache(k=FAKE + 1)) == 3


@pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls with fake pointers must not reach a GPU")
@pytest.mark.parametrize("kw", [{}, dict(H=0, q=None, out=None), dict(rotary_dim=0, freq=None), dict(start=None), dict(k_weight=None, q_weight=None, eps=0.0)],
                         ids=str)
def test_valid_appends_reach_the_device(lib, kw):
    assert _append(lib, _cache(), **kw) in (2, 4)


@pytest.mark.parametrize("kw,code", [
    (dict(tree=None), 1), (dict(Nq=513), 1), (dict(Nq=0), 1), (dict(tree=FAKE + 2), 3), (dict(stride=39), 1), (dict(stride=-40), 1),
    (dict(scale=0.0), 1), (dict(ws=None), 6), (dict(ws=FAKE + 128), 3), (dict(lens=None), 1), (dict(H=3), 1), (dict(q=None), 1),
    (dict(dtype=5), 1),
], ids=str)
def test_tree_rules(lib, kw, code):
    f = dict(q=FAKE, tree=FAKE, stride=40, lens=FAKE, H=4, Nq=40, scale=0.1, dtype=0, ws=FAKE)
    f.update(kw)
    st, vp = exattn.Strides(8192, 4096, 64), ctypes.c_void_p
    if "stride" not in kw:
        f["stride"] = 80
    got = lib.attn_fwd_cache_tree(vp(f["q"]), st, ctypes.byref(_cache()), vp(f["lens"]), vp(f["tree"]), f["stride"], vp(FAKE), st, vp(FAKE), 2,
                                  f["H"], f["Nq"], f["scale"], f["dtype"], vp(f["ws"]), 1 << 40, None)
    assert got == code


@pytest.mark.parametrize("args,code", [((None, FAKE, FAKE, 1, 4), 1), ((FAKE, None, FAKE, 1, 4), 1), ((FAKE, FAKE, None, 1, 4), 1), ((FAKE, FAKE, FAKE, 0, 4), 1),
                                       ((FAKE, FAKE, FAKE, 1, 0), 1), ((FAKE, FAKE, FAKE, 1, 513), 1), ((FAKE + 2, FAKE, FAKE, 1, 4), 3),
                                       ((FAKE, FAKE + 1, FAKE, 1, 4), 3), ((FAKE, FAKE, FAKE + 2, 1, 4), 3)], ids=str)
def test_draft_tree_rules(lib, args, code):
    assert lib.attn_draft_tree(*map(ctypes.c_void_p, args[:3]), *args[3:], None) == code


def test_tree_status(lib):
    assert exattn.STATUS_NAMES[9] == "ATTN_ERR_TREE" and "parent" in exattn.status_string(9)


def test_binding_refuses_what_it_cannot_pass_on(lib):
    """On the CPU, before any device is touched."""
    q = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    freq = exattn.rope_frequencies(64, device="cpu")[0]
    for call in (lambda: exattn.rope_forward(q, q, freq), lambda: exattn.rope_forward(None, None, freq), lambda: exattn.rope_forward(q, q, freq, layout="x"),
                 lambda: exattn.rope_backward(q, None, None, None, freq), lambda: exattn.draft_tree(torch.zeros((1, 3), dtype=torch.int32)),
                 lambda: exattn.rope_forward(q, None, freq, out=(None, None))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: exattn.rope_forward(3, q, freq), lambda: exattn.draft_tree(None), lambda: exattn.rope_forward(q, q, freq, amplitude="x")):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_a_stream_of_another_device_is_refused(lib):
    """On the CPU: the tensors' device is compared with the stream's before either is touched."""
    class Stream:
        device = torch.device("cuda", 7)

    class Cache:
        device = torch.device("cuda", 0)
        address = index = B = 0

    q, freq = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16), None
    for call in (lambda s: exattn.rope_forward(q, None, freq, stream=s), lambda s: exattn.rope_forward(None, q, freq, stream=s),
                 lambda s: exattn.rope_backward(q, None, q, None, freq, stream=s), lambda s: exattn.draft_tree(q, stream=s),
                 lambda s: exattn.cache_append(Cache(), q, q, freq, stream=s),
                 lambda s: exattn.forward_cache_tree(q, Cache(), None, None, stream=s)):
        with pytest.raises(ValueError, match="another device"):
            call(Stream())
