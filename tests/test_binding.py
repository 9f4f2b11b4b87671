"""The 8-bit cache without the compiled binding, and the binding's own conditions: a copy of the package in a process of its own."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

from exact_head_attention_gb300 import build

REFUSALS = """
k = torch.zeros((4, 2, 16, 64), dtype=torch.int8, device=dev)
s = torch.zeros((4, 2), device=dev)
t = torch.zeros((1, 2), dtype=torch.int32, device=dev)
for args in [(k.float(), k, s, s, t), (k, k.view(torch.float8_e4m3fn), s, s, t), (k, k, s.double(), s, t), (k, k, s, s, t.long()),
             (None, k, s, s, t), (k, k, s, s, 3)]:
    with pytest.raises(TypeError):
        exattn.QuantCache(*args)
for args in [(k[0], k[0], s, s, t), (k, k[:3], s, s, t), (k, k, s[:3], s, t), (k, k, s, s, t[0]), (k, k, s, s, t.cpu()),
             (k.transpose(0, 1), k.transpose(0, 1), s.T.contiguous(), s.T.contiguous(), t)]:
    with pytest.raises(ValueError):
        exattn.QuantCache(*args)
"""
NEEDS_BINDING = """
q = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16, device=dev)
for call in (lambda: exattn.rope_forward(q, q, None), lambda: exattn.draft_tree(torch.zeros(3, dtype=torch.int32, device=dev))):
    with pytest.raises(OSError, match=says):
        call()
"""
WORKS = """
g = torch.Generator().manual_seed(1)
table = torch.tensor([[3, 0, 5], [1, 2, 4]], dtype=torch.int32, device=dev)
cache = exattn.QuantCache.empty(6, 2, 16, 64, table)
k, v = (torch.randn((2, 2, 40, 64), generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
q = torch.randn((2, 4, 3, 64), generator=g).to(torch.bfloat16).to(dev)
lens = torch.tensor([40, 33], dtype=torch.int32, device=dev)
exattn.cache_write(cache, k, v, None, lens)
out = [*exattn.forward_cache(q, cache, lens), *exattn.cache_read(cache, lens, rows=40), cache.k_scale, cache.v_scale]
assert exattn.check_device_error() == 0
"""
OTHERS = {
    "missing": "",
    "other library": "import shutil\nshutil.copy(exattn.LIB_PATH, path + '/other.so')\nexattn.load(path + '/other.so')\n",
    "other torch": "",
}
SAYS = {"missing": "_binding.so not found", "other library": "is loaded", "other torch": "is of torch"}


def run(tmp_path, which, dev, code):
    """`code` in a process that has a copy of the package, as `which` says."""
    build.build()
    pkg = tmp_path / "exact_head_attention_gb300"
    shutil.copytree(build.PKG, pkg, ignore=shutil.ignore_patterns("csrc", "_build", "__pycache__"))
    if which == "missing":
        os.remove(pkg / "_binding.so")
    if which == "other torch":
        os.mkdir(pkg / "_build")
        (pkg / "_build" / "binding.torch").write_text("0.0 3.0")
    head = (f"import sys\nsys.path.insert(0, {str(tmp_path)!r})\nimport pytest, torch\nfrom exact_head_attention_gb300 import exattn\n"
            f"path, dev, says = {str(tmp_path)!r}, {dev!r}, {SAYS[which]!r}\nassert exattn.LIB_PATH.startswith(path)\n")
    r = subprocess.run([sys.executable, "-c", head + OTHERS[which] + code], capture_output=True, text=True, cwd=tmp_path)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("which", OTHERS)
def test_refusals_without_the_binding(which, tmp_path):
    """On the CPU: what the cache refuses, and that the calls of the binding say why they are not to be had."""
    run(tmp_path, which, "cpu", REFUSALS + NEEDS_BINDING)


@pytest.mark.gpu
@pytest.mark.parametrize("which", OTHERS)
def test_cache_without_the_binding(which, tmp_path):
    """Writing, reading and attending give the same bits as with it."""
    run(tmp_path, which, "cuda:0", REFUSALS + NEEDS_BINDING + WORKS + "torch.save([t.cpu() for t in out], path + '/out')\n")
    from exact_head_attention_gb300 import exattn
    exattn.binding()
    here = {"torch": torch, "exattn": exattn, "dev": "cuda:0"}
    exec(WORKS, here)
    for a, b in zip(here["out"], torch.load(tmp_path / "out")):
        assert torch.equal(a.cpu(), b)
