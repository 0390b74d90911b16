"""What the paged-cache and linear entry points refuse on the host, before
anything is launched (no GPU needed), and the quantisation rule."""
import ctypes
import math
import os
import shutil
import subprocess
import sys

import pytest
import torch

import speculative_flash_decoding_b200 as sfd
from speculative_flash_decoding_b200 import alspec as ab
from paged_reference import quantise

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = (ab.ALSPEC_OK, ab.ALSPEC_ERR_INVALID_ARG,
                                       ab.ALSPEC_ERR_UNSUPPORTED, ab.ALSPEC_ERR_WORKSPACE)
P = 1 << 20  # stands for a device address


def cache(**kw):
    f = dict(k_pages=P, v_pages=P, k_scales=P, v_scales=P, page_stride=0, head_stride=0,
             token_stride=0, n_pages=10, page_size=16, n_kv_heads=4, head_dim=128,
             dtype=ab.ALSPEC_BF16, reserved=0)
    f.update(kw)
    return ab.alspec_paged_cache(**f)


def append(c, **kw):
    a = dict(k=P, v=P, src=ab.ALSPEC_BF16, ks=0, vs=0, pos=P, seq=P, n=4, table=P, batch=3,
             pages=5, err=P)
    a.update(kw)
    return ab.alspec_paged_append(c, a["k"], a["v"], a["src"], a["ks"], a["vs"], a["pos"],
                                  a["seq"], a["n"], a["table"], a["batch"], a["pages"], a["err"],
                                  0)


def gather(c, **kw):
    a = dict(table=P, pages=5, lens=P, batch=3, length=70, dtype=ab.ALSPEC_BF16, k=P, v=P, err=P)
    a.update(kw)
    return ab.alspec_paged_gather(c, a["table"], a["pages"], a["lens"], a["batch"], a["length"],
                                  a["dtype"], a["k"], a["v"], a["err"], 0)


def decode(c, **kw):
    a = dict(q=P, qs=0, hq=8, table=P, pages=5, lens=P, batch=3, S=0, W=0, scale=0.0,
             dtype=ab.ALSPEC_F32, out=P, lse=P, ms=0, ws=P, wsb=1 << 30)
    a.update(kw)
    return ab.alspec_paged_decode(c, a["q"], a["qs"], a["hq"], a["table"], a["pages"], a["lens"],
                                  a["batch"], a["S"], a["W"], a["scale"], a["dtype"], a["out"],
                                  a["lse"], a["ms"], a["ws"], a["wsb"], 0)


def linear(**kw):
    a = dict(x=P, xs=0, w=P, bias=P, res=P, y=P, dtype=ab.ALSPEC_BF16, act=0, rows=4, n=100,
             k=64, err=P)
    a.update(kw)
    return ab.alspec_linear(a["x"], a["xs"], a["w"], a["bias"], a["res"], a["y"], a["dtype"],
                            a["act"], a["rows"], a["n"], a["k"], a["err"], 0)


@pytest.mark.parametrize("kw,code", [
    (dict(k_pages=0), INVALID), (dict(v_pages=0), INVALID), (dict(k_pages=P + 8), INVALID),
    (dict(n_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(n_kv_heads=0), INVALID),
    (dict(head_dim=-1), INVALID), (dict(dtype=3), INVALID), (dict(reserved=1), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(page_size=12), UNSUPPORTED),
    (dict(page_size=1), UNSUPPORTED),
    (dict(dtype=ab.ALSPEC_E4M3, k_scales=0), INVALID),
    (dict(dtype=ab.ALSPEC_E4M3, v_scales=P + 2), INVALID),
    # Strides: one missing, rows that overlap, not a multiple of 16 bytes.
    (dict(page_stride=8192), INVALID),
    (dict(page_stride=8192, head_stride=2048, token_stride=64), INVALID),
    (dict(page_stride=8192, head_stride=2048, token_stride=132), INVALID),
    (dict(page_stride=8192, head_stride=2052, token_stride=128), INVALID),
    (dict(page_stride=1 << 40, head_stride=2048, token_stride=128), INVALID),
    (dict(page_stride=-8192, head_stride=2048, token_stride=128), INVALID),
])
def test_every_entry_point_refuses_a_bad_cache(kw, code):
    c = cache(**kw)
    assert append(c) == code and gather(c) == code and decode(c) == code
    if not any(s in kw for s in ("k_pages", "v_pages", "k_scales", "v_scales")):
        assert ab.alspec_paged_workspace_size(c, 3, 8) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), INVALID), (dict(v=P + 4), INVALID), (dict(src=ab.ALSPEC_E4M3), INVALID),
    (dict(ks=511), INVALID), (dict(vs=516), INVALID), (dict(vs=256), INVALID),
    (dict(pos=0), INVALID), (dict(pos=P + 2), INVALID), (dict(seq=P + 1), INVALID),
    (dict(seq=0, n=4), INVALID),          # more tokens than sequences
    (dict(n=-1), INVALID), (dict(table=0), INVALID), (dict(table=P + 2), INVALID),
    (dict(batch=0), INVALID), (dict(pages=0), INVALID), (dict(err=P + 3), INVALID),
    (dict(n=0, k=0, v=0), OK),
])
def test_append_refuses(kw, code):
    assert append(cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(table=0), INVALID), (dict(lens=0), INVALID), (dict(lens=P + 2), INVALID),
    (dict(batch=0), INVALID), (dict(length=0), INVALID), (dict(dtype=ab.ALSPEC_E4M3), INVALID),
    (dict(k=0), INVALID), (dict(v=P + 4), INVALID), (dict(err=P + 1), INVALID),
    (dict(batch=1 << 20, length=1 << 20), UNSUPPORTED),
])
def test_gather_refuses(kw, code):
    assert gather(cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), INVALID), (dict(q=P + 8), INVALID), (dict(qs=1000), INVALID),
    (dict(qs=1028), INVALID), (dict(hq=6), INVALID), (dict(hq=0), INVALID),
    (dict(table=0), INVALID), (dict(pages=0), INVALID), (dict(lens=0), INVALID),
    (dict(batch=0), INVALID), (dict(batch=65536), UNSUPPORTED), (dict(S=-1), INVALID),
    (dict(W=-1), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(dtype=ab.ALSPEC_E4M3), INVALID), (dict(out=0), INVALID), (dict(out=P + 4), INVALID),
    (dict(lse=P + 2), INVALID), (dict(ms=-1), INVALID), (dict(ws=0), WORKSPACE),
    (dict(ws=P + 4), WORKSPACE), (dict(wsb=4096), WORKSPACE),
])
def test_decode_refuses(kw, code):
    assert decode(cache(), **kw) == code


@pytest.mark.parametrize("c,kw", [
    (dict(), dict(batch=65535, pages=1 << 20)),
    (dict(dtype=ab.ALSPEC_F32), dict(batch=65535, pages=1 << 15)),
    (dict(n_kv_heads=128), dict(hq=128, pages=1 << 27)),
    (dict(n_kv_heads=1), dict(hq=1024, pages=1 << 27)),
])
def test_decode_refuses_more_tiles_than_it_can_number(c, kw):
    assert decode(cache(**c), **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), INVALID), (dict(x=P + 8), INVALID), (dict(w=0), INVALID), (dict(w=P + 2), INVALID),
    (dict(y=0), INVALID), (dict(y=P + 1), INVALID), (dict(bias=P + 1), INVALID),
    (dict(res=P + 1), INVALID), (dict(dtype=ab.ALSPEC_F32, y=P + 2), INVALID),
    (dict(dtype=ab.ALSPEC_E4M3), INVALID), (dict(act=4), INVALID), (dict(act=-1), INVALID),
    (dict(rows=-1), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(k=68), INVALID),
    (dict(xs=32), INVALID), (dict(xs=68), INVALID), (dict(err=P + 2), INVALID),
    (dict(rows=0, x=0, y=0), OK),
])
def test_linear_refuses(kw, code):
    assert linear(**kw) == code


def test_workspace_does_not_grow_with_the_batch():
    c = cache()
    n = ab.alspec_paged_workspace_size(c, 1, 8)
    assert n > 0 and n % 256 == 0
    assert ab.alspec_paged_workspace_size(c, 4096, 32) == n
    assert ab.alspec_paged_workspace_size(c, 1, 6) == 0


def test_python_layer_refuses_without_a_gpu():
    x = torch.zeros(4, 2, 16, 64)
    with pytest.raises(ValueError, match="CUDA"):
        sfd.PagedCache.from_tensors(x, x)
    with pytest.raises(ValueError, match="dtype"):
        sfd.PagedCache(4, 16, 2, 64, "int8")
    with pytest.raises(ValueError, match="weight"):
        sfd.Linear(torch.zeros(8, 8, dtype=torch.bfloat16))


def test_quantisation_rule_on_the_cpu():
    """scale = max(amax / 448, 2^-126); the largest value becomes 448, zeros
    stay zero, and the value read back is within half an e4m3 step (2^-4
    relative, 2^-10 of the scale for the smallest codes)."""
    x = torch.randn(50, 3, 64, generator=torch.Generator().manual_seed(0))
    x[0, 0] = 0
    code, s = quantise(x)
    assert code.float()[0, 0].abs().max() == 0 and s[0, 0] == 2.0 ** -126
    top = code.float().abs().amax(-1)
    assert bool((top[1:] == 448).all())
    back = code.double() * s.double()[..., None]
    bound = torch.maximum(x.abs().double() * 2.0 ** -4, s.double()[..., None] * 2.0 ** -10)
    assert bool(((back - x.double()).abs() <= bound * (1 + 2.0 ** -20)).all())


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not installed")
def test_c_sees_the_same_cache_description(tmp_path):
    src = tmp_path / "size.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "alspec.h"\nint main(void) '
                   '{ printf("%zu %zu %zu\\n", sizeof(alspec_paged_cache), '
                   'offsetof(alspec_paged_cache, page_stride), '
                   'offsetof(alspec_paged_cache, dtype)); return 0; }\n')
    exe = tmp_path / "size"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [ctypes.sizeof(ab.alspec_paged_cache), ab.alspec_paged_cache.page_stride.offset,
                   ab.alspec_paged_cache.dtype.offset]


_BLOCKED = """
import sys
sys.modules["torch"] = None          # as where torch is not installed
import speculative_flash_decoding_b200 as sfd
c = sfd.alspec_paged_cache(n_pages=10, page_size=16, n_kv_heads=4, head_dim=128, dtype=sfd.ALSPEC_BF16)
assert sfd.alspec_paged_workspace_size(c, 3, 8) > 0
for name in ("PagedCache", "PagedDecoder", "Linear"):
    assert name in dir(sfd)
    try:
        getattr(sfd, name)
    except ImportError:
        pass
    else:
        raise SystemExit(name)
"""

_STAR = """
from speculative_flash_decoding_b200 import *
assert Linear and PagedCache and PagedDecoder and Decoder and alspec_linear and SIGNATURES
"""

_STAR_BLOCKED = """
import sys
sys.modules["torch"] = None
from speculative_flash_decoding_b200 import *
assert Decoder and alspec_linear and "Linear" not in globals()
"""

_CPU_TORCH = """
import sys, torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)      # as in a build of torch without CUDA
import speculative_flash_decoding_b200 as sfd
assert sfd.Linear is sfd.linear.Linear and sfd.PagedCache is sfd.paged.PagedCache
try:
    sfd.PagedCache.from_tensors(torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 16, 64))
except ValueError:
    pass
"""

_LATE = """
import sys
import speculative_flash_decoding_b200 as sfd
assert "torch" not in sys.modules
from speculative_flash_decoding_b200 import Linear, PagedCache, PagedDecoder
assert "torch" in sys.modules and sfd.PagedDecoder is PagedDecoder
"""


@pytest.mark.parametrize("code", [_BLOCKED, _CPU_TORCH, _LATE, _STAR, _STAR_BLOCKED],
                         ids=["no torch", "cpu torch", "late", "star", "star, no torch"])
def test_the_binding_loads_without_torch(code):
    """torch is needed where its tensors are: the ctypes binding takes plain
    addresses."""
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert p.returncode == 0, p.stderr


def test_unknown_names_are_refused():
    with pytest.raises(AttributeError, match="no attribute 'Lineal'"):
        sfd.Lineal


_PLAN = r'''
#include <cstdio>
#include <cstdlib>
#include "linear_plan.h"
// argv: clusters of 1 .. 8 CTAs that fit; then per line of stdin: tiles kblocks ctas
int main(int argc, char** argv) {
    alspec::LinClusters fit{};
    for (int c = 1; c <= 8; ++c) fit.n[c] = std::atoi(argv[c]);
    std::printf("%d %d %d\n", alspec::lin_pairs(fit, 160, 1000), alspec::lin_pairs(fit, 128, 1000),
                alspec::lin_pairs(fit, 160, 128));
    long long tiles;
    int kblocks, ctas;
    while (std::scanf("%lld %d %d", &tiles, &kblocks, &ctas) == 3)
        std::printf("%d\n", alspec::lin_split(fit, tiles, kblocks, ctas));
}
'''


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
@pytest.mark.parametrize("fit", [
    [148, 74, 45, 33, 26, 22, 17, 15],   # a whole device
    [28, 14, 8, 7, 4, 3, 2, 0],          # parts without eight SMs together
    [14, 7, 3, 2, 0, 0, 0, 0],
    [5, 0, 0, 0, 0, 0, 0, 0],            # no pairs either
    [0, 0, 0, 0, 0, 0, 0, 0],            # nothing known
])
def test_linear_takes_the_cluster_sizes_that_fit(tmp_path, fit):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(_PLAN)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "speculative_flash_decoding_b200", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    asked = [(t, kb, c) for t in (1, 3, 32, 48, 64, 400, 1 << 33) for kb in (1, 7, 8, 64, 128)
             for c in (1, 2) if fit[c - 1] > 0 or c == 1]
    out = subprocess.run([str(exe), *map(str, fit)], capture_output=True, text=True, check=True,
                         input="".join("%d %d %d\n" % a for a in asked)).stdout.split()
    assert [int(x) for x in out[:3]] == [int(fit[1] > 0), 0, 0]
    for (tiles, kb, ctas), got in zip(asked, map(int, out[3:]), strict=True):
        size = got * ctas
        assert 1 <= size <= 8 and (size == 1 or fit[size - 1] > 0)

        def cost(c):
            return -(-tiles // max(1, fit[c * ctas - 1])) * (-(-kb // c) + (20 if c > 1 else 16))

        able = [c for c in range(1, 9 // ctas + 1) if c * ctas <= 8 and c <= max(1, kb // 4)
                and (c * ctas == 1 or fit[c * ctas - 1] > 0)]
        assert cost(got) == min(map(cost, able))
