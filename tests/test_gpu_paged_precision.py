"""Precision of the paged attention where weights, scales or values differ by
many orders of magnitude: attention sinks with small values, tokens of a large
V scale and almost no weight."""
import math

import pytest
import torch

from paged_reference import U, attention, attention_bound, make_cache

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _half_step(x, dtype):
    """Half the distance between neighbouring values of dtype around x: 2^-9
    (bf16) or 2^-25 (fp32) of the power of two above it."""
    top = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=1e-30))))
    return top * U[dtype]


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("nats,v_size", [
    (0, 1.0),                                       # no outlier
    (10, 2.0 ** -6), (14, 2.0 ** -10), (20, 2.0 ** -20),   # a sink whose value is small
    (-20, 2.0 ** 10), (-20, 2.0 ** 20),             # almost no weight, a large scale
])
@pytest.mark.parametrize("at", [0, 700])
def test_one_token_far_from_the_others(cuda_device, out_dtype, nats, v_size, at):
    """1184 sequences and KV heads, so that a warp's share is a sequence and a
    running reference meets the token early and late.  Besides the output's
    rounding, each result is within 2^-17 of A = sum p |v|: scores of at most 20
    are within 2^-21 of the nats they are (4 steps of 2^-23 of the running sum
    of a score, most of them far below 20) and exp2 within 2^-22, which moves
    numerator and denominator by 2^-20 each; a weight is within 2^-22 of
    itself; the running sums take 64 steps that lose half of 2^-23 on the
    average, 2^-18."""
    from speculative_flash_decoding_b200 import PagedCache, PagedDecoder
    B, hkv, n, d, page = 37, 32, 1024, 64, 64
    g = torch.Generator(device="cuda").manual_seed(abs(nats) + at)
    q = torch.randn(B, hkv, d, generator=g, device="cuda").to(BF16)
    k = torch.randn(B, hkv, n, d, generator=g, device="cuda")
    v = 1.0 + torch.randn(B, hkv, n, d, generator=g, device="cuda")
    if nats:
        u = q.float() / q.float().square().sum(-1, keepdim=True)
        k[:, :, at] = nats * math.sqrt(d) * u
        v[:, :, at] *= v_size

    def rows(x):  # codes and scales of alspec_paged_append, on the GPU
        s = (x.abs().amax(-1).double() / 448).float()
        c = (x.double() / s.double()[..., None]).float().clamp(-448, 448).to(torch.float8_e4m3fn)
        return c, s

    def pages(x):  # [B, hkv, n, ...] -> [B * n / page, hkv, page, ...]
        return x.unflatten(2, (n // page, page)).transpose(1, 2).flatten(0, 1).contiguous()

    (kc, ks), (vc, vs) = rows(k), rows(v)
    cache = PagedCache.from_tensors(*(pages(x.view(torch.uint8)).view(x.dtype) for x in (kc, vc)),
                                    pages(ks), pages(vs))
    table = torch.arange(B * n // page, dtype=torch.int32, device="cuda").view(B, -1)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    dec = PagedDecoder(cache, B, hkv)
    got = dec.decode(q, table, lens, out=torch.empty(B, hkv, d, dtype=out_dtype, device="cuda"))
    assert dec.device_error() == (0, 0)
    k64, v64 = kc.double() * ks.double()[..., None], vc.double() * vs.double()[..., None]
    p = torch.softmax(torch.einsum("bhd,bhld->bhl", q.double(), k64) / math.sqrt(d), -1)
    want = torch.einsum("bhl,bhld->bhd", p, v64)
    A = torch.einsum("bhl,bhld->bhd", p, v64.abs())
    err = ((got.double() - want).abs() - _half_step(want, out_dtype)).clamp(min=0) / A
    assert float(err.max()) <= 2.0 ** -17, float(err.max())


@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_v_scales_over_a_wide_range(cuda_device, out_dtype):
    """V scales that differ by 2^80 between tokens, under the bound of
    ordinary caches."""
    from speculative_flash_decoding_b200 import PagedCache, PagedDecoder
    lens = [700, 64, 5]
    c = make_cache("e4m3", lens, 16, 2, 64, seed=6, v_scale_span=40.0)
    q = torch.randn(3, 6, 64, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    dec = PagedDecoder(PagedCache.from_tensors(c["k"], c["v"], c["ks"], c["vs"]), 3, 6)
    got = dec.decode(q, c["table"], torch.tensor(lens, dtype=torch.int32, device="cuda"),
                     out=torch.empty(3, 6, 64, dtype=out_dtype, device="cuda"))
    ref = attention(q, c["k64"], c["v64"], lens)
    bound, _ = attention_bound(ref, lens, 64, "e4m3", out_dtype)
    err = (got.double().cpu() - ref[0]).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


# NaN as fp32 arithmetic makes it (0x7fffffff), as math.nan (0x7fc00000), with
# the least payload, and negative ones.
NANS = [0x7fffffff, 0x7fc00000, 0x7ffff000, 0x7f800001, -1, -(0x7fffff)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", NANS)
def test_every_nan_reaches_its_heads_over_fp32_pages(cuda_device, d, bits):
    from speculative_flash_decoding_b200 import PagedCache, PagedDecoder
    lens = [200, 150, 40]
    c = make_cache("f32", lens, 16, 2, d, seed=2)
    q = torch.randn(3, 4, d, generator=torch.Generator().manual_seed(0)).cuda()

    def poke(x, *at):
        x.view(torch.int32)[at] = bits

    for name, b, h, t in (("k", 0, 1, 100), ("v", 1, 0, 100)):
        poke(c[name], c["table"][b, t // 16].long(), h, t % 16, 5)
    poke(q, 2, 3, 7)
    dec = PagedDecoder(PagedCache.from_tensors(c["k"], c["v"]), 3, 4)
    lse = torch.empty(3, 4, device="cuda")
    out = dec.decode(q, c["table"], torch.tensor(lens, dtype=torch.int32, device="cuda"), lse=lse)
    bad = torch.zeros(3, 4, d, dtype=torch.bool, device="cuda")
    bad[0, 2:] = True     # a NaN key
    bad[1, :2, 5] = True  # a NaN value
    bad[2, 3] = True      # a NaN query
    assert torch.equal(out.isnan(), bad)
    of_scores = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    of_scores[0, 2:] = of_scores[2, 3] = True
    assert torch.equal(lse.isnan(), of_scores)


@pytest.mark.parametrize("bits", [0x7f7fffff, 0x7f7ff000, 0x7f7fefff, 0x7f7fe000])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_values_near_the_largest_over_fp32_pages(cuda_device, bits, sign):
    """Finite keys, values and queries up to the largest fp32 stay finite:
    here a key meets a query element of 2^-124, a value a weight of e^-60, a
    query element keys of 2^-112."""
    from speculative_flash_decoding_b200 import PagedCache, PagedDecoder
    d, lens = 64, [150, 90, 40]
    big = sign * float(torch.tensor(bits, dtype=torch.int32).view(torch.float32))
    c = make_cache("f32", lens, 16, 1, d, seed=5)
    q = torch.randn(3, 4, d, generator=torch.Generator().manual_seed(3))

    def put(name, b, t, e, x):
        c[name][c["table"][b, t // 16].long(), 0, t % 16, e] = x
        c[name + "64"][b, 0, t, e] = x

    q[0, :, 5] = 2.0 ** -124
    put("k", 0, 100, 5, big)
    q[1] = q[1, :1]  # heads alike, so that one key is at -60 for all
    u = q[1, 0].clone()
    for e in range(d):
        put("k", 1, 30, e, float(-60.0 * math.sqrt(d) * u[e] / (u @ u)))
    put("v", 1, 30, 9, big)
    q[2] *= 2.0 ** 16
    q[2, :, 7] = big
    for t in range(lens[2]):
        put("k", 2, t, 7, float(c["k64"][2, 0, t, 7] * 2.0 ** -112))
        for e in range(d):
            if e != 7:
                put("k", 2, t, e, float(c["k64"][2, 0, t, e] * 2.0 ** -16))
    q = q.cuda()
    dec = PagedDecoder(PagedCache.from_tensors(c["k"], c["v"]), 3, 4)
    got = dec.decode(q, c["table"], torch.tensor(lens, dtype=torch.int32, device="cuda"))
    ref = attention(q, c["k64"], c["v64"], lens)
    bound, _ = attention_bound(ref, lens, d, "f32", F32)
    err = (got.double().cpu() - ref[0]).abs()
    assert bool(got.isfinite().all())
    assert bool((err <= bound).all()), float((err / bound).max())
