"""The paged cache on the GPU: rows written (and quantised), read back, and
attention of one new token per sequence, against plain 64-bit forms."""
import math

import pytest
import torch

from paged_reference import DTYPES, attention, check_attention, make_cache, quantise

pytestmark = pytest.mark.gpu


def _cache(c):
    from speculative_flash_decoding_b200 import PagedCache
    return PagedCache.from_tensors(c["k"], c["v"], c["ks"], c["vs"])


# ------------------------------------------------------------------- append

def _append_case(dtype, src, d, hkv, page, token_major, n, batch, seed, fused=False):
    """A cache with known old contents, tokens for distinct places, and what
    the pools hold afterwards."""
    g = torch.Generator().manual_seed(seed)
    lens = [page * 3] * batch
    c = make_cache(dtype, lens, page, hkv, d, token_major, seed=seed + 1)
    row = hkv * d
    wide = torch.randn((n, 2 * row + (32 if fused else 0)), generator=g).to(DTYPES[src])
    wide[0, :d] = 0            # a row of zeros
    wide[n // 2, :d] *= 2.0 ** -110  # tiny values
    wide = wide.cuda()
    k = wide[:, :row].unflatten(1, (hkv, d))
    v = wide[:, row: 2 * row].unflatten(1, (hkv, d))
    places = torch.randperm(batch * page * 3, generator=g)[:n]
    seq, pos = (places // (page * 3)).int(), (places % (page * 3)).int()
    if n > 3:
        pos[2] = -1            # padding
    return c, k, v, seq, pos


def _expect(c, name, x, seq, pos, page):
    """Pools after the append, on the CPU."""
    pool = c[name].cpu().contiguous()
    scale = c[name + "s"].cpu() if c[name + "s"] is not None else None
    code, s = quantise(x) if scale is not None else (x.cpu().to(pool.dtype), None)
    for i in range(len(pos)):
        if pos[i] < 0:
            continue
        pg, off = int(c["table"][int(seq[i]), int(pos[i]) // page]), int(pos[i]) % page
        if scale is not None:
            pool.view(torch.uint8)[pg, :, off] = code[i].view(torch.uint8)
            scale[pg, :, off] = s[i]
        else:
            pool[pg, :, off] = code[i]
    return pool, scale


def _bits(x):
    x = x.cpu().contiguous()
    return x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


@pytest.mark.parametrize("dtype,src,d,hkv,page,token_major,n,batch,fused", [
    ("bf16", "bf16", 128, 8, 16, False, 33, 7, True),
    ("bf16", "f32", 64, 3, 8, True, 20, 4, False),
    ("f32", "f32", 128, 1, 24, False, 5, 2, False),
    ("f32", "bf16", 64, 2, 16, False, 9, 3, True),
    ("e4m3", "bf16", 128, 8, 16, False, 70, 9, True),
    ("e4m3", "f32", 128, 2, 32, True, 41, 3, False),
    ("e4m3", "bf16", 64, 5, 8, True, 1, 1, False),
    ("e4m3", "f32", 64, 1, 24, False, 17, 2, True),
])
def test_append_writes_exactly_its_rows(cuda_device, dtype, src, d, hkv, page, token_major, n,
                                        batch, fused):
    c, k, v, seq, pos = _append_case(dtype, src, d, hkv, page, token_major, n, batch, n, fused)
    want = [_expect(c, w, x, seq, pos, page) for w, x in (("k", k), ("v", v))]
    cache = _cache(c)
    cache.append(k, v, pos.cuda(), c["table"], seq_ids=seq.cuda())
    for (pool, scale), w in zip(want, "kv"):
        assert torch.equal(_bits(c[w]), _bits(pool))
        if scale is not None:
            assert torch.equal(_bits(c[w + "s"]), _bits(scale))
    assert cache.device_error() == (0, 0)


def test_append_step_without_sequence_ids(cuda_device):
    c, k, v, _, _ = _append_case("e4m3", "bf16", 128, 4, 16, False, 6, 6, 5)
    pos = torch.tensor([0, 47, -1, 15, 16, 31], dtype=torch.int32)
    seq = torch.arange(6)
    want, scale = _expect(c, "k", k, seq, pos, 16)
    cache = _cache(c)
    cache.append(k, v, pos.cuda(), c["table"])
    assert torch.equal(_bits(c["k"]), _bits(want)) and torch.equal(_bits(c["ks"]), _bits(scale))


def test_append_rows_that_are_not_finite(cuda_device):
    """A row with a NaN or an infinity reads back as NaN, its neighbours do
    not."""
    c = make_cache("e4m3", [16], 16, 2, 64, seed=3)
    cache = _cache(c)
    x = torch.randn(4, 2, 64, device="cuda")
    x[1, 0, 3] = math.nan
    x[2, 1, 63] = -math.inf
    cache.append(x, x, torch.arange(4, dtype=torch.int32, device="cuda"), c["table"],
                 seq_ids=torch.zeros(4, dtype=torch.int32, device="cuda"))
    k, v = (torch.zeros(1, 2, 16, 64, device="cuda") for _ in range(2))
    cache.gather(c["table"], torch.tensor([4], dtype=torch.int32, device="cuda"), k, v)
    bad = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 2] = True
    for y in (k, v):
        assert torch.equal(y[0, :, :4].isnan().all(-1), bad)
        assert torch.equal(y[0, :, :4].isnan().any(-1), bad)


def test_append_skips_and_flags_bad_places(cuda_device):
    import speculative_flash_decoding_b200 as sfd
    c, k, v, _, _ = _append_case("bf16", "bf16", 64, 2, 8, False, 6, 3, 8)
    c["table"][1, 2] = c["n_pages"]      # a page that does not exist
    before = [_bits(c[w]).clone() for w in "kv"]
    cache = _cache(c)
    #            sequence too large, negative, position past the table, bad page x2, padding
    seq = torch.tensor([3, -1, 0, 1, 1, 2], dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 0, 24, 16, 23, -5], dtype=torch.int32, device="cuda")
    cache.append(k, v, pos, c["table"], seq_ids=seq)
    assert all(torch.equal(_bits(c[w]), x) for w, x in zip("kv", before))
    assert cache.device_error() == (sfd.ALSPEC_ERR_DEVICE_DATA, sfd.ALSPEC_DEVERR_PAGE)
    assert cache.device_error() == (0, 0)


# ------------------------------------------------------------------- gather

@pytest.mark.parametrize("dtype,out,d,hkv,page,token_major,lens,max_len", [
    ("bf16", "bf16", 128, 8, 16, False, [100, 0, 64, 1], 131),
    ("e4m3", "bf16", 128, 2, 24, True, [70, 129], 129),
    ("e4m3", "f32", 64, 3, 8, False, [1, 65, 8], 70),
    ("f32", "f32", 64, 1, 16, True, [33], 33),
    ("f32", "bf16", 128, 4, 32, False, [5, 200, 31], 256),
    ("bf16", "f32", 64, 2, 128, False, [127, 128, 129], 130),
])
def test_gather_reads_back_and_leaves_the_rest(cuda_device, dtype, out, d, hkv, page, token_major,
                                               lens, max_len):
    c = make_cache(dtype, lens, page, hkv, d, token_major, seed=len(lens))
    cache = _cache(c)
    shape = (len(lens), hkv, max_len, d)
    k, v = (torch.full(shape, 7.0, dtype=DTYPES[out], device="cuda") for _ in range(2))
    cache.gather(c["table"], torch.tensor(lens, dtype=torch.int32, device="cuda"), k, v)
    for got, want in ((k, c["k64"]), (v, c["v64"])):
        ref = torch.full(shape, 7.0, dtype=DTYPES[out])
        for b, n in enumerate(lens):
            # fp32 products of a code and its scale, then one rounding.
            ref[b, :, :n] = want[b, :, :n].float().to(DTYPES[out])
        assert torch.equal(_bits(got), _bits(ref))
    assert cache.device_error() == (0, 0)


def test_gather_flags_bad_lengths_and_pages(cuda_device):
    import speculative_flash_decoding_b200 as sfd
    c = make_cache("bf16", [40, 40], 8, 2, 64, seed=1)
    c["table"][1, 0] = -3
    cache = _cache(c)
    k, v = (torch.zeros(2, 2, 50, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache.gather(c["table"], torch.tensor([41, 9], dtype=torch.int32, device="cuda"), k, v)
    assert cache.device_error() == (sfd.ALSPEC_ERR_DEVICE_DATA,
                                    sfd.ALSPEC_DEVERR_PAGE | sfd.ALSPEC_DEVERR_SEQ_LEN)
    assert torch.equal(k[0, :, :40].double().cpu(), c["k64"][0, :, :40])
    assert not k[0, :, 40:].any() and not k[1, :, :8].any()
    assert torch.equal(k[1, :, 8].double().cpu(), c["k64"][1, :, 8])


# ------------------------------------------------------------------- decode

def _decode(c, lens, hq, d, out_dtype, n_sink=0, window=0, scale=0.0, seed=0, q_pad=0,
            dtype="bf16", with_lse=True):
    from speculative_flash_decoding_b200 import PagedDecoder
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    wide = 2.0 * torch.randn((B, hq * d + q_pad), generator=g)
    wide = wide.to(torch.float32 if dtype == "f32" else torch.bfloat16).cuda()
    q = wide[:, : hq * d].unflatten(1, (hq, d))
    dec = PagedDecoder(_cache(c), B, hq, n_sink=n_sink, window=window, scale=scale)
    out = torch.full((B, hq, d), 5.0, dtype=out_dtype, device="cuda")
    lse = torch.full((B, hq), 5.0, device="cuda") if with_lse else None
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dec.decode(q, c["table"], seq, out=out, lse=lse)
    assert dec.device_error() == (0, 0)
    return dec, q, seq, out, lse


F32, BF16 = torch.float32, torch.bfloat16
DECODE = [
    # dtype, d, page, hkv, group, lens, sink, window, out, token_major, q_pad
    ("bf16", 128, 16, 1, 1, [1], 0, 0, F32, False, 0),
    ("bf16", 128, 64, 8, 4, [513, 1, 0, 31, 32, 33], 0, 0, BF16, False, 64),
    ("bf16", 128, 24, 2, 8, [700, 95, 96, 97], 0, 0, F32, True, 0),
    ("bf16", 64, 8, 3, 3, [1, 8, 9, 100, 257], 0, 0, F32, False, 8),
    ("bf16", 64, 128, 1, 16, [2000, 3], 0, 0, BF16, False, 0),
    ("bf16", 128, 32, 2, 9, [300, 41], 0, 0, F32, False, 0),
    ("bf16", 128, 16, 8, 4, [40000], 0, 0, F32, False, 0),
    ("bf16", 64, 16, 1, 7, [4, 100, 5, 300], 4, 64, F32, False, 0),
    ("bf16", 128, 16, 2, 8, [1000, 50, 0, 131, 77], 33, 31, BF16, True, 0),
    ("bf16", 128, 64, 2, 2, [500, 20], 40, 0, F32, False, 0),
    ("bf16", 64, 64, 2, 2, [500, 20, 1], 0, 1, F32, False, 0),
    ("e4m3", 128, 16, 8, 4, [513, 1, 0, 31, 32, 33], 0, 0, BF16, False, 0),
    ("e4m3", 128, 24, 1, 8, [3000], 0, 0, F32, True, 0),
    ("e4m3", 64, 8, 2, 5, [65, 1, 7, 400], 0, 0, F32, False, 0),
    ("e4m3", 64, 64, 4, 1, [129, 1000], 5, 100, F32, True, 0),
    ("e4m3", 128, 32, 2, 12, [20000, 100], 0, 0, F32, False, 0),
    ("f32", 64, 16, 1, 4, [1024], 0, 0, F32, False, 0),
    ("f32", 128, 8, 2, 3, [1, 31, 32, 33, 0, 333], 0, 0, F32, False, 4),
    ("f32", 128, 48, 1, 8, [5000, 17], 0, 0, F32, True, 0),
    ("f32", 64, 64, 3, 10, [200, 190], 3, 50, BF16, False, 0),
]


@pytest.mark.parametrize("dtype,d,page,hkv,group,lens,n_sink,window,out,token_major,q_pad", DECODE)
def test_decode(cuda_device, dtype, d, page, hkv, group, lens, n_sink, window, out, token_major,
                q_pad):
    c = make_cache(dtype, lens, page, hkv, d, token_major, seed=sum(lens))
    dec, q, seq, got, lse = _decode(c, lens, hkv * group, d, out, n_sink, window, seed=page,
                                    q_pad=q_pad, dtype=dtype)
    ref = attention(q, c["k64"], c["v64"], lens, n_sink, window)
    check_attention(got, lse, ref, lens, d, dtype, out)
    # Again on the same workspace, bit for bit.
    again = torch.empty_like(got)
    dec.decode(q, c["table"], seq, out=again)
    assert torch.equal(_bits(again), _bits(got))


@pytest.mark.parametrize("page,token_major", [(8, False), (16, True), (24, False), (64, True)])
@pytest.mark.parametrize("n_sink,window", [(0, 0), (3, 20), (17, 15), (40, 0), (0, 1)])
def test_decode_wide_rows(cuda_device, page, token_major, n_sink, window):
    """fp32 rows of 128 elements come in shorter tiles: ends of sequences, of
    the sink set and of pages on all sides of theirs."""
    lens = [15, 16, 17, 0, 31, 32, 33, 49, 700, 1]
    c = make_cache("f32", lens, page, 3, 128, token_major, seed=page + n_sink)
    _, q, _, got, lse = _decode(c, lens, 15, 128, F32, n_sink, window, seed=page, dtype="f32")
    ref = attention(q, c["k64"], c["v64"], lens, n_sink, window)
    check_attention(got, lse, ref, lens, 128, "f32", F32)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_decode_many_sequences(cuda_device, dtype):
    """More sequences than warps, most of them short, some empty."""
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 70, (900,), generator=g).tolist()
    c = make_cache(dtype, lens, 16, 2, 64, seed=9)
    _, q, _, got, lse = _decode(c, lens, 4, 64, F32, dtype=dtype)
    check_attention(got, lse, attention(q, c["k64"], c["v64"], lens), lens, 64, dtype, F32)


def test_decode_all_rows_padded(cuda_device):
    c = make_cache("bf16", [0, 0, 0], 16, 2, 128)
    _, _, _, got, lse = _decode(c, [0, 0, 0], 8, 128, BF16)
    assert not got.any() and bool((lse == -math.inf).all())


def test_decode_scale_and_no_lse(cuda_device):
    lens = [77, 300]
    c = make_cache("bf16", lens, 16, 2, 64, seed=2)
    _, q, _, got, _ = _decode(c, lens, 4, 64, F32, scale=0.03, with_lse=False)
    ref = attention(q, c["k64"], c["v64"], lens, scale=0.03)
    check_attention(got, None, ref, lens, 64, "bf16", F32)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("scale", [-0.2, 1e-30])
def test_decode_unusual_scales(cuda_device, dtype, scale):
    """A negative scale, and one that makes every weight equal."""
    lens = [65, 300]
    c = make_cache(dtype, lens, 16, 2, 64, seed=2)
    _, q, _, got, lse = _decode(c, lens, 6, 64, F32, scale=scale, dtype=dtype, n_sink=3, window=50)
    ref = attention(q, c["k64"], c["v64"], lens, 3, 50, scale=scale)
    check_attention(got, lse, ref, lens, 64, dtype, F32)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_decode_values_that_are_not_finite(cuda_device, dtype):
    """NaN among the attended keys or values reaches the heads that read them
    and no others; behind the end of a sequence, or outside the sink set, it
    reaches nobody."""
    from speculative_flash_decoding_b200 import PagedDecoder
    lens = [200, 150]
    c = make_cache(dtype, lens, 16, 2, 64, seed=2)
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(0))
    q = q.to(F32 if dtype == "f32" else BF16).cuda()
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    nan = 0x7F if dtype == "e4m3" else math.nan

    def poke(name, b, h, t):
        x = c[name].view(torch.uint8) if dtype == "e4m3" else c[name]
        x[c["table"][b, t // 16].long(), h, t % 16, 5] = nan

    poke("k", 0, 1, 100)
    poke("v", 1, 0, 100)
    sinks = PagedDecoder(_cache(c), 2, 4, n_sink=4, window=40)
    out = sinks.decode(q, c["table"], seq, out=torch.empty(2, 4, 64, device="cuda"))
    assert bool(out.isfinite().all())
    out = PagedDecoder(_cache(c), 2, 4).decode(q, c["table"], seq,
                                               out=torch.empty(2, 4, 64, device="cuda"))
    bad = torch.zeros(2, 4, 64, dtype=torch.bool, device="cuda")
    bad[0, 2:] = True           # a NaN score
    bad[1, :2, 5] = True        # a NaN value
    assert torch.equal(out.isnan(), bad)


def test_decode_v_scales_over_a_wide_range(cuda_device):
    """V scales that differ by 2^80 between tokens: the running power of two
    keeps every weight in range."""
    lens = [700, 64]
    c = make_cache("e4m3", lens, 16, 2, 64, seed=6, v_scale_span=40.0)
    _, q, _, got, lse = _decode(c, lens, 6, 64, F32, dtype="e4m3")
    ref = attention(q, c["k64"], c["v64"], lens)
    # A weight (probability times V scale) below 2^-14 of the largest one is
    # held to 2^-25 of that largest: at most n * 2^-25 * 448 * max scale over
    # the sums, relative to A no more than 2^-21 of the largest product.
    out, _, A, _ = ref
    peak = torch.stack([c["v64"][b, :, :n].abs().amax() for b, n in enumerate(lens)])
    from paged_reference import attention_bound
    bound, _ = attention_bound(ref, lens, 64, "e4m3", F32)
    bound = bound + peak[:, None, None] * torch.tensor(lens)[:, None, None] * 2.0 ** -24
    assert bool(((got.double().cpu() - out).abs() <= bound).all())
    assert torch.isfinite(got).all()


def test_decode_extreme_queries(cuda_device):
    """Scores far apart: one token takes all the weight, and queries whose
    magnitudes differ by 2^60 between heads (e4m3 pages scale them)."""
    lens = [200]
    for dtype in ("bf16", "e4m3", "f32"):
        c = make_cache(dtype, lens, 16, 1, 64, seed=12)
        from speculative_flash_decoding_b200 import PagedDecoder
        q = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(1))
        q[0, 1] *= 200.0
        q[0, 2] *= 2.0 ** -60
        q[0, 3] = 0
        q = q.to(F32 if dtype == "f32" else BF16).cuda()
        dec = PagedDecoder(_cache(c), 1, 4)
        out = torch.empty(1, 4, 64, device="cuda")
        dec.decode(q, c["table"], torch.tensor(lens, dtype=torch.int32, device="cuda"), out=out)
        ref = attention(q, c["k64"], c["v64"], lens)
        check_attention(out, None, ref, lens, 64, dtype, F32)


def test_decode_flags_bad_pages_and_lengths(cuda_device):
    """Bad table entries and lengths set the error word; the other sequences
    are right."""
    import speculative_flash_decoding_b200 as sfd
    lens = [100, 64, 90]
    c = make_cache("bf16", lens, 16, 2, 64, seed=3)
    table = c["table"].clone()
    table[1, 1] = c["n_pages"] + 5
    from speculative_flash_decoding_b200 import PagedDecoder
    dec = PagedDecoder(_cache(c), 3, 4)
    q = torch.randn(3, 4, 64, device="cuda").to(BF16)
    out = torch.empty(3, 4, 64, device="cuda")
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dec.decode(q, table, seq, out=out)
    assert dec.device_error() == (sfd.ALSPEC_ERR_DEVICE_DATA, sfd.ALSPEC_DEVERR_PAGE)
    ref = attention(q, c["k64"], c["v64"], lens)
    pick = [0, 2]
    check_attention(out[pick], None, tuple(x[pick] for x in ref), [100, 90], 64, "bf16", F32)
    dec.decode(q, c["table"], torch.tensor([100, -2, 1000], dtype=torch.int32, device="cuda"),
               out=out)
    assert dec.device_error()[1] & sfd.ALSPEC_DEVERR_SEQ_LEN
    assert not out[1].any()
    check_attention(out[:1], None, tuple(x[:1] for x in ref), [100], 64, "bf16", F32)
    # The workspace is as good as new.
    dec.decode(q, c["table"], seq, out=out)
    assert dec.device_error() == (0, 0)
    check_attention(out, None, ref, lens, 64, "bf16", F32)


def test_decode_writes_only_its_outputs(cuda_device):
    lens = [90, 0, 33, 1500]
    c = make_cache("bf16", lens, 16, 3, 128, seed=3)
    before = [_bits(c[w]).clone() for w in "kv"]
    from speculative_flash_decoding_b200 import PagedDecoder
    dec = PagedDecoder(_cache(c), 4, 15)
    buf = torch.full((dec.workspace_bytes + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = buf[4096: 4096 + dec.workspace_bytes]
    ws.zero_()
    dec.workspace = ws
    n = 4 * 15 * 128
    o = torch.full((n + 256,), 3.0, device="cuda")
    l = torch.full((60 + 64,), 3.0, device="cuda")
    q = torch.randn(4, 15, 128, device="cuda").to(BF16)
    dec.decode(q, c["table"], torch.tensor(lens, dtype=torch.int32, device="cuda"),
               out=o[128: 128 + n].view(4, 15, 128), lse=l[32:92].view(4, 15))
    torch.cuda.synchronize()
    assert bool((buf[:4096] == 0xA5).all()) and bool((buf[4096 + dec.workspace_bytes:] == 0xA5).all())
    assert bool((o[:128] == 3).all()) and bool((o[128 + n:] == 3).all())
    assert bool((l[:32] == 3).all()) and bool((l[92:] == 3).all())
    assert all(torch.equal(_bits(c[w]), x) for w, x in zip("kv", before))


def test_decode_in_graphs_that_share_a_workspace(cuda_device):
    """Two captured calls on one workspace, replayed one after the other, and
    with new lengths, pages and queries in the same buffers."""
    lens = [500, 77, 0, 260]
    c = make_cache("e4m3", lens, 16, 2, 128, seed=5)
    from speculative_flash_decoding_b200 import PagedDecoder
    dec = PagedDecoder(_cache(c), 4, 8)
    full = PagedDecoder(_cache(c), 4, 8, n_sink=4, window=40)
    full.workspace = dec.workspace
    q = torch.randn(4, 8, 128, device="cuda").to(BF16)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    outs = [torch.empty(4, 8, 128, device="cuda") for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        for d, o in zip((dec, full), outs):
            d.decode(q, c["table"], seq, out=o)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                d.decode(q, c["table"], seq, out=o)
            graphs.append(g)
    torch.cuda.synchronize()
    for trial in range(3):
        q.copy_(torch.randn(4, 8, 128, generator=torch.Generator().manual_seed(trial)))
        now = [max(0, n - 13 * trial) for n in lens]
        seq.copy_(torch.tensor(now, dtype=torch.int32))
        for o, g in zip(outs, graphs):
            o.zero_()
            g.replay()
        torch.cuda.synchronize()
        for o, (a, w) in zip(outs, ((0, 0), (4, 40))):
            ref = attention(q, c["k64"], c["v64"], now, a, w)
            check_attention(o, None, ref, now, 128, "e4m3", F32)
    assert dec.device_error() == (0, 0)


def test_decode_on_two_streams_at_once(cuda_device):
    lens = [3000, 1000]
    c = make_cache("bf16", lens, 16, 4, 64, seed=5)
    from speculative_flash_decoding_b200 import PagedDecoder
    cache = _cache(c)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    runs = []
    for i in range(2):
        runs.append((PagedDecoder(cache, 2, 8), torch.cuda.Stream(),
                     torch.randn(2, 8, 64, device="cuda").to(BF16),
                     torch.empty(2, 8, 64, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for dec, s, q, o in runs:
            dec.decode(q, c["table"], seq, out=o, stream=s)
    torch.cuda.synchronize()
    for dec, s, q, o in runs:
        check_attention(o, None, attention(q, c["k64"], c["v64"], lens), lens, 64, "bf16", F32)


def test_new_output_comes_from_the_memory_of_its_stream(cuda_device):
    """Freed memory that the current stream still writes is not handed to a
    call on another stream."""
    from speculative_flash_decoding_b200 import Linear, PagedCache, PagedDecoder
    side = torch.cuda.Stream()
    lin = Linear(torch.ones(4096, 64, dtype=BF16, device="cuda"))
    x = torch.ones(64, 64, dtype=BF16, device="cuda")
    dec = PagedDecoder(PagedCache(8, 16, 2, 64), 64, 64)
    q = torch.ones((64, 64, 64), dtype=BF16, device="cuda")
    table = torch.zeros((64, 1), dtype=torch.int32, device="cuda")
    lens = torch.zeros(64, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for shape, call, value in (((64, 4096), lambda: lin.apply(x, stream=side), 64.0),
                               ((64, 64, 64), lambda: dec.decode(q, table, lens, stream=side), 0.0)):
        old = torch.empty(shape, dtype=BF16, device="cuda")
        at = old.data_ptr()
        torch.cuda._sleep(20_000_000)  # some milliseconds
        old.fill_(7.0)
        del old
        out = call()
        assert out.data_ptr() != at
        torch.cuda.synchronize()
        assert torch.equal(out, torch.full_like(out, value))


def test_broadcast_rows_are_refused(cuda_device):
    """A stride of 0 means contiguous rows to the C entry points."""
    from speculative_flash_decoding_b200 import PagedCache, PagedDecoder
    cache = PagedCache(8, 16, 2, 64)
    table = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    one = torch.zeros((1, 2, 64), dtype=BF16, device="cuda")
    for k, v in ((one.expand(3, 2, 64), one.repeat(3, 1, 1)),
                 (one.repeat(3, 1, 1), one.expand(3, 2, 64))):
        with pytest.raises(ValueError, match="broadcast"):
            cache.append(k, v, pos, table)
    with pytest.raises(ValueError, match="broadcast"):
        PagedDecoder(cache, 3, 2).decode(one.expand(3, 2, 64), table, pos)
    pool = one.reshape(2, 1, 1, 64)[:1].expand(4, 2, 16, 64)
    with pytest.raises(ValueError, match="strides"):
        PagedCache.from_tensors(pool, pool)
    # One row has no stride to be broadcast by.
    cache.append(one.expand(1, 2, 64), one, pos[:1], table[:1])
    assert cache.device_error() == (0, 0)


def test_offsets_past_32_bits(cuda_device):
    """Pages whose element offsets pass 2^32: written, read back, attended."""
    from speculative_flash_decoding_b200 import PagedCache, PagedDecoder
    page, hkv, d = 64, 8, 128
    n_pages = (1 << 32) // (page * hkv * d) + 3
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    k, v = (torch.empty((n_pages, hkv, page, d), dtype=BF16, device="cuda") for _ in range(2))
    cache = PagedCache.from_tensors(k, v)
    n = 100
    x = torch.randn(2, n, hkv, d, generator=torch.Generator().manual_seed(0)).to(BF16)
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device="cuda")
    xs = x.cuda()
    cache.append(xs[0], xs[1], torch.arange(n, dtype=torch.int32, device="cuda"), table,
                 seq_ids=torch.zeros(n, dtype=torch.int32, device="cuda"))
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    ko, vo = (torch.empty(1, hkv, n, d, dtype=BF16, device="cuda") for _ in range(2))
    cache.gather(table, lens, ko, vo)
    assert torch.equal(ko[0].transpose(0, 1).cpu(), x[0])
    assert torch.equal(vo[0].transpose(0, 1).cpu(), x[1])
    q = torch.randn(1, 16, d, device="cuda").to(BF16)
    out = PagedDecoder(cache, 1, 16).decode(q, table, lens, out=torch.empty(1, 16, d, device="cuda"))
    ref = attention(q, x[0].double().transpose(0, 1)[None], x[1].double().transpose(0, 1)[None], [n])
    check_attention(out, None, ref, [n], d, "bf16", F32)


@pytest.mark.parametrize("dtype,out", [("f32", F32), ("bf16", F32), ("e4m3", F32)])
def test_long_sums_keep_fp32(cuda_device, dtype, out):
    """Many tiles a warp: the result as a whole is within 2^-19.  A tile's
    products lose at most eight steps of 2^-23 (towards zero, so the whole
    shrinks by 2^-20 at most), tiles are added rounding to nearest (2^-24
    each, without a direction), and scores and exponentials are within 2^-21
    on the average."""
    lens = [30000] * 8
    c = make_cache(dtype, lens, 64, 2, 64, seed=21)
    _, q, _, got, _ = _decode(c, lens, 4, 64, out, dtype=dtype)
    ref = attention(q, c["k64"], c["v64"], lens)[0]
    rel = float((got.double().cpu() - ref).norm() / ref.norm())
    assert rel <= 2.0 ** -19, rel


def test_shared_pages(cuda_device):
    """Two sequences that share their first pages."""
    c = make_cache("bf16", [160, 64], 16, 2, 64, seed=8)
    c["table"][1, :4] = c["table"][0, :4]
    c["k64"][1, :, :64], c["v64"][1, :, :64] = c["k64"][0, :, :64], c["v64"][0, :, :64]
    _, q, _, got, lse = _decode(c, [160, 64], 4, 64, F32)
    check_attention(got, lse, attention(q, c["k64"], c["v64"], [160, 64]), [160, 64], 64, "bf16", F32)




@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("f32", 128)])
@pytest.mark.parametrize("page", [8, 16, 24, 64])
@pytest.mark.parametrize("n_sink,window", [(4, 20), (0, 1), (40, 0), (4, 0), (1, 64), (33, 31)])
def test_sink_set_of_a_cache_that_has_freed_the_rest(cuda_device, dtype, d, page, n_sink, window):
    """Table entries without a token of the sink set are not looked at: a
    sequence may have given those pages back."""
    from paged_reference import attended
    lens = [700, 65, 24, 1, 0, 333, 96, 1000, 21, 30]
    c = make_cache(dtype, lens, page, 2, d, token_major=page == 24, seed=page + window)
    table = torch.full_like(c["table"], -1)
    for b, n in enumerate(lens):
        kept = attended(n, n_sink, window).div(page, rounding_mode="floor").unique().cuda()
        table[b, kept] = c["table"][b, kept]
    assert bool((table != c["table"]).any())
    c["table"] = table
    for out in (F32, BF16):
        # (Also checks that the error word is clear.)
        _, q, _, got, lse = _decode(c, lens, 6, d, out, n_sink, window, seed=page, dtype=dtype)
        ref = attention(q, c["k64"], c["v64"], lens, n_sink, window)
        check_attention(got, lse, ref, lens, d, dtype, out)
