"""Plain 64-bit forms of the paged-cache operators, and inputs for their tests.

Rounding units (half a step, relative): bf16 2^-8 of a value's power of two,
written U_BF16; fp32 2^-24; see the bounds beside each use.
"""
import math

import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def make_cache(dtype, lens, page, hkv, d, token_major=False, seed=0, device="cuda", spare=3,
               v_scale_span=0.0):
    """Pools, table (unused entries -1, pages in random order) and the values
    [B, Hkv, max(len), d] in fp64.  Unwritten rows hold NaN.  v_scale_span:
    the V scales of an e4m3 cache spread over 2^+-span."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    used = [-(-n // page) for n in lens]
    n_pages = sum(used) + spare
    order = torch.randperm(n_pages, generator=g)
    width = max(1, max(used))
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    shape = (n_pages, page, hkv, d) if token_major else (n_pages, hkv, page, d)
    pools, scales = [], []
    for w in range(2):
        x = torch.randn(shape, generator=g)
        if dtype == "e4m3":
            x = (x * 100).clamp(-448, 448)
            s = torch.rand((n_pages, hkv, page), generator=g) * 0.01 + 0.005
            if w == 1 and v_scale_span:
                s = s * torch.exp2((torch.rand(s.shape, generator=g) * 2 - 1) * v_scale_span)
            scales.append(s)
        x = x.to(DTYPES[dtype])
        pools.append(x.transpose(1, 2) if token_major else x)
    at = 0
    values = [torch.zeros(len(lens), hkv, max(1, max(lens)), d, dtype=torch.float64)
              for _ in range(2)]
    for b, n in enumerate(lens):
        table[b, : used[b]] = order[at: at + used[b]].int()
        at += used[b]
        for i in range(used[b]):
            p = int(table[b, i])
            rows = min(page, n - i * page)
            for w in range(2):
                x = pools[w][p, :, :rows].double()
                if dtype == "e4m3":
                    x = x * scales[w][p, :, :rows].double()[..., None]
                    pools[w].view(torch.uint8)[p, :, rows:] = 0x7F
                    scales[w][p, :, rows:] = math.nan
                else:
                    pools[w][p, :, rows:] = math.nan
                values[w][b, :, i * page: i * page + rows] = x
    dev = torch.device(device)

    def move(x):  # keeps the strides of a token-major pool
        return x.transpose(1, 2).contiguous().to(dev).transpose(1, 2) if token_major else x.to(dev)

    return dict(k=move(pools[0]), v=move(pools[1]),
                ks=scales[0].to(dev) if scales else None, vs=scales[1].to(dev) if scales else None,
                table=table.to(dev), k64=values[0], v64=values[1], n_pages=n_pages)


def attended(n, n_sink, window):
    t = torch.arange(n)
    if n_sink + window == 0:
        return t
    return t[(t < n_sink) | (t >= n - window)]


def attention(q, k64, v64, lens, n_sink=0, window=0, scale=None):
    """(out, lse, A, E) in fp64: A = sum_t p_t |v_t|, E = the largest
    sum_i |q_i k_ti| * scale of a head (what a score's rounding is relative
    to)."""
    B, Hq, d = q.shape
    hkv = k64.shape[1]
    g = Hq // hkv
    scale = scale or 1 / math.sqrt(d)
    out = torch.zeros(B, Hq, d, dtype=torch.float64)
    A = torch.zeros_like(out)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    E = torch.zeros(B, Hq, dtype=torch.float64)
    q = q.double().cpu().view(B, hkv, g, d)
    for b, n in enumerate(lens):
        t = attended(n, n_sink, window)
        if not len(t):
            continue
        k, v = k64[b][:, t], v64[b][:, t]
        s = torch.einsum("hgd,hld->hgl", q[b], k) * scale
        E[b] = (torch.einsum("hgd,hld->hgl", q[b].abs(), k.abs()) * abs(scale)).amax(-1).flatten()
        p = torch.softmax(s, -1)
        lse[b] = torch.logsumexp(s, -1).flatten()
        out[b] = torch.einsum("hgl,hld->hgd", p, v).reshape(Hq, d)
        A[b] = torch.einsum("hgl,hld->hgd", p, v.abs()).reshape(Hq, d)
    return out, lse, A, E


def attention_bound(ref, lens, d, dtype, out_dtype):
    """Largest admissible error of (out, lse).

    fp32 MMA sums lose at most 2^-23 of the running magnitude per step (the
    accumulators may truncate): a score has d / 8 steps at most (twice that
    with a split operand), and the split query and tf32 terms lose 2^-22 more;
    its error es moves every weight by es relative, numerator and denominator
    alike (2 es).  exp2 and the scale's product: 2^-22 of a weight and 2^-23
    of a score.  A weight held as two bf16 terms loses 2^-18, as three 2^-26,
    as two f16 or tf32 terms 2^-22 (f16 below its normal range: 2^-25 of the
    largest).  Sums over n tokens: n / 8 + 64 steps of 2^-23 (tiles, warps and
    CTAs joined).  The output is then rounded once (U)."""
    out, lse, A, E = ref
    n = torch.tensor(lens, dtype=torch.float64)[:, None]
    es = E * ((d / 4 + 8) * 2.0 ** -23) + 2.0 ** -21
    weight = 2.0 ** -21 if dtype != "bf16" or out_dtype is torch.float32 else 2.0 ** -18
    rel = 2 * es + weight + (n / 8 + 64) * 2.0 ** -23
    lse_bound = es + (n / 8 + 64) * 2.0 ** -23 + lse.abs().nan_to_num(posinf=0.0) * 2.0 ** -22
    return U[out_dtype] * out.abs() + rel[..., None] * A + 1e-37, lse_bound


def check_attention(got, got_lse, ref, lens, d, dtype, out_dtype):
    bound, lse_bound = attention_bound(ref, lens, d, dtype, out_dtype)
    err = (got.double().cpu() - ref[0]).abs()
    assert bool((err <= bound).all()), f"largest error / bound {(err / bound).max():.3g}"
    if got_lse is not None:
        empty = torch.tensor(lens) == 0
        got_lse = got_lse.double().cpu()
        assert bool((got_lse[empty] == -math.inf).all())
        e = (got_lse - ref[1])[~empty].abs()
        assert bool((e <= lse_bound[~empty]).all()), f"{(e / lse_bound[~empty]).max():.3g}"


def quantise(x):
    """(codes, scales) of alspec_paged_append for fp32 or bf16 rows, on CPU:
    every step in fp32 (a quotient of fp32 values taken in fp64 and rounded to
    fp32 is the fp32 quotient)."""
    x = x.cpu().double()
    amax = x.abs().amax(-1)
    s = (amax / 448.0).float().double().clamp(min=2.0 ** -126)
    code = (x / s[..., None]).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    return code, s.float()
