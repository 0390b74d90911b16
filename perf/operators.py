"""Serving operators around a paged key-value cache, as cases to measure.

Four operators, as one decode layer uses them:
  append  the new tokens' keys and values written into their pages (e4m3
          pages: quantised with one scale per token and KV head);
  decode  softmax attention of one new token per sequence over its pages;
  linear  y = activation(x W^T + bias) + residual for a decode batch;
  gather  pages read back (dequantised) into one contiguous cache.

``run`` computes them in elementary torch operations, or, with ``own`` set,
with the package's PagedCache, PagedDecoder and Linear.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the smallest scale that append writes


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One decode step of a batch of 96 sequences (two of its rows are
        # padding): the new token of each goes into e4m3 pages; k and v are
        # slices of one fused projection's rows.
        dict(name="append-step", op="append", tokens=96, batch=96, hkv=8, d=128, page=16,
             cache="e4m3", src="bf16", padded=2, lo=1, hi=4096, fused=True, token_major=False),
        # A prompt chunk of three sequences, 16411 tokens in all.
        dict(name="append-prompt", op="append", tokens=16411, batch=3, hkv=8, d=128, page=64,
             cache="e4m3", src="bf16", padded=0, lo=0, hi=20000, fused=False, token_major=False),
        # Reading back one short sequence of fp32 pages.
        dict(name="gather-short", op="gather", batch=1, hkv=4, d=64, page=16, cache="f32",
             out="f32", lo=777, hi=777, token_major=False),
        # A ragged batch of 8 (16K to 64K tokens) from e4m3 pages into the
        # contiguous bf16 cache that the speculative decode reads.
        dict(name="gather-ragged", op="gather", batch=8, hkv=8, d=128, page=16, cache="e4m3",
             out="bf16", lo=16384, hi=65536, token_major=False),
        # The smallest call: one sequence of 1K tokens, one KV head, fp32.
        dict(name="decode-one-1k", op="decode", batch=1, hq=4, hkv=1, d=64, page=16, cache="f32",
             out="f32", lo=1024, hi=1024, empty=0, n_sink=0, window=0, token_major=False),
        # A long context alone: 128K tokens, 32 query heads on 8 KV heads.
        dict(name="decode-one-128k", op="decode", batch=1, hq=32, hkv=8, d=128, page=64,
             cache="bf16", out="bf16", lo=131072, hi=131072, empty=0, n_sink=0, window=0,
             token_major=False),
        # A ragged batch of long contexts over a quantised cache.
        dict(name="decode-ragged-e4m3", op="decode", batch=8, hq=32, hkv=8, d=128, page=16,
             cache="e4m3", out="bf16", lo=16384, hi=65536, empty=0, n_sink=0, window=0,
             token_major=False),
        # Chat traffic: 128 short sequences of odd lengths, five rows of the
        # batch unused, token-major pages of 24 tokens, 3 query heads a KV head.
        dict(name="decode-batch-short", op="decode", batch=128, hq=24, hkv=8, d=64, page=24,
             cache="bf16", out="f32", lo=1, hi=900, empty=5, n_sink=0, window=0,
             token_major=True),
        # Attention over the sink set alone (first 4 and last 1024 tokens).
        dict(name="decode-sink-set", op="decode", batch=32, hq=64, hkv=8, d=128, page=16,
             cache="bf16", out="bf16", lo=8192, hi=32768, empty=0, n_sink=4, window=1024,
             token_major=False),
        # The output projection of one token with its residual.
        dict(name="linear-one", op="linear", rows=1, k=4096, n=4096, act="none", bias=False,
             residual=True, out="f32", pad=0),
        # The fused query, key and value projection of a batch of 33.
        dict(name="linear-qkv-33", op="linear", rows=33, k=4096, n=6144, act="none", bias=True,
             residual=False, out="bf16", pad=64),
        # A large decode batch through a square layer with activation.
        dict(name="linear-square-250", op="linear", rows=250, k=8192, n=8192, act="silu",
             bias=True, residual=True, out="bf16", pad=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "gather", "decode", "decode", "decode", "linear", "linear"])
    if op == "linear":
        k = 8 * _log(rng, 1, 1024)
        n = _log(rng, 1, 8192)
        return dict(op=op, rows=_log(rng, 1, 512), k=k, n=n,
                    act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "f32"]),
                    pad=rng.choice([0, 0, 8]))
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128])
    cache = rng.choice(["bf16", "bf16", "e4m3", "e4m3", "f32"])
    token_major = rng.random() < 0.3
    if op == "append":
        if rng.random() < 0.5:
            batch = tokens = _log(rng, 1, 512)
        else:
            batch, tokens = _log(rng, 1, 9), _log(rng, 16, 16384)
        return dict(op=op, tokens=tokens, batch=batch, hkv=hkv, d=d, page=page, cache=cache,
                    src=rng.choice(["bf16", "bf16", "f32"]),
                    padded=rng.randrange(3) if tokens == batch and tokens > 4 else 0,
                    lo=1 if tokens == batch else 0, hi=_log(rng, 64, 8192) + (tokens if tokens != batch else 0),
                    fused=rng.random() < 0.5, token_major=token_major)
    batch = _log(rng, 1, 192)
    most = 1 << (26 if op == "gather" else 27)  # values of one pool
    hi = _log(rng, 1, max(1, min(131072, most // (batch * hkv * d))))
    lo = hi if rng.random() < 0.3 else rng.randint(max(1, hi // 8), hi)
    if op == "gather":
        return dict(op=op, batch=batch, hkv=hkv, d=d, page=page, cache=cache,
                    out=rng.choice(["bf16", "f32"]), lo=lo, hi=hi, token_major=token_major)
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16])
    sinks = rng.random() < 0.25
    return dict(op=op, batch=batch, hq=hkv * group, hkv=hkv, d=d, page=page, cache=cache,
                out="f32" if cache == "f32" else rng.choice(["bf16", "bf16", "f32"]), lo=lo, hi=hi,
                empty=rng.randrange(1, 4) if batch > 6 and rng.random() < 0.4 else 0,
                n_sink=rng.choice([0, 4, 33]) if sinks else 0,
                window=_log(rng, 1, 2048) if sinks else 0, token_major=token_major)


def _rng(case):
    """Lengths and page numbers are the case's, whatever the seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lens(case):
    r = _rng(case)
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    if case["op"] != "append":
        lens[r.randrange(case["batch"])] = case["hi"]
        for b in r.sample(range(case["batch"]), case.get("empty", 0)):
            lens[b] = 0
    return lens


def _append_plan(case):
    """(sequence, position) of every token; position -1 is padding."""
    r = _rng(case)
    batch, tokens = case["batch"], case["tokens"]
    if tokens == batch:
        pos = [n - 1 for n in _lens(case)]
        for b in r.sample(range(batch), case["padded"]):
            pos[b] = -1
        return list(range(batch)), pos
    cuts = sorted(r.randint(0, tokens) for _ in range(batch - 1))
    seq, pos = [], []
    for b, (x, y) in enumerate(zip([0] + cuts, cuts + [tokens])):
        start = r.randint(0, max(0, case["hi"] - tokens))
        seq += [b] * (y - x)
        pos += range(start, start + y - x)
    return seq, pos


# ---------------------------------------------------------------- prepare

def _pages(case, lens, gen):
    """Pages in random order, the table of each sequence, and pages' values
    N(0, 1); the unwritten rows of a last page hold NaN, unused table
    entries -1."""
    dev = torch.device("cuda")
    hkv, d, page = case["hkv"], case["d"], case["page"]
    used = [-(-n // page) for n in lens]
    width = max(1, max(used))
    n_pages = sum(used) + 5
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    row = torch.tensor(used, device=dev)[:, None] > torch.arange(width, device=dev)[None, :]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=dev)
    table[row] = order[: sum(used)]
    # One page more than the cache has: the plain form of append drops its
    # padding tokens there.
    shape = (n_pages + 1, page, hkv, d) if case["token_major"] else (n_pages + 1, hkv, page, d)

    def pool():
        x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16
                        if case["cache"] == "bf16" else torch.float32)
        if case["cache"] == "e4m3":
            x = (x * 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return x.transpose(1, 2) if case["token_major"] else x

    def scales():
        if case["cache"] != "e4m3":
            return None
        return torch.rand((n_pages + 1, hkv, page), generator=gen, device=dev) * 0.01 + 0.005

    k, v = pool(), pool()
    ks, vs = scales(), scales()
    if case["op"] != "append":
        at = torch.arange(width * page, device=dev).view(1, width, page)
        stale = row[:, :, None] & (at >= torch.tensor(lens, device=dev)[:, None, None])
        b, p, off = stale.nonzero(as_tuple=True)
        ids = table[b, p].long()
        nan = 0x7F if case["cache"] == "e4m3" else float("nan")
        for x in (k, v):
            (x.view(torch.uint8) if case["cache"] == "e4m3" else x)[ids, :, off] = nan
    return dict(k_all=k, v_all=v, ks_all=ks, vs_all=vs, table=table, n_pages=n_pages)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    st = dict(case=case)
    if case["op"] == "linear":
        rows, k, n = case["rows"], case["k"], case["n"]
        x = torch.randn((rows, k + case["pad"]), generator=gen, device=dev).to(torch.bfloat16)
        st["x"] = x[:, :k]
        st["w"] = (torch.randn((n, k), generator=gen, device=dev) / math.sqrt(k)).to(torch.bfloat16)
        st["bias"] = (torch.randn(n, generator=gen, device=dev).to(torch.bfloat16)
                      if case["bias"] else None)
        st["residual"] = (torch.randn((rows, n), generator=gen, device=dev).to(DTYPES[case["out"]])
                          if case["residual"] else None)
        st["out"] = torch.empty((rows, n), device=dev, dtype=DTYPES[case["out"]])
        if own:
            from speculative_flash_decoding_b200 import Linear
            st["linear"] = Linear(st["w"], bias=st["bias"], activation=case["act"])
        return st
    if case["op"] == "append":
        seq, pos = _append_plan(case)
        lens = [0] * case["batch"]
        for s, p in zip(seq, pos):
            lens[s] = max(lens[s], p + 1)
        st |= _pages(case, lens, gen)
        n, row = case["tokens"], case["hkv"] * case["d"]
        wide = torch.randn((n, 2 * row + (64 if case["fused"] else 0)), generator=gen, device=dev)
        wide = wide.to(DTYPES[case["src"]])
        st["k"] = wide[:, :row].unflatten(1, (case["hkv"], case["d"]))
        st["v"] = wide[:, row:2 * row].unflatten(1, (case["hkv"], case["d"]))
        if not case["fused"]:
            st["k"], st["v"] = st["k"].contiguous(), st["v"].contiguous()
        st["positions"] = torch.tensor(pos, dtype=torch.int32, device=dev)
        # A decode step's token i is sequence i's: it needs no sequence ids.
        st["seq_ids"] = (torch.tensor(seq, dtype=torch.int32, device=dev)
                         if case["tokens"] != case["batch"] else None)
    else:
        lens = _lens(case)
        st |= _pages(case, lens, gen)
        st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        if case["op"] == "gather":
            shape = (case["batch"], case["hkv"], max(lens), case["d"])
            st["k_out"] = torch.randn(shape, generator=gen, device=dev, dtype=DTYPES[case["out"]])
            st["v_out"] = torch.randn(shape, generator=gen, device=dev, dtype=DTYPES[case["out"]])
        else:
            qt = torch.float32 if case["cache"] == "f32" else torch.bfloat16
            shape = (case["batch"], case["hq"], case["d"])
            # Logits of standard deviation 2: some tokens stand out.
            st["q"] = (2.0 * torch.randn(shape, generator=gen, device=dev)).to(qt)
            st["out"] = torch.empty(shape, device=dev, dtype=DTYPES[case["out"]])
            st["lse"] = torch.empty(shape[:2], device=dev, dtype=torch.float32)
    m = st["n_pages"]
    for name in ("k", "v"):
        st[name + "_pages"] = st[name + "_all"][:m]
        s = st[name + "s_all"]
        st[name + "_scales"] = None if s is None else s[:m]
    if own:
        from speculative_flash_decoding_b200 import PagedCache, PagedDecoder
        st["cache"] = PagedCache.from_tensors(st["k_pages"], st["v_pages"], st["k_scales"],
                                              st["v_scales"])
        if case["op"] == "decode":
            st["decoder"] = PagedDecoder(st["cache"], case["batch"], case["hq"],
                                         n_sink=case["n_sink"], window=case["window"])
    return st


# -------------------------------------------------------------------- run

def _read(pages, scales, table):
    """[B, H, L, d] in fp32 of every table entry's page (unused: page 0)."""
    ids = table.clamp(min=0).long()
    x = pages.view(torch.uint8)[ids].view(pages.dtype) if scales is not None else pages[ids]
    x = x.float()
    if scales is not None:
        x = x * scales[ids][..., None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _attended(st, length):
    case, lens = st["case"], st["seq_lens"].long()[:, None]
    at = torch.arange(length, device=lens.device)[None, :]
    ok = at < lens
    if case["n_sink"] or case["window"]:
        ok = ok & ((at < case["n_sink"]) | (at >= lens - case["window"]))
    return ok


def _decode(st):
    case = st["case"]
    b, hq, d = st["q"].shape
    hkv = case["hkv"]
    k = _read(st["k_pages"], st["k_scales"], st["table"])
    ok = _attended(st, k.shape[2])[:, None, None, :]
    q = st["q"].float().view(b, hkv, hq // hkv, d)
    s = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    del k
    s = torch.where(ok, s, -torch.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.where(ok, torch.exp(s - torch.where(m == -torch.inf, 0.0, m)), 0.0)
    total = p.sum(-1, keepdim=True)
    v = _read(st["v_pages"], st["v_scales"], st["table"])
    v = torch.where(ok.transpose(2, 3), v, 0.0)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return dict(out=o.view(b, hq, d).to(st["out"].dtype),
                lse=(m + torch.log(total)).view(b, hq))


def _quantise(x):
    """e4m3 codes and one scale per row: amax / 448, at least 2^-126."""
    x = x.float()
    amax = x.abs().amax(-1)
    scale = (amax / torch.full_like(amax, E4M3_MAX)).clamp(min=TINY)
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _append(st):
    case, pos = st["case"], st["positions"].long()
    seq = st["seq_ids"].long() if st["seq_ids"] is not None else torch.arange(
        case["tokens"], device=pos.device)
    kept = pos >= 0
    page = st["table"][seq, pos.clamp(min=0) // case["page"]].long()
    page = torch.where(kept, page, st["n_pages"])
    off = pos.clamp(min=0) % case["page"]
    for name in ("k", "v"):
        pages = st[name + "_all"]
        if case["cache"] == "e4m3":
            code, scale = _quantise(st[name])
            pages.view(torch.uint8)[page, :, off] = code.view(torch.uint8)
            st[name + "s_all"][page, :, off] = scale
        else:
            pages[page, :, off] = st[name].to(pages.dtype)
    return _append_out(st)


def _append_out(st):
    return {name: st[name] for name in ("k_pages", "v_pages", "k_scales", "v_scales")
            if st[name] is not None}


def _gather(st):
    for name in ("k", "v"):
        out = st[name + "_out"]
        x = _read(st[name + "_pages"], st[name + "_scales"], st["table"])[:, :, : out.shape[2]]
        ok = (torch.arange(out.shape[2], device=x.device) < st["seq_lens"][:, None])[:, None, :, None]
        out.copy_(torch.where(ok, x.to(out.dtype), out))
    return dict(k=st["k_out"], v=st["v_out"])


def _activate(y, act):
    if act == "relu":
        return torch.where(y < 0, 0.0, y)
    if act == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    if act == "silu":
        return y / (1.0 + torch.exp(-y))
    return y


def _linear(st):
    y = torch.matmul(st["x"].float(), st["w"].float().t())
    if st["bias"] is not None:
        y = y + st["bias"].float()
    y = _activate(y, st["case"]["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(st["out"].dtype)


def _own(st):
    op = st["case"]["op"]
    if op == "linear":
        return st["linear"].apply(st["x"], residual=st["residual"], out=st["out"])
    if op == "append":
        st["cache"].append(st["k"], st["v"], st["positions"], st["table"], seq_ids=st["seq_ids"])
        return _append_out(st)
    if op == "gather":
        st["cache"].gather(st["table"], st["seq_lens"], st["k_out"], st["v_out"])
        return dict(k=st["k_out"], v=st["v_out"])
    out = st["decoder"].decode(st["q"], st["table"], st["seq_lens"], out=st["out"], lse=st["lse"])
    return dict(out=out, lse=st["lse"])


def run(state):
    if own:
        return _own(state)
    return {"linear": _linear, "append": _append, "gather": _gather,
            "decode": _decode}[state["case"]["op"]](state)


# ------------------------------------------------------------------- work

def work(case):
    size = {"f32": 4, "bf16": 2, "e4m3": 1}
    if case["op"] == "linear":
        rows, k, n, out = case["rows"], case["k"], case["n"], size[case["out"]]
        return dict(bytes=2 * n * k + 2 * rows * k + rows * n * out * (2 if case["residual"] else 1)
                    + (2 * n if case["bias"] else 0), flops=2 * rows * n * k)
    row = case["d"] * size[case["cache"]] + (4 if case["cache"] == "e4m3" else 0)
    if case["op"] == "append":
        n = (case["tokens"] - case["padded"]) * case["hkv"] * 2
        return dict(bytes=n * (case["d"] * size[case["src"]] + row) + 12 * case["tokens"],
                    flops=2 * n * case["d"])
    lens = _lens(case)
    if case["op"] == "gather":
        n = sum(lens) * case["hkv"] * 2
        return dict(bytes=n * (row + case["d"] * size[case["out"]]), flops=n * case["d"])
    if case["n_sink"] or case["window"]:
        lens = [min(x, case["n_sink"] + case["window"]) for x in lens]
    out = case["batch"] * case["hq"] * (case["d"] * (size[case["out"]] + (
        4 if case["cache"] == "f32" else 2)) + 4)
    return dict(bytes=2 * sum(lens) * case["hkv"] * row + out,
                flops=4 * sum(lens) * case["hq"] * case["d"])


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """The operators' definitions in 64 bits, one sequence at a time."""
    st = prepare(case, seed)
    if case["op"] == "linear":
        y = torch.einsum("rk,nk->rn", st["x"].double(), st["w"].double())
        if case["bias"]:
            y += st["bias"].double()[None]
        if case["act"] == "relu":
            y = y.clamp(min=0)
        elif case["act"] == "gelu":
            y = y * (1 + torch.special.erf(y / math.sqrt(2))) / 2
        elif case["act"] == "silu":
            y = y * torch.special.expit(y)
        return y + st["residual"].double() if case["residual"] else y
    page = case["page"]
    if case["op"] == "append":
        seq, pos = _append_plan(case)
        keep = torch.tensor([i for i, p in enumerate(pos) if p >= 0], device="cuda")
        s, p = (torch.tensor(x, device="cuda")[keep] for x in (seq, pos))
        ids, off = st["table"][s, p // page].long(), p % page
        out = {}
        for name in ("k", "v"):
            x = st[name][keep].double()
            if case["cache"] != "e4m3":
                y = st[name + "_pages"].double()
                # A cache of fewer bits holds the value rounded to its type.
                y[ids, :, off] = x
                out[name + "_pages"] = y
                continue
            # The scale is held in 32 bits; a code is the e4m3 value nearest
            # to the 32-bit quotient.
            scale = (x.abs().amax(-1) / E4M3_MAX).float().double().clamp(min=TINY)
            code = (x / scale[..., None]).float().to(torch.float8_e4m3fn)
            y, z = st[name + "_pages"].float().double(), st[name + "_scales"].double()
            y[ids, :, off], z[ids, :, off] = code.float().double(), scale
            out[name + "_pages"], out[name + "_scales"] = y, z
        return out
    lens = _lens(case)

    def rows(name, b, which):
        at = st["table"][b, which // page].long(), which % page
        x = st[name + "_pages"].view(torch.uint8)[at[0], :, at[1]].view(
            torch.float8_e4m3fn) if case["cache"] == "e4m3" else st[name + "_pages"][at[0], :, at[1]]
        x = x.double()
        if case["cache"] == "e4m3":
            x = x * st[name + "_scales"][at[0], :, at[1]].double()[..., None]
        return x  # [tokens, H, d]

    if case["op"] == "gather":
        out = {}
        for name in ("k", "v"):
            y = st[name + "_out"].double()
            for b, n in enumerate(lens):
                y[b, :, :n] = rows(name, b, torch.arange(n, device="cuda")).transpose(0, 1)
            out[name] = y
        return out
    group = case["hq"] // case["hkv"]
    out = torch.zeros((case["batch"], case["hq"], case["d"]), dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], case["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        which = torch.arange(n, device="cuda")
        if case["n_sink"] or case["window"]:
            which = which[(which < case["n_sink"]) | (which >= n - case["window"])]
        if not len(which):
            continue
        k, v = rows("k", b, which), rows("v", b, which)
        q = st["q"][b].double().view(case["hkv"], group, case["d"])
        s = torch.einsum("hgd,lhd->hgl", q, k) / math.sqrt(case["d"])
        lse[b] = torch.logsumexp(s, -1).flatten()
        out[b] = torch.einsum("hgl,lhd->hgd", torch.softmax(s, -1), v).reshape(case["hq"], case["d"])
    return dict(out=out, lse=lse)
