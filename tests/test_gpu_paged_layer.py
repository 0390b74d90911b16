"""The paged operators together, as one decode layer uses them: the fused
projection of a batch's hidden states, its keys and values appended to their
pages, attention over the pages, the output projection with its residual --
eagerly and captured in one graph -- and pages read back for the speculative
decode over a contiguous cache."""
import math

import pytest
import torch

from paged_reference import attention, attention_bound, check_attention, make_cache, quantise
from test_gpu_linear import _check as check_linear

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


class Layer:
    """A decode layer of `hq` query and `hkv` KV heads over a paged cache."""

    def __init__(self, dtype, batch, hq, hkv, d, page, max_pages, seed):
        import speculative_flash_decoding_b200 as sfd
        g = torch.Generator().manual_seed(seed)
        self.batch, self.hq, self.hkv, self.d, self.hidden = batch, hq, hkv, d, hq * d
        self.dtype = dtype
        n = (hq + 2 * hkv) * d
        self.w_qkv = (torch.randn(n, self.hidden, generator=g) / math.sqrt(self.hidden)).to(BF16).cuda()
        self.b_qkv = torch.randn(n, generator=g).to(BF16).cuda()
        self.w_o = (torch.randn(self.hidden, self.hidden, generator=g) / math.sqrt(self.hidden)).to(BF16).cuda()
        self.qkv_proj, self.o_proj = sfd.Linear(self.w_qkv, self.b_qkv), sfd.Linear(self.w_o)
        self.cache = sfd.PagedCache(batch * max_pages + 2, page, hkv, d, dtype)
        self.table = (torch.randperm(batch * max_pages, generator=g).int().view(batch, max_pages) + 1).cuda()
        self.decoder = sfd.PagedDecoder(self.cache, batch, hq)
        new = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
        self.qkv, self.attn, self.out = new(batch, n), new(batch, hq, d), new(batch, self.hidden)

    def step(self, x, positions, lens):
        hq, hkv, d = self.hq, self.hkv, self.d
        self.qkv_proj.apply(x, out=self.qkv)
        q, k, v = self.qkv.split([hq * d, hkv * d, hkv * d], dim=1)
        q, k, v = q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))
        self.cache.append(k, v, positions, self.table)
        self.decoder.decode(q, self.table, lens, out=self.attn)
        self.o_proj.apply(self.attn.view(self.batch, -1), residual=x, out=self.out)
        return self.out

    def check(self, x, k64, v64, lens):
        """Every stage against its definition on the inputs that it had."""
        hq, d = self.hq, self.d
        check_linear(self.qkv, x, self.w_qkv, self.b_qkv, None, "none")
        q = self.qkv[:, : hq * d].unflatten(1, (hq, d))
        check_attention(self.attn, None, attention(q, k64, v64, lens), lens, d,
                        self.dtype, BF16)
        check_linear(self.out, self.attn.view(self.batch, -1), self.w_o, None, x, "none")

    def new_rows(self):
        """What the cache holds of this step's keys and values, in fp64."""
        kv = self.qkv[:, self.hq * self.d:].unflatten(1, (2, self.hkv, self.d))
        out = []
        for w in range(2):
            x = kv[:, w]
            if self.dtype == "e4m3":
                code, s = quantise(x)
                out.append(code.double() * s.double()[..., None])
            else:
                out.append(x.double().cpu())
        return out


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("captured", [False, True])
def test_decode_steps(cuda_device, dtype, captured):
    """Eleven steps from empty caches, over the end of a page; one row of the batch stays padding."""
    B, hq, hkv, d, page, pages = 5, 12, 3, 64, 8, 2
    layer = Layer(dtype, B, hq, hkv, d, page, pages, seed=3)
    x = torch.zeros(B, hq * d, dtype=BF16, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    graph = None
    if captured:
        pos.fill_(-1)
        layer.step(x, pos, lens)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.step(x, pos, lens)
    k64 = torch.zeros(B, hkv, page * pages, d, dtype=torch.float64)
    v64 = torch.zeros_like(k64)
    for t in range(11):
        x.copy_(torch.randn(B, hq * d, generator=torch.Generator().manual_seed(t)))
        live = [t + 1] * (B - 1) + [0]
        pos.copy_(torch.tensor([t] * (B - 1) + [-1], dtype=torch.int32))
        lens.copy_(torch.tensor(live, dtype=torch.int32))
        graph.replay() if captured else layer.step(x, pos, lens)
        torch.cuda.synchronize()
        k, v = layer.new_rows()
        k64[:-1, :, t], v64[:-1, :, t] = k[:-1], v[:-1]
        layer.check(x, k64, v64, live)
        assert not layer.attn[-1].any()
    assert layer.decoder.device_error() == (0, 0)
    assert layer.cache.device_error() == (0, 0)


def test_pages_read_back_for_the_speculative_decode(cuda_device):
    """gather() makes the contiguous cache that Decoder takes: its O_exact
    and the paged attention agree with the same reference, its O_spec with
    the paged attention over the sink set."""
    import speculative_flash_decoding_b200 as sfd
    lens, S, W = [700, 260], 4, 128
    c = make_cache("bf16", lens, 16, 2, 128, seed=4)
    cache = sfd.PagedCache.from_tensors(c["k"], c["v"])
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(2, 2, 704, 128, dtype=BF16, device="cuda") for _ in range(2))
    cache.gather(c["table"], seq, k, v)
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    spec = sfd.Decoder(2, 8, 2, 128, 704, "bf16", S, W).decode(q, k, v, seq, 0.1)
    for name, (a, w) in (("out_exact", (0, 0)), ("out_spec", (S, W))):
        paged = sfd.PagedDecoder(cache, 2, 8, n_sink=a, window=w).decode(
            q, c["table"], seq, out=torch.empty(2, 8, 128, device="cuda"))
        ref = attention(q, c["k64"], c["v64"], lens, a, w)
        check_attention(paged, None, ref, lens, 128, "bf16", F32)
        # The contiguous decode holds weights to 16 bits, as bf16 outputs do.
        bound, _ = attention_bound(ref, lens, 128, "bf16", BF16)
        assert bool(((spec[name].double().cpu() - ref[0]).abs() <= bound).all())


def test_partial_attentions_join_by_their_lse(cuda_device):
    """A shared prefix attended to apart: the halves, weighted by their lse,
    make the whole."""
    import speculative_flash_decoding_b200 as sfd
    lens = [512, 512]
    c = make_cache("bf16", lens, 64, 2, 64, seed=4)
    cache = sfd.PagedCache.from_tensors(c["k"], c["v"])
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    dec = sfd.PagedDecoder(cache, 2, 4)
    n = torch.tensor([256, 256], dtype=torch.int32, device="cuda")
    parts = []
    for table in (c["table"][:, :4].contiguous(), c["table"][:, 4:].contiguous()):
        o, l = torch.empty(2, 4, 64, device="cuda"), torch.empty(2, 4, device="cuda")
        dec.decode(q, table, n, out=o, lse=l)
        parts.append((o.double(), l.double()))
    w = torch.softmax(torch.stack([l for _, l in parts]), 0)[..., None]
    got = (w * torch.stack([o for o, _ in parts])).sum(0)
    ref = attention(q, c["k64"], c["v64"], lens)
    bound, _ = attention_bound(ref, lens, 64, "bf16", F32)
    # Each half obeys its own bound, the weights move by the errors of two lse.
    assert bool(((got.cpu() - ref[0]).abs() <= 4 * bound).all())
