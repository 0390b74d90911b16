"""The linear layer with its epilogue on the GPU against its 64-bit form."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def _inputs(rows, n, k, pad=0, seed=0, bias=True, residual=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, k + pad), generator=g).to(BF16).cuda()[:, :k]
    w = (torch.randn((n, k), generator=g) / math.sqrt(k)).to(BF16).cuda()
    b = torch.randn(n, generator=g).to(BF16).cuda() if bias else None
    r = torch.randn((rows, n), generator=g).to(residual).cuda() if residual else None
    return x, w, b, r


ACT = {"none": lambda y: y, "relu": lambda y: y.clamp(min=0),
       "gelu": lambda y: 0.5 * y * (1 + torch.erf(y / math.sqrt(2))),
       "silu": lambda y: y * torch.sigmoid(y)}
# The largest slope of each activation, and what its own evaluation loses
# relative to its argument (erff and expf: a few units of 2^-23).
SLOPE = {"none": 1.0, "relu": 1.0, "gelu": 1.13, "silu": 1.1}


def _check(y, x, w, b, r, act):
    x, w = x.double(), w.double()
    z = x @ w.t()
    size = x.abs() @ w.abs().t()
    if b is not None:
        z, size = z + b.double(), size + b.double().abs()
    want = ACT[act](z)
    if r is not None:
        want = want + r.double()
    # fp32 sums of k exact products in steps of 16, each step losing at most
    # 2^-23 of the running magnitude, and up to 8 more for the split, bias and
    # residual; 2^-21 for the activation; the output's rounding.
    k = x.shape[1]
    extra = 0 if r is None else r.double().abs() * 2.0 ** -23
    bound = (SLOPE[act] * size * (k / 16 + 16) * 2.0 ** -23 + size * 2.0 ** -21 + extra
             + U[y.dtype] * want.abs() + 1e-37)
    err = (y.double() - want).abs()
    assert bool((err <= bound).all()), f"largest error / bound {(err / bound).max():.3g}"


@pytest.mark.parametrize("rows,n,k,act,out,bias,residual,pad", [
    (1, 1, 8, "none", F32, True, True, 0),
    (1, 4096, 4096, "none", F32, False, True, 0),
    (1, 130, 72, "relu", BF16, True, False, 8),
    (3, 257, 520, "gelu", F32, True, True, 0),
    (16, 128, 64, "none", F32, False, False, 0),
    (17, 1000, 4104, "silu", BF16, True, True, 64),
    (33, 6144, 4096, "none", BF16, True, False, 0),
    (64, 2048, 1024, "gelu", BF16, False, False, 0),
    (250, 512, 8192, "silu", F32, True, True, 0),
    (256, 384, 200, "relu", BF16, True, True, 0),
    (257, 300, 96, "none", F32, True, False, 0),
    (700, 129, 1032, "silu", BF16, True, True, 8),
    (2, 20000, 136, "none", F32, True, False, 0),
    # Pairs of CTAs: batches of more than 128 rows with bf16 outputs.
    (250, 256, 512, "none", BF16, False, False, 0),
    (129, 257, 64, "gelu", BF16, True, True, 0),
    (200, 1000, 4096, "silu", BF16, True, True, 8),
    (250, 8192, 1024, "none", BF16, True, False, 0),
    (1000, 140, 72, "relu", BF16, True, True, 0),
])
def test_linear(cuda_device, rows, n, k, act, out, bias, residual, pad):
    from speculative_flash_decoding_b200 import Linear
    x, w, b, r = _inputs(rows, n, k, pad, seed=rows + n, bias=bias,
                         residual=out if residual else None)
    layer = Linear(w, bias=b, activation=act)
    y = torch.full((rows, n), 9.0, dtype=out, device="cuda")
    assert layer.apply(x, residual=r, out=y) is y
    assert layer.device_error() == (0, 0)
    _check(y, x, w, b, r, act)
    again = layer.apply(x, residual=r, out=torch.empty_like(y))
    assert torch.equal(again, y)


def test_residual_in_place_and_guards(cuda_device):
    from speculative_flash_decoding_b200 import Linear
    rows, n, k = 5, 203, 328
    x, w, b, _ = _inputs(rows, n, k)
    buf = torch.randn(rows * n + 512, device="cuda")
    keep = buf.clone()
    y = buf[256: 256 + rows * n].view(rows, n)
    r = y.clone()
    Linear(w, bias=b).apply(x, residual=y, out=y)
    _check(y, x, w, b, r, "none")
    assert torch.equal(buf[:256], keep[:256]) and torch.equal(buf[-256:], keep[-256:])


def test_rows_of_one_do_not_touch_others(cuda_device):
    """NaN in one row of x stays in that row of y, in one row of W in that
    column."""
    from speculative_flash_decoding_b200 import Linear
    x, w, _, _ = _inputs(20, 150, 96, bias=False)
    x[7, 3] = math.nan
    w[149, 0] = math.nan
    y = Linear(w).apply(x, out_dtype=F32)
    bad = torch.zeros(20, 150, dtype=torch.bool, device="cuda")
    bad[7] = True
    bad[:, 149] = True
    assert torch.equal(y.isnan(), bad)
    z = Linear(w, activation="relu").apply(x, out_dtype=F32)
    assert torch.equal(z.isnan(), bad)


def test_activation_far_out(cuda_device):
    """Large arguments of either sign, and infinities."""
    from speculative_flash_decoding_b200 import Linear
    w = torch.eye(8, device="cuda").to(BF16)
    x = torch.tensor([[0.0, 1e30, -1e30, 100.0, -100.0, -88.0, 1e-30, -1e-30]], device="cuda").to(BF16)
    for act in ("gelu", "silu", "relu"):
        y = Linear(w, activation=act).apply(x, out_dtype=F32)
        want = ACT[act](x.double())
        assert bool(((y.double() - want).abs() <= 2.0 ** -20 * x.double().abs()).all()), act


def test_broadcast_rows_are_refused(cuda_device):
    """A stride of 0 means contiguous rows to the C entry point."""
    from speculative_flash_decoding_b200 import Linear
    lin = Linear(torch.zeros(16, 64, dtype=torch.bfloat16, device="cuda"))
    x = torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="broadcast"):
        lin.apply(x.expand(5, 64))
    assert lin.apply(x.expand(1, 64)).shape == (1, 16)


def test_no_rows(cuda_device):
    from speculative_flash_decoding_b200 import Linear
    _, w, b, _ = _inputs(1, 64, 64)
    assert Linear(w, bias=b).apply(torch.empty(0, 64, dtype=BF16, device="cuda")).shape == (0, 64)


def test_captured_and_on_two_streams(cuda_device):
    from speculative_flash_decoding_b200 import Linear
    x, w, b, r = _inputs(9, 600, 512, residual=BF16)
    layer = Linear(w, bias=b, activation="silu")
    y = torch.zeros(9, 600, dtype=BF16, device="cuda")
    layer.apply(x, residual=r, out=y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.apply(x, residual=r, out=y)
    x.copy_(torch.randn(9, 512, generator=torch.Generator().manual_seed(9)).to(BF16))
    g.replay()
    torch.cuda.synchronize()
    _check(y, x, w, b, r, "silu")
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.zeros_like(y) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o in zip(streams, ys):
            layer.apply(x, residual=r, out=o, stream=s)
    torch.cuda.synchronize()
    for o in ys:
        assert torch.equal(o, y)


@pytest.mark.parametrize("rows", [1, 200])
def test_silu_keeps_its_relative_error_far_below_zero(cuda_device, rows):
    """Every result that fp32 holds as a normal number is within 2^-20 +
    |x| 2^-23 of itself: an exponential of x / 2 is off by 2^-22 and by the
    rounding of its argument, |x| 2^-25, its square by twice that, the quotient
    by 2^-22.  What is below 2^-126 may be anything as small."""
    from speculative_flash_decoding_b200 import Linear
    at = torch.tensor([-87.0, -87.5, -88.0, -89.0, -90.0, -91.5, -92.0, -95.0, -110.0, -1e30,
                       -60.0, -20.0, -3.0, -0.01, 0.0, 0.5, 7.0, 88.0, 90.0, 1e30, 1e-38, -1e-38,
                       30.0, -30.0]).to(BF16)
    w = torch.eye(len(at), device="cuda").to(BF16)
    x = at.cuda().repeat(rows, 1)
    y = Linear(w, activation="silu").apply(x, out_dtype=F32).double()
    z = x.double()
    want = z * torch.exp(-torch.nn.functional.softplus(-z))
    bound = want.abs() * (2.0 ** -20 + z.abs().clamp(max=200.0) * 2.0 ** -23) + 2.0 ** -126
    err = (y - want).abs()
    assert bool((err <= bound).all()), (err / bound)[0].tolist()
    # Infinities and NaN as the formula has them.
    x = torch.tensor([[math.inf, 1.0], [-math.inf, 1.0], [math.nan, 1.0]]).to(BF16).cuda()
    w = torch.zeros(2, 8, device="cuda", dtype=BF16)
    w[0, 0] = 1
    xs = torch.zeros(3, 8, device="cuda", dtype=BF16)
    xs[:, 0] = x[:, 0]
    y = Linear(w[:1].contiguous(), activation="silu").apply(xs, out_dtype=F32)[:, 0]
    assert y[0] == math.inf and bool(y[1:].isnan().all())


@pytest.mark.parametrize("rows", [1, 16, 200])
def test_long_sums_keep_fp32(cuda_device, rows):
    """fp32 outputs over 8192 columns: their blocks go round several
    accumulators (as many of a tile's batch rows as 512 TMEM columns hold, up
    to eight), because each of a chain's steps of 16 columns cuts the running
    sum off, by half of 2^-23 on the average, and that sum is two thirds of
    its end on the average: the whole shrinks by steps * 2 / 3 * 2^-24 at the
    most, and eight more roundings of 2^-24 join the parts.  (With one
    accumulator it is off by 4e-6 at 16 rows and twice that at 200.)"""
    from speculative_flash_decoding_b200 import Linear
    k, n = 8192, 8192
    x, w, _, _ = _inputs(rows, n, k, seed=3, bias=False)
    tiles = -(-rows // 128)
    nt = -(-math.ceil(rows / tiles) // 16) * 16  # batch rows of a tile
    cols = 32
    while cols < nt:
        cols *= 2
    steps = k // 16 // min(8, 512 // cols)
    y = Linear(w).apply(x, out_dtype=F32).double()
    want = x.double() @ w.double().t()
    rel = float((y - want).norm() / want.norm())
    assert rel <= (steps * 2 / 3 + 8) * 2.0 ** -24, (rel, steps)
