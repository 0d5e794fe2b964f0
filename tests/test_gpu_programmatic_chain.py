"""Kernels that overlap their start with the kernel before them, in chains that
rewrite the same scale, code and bias buffers: each result has to be the one
of the same calls with the device idle in between, bit for bit."""
import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu

EPS = 1e-5


def operands(m, n, k, sfmt, count):
    g = torch.Generator(device="cuda").manual_seed(m + n)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    F = lib()
    # rows whose magnitude changes from one iteration to the next by powers of
    # two and more: a stale scale is off by that factor
    xs = [(rn(m, k) * 4.0 ** (i % 5)).bfloat16() for i in range(count)]
    biases = [rn(n) * (i + 1) for i in range(count)]
    w = (rn(n, k) * k ** -0.5).bfloat16()
    st = torch.float32 if sfmt == F.SCALE_F32 else torch.uint8
    q = torch.empty((n, k), dtype=torch.uint8, device="cuda")
    s = torch.empty(((n + 127) // 128, k // 128), dtype=st, device="cuda")
    F.fp8_quantize_block(w, F.E4M3, sfmt, q, s)
    return xs, biases, q, s, st


# the few-row kernel with and without split K, its two halves, 128-wide tiles
# of the general kernel (FP32 scales), block-scaled tiles behind the word
# conversion, CTA pairs
SHAPES = [(1, 2048, 1024), (16, 512, 2048), (64, 2600, 384), (100, 640, 1024), (300, 520, 1024),
          (900, 2600, 512)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("sfmt", [0, 1])
def test_norm_then_group_product(m, n, k, sfmt):
    """Codes, scales and bias rewritten before every product."""
    F = lib()
    count = 24
    xs, biases, wq, ws, st = operands(m, n, k, sfmt, count)
    q = torch.empty((m, k), dtype=torch.uint8, device="cuda")
    s = torch.empty((k // 128, m), dtype=st, device="cuda")
    bias = torch.empty(n, device="cuda")

    def run(sync):
        outs = [torch.empty((m, n), dtype=torch.bfloat16, device="cuda") for _ in xs]
        torch.cuda.synchronize()
        for x, b, out in zip(xs, biases, outs):
            bias.copy_(b)
            sync()
            F.fp8_rmsnorm_quantize(x, None, EPS, F.E4M3, q, scales=s, sfmt=sfmt)
            sync()
            F.fp8_gemm_group_epilogue(q, s, wq, ws, sfmt, out, bias=bias, act=F.ACT_SILU)
            sync()
        torch.cuda.synchronize()
        return outs

    want = run(torch.cuda.synchronize)
    assert not torch.equal(want[0], want[1])
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("sfmt", [0, 1])
def test_quantize_then_group_product(m, n, k, sfmt):
    """The same behind the group quantizer, with the plain product's bias path."""
    F = lib()
    count = 24
    xs, biases, wq, ws, st = operands(m, n, k, sfmt, count)
    q = torch.empty((m, k), dtype=torch.uint8, device="cuda")
    s = torch.empty((k // 128, m), dtype=st, device="cuda")

    def run(sync):
        outs = [torch.empty((m, n), dtype=torch.bfloat16, device="cuda") for _ in xs]
        torch.cuda.synchronize()
        for x, b, out in zip(xs, biases, outs):
            F.fp8_quantize_token_group(x, F.E4M3, sfmt, q, s)
            sync()
            F.fp8_gemm_group(q, s, wq, ws, sfmt, out, bias=b)
            sync()
        torch.cuda.synchronize()
        return outs

    want = run(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))


@pytest.mark.parametrize("m", [1, 48])
def test_product_then_quantize(m):
    """The quantizer reads what the product before it writes, over and over in
    one buffer (the feed-forward block's middle)."""
    F = lib()
    n, k, count = 1024, 512, 24
    xs, _, wq, ws, st = operands(m, n, k, 0, count)
    xq = torch.empty((m, k), dtype=torch.uint8, device="cuda")
    xsc = torch.empty((k // 128, m), device="cuda")
    a = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")

    def run(sync):
        outs = [(torch.empty((m, n), dtype=torch.uint8, device="cuda"),
                 torch.empty((n // 128, m), device="cuda")) for _ in xs]
        torch.cuda.synchronize()
        for x, (q, s) in zip(xs, outs):
            F.fp8_rmsnorm_quantize(x, None, 0.5, F.E4M3, xq, scales=xsc)
            sync()
            F.fp8_gemm_group_epilogue(xq, xsc, wq, ws, 0, a, act=F.ACT_RELU)
            sync()
            F.fp8_quantize_token_group(a, F.E4M3, 0, q, s)
            sync()
        torch.cuda.synchronize()
        return outs

    want = run(torch.cuda.synchronize)
    for _ in range(3):
        for (q, s), (wq_, ws_) in zip(run(lambda: None), want):
            assert torch.equal(q, wq_) and torch.equal(s, ws_)
