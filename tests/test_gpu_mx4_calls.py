"""Calls that make their outputs (the extension module) and calls that are given them (ctypes) agree, and
whatever is not ordinary meets the binding's checks."""

import pytest

pytestmark = pytest.mark.gpu

fo = pytest.importorskip("gemm_tile_signaling_amd")
torch = pytest.importorskip("torch")


def _x(rows, cols, dtype=torch.bfloat16):
    return torch.randn(rows, cols, device="cuda").to(dtype)


@pytest.mark.parametrize("rows, cols, dtype", [(1, 1, "bf16"), (5, 33, "fp16"), (64, 512, "bf16"), (0, 40, "fp16")])
def test_same_bits(rows, cols, dtype):
    t = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    x = _x(rows, cols, t)
    made = fo.mx4_quantize(x)
    given = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in fo.mx4_shapes(rows, cols)]
    fo.mx4_quantize(x, *given)
    assert all(torch.equal(a, b) for a, b in zip(made, given))
    for name, out in (("bf16", torch.bfloat16), ("fp16", torch.float16), ("fp32", torch.float32)):
        o = torch.empty(rows, cols, dtype=out, device="cuda")
        fo.mx4_dequantize(*made, cols, dtype=name, out=o)
        y = fo.mx4_dequantize(*made, cols, dtype=name)
        assert y.dtype == out and torch.equal(y, o)
    if rows:
        w = fo.mx4_quantize(_x(16, cols, t))
        o = torch.empty(rows, 16, dtype=t, device="cuda")
        fo.mx4_gemm(*made, *w, dtype=dtype, out=o)
        assert torch.equal(fo.mx4_gemm(*made, *w, dtype=dtype), o)


def test_parameters_views_and_streams():
    x = _x(40, 96)
    want = fo.mx4_quantize(x)
    assert all(torch.equal(a, b) for a, b in zip(fo.mx4_quantize(torch.nn.Parameter(x)), want))
    wide = torch.zeros(40, 200, device="cuda", dtype=torch.bfloat16)
    wide[:, 7:103] = x
    assert all(torch.equal(a, b) for a, b in zip(fo.mx4_quantize(wide[:, 7:103]), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = fo.mx4_gemm(*want, *want)
    by_name = fo.mx4_gemm(*want, *want, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(on_side, fo.mx4_gemm(*want, *want)) and torch.equal(on_side, by_name)


@pytest.mark.parametrize("call, error", [
    (lambda x, c, s, e: fo.mx4_quantize(x.float()), ValueError),
    (lambda x, c, s, e: fo.mx4_quantize(x.t()), ValueError),
    (lambda x, c, s, e: fo.mx4_quantize(x[0]), ValueError),
    (lambda x, c, s, e: fo.mx4_quantize(x.cpu()), ValueError),
    (lambda x, c, s, e: fo.mx4_quantize(x.to_sparse()), (ValueError, RuntimeError)),
    (lambda x, c, s, e: fo.mx4_dequantize(c, s, 65), ValueError),
    (lambda x, c, s, e: fo.mx4_dequantize(c, s, 0), ValueError),
    (lambda x, c, s, e: fo.mx4_dequantize(c, s, 2 ** 62), ValueError),
    (lambda x, c, s, e: fo.mx4_dequantize(c, s.cpu(), 64), ValueError),
    (lambda x, c, s, e: fo.mx4_dequantize(c, s[:, :4], 64), ValueError),
    (lambda x, c, s, e: fo.mx4_gemm(c, s, c[:, :16], s), ValueError),
    (lambda x, c, s, e: fo.mx4_gemm(c, s, c.t().contiguous().t(), s), ValueError),
    (lambda x, c, s, e: fo.mx4_gemm(c, s, c, s.view(8, 1, 8)), ValueError),
    (lambda x, c, s, e: fo.mx4_gemm(c, s.float(), c, s), ValueError),
    (lambda x, c, s, e: fo.mx4_gemm(c, s, c, s, row_ends=e.long()), ValueError),
    (lambda x, c, s, e: fo.mx4_gemm(c, s, c, s, row_ends=e.cpu()), ValueError),
    (lambda x, c, s, e: fo.mx4_gemm(c, s, c, s, row_ends=e.repeat(3)), ValueError),
    (lambda x, c, s, e: fo.mx4_gemm(c, s, c[:4], s[:, :4].contiguous()), fo.FoError),   # N = 4
    (lambda x, c, s, e: fo.mx4_gemm(c.flatten()[1:129].view(4, 32), s[:, :4].contiguous(), c, s), fo.FoError),  # alignment
])
def test_refusals(call, error):
    x = _x(8, 64)
    c, s = fo.mx4_quantize(x)
    with pytest.raises(error):
        call(x, c, s, torch.tensor([8], dtype=torch.int32, device="cuda"))


def test_repeated_calls_keep_no_reference():
    """Outputs are freed with their last name: a thousand calls stay within a few allocations."""
    x = _x(64, 512)
    fo.mx4_quantize(x)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(1000):
        c, s = fo.mx4_quantize(x)
        y = fo.mx4_dequantize(c, s, 512)
        z = fo.mx4_gemm(c, s, c, s)
    del c, s, y, z
    assert torch.cuda.memory_allocated() == before
