"""Tensors of another type than the call's are refused; integers of the same size hold the bits."""

import pytest

pytestmark = pytest.mark.gpu

fo = pytest.importorskip("gemm_tile_signaling_amd")
torch = pytest.importorskip("torch")


def _operand(rows, cols):
    return fo.mx4_quantize(torch.randn(rows, cols, device="cuda").bfloat16())


@pytest.mark.parametrize("dtype, other", [("bf16", torch.float16), ("fp16", torch.bfloat16)])
def test_outputs(dtype, other):
    a, b = _operand(5, 64), _operand(16, 64)
    bits = torch.empty(5, 16, dtype=torch.int16, device="cuda")
    want = fo.mx4_gemm(*a, *b, dtype=dtype)
    assert torch.equal(fo.mx4_gemm(*a, *b, dtype=dtype, out=bits).view(want.dtype), want)
    with pytest.raises(ValueError, match="out"):
        fo.mx4_gemm(*a, *b, dtype=dtype, out=torch.empty(5, 16, dtype=other, device="cuda"))
    with pytest.raises(ValueError, match="out"):
        fo.mx4_dequantize(*a, 64, dtype=dtype, out=torch.empty(5, 64, dtype=other, device="cuda"))


def test_layer():
    layer = fo.Moe(64, 32, 4, 2)
    make = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    args = dict(x=make(3, 64), router=make(4, 64), gate_up=make(4, 64, 64), down=make(4, 64, 32),
                workspace=layer.new_workspace())
    assert layer.forward(**args).abs().max() == 0
    for name in ("x", "router", "gate_up", "down"):
        with pytest.raises(ValueError, match=name):
            layer.forward(**dict(args, **{name: args[name].half()}))
    with pytest.raises(ValueError, match="out"):
        layer.forward(**args, out=make(3, 64, t=torch.float16))
