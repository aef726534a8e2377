"""4-bit experts with enough values that a wave of the second product takes several row blocks: token counts of
every form, hidden sizes that no workgroup divides, and experts picked by every token."""

import pytest

from tests.gpu_util import say
from tests.test_gpu_moe import U, device_case

pytestmark = pytest.mark.gpu

fo = pytest.importorskip("gemm_tile_signaling_amd")
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T, D, F, E, k, first, local", [
    (1, 2080, 8224, 8, 4, 0, 8), (2, 4064, 4128, 5, 2, 0, 5),                          # two row blocks, one token and two
    (7, 2080, 8224, 20, 4, 0, 20), (8, 4000, 9760, 12, 3, 2, 8),                        # four
    (13, 2080, 2080, 20, 2, 0, 20), (27, 2016, 2080, 24, 2, 1, 23), (50, 2080, 1056, 60, 2, 0, 50)])
def test_row_blocks(T, D, F, E, k, first, local, dtype):
    say(f"moe rows T={T} D={D} F={F} E={E} k={k} first={first} local={local} {dtype}")
    device_case(T, D, F, E, k, first, local, "mx4", dtype, T % 2 == 0, T * D + F)


@pytest.mark.parametrize("T", [8, 14, 20, 32, 45, 64])
def test_every_token_on_two_of_many_experts(T):
    """A router of zeros: equal logits, so every token picks experts 0 and 1 with weights 1/2.  Against 64 bits; the
    bound is that of the layer's other tests, with exact weights."""
    D, F, E = 2080, 1056, 60
    say(f"moe rows, two experts of {E} T={T}")
    g = torch.Generator(device="cuda").manual_seed(T)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = normal(T, D).bfloat16()
    gu = fo.mx4_quantize((normal(E * 2 * F, D) * D ** -0.5).bfloat16())
    dn = fo.mx4_quantize((normal(E * D, F) * F ** -0.5).bfloat16())
    layer = fo.Moe(D, F, E, 2, weights="mx4")
    out = layer.forward(x, torch.zeros(E, D, dtype=torch.bfloat16, device="cuda"), gu, dn, layer.new_workspace())
    want = bound = 0
    xd = x.double()
    wide_gu = fo.mx4_dequantize(*gu, D, dtype="fp32").view(E, 2 * F, D)
    wide_dn = fo.mx4_dequantize(*dn, F, dtype="fp32").view(E, D, F)
    for e in range(2):
        w = wide_gu[e].double()
        a, b = (xd @ w.t()).split(F, 1)
        da, db = (D * U * (xd.abs() @ w.abs().t())).split(F, 1)
        s = a * torch.sigmoid(a)
        h = s * b
        dh = 1.1 * b.abs() * da + s.abs() * db + h.abs() * ((a.abs() + 8) * U + 2.0 ** -16)
        d = wide_dn[e].double()
        want = want + 0.5 * (h @ d.t())
        bound = bound + 0.5 * (dh @ d.abs().t() + (F + 32) * U * (h.abs() @ d.abs().t())) + (E + 4) * U * (h @ d.t()).abs()
    bound = bound + 2.0 ** -8 * (want.abs() + bound)
    assert ((out.double() - want).abs() <= bound).all()
