"""Arguments that the mixture-of-experts layer refuses, with the documented codes -- all without a GPU."""

import ctypes as C

import pytest

fo = pytest.importorskip("gemm_tile_signaling_amd")
torch = pytest.importorskip("torch")
from gemm_tile_signaling_amd import moe  # noqa: E402

INVALID, UNSUPPORTED = fo.FO_ERR_INVALID, fo.FO_ERR_UNSUPPORTED
DESC = dict(hidden=64, ffn=96, experts=8, top_k=2, first_expert=2, local_experts=4, dtype=0, weights=0, renormalize=1,
            max_tokens=4)


def _bytes(**change):
    n = C.c_int64(-1)
    d = moe._MoeDesc(**dict(DESC, **change))
    return moe._ops().fo_moe_workspace_bytes(C.byref(d), C.byref(n)), n.value


@pytest.mark.parametrize("change, code", [
    (dict(hidden=0), INVALID), (dict(hidden=60), INVALID), (dict(ffn=-8), INVALID), (dict(ffn=12), INVALID),
    (dict(weights=1, hidden=72), INVALID), (dict(weights=1, ffn=104), INVALID), (dict(weights=2), INVALID),
    (dict(dtype=2), INVALID), (dict(experts=0), INVALID), (dict(top_k=0), INVALID), (dict(top_k=9), INVALID),
    (dict(first_expert=-1), INVALID), (dict(first_expert=5), INVALID), (dict(local_experts=0), INVALID),
    (dict(first_expert=2 ** 31 - 1, local_experts=2), INVALID), (dict(renormalize=2), INVALID),
    (dict(max_tokens=0), INVALID), (dict(max_tokens=65), UNSUPPORTED), (dict(experts=1025), UNSUPPORTED),
    (dict(experts=64, top_k=17), UNSUPPORTED), (dict(hidden=1 << 20), UNSUPPORTED), (dict(ffn=1 << 20), UNSUPPORTED),
])
def test_description(change, code):
    assert _bytes(**change) == (code, -1)


def test_workspace_size():
    rc, n = _bytes()
    assert rc == 0 and n % 256 == 0 and n >= 4 * 4 * 2 * 96
    # 4-bit weights: the tokens laid out in panels of 256 values, fp16 ones as two bf16 values
    assert _bytes(weights=1, dtype=1)[1] == _bytes(weights=1, dtype=0)[1] + 2 * 4 * 256
    assert moe._ops().fo_moe_workspace_bytes(None, None) == INVALID
    layer = fo.Moe(64, 96, 8, 2, first_expert=2, max_tokens=4)
    assert layer.local_experts == 6


ARGS = dict(tokens=2, x=256, router=256, gate_up=256, gus=0, down=256, dns=0, out=256, ids=0, weights=0, workspace=256)


@pytest.mark.parametrize("desc, change, code", [
    ({}, dict(tokens=-1), INVALID), ({}, dict(tokens=5), UNSUPPORTED), ({}, dict(x=0), INVALID),
    ({}, dict(x=264), INVALID), ({}, dict(router=0), INVALID), ({}, dict(gate_up=8), INVALID),
    ({}, dict(down=0), INVALID), ({}, dict(out=0), INVALID), ({}, dict(workspace=128), INVALID),
    ({}, dict(workspace=0), INVALID), ({}, dict(ids=2), INVALID), ({}, dict(weights=6), INVALID),
    ({}, dict(gus=256), INVALID), (dict(weights=1), {}, INVALID), (dict(weights=1), dict(gus=256), INVALID),
    (dict(weights=1), dict(gus=256, dns=8), INVALID), ({}, dict(tokens=0, x=0, out=0), 0),
    (dict(top_k=0), {}, INVALID),
])
def test_forward(desc, change, code):
    d = moe._MoeDesc(**dict(DESC, **desc))
    assert moe._ops().fo_moe_forward(C.byref(d), *dict(ARGS, **change).values(), None) == code
    assert moe._ops().fo_moe_forward(None, *ARGS.values(), None) == INVALID


def test_binding():
    with pytest.raises(ValueError, match="dtype"):
        fo.Moe(64, 96, 8, 2, dtype="fp32")
    with pytest.raises(ValueError, match="weights"):
        fo.Moe(64, 96, 8, 2, weights="fp8")
    with pytest.raises(fo.FoError) as e:
        fo.Moe(64, 96, 8, 9)
    assert e.value.code == INVALID
    layer = fo.Moe(64, 96, 8, 2, max_tokens=2)
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        layer.forward(x, x, x, x, x)
    with pytest.raises(ValueError, match="shape"):
        layer.forward(x[:, :32], x, x, x, x)
