"""The mixture-of-experts layer against the oracle.

Tolerance, element by element, derived from the arithmetic (u = 2^-23 bounds
one unit in the last place of an fp32 partial sum, so a sum of n products is off
by at most n u times the sum of their magnitudes):
  logits            dl = D u sum |router| |x|
  weights           relative 2 dl + (|l - max| + E + 4) u          (exp, sums, division)
  gate, up          dg, du = D u sum |w| |x|
  h                 dh = 1.1 |u| dg + |silu(g)| du + |h| ((|g| + 8) u + 2^-16), the slope of silu being at most 1.1,
                    and 2^-16 for the 16-bit pair (2^-25 absolute where the pair is fp16)
  out               sum_j w_j (sum |down| dh + (F + 32) u sum |down| |h|) + dw_j |y_j|, and one rounding to p bits.
"""

import numpy as np
import pytest

import oracle
from oracle import moe as omoe
from oracle import mx4
from tests.gpu_util import say
from workloads import to_bits

pytestmark = pytest.mark.gpu

fo = pytest.importorskip("gemm_tile_signaling_amd")
torch = pytest.importorskip("torch")
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -23


def rounded(rng, shape, scale, dtype):
    """(bits, fp64 values) of normal draws."""
    b = to_bits((rng.standard_normal(shape) * scale).astype(np.float32), dtype)
    return b, oracle.decode_bits(b, dtype)


def up16(b, dtype):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16).copy()).view(TORCH[dtype]).to("cuda")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


class Case:
    def __init__(self, T, D, F, E, k, first=0, local=None, weights="16", dtype="bf16", renorm=True, seed=0):
        rng = np.random.default_rng(seed + 1000 * T + D + F)
        self.T, self.D, self.F, self.E, self.k, self.first, self.renorm = T, D, F, E, k, first, renorm
        self.local = L = E - first if local is None else local
        self.dtype, self.kind = dtype, weights
        self.xb, self.x = rounded(rng, (T, D), 1.0, dtype)
        self.rb, self.router = rounded(rng, (E, D), D ** -0.5, dtype)
        if weights == "16":
            self.gb, gu = rounded(rng, (L * 2 * F, D), D ** -0.5, dtype)
            self.db, dn = rounded(rng, (L * D, F), F ** -0.5, dtype)
        else:
            form = lambda rows, cols: (rng.integers(0, 16, (rows, cols)).astype(np.uint8),  # noqa: E731
                                       rng.integers(118, 123, (rows, cols // 32)).astype(np.uint8))
            self.gb, self.db = form(L * 2 * F, D), form(L * D, F)
            gu, dn = mx4.values(*self.gb), mx4.values(*self.db)
        self.gu, self.dn = gu.reshape(L, 2 * F, D), dn.reshape(L, D, F)

    def layer(self, **kw):
        return fo.Moe(self.D, self.F, self.E, self.k, dtype=self.dtype, weights=self.kind, renormalize=self.renorm,
                      first_expert=self.first, local_experts=self.local, **kw)

    def matrices(self):
        if self.kind == "16":
            return up16(self.gb, self.dtype), up16(self.db, self.dtype)
        out = []
        for f in (self.gb, self.db):
            p, q = mx4.pack(*f)
            if f[1].shape[1] % 8:
                q[-1, :, f[1].shape[1] % 8:] = 255     # bytes without a block carry no meaning
            out.append((dev(p), dev(q)))
        return out

    def run(self, layer=None, ws=None, **kw):
        say(f"moe T={self.T} D={self.D} F={self.F} E={self.E} k={self.k} first={self.first} local={self.local} "
            f"{self.kind} {self.dtype}")
        layer = layer or self.layer()
        ws = layer.new_workspace() if ws is None else ws
        out = torch.full((self.T + 1, self.D), -7.0, dtype=TORCH[self.dtype], device="cuda")
        ids = torch.full((self.T + 1, self.k), -7, dtype=torch.int32, device="cuda")
        wts = torch.full((self.T + 1, self.k), -7.0, dtype=torch.float32, device="cuda")
        layer.forward(up16(self.xb, self.dtype), up16(self.rb, self.dtype), *self.matrices(), ws, out=out[:self.T],
                      picks=(ids[:self.T], wts[:self.T]), **kw)
        torch.cuda.synchronize()
        assert (out[self.T:] == -7).all() and (ids[self.T:] == -7).all() and (wts[self.T:] == -7).all()
        o = oracle.decode_bits(out[:self.T].view(torch.int16).cpu().numpy().view(np.uint16), self.dtype)
        return o, ids[:self.T].cpu().numpy(), wts[:self.T].cpu().numpy().astype(np.float64)

    def check(self, got):
        o, ids, wts = got
        # the picks: distinct, in descending order and none of the others larger, up to the logits' own error
        assert all(len(set(i)) == self.k for i in ids.tolist()) and ids.min() >= 0 and ids.max() < self.E
        r = omoe.layer(self.x, self.router, self.gu, self.dn, self.k, self.renorm, self.first, ids=ids)
        dl = self.D * U * (np.abs(self.x) @ np.abs(self.router).T)
        picked, open_ = np.take_along_axis(r["logits"], ids, 1), 2 * dl.max(1, keepdims=True)
        assert (picked[:, :-1] - picked[:, 1:] >= -open_).all()
        others = r["logits"].copy()
        np.put_along_axis(others, ids, -np.inf, 1)
        assert (picked[:, -1:] - others >= -open_).all()
        top = r["logits"].max(1, keepdims=True)
        rel = 4 * dl.max(1, keepdims=True) + (np.abs(np.take_along_axis(r["logits"], ids, 1) - top) + self.E + 4) * U
        assert (np.abs(wts - r["weights"]) <= rel * r["weights"]).all()
        bound = np.zeros_like(o)
        p = oracle.DTYPES[self.dtype]["p"]
        pair = 2.0 ** -25 if self.dtype == "fp16" and self.kind == "16" else 0.0
        for (t, j), (g, u, h, y) in r["parts"].items():
            e = ids[t, j] - self.first
            a = self.D * U * (np.abs(self.gu[e]) @ np.abs(self.x[t]))
            s = np.abs(g / (1 + np.exp(-g)))
            dh = 1.1 * np.abs(u) * a[:self.F] + s * a[self.F:] + np.abs(h) * ((np.abs(g) + 8) * U + 2.0 ** -16) + pair
            w = np.abs(self.dn[e])
            bound[t] += r["weights"][t, j] * (w @ dh + (self.F + 32) * U * (w @ np.abs(h))) \
                + rel[t, j] * r["weights"][t, j] * np.abs(y)
        bound += 2.0 ** -p * (np.abs(r["out"]) + bound) + 2.0 ** (-133 if self.dtype == "bf16" else -25)
        bad = np.abs(o - r["out"]) > bound
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), np.abs(o - r["out"]).max(), bound.max())
        return r


SIZES = [
    # T, D, F, E, k, first, local
    (1, 64, 96, 4, 2, 0, 4), (1, 256, 512, 8, 2, 0, 8), (2, 32, 32, 2, 1, 0, 2), (3, 96, 64, 5, 5, 0, 5),
    (7, 512, 160, 16, 4, 0, 16), (16, 288, 224, 8, 2, 0, 8), (17, 128, 544, 33, 3, 0, 33), (31, 1056, 96, 20, 6, 0, 20),
    (33, 160, 1120, 8, 2, 0, 8), (48, 64, 64, 130, 8, 0, 130), (64, 256, 256, 64, 6, 16, 8), (64, 96, 128, 3, 3, 0, 3),
    (5, 128, 128, 64, 2, 40, 7), (64, 64, 32, 1024, 16, 0, 1024), (13, 2080, 32, 12, 8, 11, 1), (4, 32, 4128, 6, 2, 0, 6),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("weights", ["16", "mx4"])
@pytest.mark.parametrize("T, D, F, E, k, first, local", SIZES)
def test_layer(T, D, F, E, k, first, local, weights, dtype):
    c = Case(T, D, F, E, k, first, local, weights, dtype, renorm=T % 2 == 1)
    r = c.check(c.run())
    held = ((r["ids"] >= first) & (r["ids"] < first + local)).any(1)
    if local < E:
        assert not c.run()[0][~held].any()             # nothing held here: zeros


def device_case(T, D, F, E, k, first, local, weights, dtype, renorm, seed):
    """Inputs made on the device, and the layer in 64 bits with the error bound of the module's docstring, there as well."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *sh: torch.randn(*sh, generator=g, device="cuda")  # noqa: E731
    x, router = normal(T, D).to(TORCH[dtype]), (normal(E, D) * D ** -0.5).to(TORCH[dtype])
    mats, values = [], []
    for rows, cols in ((local * 2 * F, D), (local * D, F)):
        if weights == "16":
            w = (normal(rows, cols) * cols ** -0.5).to(TORCH[dtype])
            mats.append(w)
            values.append(lambda lo, hi, w=w: w[lo:hi].double())
        else:
            nb = cols // 32
            codes = torch.randint(0, 256, (rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
            scales = torch.randint(118, 122, ((nb + 7) // 8, rows, 8), generator=g, device="cuda", dtype=torch.uint8)
            if nb % 8:
                scales[-1, :, nb % 8:] = 255
            mats.append((codes, scales))
            table = torch.tensor(np.concatenate([mx4.MAGNITUDES, -mx4.MAGNITUDES]), device="cuda")

            def part(lo, hi, codes=codes, scales=scales, nb=nb, table=table):
                c = codes[lo:hi].int()
                v = torch.stack([table[c & 15], table[c >> 4]], -1).reshape(hi - lo, nb, 32)
                e = scales[:, lo:hi].permute(1, 0, 2).reshape(hi - lo, -1)[:, :nb].double() - 127
                return (v * torch.exp2(e)[..., None]).reshape(hi - lo, -1)
            values.append(part)
    layer = fo.Moe(D, F, E, k, dtype=dtype, weights=weights, renormalize=renorm, first_expert=first, local_experts=local)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    wts = torch.empty(T, k, dtype=torch.float32, device="cuda")
    out = layer.forward(x, router, *mats, layer.new_workspace(), picks=(ids, wts))
    xd, rd = x.double(), router.double()
    logits = xd @ rd.t()
    dl = (D * U * (xd.abs() @ rd.abs().t())).amax(1, keepdim=True)
    order = logits.gather(1, ids.long())
    assert (order[:, :-1] - order[:, 1:] >= -2 * dl).all()
    assert (order[:, -1:] - logits.scatter(1, ids.long(), -float("inf")) >= -2 * dl).all()
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    w = p.gather(1, ids.long())
    w = w / (w.sum(1, keepdim=True) if renorm else p.sum(1, keepdim=True))
    rel = 4 * dl + ((order - logits.amax(1, keepdim=True)).abs() + E + 4) * U
    want, bound = torch.zeros_like(xd), torch.zeros_like(xd)
    pair = 2.0 ** -25 if dtype == "fp16" and weights == "16" else 0.0
    for e in range(local):
        t, j = (ids == first + e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        gu = values[0](e * 2 * F, (e + 1) * 2 * F)
        gate, up = (xd[t] @ gu.t()).split(F, 1)
        da, du = (D * U * (xd[t].abs() @ gu.abs().t())).split(F, 1)
        del gu
        s = gate / (1 + torch.exp(-gate))
        h = s * up
        dh = 1.1 * up.abs() * da + s.abs() * du + h.abs() * ((gate.abs() + 8) * U + 2.0 ** -16) + pair
        dn = values[1](e * D, (e + 1) * D)
        y = h @ dn.t()
        dy = dh @ dn.abs().t() + (F + 32) * U * (h.abs() @ dn.abs().t()) + rel[t, j, None] * y.abs()
        want.index_add_(0, t, w[t, j, None] * y)
        bound.index_add_(0, t, w[t, j, None] * dy)
    bits = oracle.DTYPES[dtype]["p"]
    bound += 2.0 ** -bits * (want.abs() + bound) + 2.0 ** (-133 if dtype == "bf16" else -25)
    bad = (out.double() - want).abs() > bound
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist(), float((out.double() - want).abs().max()))


@pytest.mark.parametrize("T, D, F, E, k, first, local, weights, dtype", [
    # enough values for the forms that large 4-bit experts take: a few, some and all tokens on an expert (past 16 and
    # 32 of them the columns take more tiles and a second pass), partial panels, a share of the experts
    (16, 2080, 3232, 40, 8, 0, 40, "mx4", "fp16"), (24, 2048, 4160, 33, 5, 1, 32, "mx4", "bf16"),
    (64, 4096, 8224, 8, 2, 0, 8, "mx4", "bf16"), (64, 2080, 16160, 8, 8, 0, 8, "mx4", "fp16"),
    (30, 4096, 14336, 5, 5, 0, 5, "mx4", "bf16"), (12, 2048, 4128, 36, 12, 0, 36, "mx4", "bf16"),
    (64, 4096, 4104, 8, 4, 0, 8, "16", "bf16"), (40, 2056, 1032, 9, 3, 3, 4, "16", "fp16"),
    (3, 4096, 14336, 4, 2, 0, 4, "16", "bf16"), (8, 4096, 4096, 16, 2, 0, 16, "mx4", "fp16")])
def test_large_experts(T, D, F, E, k, first, local, weights, dtype):
    say(f"moe large T={T} D={D} F={F} E={E} k={k} first={first} local={local} {weights} {dtype}")
    device_case(T, D, F, E, k, first, local, weights, dtype, T % 2 == 0, T + D)


@pytest.mark.parametrize("weights", ["16", "mx4"])
@pytest.mark.parametrize("T", [9, 33, 64])
def test_every_token_on_every_expert(T, weights):
    """top_k == experts: every expert has all the tokens (two passes over its rows past 32)."""
    c = Case(T, 256, 544, 3, 3, weights=weights)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T, D, F, E, k", [(3, 8, 8, 4, 2), (18, 72, 40, 9, 3), (64, 1000, 776, 4, 1), (1, 24, 2056, 7, 7)])
def test_sizes_that_are_multiples_of_8_only(T, D, F, E, k, dtype):
    c = Case(T, D, F, E, k, dtype=dtype)
    c.check(c.run())


def test_ties_go_to_the_lowest_index():
    """Logits are exact small integers with many ties, and zeros of both signs."""
    c = Case(24, 64, 32, 70, 5)
    rng = np.random.default_rng(1)
    c.xb[:] = 0
    c.xb[:, 0] = to_bits(np.where(np.arange(24) % 2, 1.0, -1.0).astype(np.float32), "bf16")
    c.rb[:] = 0
    c.rb[:, 0] = to_bits(rng.integers(-2, 3, 70).astype(np.float32), "bf16")
    c.x, c.router = oracle.decode_bits(c.xb, "bf16"), oracle.decode_bits(c.rb, "bf16")
    _, ids, wts = c.run()
    want, w = omoe.route(c.x @ c.router.T + 0.0, 5, True)
    assert np.array_equal(ids, want) and np.allclose(wts, w, rtol=1e-5)


@pytest.mark.parametrize("weights", ["16", "mx4"])
def test_one_expert_for_every_token(weights):
    """All 64 tokens on one expert, and on one of two shares none at all."""
    c = Case(64, 64, 96, 8, 1, weights=weights)
    c.rb[:] = 0
    c.rb[3, 0] = to_bits(np.float32([40.0]), "bf16")[0]
    c.xb[:, 0] = to_bits(np.abs(c.x[:, 0]).astype(np.float32) + 1, "bf16")
    c.x, c.router = oracle.decode_bits(c.xb, "bf16"), oracle.decode_bits(c.rb, "bf16")
    got = c.run()
    assert (got[1] == 3).all()
    c.check(got)
    c.first, c.local = 4, 4
    c.gb, c.db = ((f[0][-len(f[0]) // 2:], f[1][-len(f[1]) // 2:]) if weights == "mx4" else f[-len(f) // 2:] for f in (c.gb, c.db))
    o, ids, _ = c.run()
    assert (ids == 3).all() and not o.any()


@pytest.mark.parametrize("weights", ["16", "mx4"])
def test_nan_and_infinity_stay_with_their_tokens(weights):
    """A NaN token spoils its own row; NaN or infinite weights of an expert spoil the tokens that picked it, and no other."""
    c = Case(20, 64, 96, 6, 2, weights=weights)
    clean, ids, _ = c.run()
    bad = int(ids[0, 0])
    hit = (ids == bad).any(1)
    assert hit.any() and not hit.all()
    if weights == "16":
        c.db.reshape(6, 64, 96)[bad, 5, :] = 0x7F80          # infinities in one row of down
        c.gb.reshape(6, 192, 64)[bad, 9, 3] = 0x7FC0         # a NaN in one gate row
    else:
        c.gb[1].reshape(6, 192, 2)[bad, 9, 1] = 255
    o, ids2, _ = c.run()
    assert np.array_equal(ids, ids2)
    assert np.array_equal(o[~hit], clean[~hit]) and np.isnan(o[hit]).all()
    c = Case(20, 64, 96, 6, 2, weights=weights)
    c.xb[7, 11] = 0x7FC0
    o, _, w = c.run()
    other = np.arange(20) != 7
    assert np.isnan(o[7]).all() and np.isnan(w[7]).all() and np.array_equal(o[other], clean[other])


def test_experts_masked_by_minus_infinity():
    """Router rows of the type's lowest values give logits of -infinity: never picked while another is left, weight 0 after."""
    c = Case(6, 64, 32, 4, 3)
    c.xb[:] = to_bits(np.abs(c.x).astype(np.float32) + 1, "bf16")
    c.rb[1:3] = 0xFF7F                                         # lowest finite value: the sum overflows to -infinity
    c.x, c.router = oracle.decode_bits(c.xb, "bf16"), oracle.decode_bits(c.rb, "bf16")
    o, ids, w = c.run()
    assert all(set(r[:2]) == {0, 3} and r[2] == 1 for r in ids.tolist()) and (w[:, 2] == 0).all()
    assert np.allclose(w.sum(1), 1, rtol=1e-5) and np.isfinite(o).all()


def test_fp16_tokens_with_4_bit_weights_keep_their_bits():
    """fp16 tokens are split exactly: with weights 1 on one value and 0 elsewhere the gate is the token's value itself."""
    c = Case(8, 64, 32, 2, 2, weights="mx4", dtype="fp16")
    for f in (c.gb, c.db):
        f[0][:] = 0
        f[1][:] = 127
    c.gb[0].reshape(2, 64, 64)[:, np.arange(32), np.arange(32)] = 2              # gate f = x[f]
    c.gb[0].reshape(2, 64, 64)[:, 32 + np.arange(32), np.arange(32)] = 2         # up f = x[f]
    c.db[0].reshape(2, 64, 32)[:, np.arange(32), np.arange(32)] = 2              # out d = h[d]
    c.gu, c.dn = mx4.values(*c.gb).reshape(2, 64, 64), mx4.values(*c.db).reshape(2, 64, 32)
    c.check(c.run())


@pytest.mark.parametrize("weights, dtype", [("16", "bf16"), ("mx4", "fp16")])
def test_workspace_serves_calls_of_any_size_and_streams(weights, dtype):
    """One workspace, calls of 64, 1, 17 and 0 tokens after each other, the same bits each time, also on another stream."""
    cases = [Case(t, 96, 160, 12, 3, weights=weights, dtype=dtype, seed=5) for t in (64, 1, 17)]
    layer = cases[0].layer()
    ws = layer.new_workspace()
    first = [c.run(layer, ws) for c in cases]
    for c, f in zip(cases, first):
        c.check(f)
    empty = up16(cases[0].xb, dtype)[:0]
    assert layer.forward(empty, up16(cases[0].rb, dtype), *cases[0].matrices(), ws).shape == (0, 96)
    s = torch.cuda.Stream()
    for _ in range(2):
        for c, f in zip(cases, first):
            torch.cuda.synchronize()
            for a, b in zip(c.run(layer, ws, stream=s), f):
                assert np.array_equal(a, b)


@pytest.mark.parametrize("weights", ["16", "mx4"])
def test_layer_replays_in_a_graph(weights):
    """Recorded once, replayed on new tokens with eager calls between, against the eager results."""
    c = Case(9, 128, 192, 16, 4, weights=weights)
    layer = c.layer()
    ws, ws2 = layer.new_workspace(), layer.new_workspace()
    x, router, mats = up16(c.xb, "bf16"), up16(c.rb, "bf16"), c.matrices()
    layer.forward(x, router, *mats, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer.forward(x, router, *mats, ws)
    for _ in range(4):
        x.copy_(torch.randn(9, 128, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, layer.forward(x, router, *mats, ws2))
        torch.cuda.synchronize()
