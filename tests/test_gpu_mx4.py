"""The 4-bit operators against the oracle: the format bit for bit, the product within its rounding.

Tolerance of the product: products of 4-bit values are exact, so the fp32 sum
of K of them is off by at most K * 2^-23 * sum |a| |b| in any order (each of the
additions off by at most one unit in the last place of a partial sum), and the
result is rounded once to p bits: 2^-p * |result|.  Sums that fp32 holds exactly
are compared bit for bit.
"""

import numpy as np
import pytest

import oracle
from oracle import mx4
from tests.gpu_util import say
from workloads import random_bits, to_bits

pytestmark = pytest.mark.gpu

fo = pytest.importorskip("gemm_tile_signaling_amd")
torch = pytest.importorskip("torch")
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


def bits16(b, dtype):
    return torch.from_numpy(b.view(np.int16).copy()).view(TORCH[dtype]).to("cuda")


def host(t, dtype):
    return oracle.decode_bits(t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16), dtype)


def mixed_bits(seed, rows, cols, dtype):
    """Rows of ordinary values, of every exponent, of zeros, with infinities and NaN, and of denormals."""
    rng = np.random.default_rng(seed)
    b = to_bits(rng.standard_normal((rows, cols)).astype(np.float32) * 10, dtype)
    every = random_bits(seed + 1, rows * cols, dtype).reshape(rows, cols)
    kind = np.arange(rows) % 6
    b[kind == 1] = every[kind == 1]
    b[kind == 2] &= 0x8000
    special = np.array([0x7F80, 0xFF80, 0x7FC0, 0xFFFF] if dtype == "bf16" else [0x7C00, 0xFC00, 0x7E00, 0xFFFF], np.uint16)
    for r in np.nonzero(kind == 3)[0]:
        b[r, rng.integers(0, cols)] = special[rng.integers(0, 4)]
    b[kind == 4] &= 0x807F if dtype == "bf16" else 0x83FF
    # halves of the code grid: ties everywhere
    t = np.ldexp(rng.integers(-64, 65, (rows, cols)).astype(np.float32), rng.integers(-20, 10, (rows, 1)) if dtype == "bf16"
                 else rng.integers(-12, 6, (rows, 1))).astype(np.float32)
    b[kind == 5] = to_bits(t, dtype)[kind == 5]
    return b


SIZES = [(1, 1), (1, 32), (3, 31), (2, 33), (7, 255), (12, 256), (6, 257), (65, 96), (30, 513), (19, 1000), (6, 2064)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows, cols", SIZES)
def test_quantize_is_the_oracles(rows, cols, dtype):
    say(f"mx4_quantize {rows}x{cols} {dtype}")
    b = mixed_bits(rows * 1000 + cols, rows, cols, dtype)
    want = mx4.pack(*mx4.quantize(oracle.decode_bits(b, dtype)))
    cs, ss = fo.mx4_shapes(rows, cols)
    codes = torch.full((cs[0] + 1, cs[1]), 0xA5, dtype=torch.uint8, device="cuda")     # a row of marker bytes after
    scales = torch.full(ss, 0xA5, dtype=torch.uint8, device="cuda")
    fo.mx4_quantize(bits16(b, dtype), codes[:rows], scales)
    assert np.array_equal(codes[:rows].cpu().numpy(), want[0])
    assert np.array_equal(scales.cpu().numpy(), want[1])
    assert (codes[rows:] == 0xA5).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows, cols, ld, at", [(9, 64, 72, 0), (9, 64, 72, 8), (5, 100, 131, 3), (33, 512, 515, 1), (1, 7, 7, 1),
                                                (4, 256, 258, 2)])
def test_quantize_strided_rows(rows, cols, ld, at, dtype):
    """Rows of a wider tensor, beginning on any element; the integer view of the bits as well."""
    say(f"mx4_quantize strided {rows}x{cols} of {ld} from {at} {dtype}")
    b = mixed_bits(rows + cols, rows, ld + at, dtype)[:, at:at + ld]
    flat = np.concatenate([np.full(at, 0x7F80 if dtype == "bf16" else 0x7C00, np.uint16), b.ravel()])
    x = bits16(flat, dtype)[at:].view(rows, ld)[:, :cols]
    want = mx4.pack(*mx4.quantize(oracle.decode_bits(b[:, :cols], dtype)))
    for got in (fo.mx4_quantize(x), fo.mx4_quantize(x.view(torch.int16), dtype=dtype)):
        assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_large_matrices_are_quantised_like_their_parts(dtype):
    """Past 32 MB of 16-bit values the memory accesses differ; the bits must not."""
    rows, cols = 4111, 4131
    wide = (torch.randn(rows, cols + 3, device="cuda") * 5).to(TORCH[dtype])
    wide[17, 100] = float("inf")
    x = wide[:, :cols]
    codes, scales = fo.mx4_quantize(x)
    back = fo.mx4_dequantize(codes, scales, cols, dtype=dtype)
    for a in range(0, rows, 1000):
        c, s = fo.mx4_quantize(x[a:a + 1000])
        assert torch.equal(codes[a:a + 1000], c) and torch.equal(scales[:, a:a + 1000], s)
        assert torch.equal(back[a:a + 1000].view(torch.int16), fo.mx4_dequantize(c, s, cols, dtype=dtype).view(torch.int16))


def random_form(seed, rows, k, lo=0, hi=256):
    rng = np.random.default_rng(seed)
    return rng.integers(0, 16, (rows, k)).astype(np.uint8), rng.integers(lo, hi, (rows, k // 32)).astype(np.uint8)


@pytest.mark.parametrize("rows, cols", SIZES)
def test_dequantize_every_scale(rows, cols):
    say(f"mx4_dequantize {rows}x{cols}")
    nb = -(-cols // 32)
    c, s = random_form(cols, rows, nb * 32)
    s.ravel()[: min(s.size, 4)] = [0, 255, 254, 1][: min(s.size, 4)]
    v = mx4.values(c, s)[:, :cols]
    p, q = (dev(t) for t in mx4.pack(c, s))
    got = fo.mx4_dequantize(p, q, cols, dtype="fp32").cpu().numpy()
    with np.errstate(over="ignore"):
        want = v.astype(np.float32)      # past byte 252 the largest values overflow fp32 to infinities
    assert np.array_equal(got, want, equal_nan=True)
    for dtype in ("bf16", "fp16"):
        g = host(fo.mx4_dequantize(p, q, cols, dtype=dtype), dtype)
        assert np.array_equal(g, oracle.round_to_dtype(v, dtype), equal_nan=True), dtype


def check_gemm(a, b, dtype, ends=None, what=""):
    """a, b: (element codes, scale bytes); b's rows stacked over the problems."""
    say(f"mx4_gemm {what} M={a[0].shape[0]} rows of B={b[0].shape[0]} K={a[0].shape[1]} {dtype} ends={ends}")
    M, K = a[0].shape
    P = 1 if ends is None else len(ends)
    av, bv = mx4.values(*a), mx4.values(*b).reshape(P, -1, K)
    N = bv.shape[1]
    want = mx4.gemm(av, bv, ends)
    size = mx4.gemm(np.abs(av), np.abs(bv), ends)
    out = torch.full((M + 1, N), -7.0, dtype=TORCH[dtype], device="cuda")
    e = None if ends is None else torch.tensor(ends, dtype=torch.int32, device="cuda")
    (pa, qa), (pb, qb) = mx4.pack(*a), mx4.pack(*b)
    # the bytes past a row's last block carry no meaning: NaN scales there must not reach a result
    if K % 256:
        qa[-1, :, K % 256 // 32:] = 255
        qb[-1, :, K % 256 // 32:] = 255
    fo.mx4_gemm(dev(pa), dev(qa), dev(pb), dev(qb), dtype=dtype, row_ends=e, out=out[:M])
    got = host(out, dtype)
    last = M if ends is None else min(max(ends[-1], 0), M)
    assert (got[last:] == -7.0).all()                   # rows of no problem and the row after are not written
    got, want, size = got[:last], want[:last], size[:last]
    p = oracle.DTYPES[dtype]["p"]
    with np.errstate(invalid="ignore"):
        bound = 2.0 ** -p * np.abs(want) + K * 2.0 ** -23 * size * (1 + 2.0 ** -p) + 2.0 ** (-133 if dtype == "bf16" else -25)
        ok = (np.abs(got - want) <= bound) | (np.isnan(got) & np.isnan(want))
    assert ok.all(), (what, int((~ok).sum()), np.argwhere(~ok)[:4].tolist())
    return got, want


GEMM_SIZES = [(1, 8, 32), (1, 16, 256), (1, 1032, 2752), (3, 40, 96), (16, 64, 512), (17, 72, 288), (31, 128, 1024), (33, 256, 160),
              (64, 520, 768), (65, 136, 256), (127, 264, 544), (128, 128, 4096), (200, 8, 320), (257, 264, 64), (300, 520, 1056),
              (513, 776, 512), (1, 24, 16384), (40, 16, 8192),
              (2, 8208, 1056), (16, 8200, 800), (30, 8192, 320), (4, 14336, 544), (13, 4096, 2080), (25, 1000, 96)]


# enough tiles for the larger tile shapes, with partial tiles on both edges and partial last slices
LARGE = [(1025, 4104, 32), (1100, 4240, 800), (2050, 8200, 96), (2100, 8328, 544), (4096, 4096, 256), (2305, 8200, 1312)]


@pytest.mark.parametrize("M, N, K", LARGE)
def test_gemm_large_tiles(M, N, K):
    dtype = "bf16" if K % 64 else "fp16"
    got, _ = check_gemm(random_form(M, M, K, 119, 126), random_form(N, N, K, 119, 126), dtype, what="large")


@pytest.mark.parametrize("ends", [[1200, 1201, 1201, 2500], [0, 700, 2500]])
def test_gemm_large_tiles_of_stacked_problems(ends):
    """Long stacks: the largest tiles, tiles cut at every problem's end, an empty problem, rows of no problem."""
    N, K = 4104 if len(ends) == 4 else 8200, 288
    a, b = random_form(3, 2600, K, 119, 126), random_form(4, N * len(ends), K, 119, 126)
    a[1][650, 2] = b[1][N + 77, 8] = 255
    check_gemm(a, b, "bf16", ends, what="large stacked")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M, N, K", GEMM_SIZES)
def test_gemm_within_its_rounding(M, N, K, dtype):
    check_gemm(random_form(M + 1, M, K, 117, 128), random_form(N + 2, N, K, 117, 128), dtype)


@pytest.mark.parametrize("M, N, K", GEMM_SIZES)
def test_gemm_exact_sums(M, N, K):
    """Codes of 0 and +-1 (codes 2 and 10) under scale 1: small integers, so every sum is exact in bf16 up to 256."""
    rng = np.random.default_rng(M * 7 + N + K)
    keep = min(1.0, 100 / K)
    form = lambda rows: (np.where(rng.random((rows, K)) < keep, rng.choice([2, 10], (rows, K)), 0).astype(np.uint8),  # noqa: E731
                         np.full((rows, K // 32), 127, np.uint8))
    got, want = check_gemm(form(M), form(N), "bf16", what="exact")
    assert np.abs(want).max() <= 256 and np.array_equal(got, want)


ENDS = [([0, 5, 5, 21], 21), ([40], 40), ([3, 3, 3], 3), ([0, 0, 0, 1], 1), ([1, 2, 3, 4, 5], 5), ([300, 310, 600], 640),
        ([64, 128, 256, 256, 300], 300), ([0, 0], 9), (list(range(2, 132, 2)) + [130] * 70, 140)]


@pytest.mark.parametrize("K", [64, 800])
@pytest.mark.parametrize("ends, M", ENDS + [([0, 3, 3, 20, 31], 32), ([2] * 40 + [9], 12), ([16, 16, 16], 16), ([0, 1], 1)])
def test_gemm_stacked_problems(ends, M, K):
    N = 72 if len(ends) < 20 else 16
    got, want = check_gemm(random_form(1, M, K, 120, 126), random_form(2, N * len(ends), K, 120, 126), "bf16", ends)


@pytest.mark.parametrize("N", [256, 2056])
def test_gemm_stacked_problems_large_tiles(N):
    check_gemm(random_form(1, 1500, 320, 120, 126), random_form(2, N * 3, 320, 120, 126), "fp16", [700, 700, 1400])


def test_gemm_ends_outside_the_rows_are_held():
    """Ends past M count as M and negative ones as 0, whatever the device holds."""
    a, b = random_form(1, 20, 64, 120, 126), random_form(2, 3 * 16, 64, 120, 126)
    (pa, qa), (pb, qb) = mx4.pack(*a), mx4.pack(*b)
    e = torch.tensor([-5, 12, 2 ** 30], dtype=torch.int32, device="cuda")
    got = host(fo.mx4_gemm(*map(dev, (pa, qa, pb, qb)), row_ends=e), "bf16")
    want = host(fo.mx4_gemm(*map(dev, (pa, qa, pb, qb)), row_ends=torch.tensor([0, 12, 20], dtype=torch.int32, device="cuda")),
                "bf16")
    assert np.array_equal(got, want)


@pytest.mark.parametrize("M", [1, 20, 150, 300])
def test_gemm_nan_blocks_reach_their_rows_and_columns_only(M):
    N, K = 264, 320
    a, b = random_form(1, M, K, 120, 126), random_form(2, N, K, 120, 126)
    a[1][M // 2, 3] = 255
    b[1][100, 9] = 255
    got, _ = check_gemm(a, b, "bf16", what="NaN blocks")
    nan = np.zeros((M, N), bool)
    nan[M // 2] = nan[:, 100] = True
    assert np.array_equal(np.isnan(got), nan)


@pytest.mark.parametrize("M", [2, 40, 300])
def test_gemm_range_of_scales(M):
    """Scales from 2^-67 to 2^52 (sums stay inside fp32): overflow goes to infinity with its sign as the oracle's rounding does."""
    N, K = 40, 128
    a, b = random_form(3, M, K, 60, 180), random_form(4, N, K, 60, 180)
    av, bv = mx4.values(*a), mx4.values(*b)
    want = av @ bv.T
    got = host(fo.mx4_gemm(*map(dev, mx4.pack(*a)), *map(dev, mx4.pack(*b)), dtype="fp16"), "fp16")
    size = np.abs(av) @ np.abs(bv).T
    big = (np.abs(want) > 2 * 65504) & (np.abs(want) > 1e-3 * size)
    assert big.any() and np.array_equal(got[big], np.sign(want[big]) * np.inf)


def test_gemm_same_result_every_time_and_on_another_stream():
    a, b = random_form(5, 70, 1024, 120, 126), random_form(6, 200, 1024, 120, 126)
    args = [dev(t) for t in (*mx4.pack(*a), *mx4.pack(*b))]
    first = fo.mx4_gemm(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = fo.mx4_gemm(*args, stream=s)
        s.synchronize()
        assert torch.equal(first, got)


def test_operators_replay_in_a_graph():
    """Quantise, product and dequantise recorded once and replayed on new inputs, against the eager results."""
    x = torch.randn(33, 520, device="cuda").to(torch.bfloat16)
    w = fo.mx4_quantize(torch.nn.functional.pad(torch.randn(72, 520, device="cuda"), (0, 24)).to(torch.bfloat16))
    body = lambda: (lambda q: (fo.mx4_gemm(*q, *w), fo.mx4_dequantize(*q, 520)))(fo.mx4_quantize(x))  # noqa: E731
    body()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = body()
    for i in range(4):
        x.copy_(torch.randn(33, 520, device="cuda") * (i + 1))
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, body()):
            assert torch.equal(got, want)
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Operands and an output of more than 2^32 bytes: the last rows are where 64-bit offsets are needed."""
    rows, cols = (1 << 21) + 3, 2048        # 2^32 bytes of 16-bit values and a little
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(5, cols, device="cuda").to(torch.bfloat16)
    x[-5:] = tail
    c, s = fo.mx4_quantize(x)
    cc, ss = fo.mx4_quantize(tail)
    assert torch.equal(c[-5:], cc) and torch.equal(s[:, -5:], ss) and not c[:5].any()
    back = fo.mx4_dequantize(c, s, cols)
    assert torch.equal(back[-5:], fo.mx4_dequantize(cc, ss, cols))
    del x, back
    N = 1032                                # rows * N * 2 bytes of output, past 2^32
    w = fo.mx4_quantize(torch.randn(N, cols, device="cuda").to(torch.bfloat16))
    out = fo.mx4_gemm(c, s, *w)
    assert torch.equal(out[-5:], fo.mx4_gemm(cc, ss, *w)) or torch.allclose(
        out[-5:].float(), fo.mx4_gemm(cc, ss, *w).float(), rtol=2 ** -7, atol=1e-2)
    assert not out[:5].any()
