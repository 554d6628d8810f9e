"""The microscaled 4-bit floating-point operators on the GPU against the plain
64-bit reference: quantiser, dequantiser and lookup bit for bit, the products
within error bounds that f4_reference derives."""
import os
import subprocess
import sys

import numpy as np
import pytest

import f4_reference as ref
import parity

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FORMATS = ["mx", "nv"]


@pytest.fixture(scope="module")
def torch():
    return parity.cuda_or_skip()


@pytest.fixture(scope="module")
def w4(torch):
    import w4_quant_matmul_b200
    return w4_quant_matmul_b200


def dev(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.cpu().numpy()


class Matrix:
    """A 4-bit matrix: its planes on the device and its values in 64 bits
    (without g)."""

    def __init__(self, torch, codes, scales, fmt, g=None):
        self.values = ref.values(codes, scales, fmt)
        self.g = g
        self.planes = (dev(torch, ref.pack(codes)), dev(torch, ref.tile(scales, fmt)),
                       None if g is None else torch.tensor([g], device="cuda"))

    @property
    def scaled(self):
        return self.values * (1.0 if self.g is None else float(np.float32(self.g)))


def random_matrix(torch, R, K, fmt, seed, g=0.37):
    """Random codes and scale bytes over the whole code range and a wide range of scales."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (R, K)).astype(np.uint8)
    lo, hi = (118, 136) if fmt == "mx" else (0, 127)
    scales = rng.integers(lo, hi, (R, K // ref.BLOCK[fmt])).astype(np.uint8)
    return Matrix(torch, codes, scales, fmt, g if fmt == "nv" else None)


# ---------------------------------------------------------------------------
# quantiser
# ---------------------------------------------------------------------------

def special_rows(K, fmt):
    """Rows that exercise the rounding rules: zeros, signed zeros, grids with
    every tie, powers of two and their neighbours, tiny and huge values."""
    rng = np.random.default_rng(5)
    rows = [np.zeros(K), -np.zeros(K), np.full(K, -0.0)]
    grid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1, 1.5, 2, 3, 4, 0.125, 7])
    rows.append(np.resize(grid, K))
    rows.append(-np.resize(grid, K) * 2.0 ** -20)
    rows.append(np.resize(2.0 ** np.arange(-12, 4), K))
    rows.append(np.where(np.arange(K) % ref.BLOCK[fmt] == 3, 100.0, 1e-3))
    rows.append(rng.standard_normal(K) * 2.0 ** rng.integers(-12, 12, K))
    return np.stack(rows)


def check_quantize(torch, w4, x, fmt, g=None):
    """x: a torch tensor on the device."""
    x64 = host(x.double())
    gt = None if g is None else torch.tensor([g], device="cuda")
    codes, scales, gout = w4.f4_quantize(x, fmt, tensor_scale=gt)
    torch.cuda.synchronize()
    if fmt == "nv":
        gref = float(np.float32(g)) if g is not None else ref.tensor_scale(x64)
        assert float(gout.double()) == gref
    else:
        assert gout is None
        gref = None
    c, s = ref.quantize(x64, fmt, gref)
    assert np.array_equal(host(scales), ref.tile(s, fmt)), "scales"
    assert np.array_equal(host(codes), ref.pack(c)), "codes"


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (33, 96), (130, 288), (257, 1056), (2, 8224)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_quantize_bit_exact(torch, w4, fmt, R, K, dtype):
    rng = np.random.default_rng(R * 1000 + K)
    x = rng.standard_normal((R, K)) * np.where(rng.random((R, K)) < 0.01, 20.0, 1.0)
    xt = dev(torch, x).to(getattr(torch, dtype))
    check_quantize(torch, w4, xt, fmt)
    if fmt == "nv":  # a calibrated scale that saturates, one that flushes small blocks to zero
        check_quantize(torch, w4, xt, fmt, g=3.0 / 2688)
        check_quantize(torch, w4, xt, fmt, g=9.0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_quantize_special_rows(torch, w4, fmt, dtype):
    x = dev(torch, special_rows(160, fmt)).to(getattr(torch, dtype))
    check_quantize(torch, w4, x, fmt)
    if fmt == "nv":
        check_quantize(torch, w4, x, fmt, g=1.0)
    if dtype != "float16":  # ends of the fp32 exponent range
        for scale in (2.0 ** 120, 2.0 ** -110, 2.0 ** -132):
            check_quantize(torch, w4, x * scale, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_quantize_non_finite_blocks(torch, w4, fmt, dtype):
    x = dev(torch, np.random.default_rng(2).standard_normal((3, 128))).to(getattr(torch, dtype))
    x[0, 5], x[1, 70], x[1, 127], x[2, 0] = float("nan"), float("inf"), float("-inf"), float("nan")
    check_quantize(torch, w4, x, fmt)
    codes, scales, g = w4.f4_quantize(x, fmt)
    v = host(w4.f4_dequantize(codes, scales, g, torch.float32))
    blk = ref.BLOCK[fmt]
    bad = ~np.isfinite(host(x.double())).reshape(3, -1, blk).all(-1)
    assert np.array_equal(np.isnan(v), np.repeat(bad, blk, 1))


def test_tensor_scale(torch, w4):
    for x in (np.zeros((2, 64)), np.full((1, 32), 2688.0), np.full((5, 96), -1e-35),
              np.random.default_rng(0).standard_normal((300, 4128))):
        t = dev(torch, x.astype(np.float32))
        assert float(w4.f4_tensor_scale(t)) == ref.tensor_scale(host(t))
    t = dev(torch, np.array([[1.0, np.nan, -3.0, np.inf] * 8], np.float32))
    assert float(w4.f4_tensor_scale(t)) == float(np.float32(3.0 / 2688.0))
    for shape in ((0, 64), (3, 0)):
        assert float(w4.f4_tensor_scale(torch.empty(shape, device="cuda"))) == 2.0 ** -100


def test_quantize_fills_padding(torch, w4):
    x = dev(torch, np.ones((5, 160), np.float32))
    scales = torch.full((1, 2, 512), 0xEE, dtype=torch.uint8, device="cuda")
    w4.f4_quantize(x, "mx", scales=scales)
    want = ref.tile(np.full((5, 5), 125, np.uint8), "mx")
    assert np.array_equal(host(scales), want)
    for shape in ((0, 64), (4, 0)):
        c, s, _ = w4.f4_quantize(torch.empty(shape, device="cuda"), "mx")
        assert c.shape == (shape[0], shape[1] // 2) and s.numel() == 0


# ---------------------------------------------------------------------------
# dequantiser and lookup
# ---------------------------------------------------------------------------

def expected_rows(m, rows, alpha=1.0):
    """fl((q s) fl(g alpha)): q s is exact in fp32."""
    c = np.float32(1.0 if m.g is None else m.g) * np.float32(alpha)
    return m.values[rows].astype(np.float32) * c


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("R,K", [(1, 32), (130, 96), (5, 288), (129, 1056), (3, 4128)])
def test_dequantize_bit_exact(torch, w4, fmt, R, K):
    m = random_matrix(torch, R, K, fmt, seed=R + K)
    want = expected_rows(m, np.arange(R))
    got = w4.f4_dequantize(*m.planes, out_dtype=torch.float32)
    assert np.array_equal(host(got), want)
    assert torch.equal(w4.f4_dequantize(*m.planes), dev(torch, want).bfloat16())


def test_dequantize_extreme_scales(torch, w4):
    codes = np.resize(np.arange(16), (3, 256)).astype(np.uint8)
    scales = np.array([[0, 1, 2, 3, 100, 127, 200, 251]] * 3, np.uint8)
    m = Matrix(torch, codes, scales, "mx")
    assert np.array_equal(host(w4.f4_dequantize(*m.planes, out_dtype=torch.float32)),
                          m.values.astype(np.float32))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("V,K,T", [(1, 32, 1), (300, 96, 7), (1000, 2592, 65), (50, 64, 3000)])
def test_embed(torch, w4, fmt, V, K, T):
    m = random_matrix(torch, V, K, fmt, seed=V + T)
    rng = np.random.default_rng(T)
    ids = rng.integers(0, V, T)
    ids[::5] = ids[0]                        # the same row many times
    ids[3::7] = -1                           # padding
    if T > 20:
        ids[10], ids[11], ids[12] = V, 2 ** 40, -2 ** 62
    want = expected_rows(m, np.clip(ids, 0, V - 1), alpha=50.6)
    want[(ids < 0) | (ids >= V)] = 0.0
    it = dev(torch, ids)
    got = w4.f4_embed(*m.planes, it, scale=50.6, out_dtype=torch.float32)
    assert np.array_equal(host(got), want)
    assert torch.equal(w4.f4_embed(*m.planes, it, scale=50.6), dev(torch, want).bfloat16())
    assert w4.f4_embed(*m.planes, it[:0]).shape == (0, K)


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def check_product(torch, got32, got16, want, bound):
    y = host(got32).astype(np.float64)
    assert y.shape == want.shape
    worst = (np.abs(y - want) / np.maximum(bound, 1e-300)).max()
    assert worst <= 1.0, f"error {worst:.3g} of the bound"
    # bf16 output: one rounding of the same sums
    assert torch.equal(got16, got32.bfloat16())


MM_SHAPES = [(1, 1, 32), (2, 3, 64), (16, 128, 96), (17, 129, 128), (31, 200, 160), (33, 300, 288),
             (64, 127, 1056), (65, 257, 544), (128, 256, 2560), (129, 130, 800), (255, 513, 320),
             (256, 2100, 96), (257, 130, 1056), (300, 513, 2592), (513, 1030, 512), (1, 5000, 544),
             (7, 640, 9728), (100, 384, 9728)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", MM_SHAPES)
def test_mm(torch, w4, fmt, M, N, K):
    w = random_matrix(torch, N, K, fmt, seed=M + N + K)
    a = random_matrix(torch, M, K, fmt, seed=M + N + K + 1, g=2.5)
    y = w4.f4_mm(*w.planes, *a.planes, out_dtype=torch.float32)
    y16 = w4.f4_mm(*w.planes, *a.planes)
    check_product(torch, y, y16, a.scaled @ w.scaled.T, ref.mm_bound(a.scaled, w.scaled, K))


@pytest.mark.parametrize("fmt", FORMATS)
def test_mm_longest_k(torch, w4, fmt):
    K = 131072
    w = random_matrix(torch, 3, K, fmt, seed=8)
    a = random_matrix(torch, 2, K, fmt, seed=9)
    y = w4.f4_mm(*w.planes, *a.planes, out_dtype=torch.float32)
    check_product(torch, y, w4.f4_mm(*w.planes, *a.planes), a.scaled @ w.scaled.T,
                  ref.mm_bound(a.scaled, w.scaled, K))


GEMV_SHAPES = [(1, 32), (3, 64), (128, 96), (129, 288), (300, 544), (2560, 4096), (1000, 2592),
               (20000, 160), (6151, 2560), (40, 65536)]


def activations(M, K, seed):
    """Outliers, quiet stretches and a zero block among normal values."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.where(rng.random((M, K)) < 0.01, 20.0, 1.0)
    x[:, : K // 4] *= 2.0 ** rng.integers(-20, 3, (M, K // 4))
    x[0, :32] = 0.0
    return x


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("N,K", GEMV_SHAPES)
def test_gemv(torch, w4, fmt, N, K):
    w = random_matrix(torch, N, K, fmt, seed=N + K)
    for M in range(1, 9):
        x = dev(torch, activations(M, K, seed=M + K)).bfloat16()
        x64 = host(x.double())
        y = w4.f4_gemv(*w.planes, x, out_dtype=torch.float32)
        check_product(torch, y, w4.f4_gemv(*w.planes, x), x64 @ w.scaled.T,
                      ref.gemv_bound(x64, w.scaled, K, fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tiles,K", [(296, 512), (297, 512), (297, 1056), (310, 2592), (345, 2592),
                                     (405, 1312), (590, 1056), (593, 1056)])
def test_gemv_of_one_to_two_tiles_a_cta(torch, w4, fmt, tiles, K):
    """Row counts about one and two times the CTAs that run at once, where tiles
    may be left over for clusters: 13 row tiles (1664 rows) over and over, so that
    any mix-up of tiles shows, and a last one that ends early."""
    base = random_matrix(torch, 13 * 128, K, fmt, seed=K)
    N = tiles * 128 - 37
    reps = -(-tiles // 13)
    codes = base.planes[0].repeat(reps, 1)[:N].contiguous()
    plane = base.planes[1].repeat(reps, 1, 1)[:tiles].contiguous()
    for M in (1, 2, 3, 4, 5, 6, 8):
        x = dev(torch, activations(M, K, seed=M)).bfloat16()
        x64 = host(x.double())
        room = torch.full((M * N + 64,), 7.0, device="cuda")
        y = room[:M * N].view(M, N)
        w4.f4_gemv(codes, plane, base.planes[2], x, y=y)
        y16 = w4.f4_gemv(codes, plane, base.planes[2], x)
        assert (room[M * N:] == 7.0).all()
        every = lambda a: np.tile(a, (1, reps))[:, :N]
        check_product(torch, y, y16, every(x64 @ base.scaled.T),
                      every(ref.gemv_bound(x64, base.scaled, K, fmt)))


@pytest.mark.parametrize("fmt", FORMATS)
def test_gemv_is_exact_for_small_integers(torch, w4, fmt):
    # integer weights and activations whose sums stay below 2^24: every fp32
    # partial sum is an integer, so the result has no error at all
    rng = np.random.default_rng(3)
    N, K = 200, 512
    codes = rng.choice(np.array([0, 2, 4, 5, 6, 7, 10, 12, 13, 14, 15], np.uint8), (N, K))
    one = 127 if fmt == "mx" else int(np.searchsorted(ref.E4M3, 1.0))
    w = Matrix(torch, codes, np.full((N, K // ref.BLOCK[fmt]), one, np.uint8), fmt,
               1.0 if fmt == "nv" else None)
    x = rng.integers(-128, 129, (5, K)).astype(np.float64)
    xt = dev(torch, x).bfloat16()
    y = w4.f4_gemv(*w.planes, xt, out_dtype=torch.float32)
    assert np.array_equal(host(y).astype(np.float64), x @ w.scaled.T)


@pytest.mark.parametrize("fmt", FORMATS)
def test_gemv_activation_range(torch, w4, fmt):
    # one token of subnormals, one near the top of bf16, one zero, one with a
    # single huge element
    N, K = 130, 128
    w = random_matrix(torch, N, K, fmt, seed=1, g=1.0)
    rng = np.random.default_rng(4)
    x = rng.standard_normal((4, K))
    x[0] *= 2.0 ** -128
    x[1] *= 2.0 ** 100
    x[2] = 0.0
    x[3, 40] = 2.0 ** 60
    xt = dev(torch, x.astype(np.float32)).bfloat16()
    x64 = host(xt.double())
    y = host(w4.f4_gemv(*w.planes, xt, out_dtype=torch.float32)).astype(np.float64)
    want, bound = x64 @ w.scaled.T, ref.gemv_bound(x64, w.scaled, K, fmt)
    # the smallest token's sums are fp32 subnormals: half a unit of 2^-149 for
    # each of the 8 digit columns' terms and the two factors
    assert (np.abs(y - want) <= bound + 16 * 2.0 ** -149).all()
    assert (y[2] == 0).all()


def test_gemv_small_scales(torch, w4):
    # a tensor scale and activations whose product leaves the range of fp32,
    # with weights that bring the sums back into it
    N, K = 130, 64
    codes = np.full((N, K), 7, np.uint8)                          # 6
    scales = np.full((N, K // 16), 126, np.uint8)                 # 448
    g = 2.0 ** -100
    w = Matrix(torch, codes, scales, "nv", g)
    for M in (1, 5):
        x = np.full((M, K), 2.0 ** -28)
        y = host(w4.f4_gemv(*w.planes, dev(torch, x).bfloat16(), out_dtype=torch.float32))
        # every digit, weight and partial sum is a small integer times a power
        # of two: exact
        assert np.array_equal(y.astype(np.float64), x @ w.scaled.T)


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_stays_in_its_row(torch, w4, fmt):
    N, K, M = 140, 160, 6
    rng = np.random.default_rng(6)
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    scales = rng.integers(100, 120, (N, K // ref.BLOCK[fmt])).astype(np.uint8)
    scales[133, 2] = ref.NAN_BYTE[fmt]
    w = Matrix(torch, codes, scales, fmt, 1.0 if fmt == "nv" else None)
    x = dev(torch, rng.standard_normal((M, K))).bfloat16()
    x[4, 7] = float("nan")
    x[1, 150] = float("inf")
    want = np.zeros((M, N), bool)
    want[:, 133] = True
    want[[1, 4]] = True
    y = host(w4.f4_gemv(*w.planes, x, out_dtype=torch.float32))
    assert np.array_equal(np.isnan(y), want)
    y = host(w4.f4_mm(*w.planes, *w4.f4_quantize(x, fmt), out_dtype=torch.float32))
    assert np.array_equal(np.isnan(y), want)


# ---------------------------------------------------------------------------
# as they are used
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FORMATS)
def test_a_run_of_them(torch, w4, fmt):
    """Tied vocabulary table: embed a prompt, two 4-bit layers over quantised
    activations, logits of the last tokens by the decode GEMV; every step
    against the reference on the previous step's own output."""
    V, D, F, T = 700, 256, 416, 37
    rng = np.random.default_rng(11)
    mats = {}
    for name, (r, k) in dict(table=(V, D), up=(F, D), down=(D, F)).items():
        src = dev(torch, rng.standard_normal((r, k)).astype(np.float32) * 0.05)
        planes = w4.f4_quantize(src, fmt)
        vals = host(w4.f4_dequantize(*planes, out_dtype=torch.float32)).astype(np.float64)
        mats[name] = (planes, vals)
    ids = dev(torch, rng.integers(0, V, T))
    h = w4.f4_embed(*mats["table"][0], ids, scale=16.0)
    for name in ("up", "down"):
        q = w4.f4_quantize(h, fmt)
        a = host(w4.f4_dequantize(*q, out_dtype=torch.float32)).astype(np.float64)
        y = w4.f4_mm(*mats[name][0], *q, out_dtype=torch.float32)
        want, bound = a @ mats[name][1].T, ref.mm_bound(a, mats[name][1], a.shape[1])
        # the dequantised values carry one fp32 rounding each
        assert (np.abs(host(y) - want) <= 1.01 * bound).all()
        h = y.bfloat16()
    x = h[-5:].contiguous()
    logits = w4.f4_gemv(*mats["table"][0], x, out_dtype=torch.float32)
    x64 = host(x.double())
    bound = ref.gemv_bound(x64, mats["table"][1], D, fmt)
    assert (np.abs(host(logits) - x64 @ mats["table"][1].T) <= 1.01 * bound).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_deterministic_and_independent_of_neighbours(torch, w4, fmt):
    # the same call twice gives the same bits, also while another stream runs it
    w = random_matrix(torch, 2560, 1056, fmt, seed=21)
    x = dev(torch, activations(8, 1056, 22)).bfloat16()
    a = w4.f4_quantize(dev(torch, activations(100, 1056, 23)).bfloat16(), fmt)
    ref_g, ref_m = w4.f4_gemv(*w.planes, x), w4.f4_mm(*w.planes, *a)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    out = []
    for i in range(12):
        out.append((w4.f4_gemv(*w.planes, x, stream=streams[i % 3]),
                    w4.f4_mm(*w.planes, *a, stream=streams[(i + 1) % 3])))
    torch.cuda.synchronize()
    for g, m in out:
        assert torch.equal(g, ref_g) and torch.equal(m, ref_m)


@pytest.mark.parametrize("fmt", FORMATS)
def test_captured_and_replayed(torch, w4, fmt):
    N, K, M = 300, 544, 4
    w = random_matrix(torch, N, K, fmt, seed=31)
    x = dev(torch, activations(M, K, 32)).bfloat16()
    src = dev(torch, activations(50, K, 33)).bfloat16()
    ids = dev(torch, np.array([5, 299, -1]))

    def step():
        q = w4.f4_quantize(src, fmt)
        return (w4.f4_gemv(*w.planes, x), w4.f4_mm(*w.planes, *q), w4.f4_embed(*w.planes, ids),
                w4.f4_dequantize(*q))

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs that live side by side
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for seed in (41, 42):
        x.copy_(dev(torch, activations(M, K, seed)).bfloat16())
        src.copy_(dev(torch, activations(50, K, seed + 5)).bfloat16())
        want = step()
        for g, out in graphs:
            for t in out:
                t.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            for t, r in zip(out, want):
                assert torch.equal(t, r)


@pytest.mark.parametrize("fmt", FORMATS)
def test_plain_calls_are_the_same_calls(torch, w4, fmt):
    """The extension's calls against the ctypes way, which a caller's y takes;
    on another current stream too."""
    from w4_quant_matmul_b200 import _f4call
    assert w4._calls() is _f4call
    w, a = random_matrix(torch, 300, 160, fmt, 91), random_matrix(torch, 70, 160, fmt, 92)
    x = dev(torch, activations(6, 160, 93)).bfloat16()
    ids = dev(torch, np.array([0, 299, 300, 7]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for out in (None, torch.bfloat16, torch.float32):
        dt = out or torch.bfloat16
        new = lambda *s: torch.empty(s, dtype=dt, device="cuda")
        for here in (torch.cuda.current_stream(), side):
            with torch.cuda.stream(here):
                for m in (1, 3, 6):
                    xm = x[:m].contiguous()
                    got = w4.f4_gemv(*w.planes, xm, out_dtype=out)
                    assert got.dtype == dt
                    assert torch.equal(got, w4.f4_gemv(*w.planes, xm, y=new(m, 300)))
                assert torch.equal(w4.f4_mm(*w.planes, *a.planes, out_dtype=out),
                                   w4.f4_mm(*w.planes, *a.planes, y=new(70, 300)))
                assert torch.equal(w4.f4_embed(*w.planes, ids, 2.5, out_dtype=out),
                                   w4.f4_embed(*w.planes, ids, 2.5, y=new(4, 160)))
                assert torch.equal(w4.f4_dequantize(*w.planes, out_dtype=out),
                                   w4.f4_dequantize(*w.planes, y=new(300, 160)))
    torch.cuda.synchronize()
    for src in (x, x.float(), x.half()):
        c, s, g = w4.f4_quantize(src, fmt)
        c2, s2, g2 = w4.f4_quantize(src, fmt, codes=torch.empty_like(c))
        assert torch.equal(c, c2) and torch.equal(s, s2)
        assert g is None and g2 is None or torch.equal(g, g2)
        if fmt == "nv":
            assert w4.f4_quantize(src, fmt, tensor_scale=g)[2] is g


def test_wrong_calls_fall_through_to_the_checks(torch, w4):
    w = random_matrix(torch, 300, 160, "mx", 94)
    x = dev(torch, activations(2, 160, 95)).bfloat16()
    with pytest.raises(ValueError, match="^x must be contiguous"):
        w4.f4_gemv(*w.planes, dev(torch, activations(160, 2, 95)).bfloat16().t())
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        w4.f4_gemv(*w.planes, x.cpu())
    with pytest.raises(ValueError, match="^codes must have shape"):
        w4.f4_gemv(*w.planes, x[:, :128].contiguous())
    with pytest.raises(w4.W4Error, match="W4_ERR_SHAPE"):
        w4.f4_gemv(*w.planes, x[:0])
    with pytest.raises(w4.W4Error, match="W4_ERR_SHAPE"):
        w4.f4_gemv(*w.planes, x[:1].expand(9, 160).contiguous())
    with pytest.raises(ValueError, match="unsupported out_dtype"):
        w4.f4_gemv(*w.planes, x, out_dtype=torch.float16)
    # a parameter is a tensor like any other
    p = torch.nn.Parameter(x, requires_grad=False)
    assert torch.equal(w4.f4_gemv(*w.planes, p), w4.f4_gemv(*w.planes, x))


def test_outputs_stay_inside(torch, w4):
    # guard bands around the outputs of ragged sizes
    for fmt in FORMATS:
        for M, N, K in [(3, 129, 96), (65, 7, 160), (300, 131, 288)]:
            w, a = random_matrix(torch, N, K, fmt, 51), random_matrix(torch, M, K, fmt, 52)
            buf = torch.full((M * N + 64,), 3.0, device="cuda")
            y = buf[32:32 + M * N].view(M, N)
            w4.f4_mm(*w.planes, *a.planes, y=y)
            assert (buf[:32] == 3).all() and (buf[32 + M * N:] == 3).all()
            assert torch.equal(y, w4.f4_mm(*w.planes, *a.planes, out_dtype=torch.float32))
            m = min(M, 8)
            x = dev(torch, activations(m, K, 53)).bfloat16()
            need = w4.f4_gemv_workspace_size(m, N, K, fmt)
            ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
            buf.fill_(3.0)
            y = buf[32:32 + m * N].view(m, N)
            w4.f4_gemv(*w.planes, x, y=y, workspace=ws[:need])
            assert (buf[:32] == 3).all() and (buf[32 + m * N:] == 3).all()
            assert (ws[need:] == 0x5A).all()


def test_workspace_contents_do_not_matter(torch, w4):
    for fmt in FORMATS:
        w = random_matrix(torch, 6500, 288, fmt, 61)
        x = dev(torch, activations(7, 288, 62)).bfloat16()
        need = w4.f4_gemv_workspace_size(7, 6500, 288, fmt)
        outs = []
        for fill in (0x00, 0xFF, 0x7F):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            outs.append(w4.f4_gemv(*w.planes, x, workspace=ws, out_dtype=torch.float32))
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_weights_written_just_before(torch, w4):
    # quantise, then multiply at once on the same stream: the product must see
    # the new weights
    rng = np.random.default_rng(71)
    x = dev(torch, activations(2, 512, 72)).bfloat16()
    codes = scales = None
    for i in range(4):
        src = dev(torch, rng.standard_normal((3000, 512)).astype(np.float32))
        codes, scales, _ = w4.f4_quantize(src, "mx", codes=codes, scales=scales)
        y = w4.f4_gemv(codes, scales, None, x, out_dtype=torch.float32)
        torch.cuda.synchronize()
        again = w4.f4_gemv(codes, scales, None, x, out_dtype=torch.float32)
        assert torch.equal(y, again)


@pytest.mark.parametrize("fmt", FORMATS)
def test_large_weights_written_just_before(torch, w4, fmt):
    """The same for streams of several tiles a CTA, whose first weights are
    requested before the kernel ahead has completed: planes that the quantiser or
    a copy on the stream has just written, directly ahead of the product."""
    N, K = 40000, 512
    gen = torch.Generator(device="cuda").manual_seed(9)
    srcs = [torch.randn(N, K, device="cuda", generator=gen) for _ in range(2)]
    sets = [w4.f4_quantize(s, fmt) for s in srcs]
    for M in (1, 5, 7):
        x = dev(torch, activations(M, K, 73)).bfloat16()
        torch.cuda.synchronize()
        want = []
        for p in sets:
            want.append(w4.f4_gemv(*p, x))
            torch.cuda.synchronize()
        codes, scales = (torch.empty_like(t) for t in sets[0][:2])
        y = torch.empty_like(want[0])
        for i in range(12):
            k, g = i % 2, sets[i % 2][2]
            y.fill_(float("nan"))
            w4.f4_gemv(*sets[1 - k], x)      # a kernel that lets the next start early
            if i % 4 < 2:
                w4.f4_quantize(srcs[k], fmt, g, codes, scales)
            else:
                codes.copy_(sets[k][0])
                scales.copy_(sets[k][1])
            w4.f4_gemv(codes, scales, g, x, y=y)
            torch.cuda.synchronize()
            assert torch.equal(y, want[k]), (M, i)


@pytest.mark.parametrize("fmt", FORMATS)
def test_weights_from_another_stream(torch, w4, fmt):
    """Planes and activations written late on one stream, an event, the product on
    another stream behind kernels that let it start early."""
    N, K = 40000, 512
    gen = torch.Generator(device="cuda").manual_seed(19)
    src = [torch.randn(N, K, device="cuda", generator=gen) for _ in range(2)]
    sets = [w4.f4_quantize(s, fmt) for s in src]
    xs = [dev(torch, activations(7, K, 80 + i)).bfloat16() for i in range(2)]
    torch.cuda.synchronize()
    want = {}
    for k in range(2):
        for m in (1, 5, 7):
            want[k, m] = w4.f4_gemv(*sets[k], xs[k][:m])
    codes, scales, x = (t.clone() for t in (*sets[0][:2], xs[0]))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(6):
        k = i % 2
        with torch.cuda.stream(a):
            torch.cuda._sleep(2_000_000)
            w4.f4_quantize(src[k], fmt, sets[k][2], codes, scales)
            x.copy_(xs[k])
            done = a.record_event()
        with torch.cuda.stream(b):
            w4.f4_gemv(*sets[0], xs[0])
            b.wait_event(done)
            got = {m: w4.f4_gemv(codes, scales, sets[k][2], x[:m]) for m in (1, 5, 7)}
            a.wait_stream(b)
        torch.cuda.synchronize()
        for m in (1, 5, 7):
            assert torch.equal(got[m], want[k, m]), (i, m)


def test_workspace_too_small_is_refused(torch, w4):
    w = random_matrix(torch, 6500, 96, "mx", 81)
    x = dev(torch, activations(7, 96, 82)).bfloat16()
    need = w4.f4_gemv_workspace_size(7, 6500, 96, "mx")
    y = torch.full((7, 6500), 9.0, device="cuda")
    with pytest.raises(w4.W4Error, match="W4_ERR_WORKSPACE"):
        w4.f4_gemv(*w.planes, x, y=y,
                   workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert (y == 9).all()


CAPTURE_FIRST = """
import torch, w4_quant_matmul_b200 as w4
x = torch.randn(40, 288, device="cuda").bfloat16()
w = torch.randn(300, 288, device="cuda")
ids = torch.tensor([3, -1, 299], device="cuda")
out = {}
def step():
    for fmt in ("mx", "nv"):
        p, a = w4.f4_quantize(w, fmt), w4.f4_quantize(x, fmt)
        out[fmt] = [w4.f4_mm(*p, *a), w4.f4_gemv(*p, x[:1]), w4.f4_gemv(*p, x[:8]),
                    w4.f4_embed(*p, ids), w4.f4_dequantize(*p)]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):       # the first calls of the process
    step()
graphed = {k: list(v) for k, v in out.items()}
for r in range(2):
    g.replay()
torch.cuda.synchronize()
step()
torch.cuda.synchronize()
for fmt in out:
    for a, b in zip(graphed[fmt], out[fmt]):
        assert torch.equal(a, b)
w4.w4_check_device_error()
print("captured")
"""


def test_first_calls_inside_a_capture(torch):
    r = subprocess.run([sys.executable, "-c", CAPTURE_FIRST], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, (r.stdout, r.stderr[-3000:])


def test_two_host_threads(torch, w4):
    """Two threads, each with its own stream and tensors, calling at once."""
    import threading
    bad = []

    def work(seed, fmt):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            w = random_matrix(torch, 6500, 544, fmt, seed)
            x = dev(torch, activations(7, 544, seed + 1)).bfloat16()
            src = dev(torch, activations(150, 544, seed + 2)).bfloat16()
            want = None
            for i in range(40):
                q = w4.f4_quantize(src, fmt)
                got = [w4.f4_gemv(*w.planes, x), w4.f4_gemv(*w.planes, x[:1]),
                       w4.f4_gemv(*w.planes, x[:4]),
                       w4.f4_mm(*w.planes, *q), q[0]]
                s.synchronize()
                if want is None:
                    want = got
                elif not all(torch.equal(a, b) for a, b in zip(want, got)):
                    bad.append((seed, i))

    threads = [threading.Thread(target=work, args=(100 * i, FORMATS[i % 2])) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    w4.w4_check_device_error()


@pytest.mark.parametrize("fmt", FORMATS)
def test_chain_of_dependent_products(torch, w4, fmt):
    """Products fed each other's outputs back to back, every buffer poisoned
    before: each kernel starts while the one before it still runs and has to
    wait for its results."""
    D = 512
    ws = [w4.f4_quantize(dev(torch, np.random.default_rng(i).standard_normal((D, D)) / 20)
                         .float(), fmt) for i in range(6)]
    for M in (1, 4, 7):
        x0 = dev(torch, activations(M, D, 7)).bfloat16()
        want, x = [], x0
        for p in ws:
            x = w4.f4_gemv(*p, x)
            torch.cuda.synchronize()
            want.append(x.clone())
        ys = [torch.empty((M, D), dtype=torch.bfloat16, device="cuda") for _ in ws]
        for _ in range(5):
            for y in ys:
                y.fill_(float("nan"))
            x = x0
            for p, y in zip(ws, ys):
                x = w4.f4_gemv(*p, x, y=y)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(ys, want))
    for M in (40, 300):
        x0 = dev(torch, activations(M, D, 8)).bfloat16()
        want, x = [], x0
        for p in ws:
            q = w4.f4_quantize(x, fmt)
            torch.cuda.synchronize()
            x = w4.f4_mm(*p, *q)
            torch.cuda.synchronize()
            want.append(x.clone())
        for _ in range(5):
            got, x = [], x0
            for p in ws:
                x = w4.f4_mm(*p, *w4.f4_quantize(x, fmt))
                got.append(x)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_beside_the_integer_format(torch, w4):
    """f4 kernels between the library's other kernels, which start early too:
    every result as when each kernel runs alone."""
    N, K = 512, 512
    src = dev(torch, np.random.default_rng(3).standard_normal((N, K))).float()
    x = dev(torch, activations(4, K, 4)).bfloat16()

    def step(sync):
        def done(*t):
            if sync:
                torch.cuda.synchronize()
            return t
        codes, d, m = done(*w4.w4_pack(src))
        f = w4.f4_quantize(src, "nv")
        done()
        y = w4.w4_gemv(codes, d, m, x)
        done()
        z = w4.f4_gemv(*f, y)
        done()
        q = w4.q8_quantize_act(z)
        done()
        u = w4.w4a8_mmq(codes, d, m, *q)
        done()
        v = w4.f4_mm(*f, *w4.f4_quantize(u, "nv"))
        done()
        t = w4.w4a8_gemv_bf16(codes, d, m, v)
        torch.cuda.synchronize()
        return [y, z, *q, u, v, t]

    want = step(True)
    for _ in range(8):
        assert all(torch.equal(a, b) for a, b in zip(step(False), want))


@pytest.mark.skipif(os.environ.get("W4_LIBRARY") == "debug", reason="runs this file's cases itself")
def test_small_cases_with_index_checks(torch):
    """The small cases against libw4_debug.so, whose failed index checks the
    session's fixture reports."""
    from w4_quant_matmul_b200 import build
    build.build(debug=True)
    cases = ["test_quantize_bit_exact", "test_dequantize_bit_exact", "test_embed",
             "test_outputs_stay_inside", "test_nan_stays_in_its_row", "test_a_run_of_them"]
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p",
                        "no:cacheprovider", "tests/test_f4.py", "-k", " or ".join(cases)],
                       cwd=ROOT, env=dict(os.environ, W4_LIBRARY="debug"), capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-2000:])
    assert " passed" in r.stdout
