"""Scales at the ends of their ranges: tensor scales and activations whose product
leaves the range of fp32 while the result does not, block scales 2^-127 and 2^127,
scale bytes with the unused bit set."""
import numpy as np
import pytest

import f4_reference as ref
import parity
from test_f4 import Matrix, dev, host, random_matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return parity.cuda_or_skip()


@pytest.fixture(scope="module")
def w4(torch):
    import w4_quant_matmul_b200
    return w4_quant_matmul_b200


# tokens, rows, k: one CTA a tile; K split over a cluster, rows of y on 16 bytes and
# not; several tiles a CTA; CTA pairs with 16-byte stores and without
MM_PATHS = [(20, 300, 64), (20, 300, 2592), (20, 301, 2592), (10, 38100, 64), (300, 4104, 64),
            (300, 4099, 64)]


def f32(v):
    with np.errstate(over="ignore"):
        return np.asarray(v, np.float64).astype(np.float32)


def check_mm_scales(torch, w4, M, N, K, gw, ga):
    w = random_matrix(torch, N, K, "nv", seed=5, g=gw)
    a = random_matrix(torch, M, K, "nv", seed=6, g=ga)
    zero = np.zeros((1, K), np.uint8)               # a token whose sums are all zero
    z = Matrix(torch, zero, np.ones((1, K // 16), np.uint8), "nv", ga)
    y = host(w4.f4_mm(*w.planes, *a.planes, out_dtype=torch.float32))
    want = a.scaled @ w.scaled.T
    # beside the accumulation the two scales round twice (counted in the bound), and
    # a result below the normal numbers by half a unit of 2^-149
    bound = ref.mm_bound(a.scaled, w.scaled, K) + 2.0 ** -150
    top = 2.0 ** 128 * (1 - 2.0 ** -24)
    inside, over = np.abs(want) + bound < top, np.abs(want) - bound > top
    assert (np.abs(y.astype(np.float64)[inside] - want[inside]) <= bound[inside]).all()
    assert (y[over] == np.sign(want[over]) * np.inf).all()
    y16 = w4.f4_mm(*w.planes, *a.planes)
    assert torch.equal(y16, dev(torch, y).bfloat16())
    assert (host(w4.f4_mm(*w.planes, *z.planes, out_dtype=torch.float32)) == 0).all()


@pytest.mark.parametrize("M,N,K", MM_PATHS)
@pytest.mark.parametrize("ew,ea", [(-100, -55), (-80, -62), (-62, -80), (-75, -75), (100, -100),
                                   (-100, 100), (100, 20), (64, 64), (70, 70)])
def test_mm_of_any_two_tensor_scales(torch, w4, M, N, K, ew, ea):
    check_mm_scales(torch, w4, M, N, K, float(np.float32(1.3 * 2.0 ** ew)),
                    float(np.float32(1.7 * 2.0 ** ea)))


GEMV_PATHS = [(1, 300, 64), (4, 300, 2592), (6, 300, 2592), (7, 300, 64), (7, 6500, 64),
              (1, 40000, 64), (8, 40000, 64)]


@pytest.mark.parametrize("M,N,K", GEMV_PATHS)
@pytest.mark.parametrize("eg,ex", [(-20, 115), (-100, 120), (-100, -20), (-100, -45), (60, -126),
                                   (100, -120), (100, -133), (90, 20), (20, 120)])
def test_gemv_of_any_tensor_scale_and_activations(torch, w4, M, N, K, eg, ex):
    """Integer activations times 2^ex (every digit exact)."""
    w = random_matrix(torch, N, K, "nv", seed=5, g=float(np.float32(1.3 * 2.0 ** eg)))
    rng = np.random.default_rng(7)
    x = rng.integers(-8, 9, (M, K)) * 2.0 ** ex
    if M > 1:
        x[M - 1] = 0.0                              # a token whose sums are all zero
    xt = dev(torch, x.astype(np.float32)).bfloat16()
    x64 = host(xt.double())
    y = host(w4.f4_gemv(*w.planes, xt, out_dtype=torch.float32))
    want = x64 @ w.scaled.T
    # below the normal numbers half a unit of 2^-149 for each of up to 6 K slices;
    # the slices are added in fp32, so that the magnitudes have to stay inside it
    bound = ref.gemv_bound(x64, w.scaled, K, "nv") + 6 * 2.0 ** -150
    top = 2.0 ** 128 * (1 - 2.0 ** -24)
    inside = np.abs(x64) @ np.abs(w.scaled).T + bound < top
    over = np.abs(want) - bound > top
    assert (np.abs(y.astype(np.float64)[inside] - want[inside]) <= bound[inside]).all()
    assert not np.isfinite(y[over]).any()
    if M > 1:
        assert (y[M - 1] == 0).all()
    y16 = w4.f4_gemv(*w.planes, xt)
    assert torch.equal(y16.nan_to_num(nan=1.0), dev(torch, y).bfloat16().nan_to_num(nan=1.0))


# ends of the block scales' range: sums that fp32 holds are exact (64 products of small
# integers, quarters among them)
@pytest.mark.parametrize("wb,ab", [(0, 254), (254, 0), (1, 253), (250, 10), (0, 127), (127, 0),
                                   (60, 60), (0, 0)])
@pytest.mark.parametrize("M,N", [(20, 300), (300, 4099)])
def test_mm_extreme_block_scales(torch, w4, M, N, wb, ab):
    rng = np.random.default_rng(wb + ab)
    w = Matrix(torch, rng.integers(0, 16, (N, 64)).astype(np.uint8), np.full((N, 2), wb, np.uint8), "mx")
    a = Matrix(torch, rng.integers(0, 16, (M, 64)).astype(np.uint8), np.full((M, 2), ab, np.uint8), "mx")
    y = host(w4.f4_mm(*w.planes, *a.planes, out_dtype=torch.float32))
    assert np.array_equal(y, f32(a.values @ w.values.T))


@pytest.mark.parametrize("wb,ex", [(0, 120), (0, 0), (254, -100), (240, -120), (127, -130)])
@pytest.mark.parametrize("M", [1, 7])
def test_gemv_extreme_block_scales(torch, w4, M, wb, ex):
    rng = np.random.default_rng(wb)
    w = Matrix(torch, rng.integers(0, 16, (300, 64)).astype(np.uint8),
               np.full((300, 2), wb, np.uint8), "mx")
    x = dev(torch, (rng.integers(-8, 9, (M, 64)) * 2.0 ** ex).astype(np.float32)).bfloat16()
    y = host(w4.f4_gemv(*w.planes, x, out_dtype=torch.float32))
    assert np.array_equal(y, f32(host(x.double()) @ w.values.T))


def test_bit_7_of_a_scale_byte_is_not_read(torch, w4):
    N, K = 300, 160
    rng = np.random.default_rng(9)
    scales = rng.integers(0, 128, (N, K // 16)).astype(np.uint8)   # NaN (127) among them
    scales[:8] = 56
    w = Matrix(torch, rng.integers(0, 16, (N, K)).astype(np.uint8), scales, "nv", 0.37)
    a = random_matrix(torch, 20, K, "nv", 3)
    high = lambda m: (m.planes[0], m.planes[1] | 0x80, m.planes[2])
    x = dev(torch, rng.standard_normal((7, K))).bfloat16()
    ids = dev(torch, np.array([0, 299, -1, 140]))
    want = np.where(np.isnan(w.values), np.nan, w.values).astype(np.float32) * np.float32(0.37)
    for planes, other in ((w.planes, a.planes), (high(w), high(a))):
        got = host(w4.f4_dequantize(*planes, out_dtype=torch.float32))
        assert np.array_equal(got, want, equal_nan=True)
        rows = host(w4.f4_embed(*planes, ids, out_dtype=torch.float32))
        assert np.array_equal(rows[[0, 1, 3]], want[[0, 299, 140]], equal_nan=True)
        for f, rest in ((w4.f4_mm, other), (w4.f4_gemv, (x[:2],)), (w4.f4_gemv, (x,))):
            y, ref_y = host(f(*planes, *rest, out_dtype=torch.float32)), \
                host(f(*w.planes, *(a.planes if f is w4.f4_mm else rest), out_dtype=torch.float32))
            assert np.array_equal(y, ref_y, equal_nan=True)
