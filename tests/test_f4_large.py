"""f4 operators on planes and outputs whose offsets pass 32 bits: elements beyond
2^32, code bytes beyond 2^31, outputs beyond 2^31 elements or bytes.  The last rows have to be
what the same call gives for these rows alone, or the 64-bit product of the values
that their planes stand for."""
import pytest

import parity

pytestmark = pytest.mark.gpu

FORMATS = ["mx", "nv"]


@pytest.fixture(scope="module")
def torch():
    torch = parity.cuda_or_skip()
    if torch.cuda.mem_get_info()[0] < 100e9:
        pytest.skip("needs 100 GB of device memory")
    yield torch
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def w4(torch):
    import w4_quant_matmul_b200
    return w4_quant_matmul_b200


def tail(planes, rows):
    """The last `rows` rows (whole scale tiles) of a matrix as planes of their own."""
    codes, scales, g = planes
    assert codes.shape[0] % 128 == 0 and rows % 128 == 0
    return codes[-rows:].contiguous(), scales[-(rows // 128):].contiguous(), g


def dense(w4, torch, planes):
    return w4.f4_dequantize(*planes, out_dtype=torch.float32).double()


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_past_32_bits(torch, w4, fmt):
    R, K = 313 * 128, 131072
    assert R * K > 2 ** 32 and R * K // 2 > 2 ** 31
    x = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x[:128].normal_(generator=gen)
    x[-256:].normal_(generator=gen)
    planes = w4.f4_quantize(x, fmt)
    if fmt == "nv":
        assert torch.equal(planes[2], w4.f4_tensor_scale(x[-256:]).maximum(
            w4.f4_tensor_scale(x[:128])))
    alone = w4.f4_quantize(x[-256:].contiguous(), fmt, tensor_scale=planes[2])
    end = tail(planes, 256)
    assert torch.equal(end[0], alone[0]) and torch.equal(end[1], alone[1])
    assert not planes[0][128:-256].any()
    del x
    want = w4.f4_dequantize(*alone)
    y = w4.f4_dequantize(*planes)
    assert torch.equal(y[-256:], want)
    del y
    ids = torch.full((20000,), R - 1, device="cuda")
    ids[::3] = 5
    ids[1::3] = -1
    y = w4.f4_embed(*planes, ids)
    assert y.numel() > 2 ** 31
    first = w4.f4_embed(*planes, ids[:3])
    assert torch.equal(first[2], want[-1]) and not first[1].any()
    assert torch.equal(y[:19998].view(-1, 3, K)[::1111], first.expand(6, 3, K))
    assert torch.equal(y[-1], first[19999 % 3])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 3, 8])
def test_gemv_past_32_bits(torch, w4, fmt, M):
    N, K = 782 * 128, 65536
    assert N * K // 2 > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    w[-128:].normal_(generator=gen)
    planes = w4.f4_quantize(w, fmt)
    del w
    x = torch.randn((M, K), device="cuda", generator=gen).bfloat16()
    y = w4.f4_gemv(*planes, x, out_dtype=torch.float32)
    want = x.double() @ dense(w4, torch, tail(planes, 128)).t()
    mass = x.double().abs() @ dense(w4, torch, tail(planes, 128)).abs().t()
    # 1024 steps of the accumulation, 2^-22 each, of digits up to 32 / 7 of a block's
    # largest element, which is below 6 standard deviations, mass being 0.8 of one
    assert ((y[:, -128:].double() - want).abs() <= 1040 * 2.0 ** -22 * 32 / 7 * 8 * mass).all()
    assert not y[:, :-128].any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N", [(50048, 50048), (50048, 50049), (64, 2 ** 24)])
def test_mm_past_32_bits(torch, w4, fmt, M, N):
    """K = 32: no sum has more than 32 terms, all exact in fp32 but for one rounding a
    factor, so that the corners of y can be compared closely."""
    K = 32
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = w4.f4_quantize(torch.randn((N, K), device="cuda", generator=gen).bfloat16(), fmt)
    a = w4.f4_quantize(torch.randn((M, K), device="cuda", generator=gen).bfloat16(), fmt)
    out = torch.bfloat16 if M > 64 else torch.float32
    y = w4.f4_mm(*w, *a, out_dtype=out)
    # (64 x 2^24 fp32 are 2^32 bytes exactly: the largest N at the most tokens of a tile)
    assert y.numel() * y.element_size() > 2 ** 31
    wd, ad = dense(w4, torch, w), dense(w4, torch, a)
    eps = torch.finfo(out).eps / 2
    for rows in (slice(0, 64), slice(M - 64, M), slice(M // 2 - 32, M // 2 + 32)):
        for cols in (slice(0, 300), slice(N - 300, N), slice(N // 2, N // 2 + 300)):
            want = ad[rows] @ wd[cols].t()
            mass = ad[rows].abs() @ wd[cols].abs().t()
            # the values' own rounding to fp32 and the factors: 8 of 2^-24; the step of
            # the accumulation 2^-22; the output's rounding of a value up to that
            bound = (8 * 2.0 ** -24 + 2.0 ** -22) * mass
            bound = bound + eps * (want.abs() + bound)
            assert ((y[rows, cols].double() - want).abs() <= bound).all(), (rows, cols)
