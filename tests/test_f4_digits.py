"""f4_gemv's activations digit by digit: with one weight of value 1 in a row the
output is that activation as the kernel holds it, so that every one of its 22 bits
shows.  Expected, from include/w4.h: with 2^E the power of two of the block's largest
magnitude, x rounded to the nearest multiple of 2^(E - 21), ties to even; no rounding
at all for |x| > 2^-14 of that magnitude.  No error is allowed: the digits times one,
their sum and the powers of two are exact in fp32."""
import numpy as np
import pytest

import f4_reference as ref
import parity

ONE = {"mx": 127, "nv": 56}  # scale bytes of value 1
FORMATS = ["mx", "nv"]


def held(x, fmt):
    """x as f4_gemv holds it (blocks within 2^-17 of the token's largest magnitude)."""
    top = ref.block_amax(x, fmt)
    e = np.where(top > 0, np.frexp(top)[1] - 1, 0)
    return np.ldexp(np.rint(np.ldexp(x, 21 - e)), e - 21)


def activations(M, K, fmt, seed):
    """Every block one large element and odd bf16 mantissas of both signs 2^0 to 2^-24
    below it; blocks 2^0 to 2^-9 below the token's largest."""
    rng = np.random.default_rng(seed)
    blk = ref.BLOCK[fmt]
    mantissa = 1.0 + (2 * rng.integers(0, 64, (M, K)) + 1) / 128.0
    down = rng.integers(1, 25, (M, K))
    for b in range(0, K, blk):
        down[:, b + (b // blk) % blk] = 0
    down += np.repeat(rng.integers(0, 10, (M, K // blk)), blk, 1)
    return np.where(rng.random((M, K)) < 0.5, -1.0, 1.0) * mantissa * 2.0 ** (3 - down)


def tiles(R, K, fmt):
    """The scale plane of value 1 everywhere, zeros in its padding."""
    nb = K // ref.BLOCK[fmt]
    full = np.zeros((-(-R // 128) * 128, -(-nb // 4) * 4), np.uint8)
    full[:R, :nb] = ONE[fmt]
    return np.ascontiguousarray(
        full.reshape(-1, 4, 32, full.shape[1] // 4, 4).transpose(0, 3, 2, 1, 4)).reshape(
            -1, full.shape[1] // 4, 512)


def test_the_plane_is_the_reference_s():
    for fmt in FORMATS:
        for R, K in ((5, 32), (130, 288)):
            s = np.full((R, K // ref.BLOCK[fmt]), ONE[fmt], np.uint8)
            assert np.array_equal(tiles(R, K, fmt), ref.tile(s, fmt))
            assert (ref.scale_value(s, fmt) == 1.0).all()


def test_two_digits_fewer_would_show():
    """x in eight base-8 digits -4..3 is what is held; without the lowest two of them it
    differs in most elements, so that the tests below reject it."""
    for fmt in FORMATS:
        x = activations(3, 288, fmt, 1)
        e = np.frexp(ref.block_amax(x, fmt))[1] - 1
        v = np.rint(np.ldexp(x, 21 - e)).astype(np.int64)
        rest, total, digits = v.copy(), np.zeros_like(v), []
        for j in range(8):                       # digit 7 first
            d = (rest + 4) % 8 - 4
            digits.append(d)
            total += d * 8 ** j
            rest = (rest - d) // 8
        assert (rest == 0).all() and (total == v).all()
        assert np.array_equal(np.ldexp(total.astype(float), e - 21), held(x, fmt))
        fewer = total - digits[0] - 8 * digits[1]
        assert (fewer != v).mean() > 0.5
        # and bf16 alone does not give the low digits' bits away: many elements are exact
        exact = np.abs(x) > 2.0 ** -14 * ref.block_amax(x, fmt)
        assert (held(x, fmt) == x)[exact].all() and 0.4 < exact.mean() < 0.8


@pytest.fixture(scope="module")
def torch():
    return parity.cuda_or_skip()


@pytest.fixture(scope="module")
def w4(torch):
    import w4_quant_matmul_b200
    return w4_quant_matmul_b200


# one kernel with K slices; digits in a workspace beyond 5 (4) tokens; several tiles a
# CTA; one whole tile a CTA and the others along K
@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("N,K", [(300, 288), (2560, 2560), (6500, 544), (40000, 288),
                                 (39643, 2592)])
def test_every_bit_of_an_activation(torch, w4, fmt, N, K):
    rng = np.random.default_rng(N)
    at = np.concatenate([rng.permutation(K) for _ in range(-(-N // K))])[:N]
    minus = rng.random(N) < 0.5
    codes = np.zeros((N, K // 2), np.uint8)
    codes[np.arange(N), at // 2] = np.where(minus, 10, 2) << (4 * (at % 2))
    planes = (torch.from_numpy(codes).cuda(), torch.from_numpy(tiles(N, K, fmt)).cuda(),
              torch.ones(1, device="cuda") if fmt == "nv" else None)
    x = activations(8, K, fmt, seed=K)
    xt = torch.from_numpy(x).cuda().bfloat16()
    assert np.array_equal(xt.double().cpu().numpy(), x)  # bf16 numbers all of them
    want = held(x, fmt)[:, at] * np.where(minus, -1.0, 1.0)
    for M in range(1, 9):
        # the last tokens, so that each one goes through every place
        got = w4.f4_gemv(*planes, xt[8 - M:].contiguous(), out_dtype=torch.float32)
        assert np.array_equal(got.double().cpu().numpy(), want[8 - M:]), M
    assert w4.f4_gemv_workspace_size(4, N, K, fmt) == 0
    if N > 6000:  # more than 49 row tiles: the digits of many tokens leave the kernel
        assert w4.f4_gemv_workspace_size(8, N, K, fmt) > 0
