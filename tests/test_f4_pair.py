"""f4_mm where a CTA works on several tiles: the CTA-pair kernel of many tokens,
and the 128 x 64 tiles of few tokens on more rows than CTAs run at once.  Every
shape is checked to reach its kernel by the rule that f4_mm itself evaluates;
expected values are the plain 64-bit reference's."""
import os
import subprocess
import sys

import numpy as np
import pytest

import f4_reference as ref
import parity
from test_f4 import activations, check_product, dev, host, random_matrix

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FORMATS = ["mx", "nv"]
GUARD = 64

# tokens, weight rows, k.  The pair kernel's tiles are 256 x 192: one token past a
# 64-token tile; partial token tiles; K that ends inside a stage and inside an MMA;
# odd last row tiles (their scales start in the middle of a 128-row scale tile);
# rows of y on 16 bytes for both outputs, for fp32 alone, for none
SMALL_PAIR_SHAPES = [(65, 9601, 96), (129, 6401, 288), (300, 4099, 544), (300, 4100, 32),
                     (513, 2200, 1056), (1000, 1283, 160), (10000, 1, 32), (2600, 400, 64)]
# several tiles a pair (more than 74), so that both accumulators come round
PAIR_SHAPES = SMALL_PAIR_SHAPES + [(1900, 2600, 320), (2049, 4104, 224), (257, 20001, 96),
                                   (700, 4096, 2592), (3000, 192 * 7, 9728)]
# 128 x 64 tiles: more row tiles than CTAs at once, with tokens in each tile width
MANY_TILES = [(5, 38100, 288), (17, 38016, 96), (33, 50001, 160), (64, 80000, 96)]


@pytest.fixture(scope="module")
def torch():
    return parity.cuda_or_skip()


@pytest.fixture(scope="module")
def w4(torch):
    import w4_quant_matmul_b200
    return w4_quant_matmul_b200


def pairs(w4, M, N):
    return w4.lib().w4_test_f4_mm_pairs(M, N)


def guarded(torch, M, N, dtype, value=3.0):
    """y [M][N] of poison between guard bands that keep its 16-byte start."""
    buf = torch.full((M * N + 2 * GUARD,), value, dtype=dtype, device="cuda")
    y = buf[GUARD:GUARD + M * N].view(M, N)
    y.fill_(float("nan"))
    return buf, y


def check_mm(torch, w4, fmt, M, N, K):
    w = random_matrix(torch, N, K, fmt, seed=M + N + K)
    a = random_matrix(torch, M, K, fmt, seed=M + N + K + 1, g=2.5)
    outs = []
    for dtype in (torch.float32, torch.bfloat16):
        buf, y = guarded(torch, M, N, dtype)
        w4.f4_mm(*w.planes, *a.planes, y=y)
        assert (buf[:GUARD] == 3).all() and (buf[GUARD + M * N:] == 3).all(), "guard bands"
        outs.append(y)
    check_product(torch, *outs, a.scaled @ w.scaled.T, ref.mm_bound(a.scaled, w.scaled, K))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", SMALL_PAIR_SHAPES)
def test_pairs_small(torch, w4, fmt, M, N, K):
    assert pairs(w4, M, N) == 1
    check_mm(torch, w4, fmt, M, N, K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", PAIR_SHAPES[len(SMALL_PAIR_SHAPES):])
def test_pairs_of_several_tiles(torch, w4, fmt, M, N, K):
    assert pairs(w4, M, N) == 1
    check_mm(torch, w4, fmt, M, N, K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", MANY_TILES)
def test_few_tokens_on_many_tiles(torch, w4, fmt, M, N, K):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert pairs(w4, M, N) == 0 and -(-N // 128) > 2 * sms
    check_mm(torch, w4, fmt, M, N, K)


@pytest.mark.parametrize("M,N", [(1, 1), (64, 2 ** 24), (65, 9472), (449, 2560), (0, 5), (5, 0),
                                 (2 ** 24 + 1, 1)])
def test_the_rule(torch, w4, M, N):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    inside = 1 <= M <= 2 ** 24 and 1 <= N <= 2 ** 24
    want = int(M > 64 and -(-N // 128) * -(-M // 64) > sms) if inside else -1
    assert pairs(w4, M, N) == want


@pytest.mark.parametrize("fmt", FORMATS)
def test_pairs_keep_nan_in_its_row(torch, w4, fmt):
    M, N, K = 300, 4099, 160
    assert pairs(w4, M, N) == 1
    rng = np.random.default_rng(6)
    nb = K // ref.BLOCK[fmt]
    from test_f4 import Matrix

    def matrix(rows, bad):
        scales = rng.integers(100, 120, (rows, nb)).astype(np.uint8)
        for r, b in bad:
            scales[r, b] = ref.NAN_BYTE[fmt]
        return Matrix(torch, rng.integers(0, 16, (rows, K)).astype(np.uint8), scales, fmt,
                      1.0 if fmt == "nv" else None)

    w = matrix(N, [(0, 0), (191, nb - 1), (192, 1), (319, 2), (4098, nb - 1)])
    a = matrix(M, [(31, 0), (255, nb - 1), (299, 1)])
    want = np.zeros((M, N), bool)
    want[:, [0, 191, 192, 319, 4098]] = True
    want[[31, 255, 299]] = True
    y = host(w4.f4_mm(*w.planes, *a.planes, out_dtype=torch.float32))
    assert np.array_equal(np.isnan(y), want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_pairs_in_a_chain(torch, w4, fmt):
    """Products of the pair kernel and quantisers fed each other's outputs back to
    back, eagerly and as a replayed graph, against a run with a wait after each."""
    D, M = 1024, 1300
    assert pairs(w4, M, D) == 1
    ws = [w4.f4_quantize(dev(torch, np.random.default_rng(i).standard_normal((D, D)) / 32).float(),
                         fmt) for i in range(5)]
    x0 = dev(torch, activations(M, D, 8)).bfloat16()
    ys = [torch.empty((M, D), dtype=torch.bfloat16, device="cuda") for _ in ws]

    def step(sync=False):
        x = x0
        for p, y in zip(ws, ys):
            q = w4.f4_quantize(x, fmt)
            w4.f4_mm(*p, *q, y=y)
            if sync:
                torch.cuda.synchronize()
            x = y

    def poison():
        for y in ys:
            y.fill_(float("nan"))

    poison()
    step(sync=True)
    want = [y.clone() for y in ys]
    assert all(torch.isfinite(y).all() for y in want)
    for _ in range(5):
        poison()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        poison()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys, want))


@pytest.mark.parametrize("fmt", FORMATS)
def test_pairs_on_several_streams(torch, w4, fmt):
    M, N, K = 513, 2200, 1056
    assert pairs(w4, M, N) == 1
    w, a = random_matrix(torch, N, K, fmt, 21), random_matrix(torch, M, K, fmt, 22)
    few = random_matrix(torch, 20, K, fmt, 23)
    want, want_few = w4.f4_mm(*w.planes, *a.planes), w4.f4_mm(*w.planes, *few.planes)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    out = []
    for i in range(12):
        out.append((w4.f4_mm(*w.planes, *a.planes, stream=streams[i % 3]),
                    w4.f4_mm(*w.planes, *few.planes, stream=streams[(i + 1) % 3])))
    torch.cuda.synchronize()
    for big, small in out:
        assert torch.equal(big, want) and torch.equal(small, want_few)


@pytest.mark.skipif(os.environ.get("W4_LIBRARY") == "debug", reason="runs this file's cases itself")
def test_small_pair_cases_with_index_checks(torch):
    """The small cases against libw4_debug.so, whose failed index checks the
    session's fixture reports."""
    from w4_quant_matmul_b200 import build
    build.build(debug=True)
    cases = ["test_pairs_small", "test_few_tokens_on_many_tiles", "test_pairs_keep_nan"]
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p",
                        "no:cacheprovider", "tests/test_f4_pair.py", "-k", " or ".join(cases)],
                       cwd=ROOT, env=dict(os.environ, W4_LIBRARY="debug"), capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-2000:])
    assert " passed" in r.stdout
