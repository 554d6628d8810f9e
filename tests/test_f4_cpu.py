"""The microscaled 4-bit floating-point operators without a GPU: the plain
reference's own pins, the C ABI's argument checks (nothing is enqueued) and the
binding's checks."""
import numpy as np
import pytest

import f4_reference as ref

torch = pytest.importorskip("torch")
w4 = pytest.importorskip("w4_quant_matmul_b200")

FAKE = 0x10000  # never dereferenced: validation fails first
MIS = 0x10001


@pytest.fixture(scope="module")
def lib():
    from w4_quant_matmul_b200 import build, _lib
    build.build()
    return _lib.load()


# ---------------------------------------------------------------------------
# the reference
# ---------------------------------------------------------------------------

def test_e2m1_levels_and_ties():
    v = np.array([0, .25, .26, .5, .75, 1, 1.25, 1.26, 1.5, 1.75, 2, 2.5, 2.6, 3, 3.5, 4, 5, 5.1, 6, 9])
    want = [0, 0, 1, 1, 2, 2, 2, 3, 3, 4, 4, 4, 5, 5, 6, 6, 6, 7, 7, 7]
    assert ref.e2m1_codes(v).tolist() == want
    neg = ref.e2m1_codes(-v)
    assert neg.tolist() == [c + 8 for c in want]
    assert ref.e2m1_values(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6,
                                                       0, -.5, -1, -1.5, -2, -3, -4, -6]


def test_e4m3_matches_torch():
    b = torch.arange(127, dtype=torch.uint8)
    assert torch.equal(b.view(torch.float8_e4m3fn).double(), torch.from_numpy(ref.E4M3))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_reference_quantiser_closed_forms(fmt):
    blk = ref.BLOCK[fmt]
    g = 1.0
    x = np.zeros((3, 64))
    x[0, :] = 6.0            # amax 6
    x[1, 0] = 3.0
    x[1, 1] = -1.5
    codes, scales = ref.quantize(x, fmt, g)
    if fmt == ref.MX:        # floor(log2 6) - 2 = 0; floor(log2 3) - 2 = -1; zero block: byte 0
        assert scales[0].tolist() == [127] * (64 // blk)
        assert scales[1, 0] == 126 and scales[1, 1] == 0
        assert codes[1, :2].tolist() == [7, 8 + 5]   # 3 / 0.5 = 6, -1.5 / 0.5 = -3
    else:                    # 6 / 6 = 1; 3 / 6 = 0.5; zero block: 0
        assert ref.E4M3[scales[0, 0]] == 1.0 and ref.E4M3[scales[1, 0]] == 0.5
        assert scales[1, 1] == 0
        assert codes[1, :2].tolist() == [7, 8 + 5]
    v = ref.values(codes, scales, fmt)
    assert np.array_equal(v, x)                      # all on the grid


def test_reference_tiles():
    s = np.arange(130 * 5).reshape(130, 5).astype(np.uint8)
    t = ref.tile(s, "mx")
    assert t.shape == (2, 2, 512)
    assert t[0, 0, 0] == s[0, 0] and t[0, 0, 16 + 1] == s[1, 1] and t[0, 0, 4 + 2] == s[32, 2]
    assert t[0, 1, 31 * 16 + 12] == s[127, 4] and t[1, 0, 16] == s[129, 0]
    assert t[0, 1, 1] == 0 and t[1, 0, 4] == 0       # padding


def test_bounds_catch_a_swapped_nibble():
    # the tolerance of the products must not hide a real mistake
    rng = np.random.default_rng(0)
    w, a = rng.standard_normal((40, 96)), rng.standard_normal((3, 96))
    cw, sw = ref.quantize(w, "mx")
    ca, sa = ref.quantize(a, "mx")
    wv, av = ref.values(cw, sw, "mx"), ref.values(ca, sa, "mx")
    swapped = ref.values(cw.reshape(40, -1, 2)[:, :, ::-1].reshape(40, 96), sw, "mx")
    shifted = ref.values(cw, np.roll(sw, 1, 1), "mx")
    bound = ref.mm_bound(av, wv, 96)
    for wrong in (swapped, shifted):
        assert (np.abs(av @ wrong.T - av @ wv.T) > bound).mean() > 0.5
    xb = ref.gemv_bound(a, wv, 96, "mx")
    assert (np.abs(a @ swapped.T - a @ wv.T) > xb).mean() > 0.5


def test_the_extension_is_built_and_bound(lib):
    from w4_quant_matmul_b200 import build
    import os
    assert os.path.exists(build.CALLS)
    from w4_quant_matmul_b200 import _f4call
    assert w4._calls() is _f4call
    # without tensors that it can take it leaves the call to the checks
    assert _f4call.mm(1, 2, None, 3, 4, None, None) is None
    assert _f4call.gemv(torch.zeros(2, 2), None, None, None, None) is None


# ---------------------------------------------------------------------------
# C ABI
# ---------------------------------------------------------------------------

def test_scale_bytes(lib):
    f = lib.f4_scale_bytes
    assert f(1, 32, 0) == 512 and f(128, 128, 0) == 512 and f(129, 160, 0) == 4 * 512
    assert f(1, 32, 1) == 512 and f(128, 96, 1) == 2 * 512
    assert f(0, 64, 0) == 0 and f(5, 0, 0) == 0
    assert f(5, 48, 0) == 0 and f(5, 64, 2) == 0 and f(-1, 64, 0) == 0
    assert f(2 ** 24 + 1, 64, 0) == 0 and f(1, 131104, 0) == 0


def test_quantize_validation(lib):
    from w4_quant_matmul_b200 import _lib as L
    f = lib.f4_quantize
    ok = dict(x=FAKE, t=0, R=4, K=64, fmt=1, g=FAKE, c=FAKE, s=FAKE)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["x"], a["t"], a["R"], a["K"], a["fmt"], a["g"], a["c"], a["s"], None)

    for bad in (dict(K=48), dict(K=-32), dict(K=131104), dict(R=-1), dict(R=2 ** 24 + 1),
                dict(t=3), dict(t=-1), dict(fmt=2), dict(fmt=-1)):
        assert call(**bad) == L.W4_ERR_SHAPE, bad
    for p in "xgcs":
        assert call(**{p: None}) == L.W4_ERR_NULL, p
        assert call(**{p: MIS}) == L.W4_ERR_ALIGN, p
    assert call(R=0) == L.W4_OK and call(K=0) == L.W4_OK
    g = lib.f4_tensor_scale
    assert g(FAKE, 0, 4, 48, FAKE, None) == L.W4_ERR_SHAPE
    assert g(FAKE, 5, 4, 64, FAKE, None) == L.W4_ERR_SHAPE
    assert g(None, 0, 4, 64, FAKE, None) == L.W4_ERR_NULL
    assert g(FAKE, 0, 4, 64, None, None) == L.W4_ERR_NULL
    assert g(MIS, 0, 4, 64, FAKE, None) == L.W4_ERR_ALIGN
    assert g(FAKE, 0, 4, 64, MIS, None) == L.W4_ERR_ALIGN


def test_dequantize_and_embed_validation(lib):
    from w4_quant_matmul_b200 import _lib as L
    f = lib.f4_dequantize
    assert f(FAKE, FAKE, FAKE, 4, 48, 1, FAKE, 0, None) == L.W4_ERR_SHAPE
    assert f(FAKE, FAKE, FAKE, 4, 64, 1, FAKE, 2, None) == L.W4_ERR_SHAPE
    assert f(FAKE, FAKE, None, 4, 64, 1, FAKE, 0, None) == L.W4_ERR_NULL
    assert f(FAKE, FAKE, MIS, 4, 64, 1, FAKE, 0, None) == L.W4_ERR_ALIGN
    assert f(FAKE, MIS, None, 4, 64, 0, FAKE, 0, None) == L.W4_ERR_ALIGN
    assert f(FAKE, FAKE, None, 0, 64, 0, FAKE, 0, None) == L.W4_OK
    e = lib.f4_embed
    assert e(FAKE, FAKE, None, 0, 64, 0, FAKE, 3, 1.0, FAKE, 0, None) == L.W4_ERR_SHAPE
    assert e(FAKE, FAKE, None, 9, 40, 0, FAKE, 3, 1.0, FAKE, 0, None) == L.W4_ERR_SHAPE
    assert e(FAKE, FAKE, None, 9, 64, 0, FAKE, -1, 1.0, FAKE, 0, None) == L.W4_ERR_SHAPE
    assert e(FAKE, FAKE, None, 9, 64, 0, FAKE, 3, 1.0, FAKE, 9, None) == L.W4_ERR_SHAPE
    assert e(FAKE, FAKE, None, 9, 64, 0, None, 3, 1.0, FAKE, 0, None) == L.W4_ERR_NULL
    assert e(FAKE, FAKE, None, 9, 64, 1, FAKE, 3, 1.0, FAKE, 0, None) == L.W4_ERR_NULL
    assert e(FAKE, FAKE, None, 9, 64, 0, FAKE + 4, 3, 1.0, FAKE, 0, None) == L.W4_ERR_ALIGN
    assert e(FAKE, FAKE, None, 9, 64, 0, FAKE, 0, 1.0, FAKE, 0, None) == L.W4_OK


def test_mm_validation(lib):
    from w4_quant_matmul_b200 import _lib as L
    names = ["codes", "scales", "g", "N", "K", "fmt", "qa", "sa", "ga", "M", "y", "out", "st"]
    ok = [FAKE, FAKE, FAKE, 256, 96, 1, FAKE, FAKE, FAKE, 5, FAKE, 0, None]

    def call(**kw):
        return lib.f4_mm(*[kw.get(n, v) for n, v in zip(names, ok)])

    for bad in (dict(K=48), dict(K=0), dict(K=131104), dict(N=0), dict(M=0), dict(N=2 ** 24 + 1),
                dict(M=2 ** 24 + 1), dict(fmt=2), dict(out=2)):
        assert call(**bad) == L.W4_ERR_SHAPE, bad
    for p in ("codes", "scales", "g", "qa", "sa", "ga", "y"):
        assert call(**{p: None}) == L.W4_ERR_NULL, p
        assert call(**{p: MIS}) == L.W4_ERR_ALIGN, p


def test_gemv_validation(lib):
    from w4_quant_matmul_b200 import _lib as L
    need = lib.f4_gemv_workspace_size(7, 256, 96, 1)
    assert need > 0 and lib.f4_gemv_workspace_size(2, 256, 96, 1) == 0
    names = ["codes", "scales", "g", "N", "K", "fmt", "x", "M", "y", "out", "ws", "nws", "st"]
    ok = [FAKE, FAKE, FAKE, 256, 96, 1, FAKE, 7, FAKE, 0, FAKE, need, None]

    def call(**kw):
        return lib.f4_gemv(*[kw.get(n, v) for n, v in zip(names, ok)])

    for bad in (dict(K=48), dict(K=0), dict(K=65568), dict(N=0), dict(M=0), dict(M=9), dict(fmt=3),
                dict(out=4)):
        assert call(**bad) == L.W4_ERR_SHAPE, bad
    for p in ("codes", "scales", "g", "x", "y"):
        assert call(**{p: None}) == L.W4_ERR_NULL, p
        assert call(**{p: MIS}) == L.W4_ERR_ALIGN, p
    assert call(ws=None) == L.W4_ERR_WORKSPACE
    assert call(nws=need - 1) == L.W4_ERR_WORKSPACE
    assert call(ws=MIS) == L.W4_ERR_ALIGN
    for m, n, k in [(0, 5, 64), (9, 5, 64), (1, 0, 64), (1, 5, 48), (1, 5, 65568)]:
        assert lib.f4_gemv_workspace_size(m, n, k, 0) == 0
    assert lib.f4_gemv_workspace_size(1, 5, 64, 7) == 0


def test_without_a_device_valid_calls_fail_loudly(lib):
    from w4_quant_matmul_b200 import _lib as L
    if torch.cuda.is_available() or lib.w4_check_device_error() == L.W4_OK:
        pytest.skip("a CUDA device is present; this checks the no-device branch only")
    for rc in (lib.f4_tensor_scale(FAKE, 0, 4, 64, FAKE, None),
               lib.f4_quantize(FAKE, 0, 4, 64, 0, None, FAKE, FAKE, None),
               lib.f4_dequantize(FAKE, FAKE, None, 4, 64, 0, FAKE, 0, None),
               lib.f4_embed(FAKE, FAKE, None, 4, 64, 0, FAKE, 3, 1.0, FAKE, 0, None),
               lib.f4_mm(FAKE, FAKE, None, 4, 64, 0, FAKE, FAKE, None, 2, FAKE, 0, None),
               lib.f4_gemv(FAKE, FAKE, None, 4, 64, 0, FAKE, 2, FAKE, 0, FAKE, 1 << 20, None)):
        assert rc in (L.W4_ERR_CUDA, L.W4_ERR_UNSUPPORTED_DEVICE)


# ---------------------------------------------------------------------------
# binding (CPU tensors: a call whose shapes are right stops at the device check)
# ---------------------------------------------------------------------------

def _planes(R, K, fmt):
    blk = ref.BLOCK[fmt]
    return (torch.zeros((R, K // 2), dtype=torch.uint8),
            torch.zeros((-(-R // 128), -(-K // (4 * blk)), 512), dtype=torch.uint8),
            torch.ones(1) if fmt == "nv" else None)


def _device(fn, *a, **kw):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        fn(*a, **kw)


def _shape(name, fn, *a, **kw):
    with pytest.raises(ValueError, match=rf"^{name} must have shape"):
        fn(*a, **kw)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_binding_products(fmt):
    w, a = _planes(130, 96, fmt), _planes(3, 96, fmt)
    x = torch.zeros((3, 96), dtype=torch.bfloat16)
    other = _planes(130, 96, "nv" if fmt == "mx" else "mx")
    _device(w4.f4_mm, *w, *a)
    _device(w4.f4_gemv, *w, x)
    _device(w4.f4_gemv, *w, x, y=torch.zeros((3, 130)), workspace=torch.zeros(9, dtype=torch.uint8))
    # planes of the other format, of another length, of another extent
    _shape("scales", w4.f4_mm, w[0], other[1], w[2], *a)
    _shape("scales", w4.f4_gemv, w[0], other[1], w[2], x)
    _shape("qa", w4.f4_mm, *w, *_planes(3, 128, fmt))
    _shape("codes", w4.f4_gemv, *w, torch.zeros((3, 64), dtype=torch.bfloat16))
    _shape("scales", w4.f4_mm, w[0], w[1][:1], w[2], *a)
    _shape("y", w4.f4_mm, *w, *a, y=torch.zeros((3, 131), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="both be given"):
        w4.f4_mm(*w, a[0], a[1], None if fmt == "nv" else torch.ones(1))
    with pytest.raises(TypeError, match="^x must be torch.bfloat16"):
        w4.f4_gemv(*w, x.float())
    with pytest.raises(ValueError, match="^x must be contiguous"):
        w4.f4_gemv(*w, torch.zeros((96, 3), dtype=torch.bfloat16).t())
    with pytest.raises(TypeError, match="^workspace must be torch.uint8"):
        w4.f4_gemv(*w, x, workspace=torch.zeros(64))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_binding_planes(fmt):
    w = _planes(130, 96, fmt)
    ids = torch.zeros(4, dtype=torch.int64)
    _device(w4.f4_dequantize, *w)
    _device(w4.f4_embed, *w, ids)
    with pytest.raises(TypeError, match="^ids must be torch.int64"):
        w4.f4_embed(*w, ids.int())
    _shape("ids", w4.f4_embed, *w, ids.view(2, 2))
    _shape("y", w4.f4_embed, *w, ids, y=torch.zeros((5, 96), dtype=torch.bfloat16))
    x = torch.zeros((130, 96), dtype=torch.float16)
    _device(w4.f4_quantize, x, fmt)
    _shape("codes", w4.f4_quantize, x, fmt, codes=torch.zeros((130, 96), dtype=torch.uint8))
    _shape("scales", w4.f4_quantize, x, fmt, scales=w[1][:1])
    with pytest.raises(TypeError, match="^x must be bfloat16, float16 or float32"):
        w4.f4_quantize(x.double(), fmt)
    with pytest.raises(ValueError, match="unknown format"):
        w4.f4_quantize(x, "e5m2")
    if fmt == "mx":
        with pytest.raises(ValueError, match="belongs to the nv format"):
            w4.f4_quantize(x, fmt, tensor_scale=torch.ones(1))
    else:
        _shape("tensor_scale", w4.f4_quantize, x, fmt, tensor_scale=torch.ones(2))
        _shape("g", w4.f4_dequantize, w[0], w[1], torch.ones(2))
    _device(w4.f4_tensor_scale, x)


def test_binding_leaves_format_errors_to_the_library():
    # K % 32 != 0: the scale plane's extent along K is open, the call still
    # stops at the device check on the CPU
    codes = torch.zeros((4, 24), dtype=torch.uint8)
    _device(w4.f4_dequantize, codes, torch.zeros((1, 1, 512), dtype=torch.uint8), None)
