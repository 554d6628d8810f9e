"""The f4 products against libw4_debug.so, with index checks on every store to
global memory, and guard bands where f4_gemv works with a workspace."""
import os
import subprocess
import sys

import pytest

import parity
from test_f4 import activations, dev, random_matrix

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def torch():
    return parity.cuda_or_skip()


@pytest.fixture(scope="module")
def w4(torch):
    import w4_quant_matmul_b200
    return w4_quant_matmul_b200


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,M,N,K", [("mx", 7, 6500, 96), ("mx", 8, 40000, 32),
                                       ("nv", 5, 6501, 160), ("nv", 8, 300, 16416)])
def test_gemv_stays_inside_its_workspace(torch, w4, fmt, M, N, K):
    need = w4.f4_gemv_workspace_size(M, N, K, fmt)
    assert need > 0
    w = random_matrix(torch, N, K, fmt, 51)
    x = dev(torch, activations(M, K, 53)).bfloat16()
    ws = torch.full((need + 128,), 0x5A, dtype=torch.uint8, device="cuda")
    buf = torch.full((M * N + 64,), 3.0, device="cuda")
    y = buf[32:32 + M * N].view(M, N)
    w4.f4_gemv(*w.planes, x, y=y, workspace=ws[64:64 + need])
    assert (ws[:64] == 0x5A).all() and (ws[64 + need:] == 0x5A).all()
    assert (buf[:32] == 3).all() and (buf[32 + M * N:] == 3).all()
    assert torch.equal(y, w4.f4_gemv(*w.planes, x, out_dtype=torch.float32))


@pytest.mark.gpu
@pytest.mark.skipif(os.environ.get("W4_LIBRARY") == "debug", reason="runs these cases itself")
@pytest.mark.parametrize("file,cases", [
    ("test_f4.py", "test_mm or (test_gemv and (160 or 288 or 544 or 96 or 64)) or one_to_two"),
    ("test_f4_scales.py", "any_two or any_tensor_scale"),
    ("test_f4_checks.py", "workspace")])
def test_products_with_index_checks(torch, file, cases):
    """The session's fixture reports a failed check after each case."""
    from w4_quant_matmul_b200 import build
    build.build(debug=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p",
                        "no:cacheprovider", f"tests/{file}", "-k", cases],
                       cwd=ROOT, env=dict(os.environ, W4_LIBRARY="debug"), capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-2000:])
    assert " passed" in r.stdout
