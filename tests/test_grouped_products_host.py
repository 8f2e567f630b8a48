"""Refusals of the quantizers and grouped products on the host: the C entry
points' argument checks (run where no GPU is visible, as test_capi_host.py
does, so that a lost check cannot launch anything) and the Python calls'."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import moe_gated_activation_b200 as mg
from moe_gated_activation_b200 import _capi
from moe_gated_activation_b200 import build as mbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_CHILD = os.environ.get("MOEACT_HOST_CHECKS_CHILD") == "1"
GPU_VISIBLE = (not _CHILD) and torch.cuda.is_available()


@pytest.fixture(autouse=True)
def _only_without_a_gpu(request):
    if GPU_VISIBLE and request.node.originalname != "test_host_checks_run_without_a_gpu":
        pytest.skip("runs in a child process with no GPU visible")


def test_host_checks_run_without_a_gpu():
    if not GPU_VISIBLE:
        return
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", MOEACT_HOST_CHECKS_CHILD="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.abspath(__file__)], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]


_BUF = np.zeros(1 << 16, dtype=np.uint8)
PTR = (_BUF.ctypes.data + 255) // 256 * 256


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return _capi.lib()


GEMM = dict(a=PTR, sa=PTR, la=0, M=64, K=128, ro=PTR, E=2, status=PTR, w=PTR, sw=PTR, lw=0, H=128,
            out=PTR, ldo=128, dt=0, noop=None, stream=None)
WGRAD = dict(dy=PTR, sdy=PTR, x=PTR, sx=PTR, rows=4, layout=0, M=64, H=128, K=128, ro=PTR, cb=PTR,
             E=2, status=PTR, dw=PTR, dt=1, acc=0, noop=None, stream=None)
Q4 = dict(x=PTR, ldx=128, M=64, N=128, codes=PTR, scales=PTR, layout=0, noop=None, stream=None)
D4 = dict(codes=PTR, scales=PTR, layout=0, M=64, N=128, out=PTR, ldo=128, noop=None, stream=None)

EINVAL, EALIGN, ERANGE = _capi.EINVAL, _capi.EALIGN, _capi.ERANGE


@pytest.mark.parametrize("change,status", [
    (dict(a=None), EINVAL), (dict(sa=None), EINVAL), (dict(w=None), EINVAL), (dict(sw=None), EINVAL),
    (dict(out=None), EINVAL), (dict(ro=None), EINVAL), (dict(status=None), EINVAL),
    (dict(a=PTR + 1), EALIGN), (dict(sw=PTR + 8), EALIGN), (dict(out=PTR + 8), EALIGN),
    (dict(ro=PTR + 4), EALIGN), (dict(status=PTR + 2), EALIGN), (dict(noop=PTR + 2), EALIGN),
    (dict(M=-1), EINVAL), (dict(K=0), EINVAL), (dict(K=48), EINVAL), (dict(H=100), EINVAL),
    (dict(E=0), EINVAL), (dict(E=_capi.MAX_GROUPS + 1), EINVAL), (dict(dt=2), EINVAL),
    (dict(ldo=96), EINVAL), (dict(ldo=132), EALIGN), (dict(dt=1, ldo=130), EALIGN),
    (dict(la=2), EINVAL), (dict(lw=-1), EINVAL), (dict(la=1), EINVAL),       # 64 rows: no whole tile
    (dict(lw=1, K=96), EINVAL), (dict(M=(1 << 30) + 1), ERANGE), (dict(K=1 << 25), ERANGE),
    (dict(H=1 << 24, E=2000, ldo=1 << 24), ERANGE), (dict(M=1 << 30, H=1 << 20, ldo=1 << 20), ERANGE),
])
@pytest.mark.parametrize("name", ["grouped_mxfp8_gemm", "grouped_mxfp4_gemm", "grouped_mxfp8_dgrad"])
def test_row_products_refuse(lib, name, change, status):
    a = {**GEMM, **change}
    if name == "grouped_mxfp8_dgrad" and change.get("H") == 1 << 24:
        a["K"] = 1 << 24                 # its weights are [E * K, H] in these names
    assert getattr(lib, name)(*a.values()) == status
    assert lib.moeact_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), EINVAL), (dict(sx=None), EINVAL), (dict(dw=None), EINVAL), (dict(cb=None), EINVAL),
    (dict(ro=None), EINVAL), (dict(x=PTR + 4), EALIGN), (dict(dw=PTR + 4), EALIGN),
    (dict(cb=PTR + 4), EALIGN), (dict(H=48), EINVAL), (dict(K=0), EINVAL), (dict(rows=1), EINVAL),
    (dict(layout=3), EINVAL), (dict(layout=1), EINVAL), (dict(layout=1, M=128, rows=4, H=96), EINVAL),
    (dict(dt=0, acc=1), EINVAL), (dict(acc=2), EINVAL), (dict(dt=5), EINVAL), (dict(E=0), EINVAL),
    (dict(M=-2), EINVAL), (dict(M=1 << 31), ERANGE), (dict(E=2000, H=1 << 24, K=1 << 24), ERANGE),
])
def test_wgrad_refuses(lib, change, status):
    assert lib.grouped_mxfp8_wgrad(*{**WGRAD, **change}.values()) == status
    assert lib.moeact_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), EINVAL), (dict(N=0), EINVAL), (dict(N=40), EINVAL), (dict(codes=None), EINVAL),
    (dict(scales=None), EINVAL), (dict(codes=PTR + 8), EALIGN), (dict(layout=1), EINVAL),
    (dict(layout=7), EINVAL), (dict(M=(1 << 30) + 1), ERANGE), (dict(N=1 << 25), ERANGE),
    (dict(noop=PTR + 1), EALIGN),
])
def test_mxfp4_refuses(lib, change, status):
    assert lib.mxfp4_quantize(*{**Q4, **change}.values()) == status
    assert lib.mxfp4_dequantize(*{**D4, **change}.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(x=None), EINVAL), (dict(ldx=96), EINVAL), (dict(ldx=132), EALIGN), (dict(x=PTR + 2), EALIGN)])
def test_mxfp4_quantize_refuses(lib, change, status):
    assert lib.mxfp4_quantize(*{**Q4, **change}.values()) == status


def test_no_rows_need_no_codes(lib):
    """M == 0 returns before any CUDA call."""
    for name in ("grouped_mxfp8_gemm", "grouped_mxfp4_gemm", "grouped_mxfp8_dgrad"):
        assert getattr(lib, name)(*{**GEMM, "M": 0, "a": None, "sa": None, "out": None}.values()) == 0
    assert lib.mxfp4_quantize(*{**Q4, "M": 0, "x": None}.values()) == 0


def test_plain_quantizer_refuses(lib):
    mx = _capi.MxOut(PTR, PTR, PTR, PTR, 0, None)
    row = _capi.MxOut(PTR, PTR, None, None, 0, None)
    f = lib.mxfp8_quantize
    assert f(None, 128, 64, 128, 3, mx, None) == EINVAL
    assert f(PTR, 96, 64, 128, 3, mx, None) == EINVAL
    assert f(PTR, 132, 64, 128, 3, mx, None) == EALIGN
    assert f(PTR, 128, 64, 100, 3, mx, None) == EINVAL
    assert f(PTR, 128, 64, 128, 3, row, None) == EINVAL
    assert f(PTR, 128, 64, 128, 0, row, None) == EINVAL
    assert lib.grouped_mxfp8_quantize(PTR, 128, 64, 128, 3, None, PTR, 2, PTR, mx, None) == EINVAL


def test_python_refusals():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    ro = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        mg.mxfp8_quantize(torch.zeros(4, 32, dtype=torch.bfloat16))             # not on a GPU
    with pytest.raises(TypeError):
        mg.mxfp4_quantize(torch.zeros(4, 32))
    with pytest.raises(ValueError):
        mg.mxfp4_dequantize(mg.MXFP4(u8(4, 16), u8(4, 1)))
    for codes in (None, u8(4, 32)):
        with pytest.raises(ValueError):
            mg.grouped_mxfp8_gemm(mg.MXFP8(codes, None, u8(4, 1), None),
                                  mg.MXFP8(u8(64, 32), None, u8(64, 1), None), ro)
    with pytest.raises(ValueError):
        mg.grouped_mxfp8_wgrad(mg.MXFP8(None, None, None, None), mg.MXFP8(None, None, None, None),
                               ro, ro)
