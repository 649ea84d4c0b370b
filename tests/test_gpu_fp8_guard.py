"""A library whose 8-bit product cannot run (its kernels were given fewer registers than their split among
warpgroups needs): the product says so, and everything else runs.

The library is linked from this one's objects and a copy of the product's source that asks for more registers than
any compiler gives; the kernels themselves stay as they are and are never launched."""
import ctypes
import os
import subprocess

import pytest
import torch

import linear_cross_entropy_chunked_gb300 as lce
from linear_cross_entropy_chunked_gb300 import build_lib

pytestmark = pytest.mark.gpu
OK, ERR_CUDA = 0, 6


@pytest.fixture(scope="module")
def crippled(tmp_path_factory):
    names = [os.path.splitext(s)[0] for s in build_lib.SOURCES]
    objects = {n: os.path.join(build_lib.BUILD_DIR, n + ".o") for n in names}
    if not all(map(os.path.exists, objects.values())):
        pytest.skip("the library's objects are not here")
    tmp = tmp_path_factory.mktemp("guard")
    with open(os.path.join(build_lib.CSRC, "lce_fp8.cu")) as f:
        source = f.read()
    needs = "constexpr int F8_REGS = 168,"
    assert needs in source
    src = tmp / "lce_fp8.cu"
    src.write_text(source.replace(needs, "constexpr int F8_REGS = 256,"))
    nvcc, so = build_lib._nvcc(), str(tmp / "liblce_guard.so")
    objects["lce_fp8"] = str(tmp / "lce_fp8.o")
    subprocess.run([nvcc, *build_lib.NVCC_FLAGS, "-I", build_lib.INCLUDE, "-I", build_lib.CSRC, "-c", str(src), "-o",
                    objects["lce_fp8"]], check=True, capture_output=True)
    subprocess.run([nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-o", so, *objects.values()],
                   check=True, capture_output=True)
    L, known = ctypes.CDLL(so), lce.lib()
    for name in ("lce_grad_norm", "lce_fp8_quantize", "lce_fp8_matmul", "lce_count_valid", "lce_sample_logits"):
        getattr(L, name).argtypes = getattr(known, name).argtypes
        getattr(L, name).restype = ctypes.c_int
    return L


def test_only_the_product_fails(crippled):
    L, s = crippled, torch.cuda.current_stream().cuda_stream
    x = torch.randn(300, 256, device="cuda")
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    norm = torch.zeros((), device="cuda")
    ptr, size, code = (ctypes.c_void_p * 1)(x.data_ptr()), (ctypes.c_int64 * 1)(x.numel()), (ctypes.c_int32 * 1)(1)
    assert L.lce_grad_norm(ptr, size, code, 1, 0, norm.data_ptr(), ws.data_ptr(), ws.numel(), s) == OK
    assert norm.item() == lce.grad_norm(x).item()
    tokens, u = torch.empty(300, dtype=torch.int64, device="cuda"), torch.rand(300, device="cuda")
    assert L.lce_sample_logits(x.data_ptr(), 1, 256, 300, 256, u.data_ptr(), None, None, None, None, 1.0, 0, 1.0, 0.0,
                               tokens.data_ptr(), None, s) == OK
    assert torch.equal(tokens, lce.sample_logits(x, u)[0])
    q = torch.empty(300, 256, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(2, 300, device="cuda")
    assert L.lce_fp8_quantize(x.data_ptr(), 1, 256, 300, 256, 0, q.data_ptr(), 256, scale.data_ptr(), None, 0, None, s) == OK
    out = torch.full((300, 304), 7.0, device="cuda")
    for _ in range(2):
        assert L.lce_fp8_matmul(q.data_ptr(), 256, scale.data_ptr(), 1, 300, q.data_ptr(), 256, scale.data_ptr(), 1, 300,
                                1, 300, 300, 256, out.data_ptr(), 304, 1, ws.data_ptr(), ws.numel(), s) == ERR_CUDA
    torch.cuda.synchronize()
    assert (out == 7).all()
    assert L.lce_grad_norm(ptr, size, code, 1, 0, norm.data_ptr(), ws.data_ptr(), ws.numel(), s) == OK
