"""An MXFP4 product that becomes resident while a long kernel still runs waits for it as long as it
takes: the time limit of the product's pipeline waits (two seconds) does not count its predecessor."""
import ctypes
import os
import subprocess

import pytest
import torch

import q8_block_quantized_act_gb300 as q8
from gpu_util import device_ok, ensure_built
from q8_block_quantized_act_gb300 import build as q8build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
HOLD_NS = 2_600_000_000


@pytest.fixture(scope="module")
def hold(tmp_path_factory):
    ensure_built()
    so = str(tmp_path_factory.mktemp("hold") / "long_predecessor.so")
    subprocess.run([q8build._nvcc(), *q8build.ARCH, "-O2", "-shared", "-Xcompiler", "-fPIC", "-cudart", "static",
                    os.path.join(HERE, "long_predecessor.cu"), "-o", so], check=True)
    fn = ctypes.CDLL(so).long_predecessor
    fn.argtypes = [ctypes.c_longlong, ctypes.c_void_p]
    return fn


# one token quantized by the product's own CTAs, a k shared by clusters, two CTAs to an SM, pairs
@pytest.mark.parametrize("m,n,k", [(1, 640, 1024), (1, 33, 4096), (3, 20480, 512), (395, 5120, 2304)])
def test_product_outlasts_its_predecessor(hold, m, n, k):
    g = torch.Generator(device="cuda").manual_seed(m + n)
    w, wsc = q8.quantize_mxfp4(0.02 * torch.randn((n, k), generator=g, device="cuda"))
    x = torch.randn((m, k), generator=g, device="cuda")
    xq, xsc = q8.quantize_mxfp4(x)
    fused, apart = q8.gemm_mxfp4(w, wsc, x), q8.gemm_mxfp4_preq(w, wsc, xq, xsc)
    device_ok()
    out = torch.zeros_like(fused)
    for call, want in ((lambda: q8.gemm_mxfp4(w, wsc, x, out=out), fused),
                       (lambda: q8.gemm_mxfp4_preq(w, wsc, xq, xsc, out=out), apart)):
        out.zero_()
        assert hold(HOLD_NS, torch.cuda.current_stream().cuda_stream) == 0
        call()
        device_ok()                                       # no wait has given up
        assert torch.equal(out, want)
