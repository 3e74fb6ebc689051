"""The waits of the dense layer's product run out without a GPU fault: its barriers count bytes
that no copy brings, the kernel gives up, leaves its code and ends, and the next call is right."""
import ctypes as ct
import os
import subprocess

import pytest
import torch

import layers_ref as L

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "momentum_compression_gb300", "csrc")


@pytest.fixture(scope="module")
def product(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("gemm") / "libgemm.so")
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17", "-fmad=false",
                    "-shared", "-Xcompiler", "-fPIC", f"-I{CSRC}", f"-I{ROOT}/include", "-o", out,
                    os.path.join(HERE, "cuda", "gemm_selftest.cu"), os.path.join(CSRC, "k_few.cu"),
                    os.path.join(CSRC, "attn_map.cu")], check=True)
    lib = ct.CDLL(out)
    ll = ct.c_longlong
    lib.gemm_selftest.argtypes = [ct.c_void_p] * 4 + [ll, ll, ll, ct.c_int, ct.c_uint, ct.POINTER(ct.c_uint)]

    def call(x, w, r, y, pairs, lost):
        code = ct.c_uint(99)
        assert lib.gemm_selftest(x.data_ptr(), w.data_ptr(), r.data_ptr(), y.data_ptr(), x.shape[0], w.shape[0],
                                 x.shape[1], pairs, lost, ct.byref(code)) == 0
        return code.value
    return call


@pytest.mark.parametrize("pairs,K", [(0, 64), (1, 64), (0, 768)])
def test_a_product_whose_copies_never_land_gives_up(product, pairs, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    x, w, r = mk(300, K), mk(264, K), mk(300, 264)
    (_, want), (_, err) = L.dense(x, w, None, r, "none")
    for lost in (0, 16, 0):
        y = torch.zeros_like(r)
        code = product(x, w, r, y, pairs, lost)
        if lost:
            assert code in (1, 2)  # the copies' consumer, or who waits for a free stage
        else:
            assert code == 0
            L.within(y, want, err, "y")
