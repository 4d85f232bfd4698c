"""Calls of the layer's operators at the edges of their range that `test_gpu_layer.py` does not make:
shares of a split sum, tile widths, tails of the activations, infinities, calls from several
threads.  Tolerances as there.
"""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import gated_delta_rule_deltanet_gb300 as kda
from gated_delta_rule_deltanet_gb300 import _lib, build as kbuild
from oracle import layer as ol
from test_gpu_layer import DEV, U, check, dev, host, no_error, product_tol, rng

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [3, 8, 9, 16, 17, 64])
@pytest.mark.parametrize("K,N", [(4096, 512), (1024, 256)])
@pytest.mark.parametrize("dtype,y", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_split_sums_of_few_rows_back_to_back(T, K, N, dtype, y):
    """Few rows give only some CTAs of a cluster columns to finish, and the others end once their
    shares have arrived.  Launched back to back with kernels that take over their shared memory
    at once, every call gives the same bits, and the fp64 sum."""
    r = rng(30, T, K)
    x, x64 = dev(r.standard_normal((T, K)), dtype)
    w, w64 = dev(r.standard_normal((N, K)) / np.sqrt(K), dtype)
    other, _ = dev(r.standard_normal((T + 5, K)), dtype)
    yt = torch.float32 if y == "f32" else torch.bfloat16
    outs = []
    for _ in range(40):
        outs.append(kda.linear(x, w, out_dtype=yt))
        kda.linear(other, w, out_dtype=yt)
    no_error()
    check("y", outs[0], x64 @ w64.T, product_tol(x64, w64.T, K, dtype))
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.fixture(scope="module")
def giving_up(tmp_path_factory):
    """The row kernels with waits that give up at once."""
    lib = str(tmp_path_factory.mktemp("ring") / "libring.so")
    subprocess.run([kbuild.nvcc(), *kbuild.ARCH, *kbuild.NVCC_FLAGS, "-DKDA_ROW_WAIT=0", "-shared", "-o", lib,
                    os.path.join(os.path.dirname(__file__), "ring_gives_up.cu")], check=True)
    f = ctypes.CDLL(lib).ring_gives_up
    f.argtypes = [ctypes.POINTER(_lib.KdaNormParams), ctypes.c_int] + [ctypes.c_void_p] * 10
    return f


@pytest.mark.parametrize("T,N,backward", [(15000, 96, 0), (15000, 96, 1), (5000, 2048, 0), (5000, 2048, 1),
                                          (3000, 4096, 0), (3000, 4096, 1), (1000, 16384, 1)])
def test_rows_whose_wait_gives_up_end_with_their_copies(giving_up, T, N, backward):
    """A wait that gives up is an error in the device word; the block ends only after the copies it
    asked for, so that a kernel behind it finds its own shared memory untouched."""
    r = rng(31, T, N)
    x, _ = dev(r.standard_normal((T, N)), "bf16")
    w, _ = dev(r.standard_normal(N), "f32")
    want = kda.residual_norm(x, w, residual=x) + kda.residual_norm_bwd(x, x, w, x, x)[:3]
    p = _lib.KdaNormParams(tokens=T, features=N, x_dtype=1, h_dtype=1, y_dtype=1, eps=1e-6, scale=1.0)
    n = ctypes.c_size_t(0)
    assert _lib.load().kda_norm_workspace_size(ctypes.byref(p), 0, ctypes.byref(n)) == 0
    ws = torch.empty(n.value, dtype=torch.uint8, device=DEV)
    dx, dh, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(5):
        assert giving_up(ctypes.byref(p), backward, x.data_ptr(), x.data_ptr(), w.data_ptr(), x.data_ptr(),
                         dx.data_ptr(), dh.data_ptr(), dw.data_ptr(), ws.data_ptr(), word.data_ptr(),
                         torch.cuda.current_stream().cuda_stream) == 0
        got = kda.residual_norm(x, w, residual=x) + kda.residual_norm_bwd(x, x, w, x, x)[:3]
        no_error()
        assert word.item() == _lib.KDA_DEVERR_TIMEOUT
        for a, b in zip(got, want):
            assert torch.equal(a, b)
