"""Calls of the layer's operators at the edges of their range that `test_gpu_layer.py` does not make:
shares of a split sum, tile widths, tails of the activations, infinities, calls from several
threads.  Tolerances as there.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_deltanet_gb300 as kda
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
