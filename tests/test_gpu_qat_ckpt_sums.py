"""Scale gradients of rbq_qat_backward_ckpt are 64-bit sums of the fp32 dW,
as those of rbq_qat_backward are, with the workspace and without.

The gradient of a scale is sum_j B[r][j] dW[r][j] over n columns of the dW
that the same call returns.  With the sum in 64 bits the only rounding that
counts is the last one:
  |err| <= 2^-24 |ds| + n 2^-52 sum_j |dW[r][j]|
Up to 192 tokens dW is computed in one slice of the tokens, so the dW summed
is the one returned.
"""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
from test_gpu_qat_ckpt import case, dev, t_f16, t_planes

pytestmark = pytest.mark.gpu


def signs(planes, inf):
    bits = (planes[..., None] >> np.arange(32, dtype=np.uint32)) & 1
    return bits.reshape(*planes.shape[:2], inf).astype(np.float64) * 2 - 1


SIZES = [(40, 96, 1, 0, 1), (256, 512, 2, 0, 5), (130, 1056, 3, 0, 64), (100, 128, 2, 0, 33), (70, 256, 4, 128, 20),
         (300, 416, 2, 0, 65), (384, 1024, 4, 128, 130), (513, 288, 1, 0, 190), (129, 128, 3, 128, 100),
         (2050, 2048, 2, 0, 128), (4096, 4096, 2, 0, 16), (260, 8192, 3, 128, 192)]


@pytest.mark.parametrize("out,inf,K,group,M", SIZES)
def test_scale_gradients_are_64_bit_sums(out, inf, K, group, M):
    planes, s, X, dY = case(out, inf, K, group, M, 3 * out + M)
    X = (X.view(np.float16) + np.float16(4.0)).view(np.uint16)     # sums that cancel: entries of dW of one size
    dY = (dY.view(np.float16) + np.float16(1.0)).view(np.uint16)
    a = (t_planes(planes), t_f16(s), *rbq.qat_checkpoint(t_f16(X)), t_f16(dY), group)
    n = group if group else inf
    for kwargs in ({}, {"workspace": torch.empty(0, dtype=torch.uint8, device=dev())}, {"need_dx": False}):
        _, dW, ds = rbq.qat_backward_ckpt(*a, **kwargs)
        torch.cuda.synchronize()
        w = dW.cpu().numpy().astype(np.float64)
        want = (signs(planes, inf) * w).reshape(K, out, inf // n, n).sum(3)
        tol = 2.0 ** -24 * np.abs(want) + n * 2.0 ** -52 * np.abs(w).reshape(out, inf // n, n).sum(2)
        err = np.abs(ds.cpu().numpy().astype(np.float64) - want)
        assert (err <= tol).all(), f"{(err / tol).max():.3g} of the bound"
