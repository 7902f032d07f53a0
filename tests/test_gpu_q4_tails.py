"""Products in 4 bits whose last group is short: what stands in the group before it, an
infinite token entry among them, counts once, in its own group."""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
import workloads
from test_gpu_q4 import dev, layer, t_of, to_gpu
from test_gpu_q4_kernels import near, weights

pytestmark = pytest.mark.gpu


# few-token kernels, tiled ones, ragged rows and tokens of 1 to 16 and more, one group and several
@pytest.mark.parametrize("M,out,inf", [(3, 70, 416), (16, 4200, 160), (1500, 3301, 416), (1601, 4097, 352), (1219, 4111, 416),
                                       (8200, 8001, 32), (5003, 4301, 96), (4163, 2063, 288)])
def test_infinite_entries_before_a_short_group(M, out, inf):
    codes, scales, points = layer(out, inf, M, True)
    scales[0, 0] = scales[-1, -1] = np.float16(0.01).view(np.uint16)
    g = to_gpu(codes, scales, points, True)
    w = weights(codes, scales, points)
    x = t_of(workloads.gaussian_activations(M, inf, seed=M), np.float16)
    last = max(inf - 128, 0)                        # first of the row's last 128 columns
    at = sorted({0, last, max((inf - 1) // 128 * 128 - 1, 0), inf - 1})
    tokens = [0, M // 2, M - 2, M - 1][:len(at)]
    y = x.clone()
    for m, j in zip(tokens, at):
        y[m, j] = float("inf")
    Y = rbq.gemm_q4(g[0], g[1], y, g[2], dtype=torch.float32)
    for m in set(tokens):
        # (0 of an infinite entry, or two of different signs: NaN)
        want = (w[:, [j for n, j in zip(tokens, at) if n == m]] * float("inf")).sum(1)
        assert torch.equal(torch.isnan(Y[m]), torch.isnan(want)) and torch.isinf(want).any()
        assert torch.equal(torch.where(torch.isnan(want), 0.0, Y[m].double()), torch.where(torch.isnan(want), 0.0, want))
    keep = torch.ones(M, dtype=torch.bool, device=dev())
    keep[tokens] = False
    near(Y[keep], w, x[keep])
    for dtype in (torch.float16, torch.float32):
        near(rbq.gemm_q4(g[0], g[1], x, g[2], dtype=dtype), w, x, str(dtype))
