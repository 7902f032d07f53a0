"""Empty sums of the calls on checkpoints: no rows, no columns, no tokens."""
import pytest
import torch

import gemm_rbq_encode_amd as rbq

pytestmark = pytest.mark.gpu


def dev():
    return torch.device("cuda:0")


def backward(out, inf, K, group, M):
    G = rbq.groups_per_row(inf, group)
    return rbq.qat_backward_ckpt(torch.zeros(K, out, inf // 32, dtype=torch.int32, device=dev()),
                                 torch.ones(K, out, G, dtype=torch.float16, device=dev()),
                                 *rbq.qat_checkpoint(torch.ones(M, inf, dtype=torch.float16, device=dev())),
                                 torch.ones(M, out, dtype=torch.float16, device=dev()), group)


@pytest.mark.parametrize("out,inf,M", [(0, 128, 4), (0, 128, 300), (40, 0, 4), (0, 0, 4), (40, 128, 0), (0, 128, 0)])
@pytest.mark.parametrize("group", [0, 128])
def test_backward_of_empty_layers(out, inf, M, group):
    K = 2
    dX, dW, ds = backward(out, inf, K, group, M)
    torch.cuda.synchronize()
    assert dX.shape == (M, inf) and dW.shape == (out, inf) and ds.shape == (K, out, rbq.groups_per_row(inf, group))
    assert not dX.any() and not dW.any() and not ds.any()
