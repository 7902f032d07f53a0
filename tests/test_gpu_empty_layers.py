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


@pytest.mark.parametrize("group", [0, 128])
def test_a_layer_without_columns_has_no_scale_gradients(group):
    """The fp16 backward and the one from a checkpoint alike: no groups, as the scales of such a layer."""
    K, out, M = 2, 40, 4
    planes = torch.zeros(K, out, 0, dtype=torch.int32, device=dev())
    scales = torch.ones(K, out, rbq.groups_per_row(0, group), dtype=torch.float16, device=dev())
    dY = torch.ones(M, out, dtype=torch.float16, device=dev())
    dX, dW, ds = rbq.qat_backward(planes, scales, torch.ones(M, 0, dtype=torch.float16, device=dev()), dY, group)
    torch.cuda.synchronize()
    assert dX.shape == (M, 0) and dW.shape == (out, 0) and ds.shape == scales.shape == backward(out, 0, K, group, M)[2].shape
