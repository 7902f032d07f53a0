"""Empty sums whose outputs take more than 2^32 threads, one to an element
(dW, Y) or 64 to a scale's gradient: every element is written."""
import pytest
import torch

import gemm_rbq_encode_amd as rbq

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def dev():
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def all_zero(t):
    return not any(bool(p.any()) for p in t.view(-1).split(1 << 30))


# dW of 2^32 + 2^17 elements; 2^26 + 2^10 groups of 128
@pytest.mark.parametrize("out,inf,group", [((1 << 16) + 2, 1 << 16, 0), ((1 << 20) + 16, 1 << 13, 128)])
def test_gradients_of_no_tokens(out, inf, group):
    G = rbq.groups_per_row(inf, group)
    planes = torch.zeros(1, out, inf // 32, dtype=torch.int32, device=dev())
    scales = torch.ones(1, out, G, dtype=torch.float16, device=dev())
    dW = torch.full((out, inf), 3.0, device=dev())
    ds = torch.full((1, out, G), 3.0, device=dev())
    st = rbq.lib().rbq_qat_backward_ckpt(planes.data_ptr(), scales.data_ptr(), rbq.shape(out, inf, 1, group), None,
                                         None, None, 0, None, dW.data_ptr(), ds.data_ptr(), None, 0, None,
                                         torch.cuda.current_stream().cuda_stream)
    assert st == rbq.RBQ_OK
    torch.cuda.synchronize()
    assert all_zero(dW) and not ds.any()


def test_product_of_a_layer_without_columns():
    M, out = (1 << 16) + 2, 1 << 16
    Y = torch.full((M, out), 3.0, device=dev())
    rbq.gemm_f8(torch.empty(out, 0, dtype=torch.uint8, device=dev()).view(F8), torch.empty(out // 128, 0, device=dev()),
                torch.empty(M, 0, dtype=torch.uint8, device=dev()).view(F8), torch.empty(0, M, device=dev()),
                dtype=torch.float32, Y=Y)
    torch.cuda.synchronize()
    assert all_zero(Y)
