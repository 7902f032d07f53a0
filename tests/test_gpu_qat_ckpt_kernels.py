"""Every kernel that rbq_qat_backward_ckpt can choose (by tokens, planes, tile,
slices, and whether dX, dW or both are asked for), at ragged sizes, within the
bounds of test_gpu_qat_ckpt.py.  test_f8_plans_cpu.py checks that the sizes here
and in the other tests reach every kernel."""
import pytest
import torch

import gemm_rbq_encode_amd as rbq
from oracle import f8
from test_gpu_qat_ckpt import case, check_grads, dev, t_f16, t_planes

pytestmark = pytest.mark.gpu

# (tokens, out, in, planes, group, asked for: 1 dX, 2 dW and the scales' gradients, 3 both)
KERNELS = [(75, 115, 192, 3, 0, 3), (71, 1133, 160, 3, 0, 3), (67, 79, 160, 4, 0, 3), (67, 79, 256, 4, 128, 3),
           (177, 73, 224, 1, 0, 3), (429, 75, 160, 1, 0, 3), (323, 1139, 160, 1, 0, 3), (335, 1017, 160, 2, 0, 3),
           (335, 1017, 128, 2, 128, 3), (367, 81, 160, 3, 0, 3), (159, 597, 192, 3, 0, 3), (501, 569, 160, 3, 0, 3),
           (501, 569, 256, 3, 128, 3), (347, 673, 160, 4, 0, 3),
           (67, 2313, 3552, 3, 0, 2), (67, 2313, 3584, 4, 128, 2), (3549, 11061, 160, 4, 0, 2),
           (65, 327, 192, 1, 0, 1), (73, 79, 160, 2, 0, 1), (71, 77, 192, 3, 0, 1), (87, 329, 160, 3, 0, 1),
           (65, 99, 192, 4, 0, 1), (73, 453, 160, 4, 0, 1), (73, 453, 256, 4, 128, 1), (191, 327, 160, 1, 0, 1),
           (131, 91, 160, 2, 0, 1), (155, 97, 160, 3, 0, 1), (129, 109, 192, 4, 0, 1),
           (1, 79, 160, 4, 0, 1), (7, 79, 160, 4, 0, 3), (16, 1000, 256, 4, 128, 3), (17, 87, 192, 1, 0, 1),
           (31, 300, 96, 1, 0, 3), (19, 75, 160, 2, 0, 3), (17, 103, 160, 4, 0, 1), (29, 600, 384, 4, 128, 3),
           (33, 79, 160, 1, 0, 2), (61, 500, 288, 1, 0, 3), (37, 71, 160, 2, 0, 3), (64, 700, 256, 2, 128, 3)]


@pytest.mark.parametrize("M,out,inf,K,group,ask", KERNELS)
def test_backward_kernels(M, out, inf, K, group, ask):
    planes, s, X, dY = case(out, inf, K, group, M, out + 7 * M)
    a = (t_planes(planes), t_f16(s), *rbq.qat_checkpoint(t_f16(X)), t_f16(dY), group)
    x = f8.restore(*f8.checkpoint(X))
    need = dict(need_dx=bool(ask & 1), need_dw=bool(ask & 2), need_dscales=bool(ask & 2))
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=dev())):
        got = rbq.qat_backward_ckpt(*a, **need, workspace=ws, status=st)
        again = rbq.qat_backward_ckpt(*a, **need, workspace=ws)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        assert all((u is None and v is None) or torch.equal(u, v) for u, v in zip(got, again))
        check_grads(got, planes, s, x, dY, group)
