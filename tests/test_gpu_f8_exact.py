"""Exact products with fp16 outputs (RBQ_Y_EXACT): the same sums as with fp32
outputs, rounded once, so equal bits to the fp32 result rounded to fp16; and
within the bounds of test_gpu_f8.py without the 8-bit instruction's cut."""
import pytest
import torch

import gemm_rbq_encode_amd as rbq
from test_gpu_f8 import dev, layer, t_f32, t_f8
from test_gpu_f8_kernels import bound, definition, release  # noqa: F401

pytestmark = pytest.mark.gpu

# the kinds of tiles of exact products, whole, cut and in part cut, and few tokens
SIZES = [(8937, 2848, 129), (34293, 672, 139), (17951, 320, 131), (2851, 2208, 33), (33157, 672, 39), (19935, 288, 33),
         (16681, 4064, 67), (3, 960, 35), (1001, 672, 301), (5003, 4128, 777), (8191, 288, 2047), (300, 416, 32),
         (12301, 160, 5)]


@pytest.mark.parametrize("out,inf,M", SIZES)
def test_exact_fp16_outputs_are_the_fp32_ones_rounded(out, inf, M):
    a = layer(out, inf, M, out + M + inf)
    a = (t_f8(a[0]), t_f32(a[1]), t_f8(a[2]), t_f32(a[3]))
    buf = torch.full((M * out + 4096,), float("nan"), dtype=torch.float16, device=dev())
    Y = buf[:M * out].view(M, out)
    assert rbq.gemm_f8(*a, exact=True, Y=Y) is Y
    wide = rbq.gemm_f8(*a, dtype=torch.float32)
    same = rbq.gemm_f8(*a, dtype=torch.float32, exact=True)
    none = torch.empty(0, dtype=torch.uint8, device=dev())
    Y1, wide1 = rbq.gemm_f8(*a, exact=True, workspace=none), rbq.gemm_f8(*a, dtype=torch.float32, workspace=none)
    torch.cuda.synchronize()
    assert torch.equal(Y, wide.half()) and torch.equal(wide, same) and torch.equal(Y1, wide1.half())
    assert bool(torch.isnan(buf[M * out:]).all())
    y, S, _ = definition(*a, False)
    assert bool(((Y.double() - y).abs() <= bound(S, y, inf, True, 0.0)).all())


def test_exact_products_keep_what_the_8_bit_instruction_cuts():
    """One product of +-448^2 beside seven of 2^-4 in every 8 columns: the small
    ones are below the cut, and all that is left once the large ones cancel.
    (Four large ones of one sign at most are added before the others: every
    partial sum is a multiple of 2^-4 below 2^20, so fp32 holds it.)"""
    out, inf, M = 256, 512, 64
    w8 = torch.full((out, inf), 0x28, dtype=torch.uint8, device=dev())     # 2^-2
    x8 = torch.full((M, inf), 0x28, dtype=torch.uint8, device=dev())
    w8[:, ::8] = 0x7E                                                       # 448
    x8[:, ::16], x8[:, 8::16] = 0x7E, 0xFE                                  # 448, -448: the large products cancel
    F8 = torch.float8_e4m3fn
    a = (w8.view(F8), torch.full((2, 4), 0.25, device=dev()), x8.view(F8), torch.ones(4, M, device=dev()))
    want = torch.full((M, out), inf // 8 * 7 * 2.0 ** -4 * 0.25, device=dev())
    exact = rbq.gemm_f8(*a, exact=True)
    torch.cuda.synchronize()
    assert torch.equal(exact.float(), want)
