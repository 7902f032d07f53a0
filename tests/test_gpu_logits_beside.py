"""Gradients beside their logits, as columns of one wider tensor: the bits of a gradient
in a tensor of its own, and logits that stay as they were."""
import pytest
import torch

import gemm_rbq_encode_amd as rbq
from test_gpu_logits import TYPES, dev, rows, t, teacher

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V", [(5, 777), (1030, 3001), (7, 30011), (5, 60001)])
def test_columns_of_one_tensor(M, V, dtype):
    x = rows(M, V, M + V, dtype, masked=False)
    targets = torch.randint(0, V, (M,), device=dev())
    d = torch.rand(M, device=dev()) + 0.5
    idx, v = teacher(M, V, 5, 4, 1.0)
    sl = [t(idx, torch.int32), t(v, torch.float32)]
    wide = torch.full((M, 2 * V + 7), 7.0, dtype=dtype, device=dev())
    for left in (True, False):
        a, b = wide[:, 3:3 + V], wide[:, V + 3:2 * V + 3]
        mine, other = (a, b) if left else (b, a)
        mine.copy_(x)
        for ref, call in ((rbq.token_logprobs_backward(x, targets, d, d), lambda: rbq.token_logprobs_backward(mine, targets, d, d, d_logits=other)),
                          (rbq.distill_backward(x, *sl, d, tail=True), lambda: rbq.distill_backward(mine, *sl, d, tail=True, d_logits=other))):
            other.fill_(7.0)
            got = call()
            assert all(torch.equal(p, q) for p, q in zip(ref, got)) and torch.equal(mine, x)
            assert bool((wide[:, :3] == 7).all()) and bool((wide[:, 2 * V + 3:] == 7).all())
    with pytest.raises(rbq.RbqError):
        rbq.token_logprobs_backward(wide[:, :V], targets, d, d_logits=wide[:, V - 1:2 * V - 1])
