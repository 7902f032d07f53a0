"""Gradients written over the logits where rows take no part: rows of weight 0 whose
token is a real one, as prompts and padding are.  Everything that is returned has the
bits of the call whose gradient has a buffer of its own."""
import pytest
import torch

import gemm_rbq_encode_amd as rbq
from test_gpu_logits import TYPES, dev, rows, t, teacher

pytestmark = pytest.mark.gpu

# rows by workgroups of 128, 256 and 512 threads, held in LDS (many rows) and not, and cut rows
SIZES = [(40, 3001), (700, 3001), (40, 9001), (600, 12001), (40, 30011), (600, 33001), (3, 60007)]


def tokens(M, V):
    """Targets at a row's start, inside its first turn of a workgroup, in its middle and at its end."""
    places = torch.tensor([0, 7, 8, 513, V // 3, V // 2, V - 9, V - 1], device=dev())
    return places[torch.arange(M, device=dev()) % 8]


def same(ref, got):
    for a, b in zip(ref, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V", SIZES)
def test_rows_without_weight_keep_their_log_probabilities(M, V, dtype):
    x = rows(M, V, 3 * M + V, dtype, masked=False)
    if M > 3:
        x[3] = float("-inf")
    targets = tokens(M, V)
    at = torch.arange(M, device=dev())
    for a, b in [(torch.zeros(M, device=dev()), None), ((at % 2).float(), None), ((at % 3 == 0).float(), (at % 5 == 0).float()),
                 (torch.zeros(M, device=dev()), torch.zeros(M, device=dev()))]:
        ref = rbq.token_logprobs_backward(x, targets, a, b)
        y = x.clone()
        got = rbq.token_logprobs_backward(y, targets, a, b, d_logits=y)
        assert got[0] is y
        same(ref, got)
        none = a == 0 if b is None else (a == 0) & (b == 0)
        assert not y[none].any()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("M,V", SIZES)
def test_rows_without_weight_keep_their_divergence(M, V, tail):
    x = rows(M, V, 5 * M + V, torch.float16, masked=False)
    idx, v = teacher(M, V, 20, 4, 1.0)
    sl = [t(idx, torch.int32), t(v, torch.float32)]
    d = (torch.arange(M, device=dev()) % 2).float()
    ref = rbq.distill_backward(x, *sl, d, tail=tail)
    y = x.clone()
    same(ref, rbq.distill_backward(y, *sl, d, tail=tail, d_logits=y))
    assert not y[::2].any()
