"""Which places of a gradient beside its logits are refused: those whose rows overlap,
and no others of the same stride."""
import pytest
import torch

import gemm_rbq_encode_amd as rbq

pytestmark = [pytest.mark.cpu, pytest.mark.skipif(torch.cuda.device_count() > 0, reason="stand-in addresses: only without a GPU")]
BASE = 0x1000000     # a stand-in address: checks never dereference it


def calls(kind, M, vocab, stride, at, d_stride):
    """Both gradients' answers for a gradient `at` entries from the logits."""
    L = rbq.lib()
    size = 4 if kind == rbq.RBQ_L_F32 else 2
    row = [BASE, kind, M, vocab, stride, 1.0]
    place = [BASE + at * size, d_stride]
    return {L.rbq_token_logprobs_backward(*row, BASE, BASE, None, *place, None, None, None, 0, None, None),
            L.rbq_distill_backward(*row, BASE, BASE, 5, 1, BASE, *place, None, None, 0, None, None)}


@pytest.mark.parametrize("kind", [rbq.RBQ_L_F16, rbq.RBQ_L_F32, rbq.RBQ_L_BF16])
@pytest.mark.parametrize("M,vocab,stride", [(4, 5, 5), (4, 5, 9), (4, 5, 10), (4, 5, 13), (1, 5, 5), (2, 1, 2), (3, 7, 40)])
def test_equal_strides(M, vocab, stride, kind):
    mine = {m * stride + v for m in range(M) for v in range(vocab)}
    for at in range(-M * stride - 3, M * stride + 4):
        overlap = bool(mine & {at + e for e in mine}) and at != 0
        want = rbq.RBQ_ERR_INVALID_ARG if overlap else rbq.RBQ_ERR_NO_DEVICE
        assert calls(kind, M, vocab, stride, at, stride) == {want}, at


def test_other_strides():
    for at in range(-60, 60):
        # logits of 4 rows entries 0 to 34, a gradient of 4 rows, entries at to at + 40
        want = rbq.RBQ_ERR_INVALID_ARG if -40 <= at <= 34 else rbq.RBQ_ERR_NO_DEVICE
        assert calls(rbq.RBQ_L_F16, 4, 5, 10, at, 12) == {want}, at
