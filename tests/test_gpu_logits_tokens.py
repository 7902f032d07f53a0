"""Token numbers beyond the vocabulary: reported whatever is asked of their rows, and
NaN exactly in what depends on them."""
import pytest
import torch

import gemm_rbq_encode_amd as rbq
from test_gpu_logits import dev, rows, t, teacher

pytestmark = pytest.mark.gpu
INF = float("inf")
SIZES = [(6, 3001), (600, 3001), (6, 30011), (6, 60001)]       # whole rows, and cut ones


def bad_targets(M, V):
    targets = torch.full((M,), 3, dtype=torch.int64, device=dev())
    targets[1], targets[2], targets[4] = V, 2 ** 40, 2 ** 31 + 3
    return targets


@pytest.mark.parametrize("M,V", SIZES)
def test_gradients_of_the_entropy_do_not_depend_on_tokens(M, V):
    x = rows(M, V, M + V, torch.float16, masked=False)
    targets, w = bad_targets(M, V), torch.rand(M, device=dev()) + 0.5
    ref, _, H = rbq.token_logprobs_backward(x, None, None, w)
    assert torch.isfinite(ref).all()
    a = torch.ones(M, device=dev())
    a[1] = a[2] = 0.0
    for d_logp in (None, torch.zeros(M, device=dev()), a):
        st = torch.zeros(1, dtype=torch.int32, device=dev())
        dx, logp, H2 = rbq.token_logprobs_backward(x, targets, d_logp, w, status=st)
        assert int(st.item()) == rbq.RBQ_STATUS_BAD_TOKEN
        assert torch.equal(H, H2) and torch.isnan(logp[[1, 2, 4]]).all() and torch.isfinite(logp[[0, 3, 5]]).all()
        assert torch.equal(dx[1:3], ref[1:3])
        if d_logp is a:
            assert torch.isnan(dx[4]).all() and torch.isfinite(dx[[0, 3, 5]]).all()
        else:
            assert torch.equal(dx, ref)


@pytest.mark.parametrize("M,V", SIZES)
def test_empty_rows_with_a_bad_token(M, V):
    """NaN as their log probabilities are; 0 without a weight."""
    x = rows(M, V, M + V, torch.float32, masked=False)
    x[1:4] = -INF
    targets = bad_targets(M, V)
    a = torch.ones(M, device=dev())
    a[2] = 0.0
    for w in (None, torch.ones(M, device=dev())):
        dx, logp, H = rbq.token_logprobs_backward(x, targets, a, w)
        assert torch.isnan(logp[1:3]).all() and logp[3] == -INF and not H[1:4].any()
        assert torch.isnan(dx[1]).all() and not dx[2:4].any()
    idx, v = teacher(M, V, 5, 4, 1.0)
    idx[1, 0] = idx[2, 0] = V
    for tail in (False, True):
        dx, loss = rbq.distill_backward(x, t(idx, torch.int32), t(v, torch.float32), a, tail=tail)
        assert torch.isnan(loss[1:3]).all() and loss[3] == INF
        assert torch.isnan(dx[1]).all() and not dx[2:4].any() and torch.isfinite(dx[0]).all()


@pytest.mark.parametrize("M,V", SIZES)
def test_slots_that_are_not_used_name_no_token(M, V):
    x = rows(M, V, M + V, torch.float16, masked=False)
    idx, v = teacher(M, V, 6, 4, 1.0)
    v[:, 4] = -INF
    bad = idx.copy()
    bad[::2, 4] = 2 ** 31 - 1
    d = torch.ones(M, device=dev())
    for tail in (False, True):
        ref = rbq.distill_backward(x, t(idx, torch.int32), t(v, torch.float32), d, tail=tail)
        st = torch.zeros(1, dtype=torch.int32, device=dev())
        got = rbq.distill_backward(x, t(bad, torch.int32), t(v, torch.float32), d, tail=tail, status=st)
        assert all(torch.equal(p, q) for p, q in zip(ref, got)) and torch.isfinite(got[0]).all()
        assert int(st.item()) == rbq.RBQ_STATUS_BAD_TOKEN
        assert torch.equal(ref[1], rbq.distill_forward(x, t(bad, torch.int32), t(v, torch.float32), tail=tail))


@pytest.mark.parametrize("M,V", SIZES)
def test_tokens_are_reported_where_no_log_probability_is_asked_for(M, V):
    """The C calls with logp NULL, rows without weight among them."""
    x = rows(M, V, M + V, torch.float16, masked=False)
    dx = torch.empty_like(x)
    H, zero, one = torch.empty(M, device=dev()), torch.zeros(M, device=dev()), torch.ones(M, device=dev())
    L, none = rbq.lib(), torch.full((M,), -1, dtype=torch.int64, device=dev())
    need = int(L.rbq_token_logprobs_workspace_bytes(M, V, 0))
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev())
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    for targets, want in ((bad_targets(M, V), rbq.RBQ_STATUS_BAD_TOKEN), (none, 0)):
        for n in (0, need):
            row = [x.data_ptr(), rbq.RBQ_L_F16, M, V, V, 1.0, targets.data_ptr()]
            room = [ws.data_ptr(), n]
            for call, more in ((L.rbq_token_logprobs, [None, H.data_ptr(), 0, None, None]),
                               (L.rbq_token_logprobs_backward, [zero.data_ptr(), None, dx.data_ptr(), V, None, None]),
                               (L.rbq_token_logprobs_backward, [zero.data_ptr(), zero.data_ptr(), dx.data_ptr(), V, None, None]),
                               (L.rbq_token_logprobs_backward, [None, one.data_ptr(), dx.data_ptr(), V, None, H.data_ptr()])):
                st = torch.zeros(1, dtype=torch.int32, device=dev())
                assert call(*row, *more, *room, st.data_ptr(), stream) == rbq.RBQ_OK
                assert int(st.item()) == want
