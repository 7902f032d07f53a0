"""Host-side checks of the 4-bit linears and the operators on logits: the oracles
against closed forms and torch's autograd, what the C ABI and the binding refuse
before anything is launched, and the sizes of the workspaces."""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
import workloads
from gemm_rbq_encode_amd import _binding
from oracle import logits, q4

pytestmark = pytest.mark.cpu
OK = 0x10000   # an aligned stand-in address: checks never dereference it
BAD, AL, UN = rbq.RBQ_ERR_INVALID_ARG, rbq.RBQ_ERR_ALIGNMENT, rbq.RBQ_ERR_UNSUPPORTED


# ---- the oracles ---------------------------------------------------------------

def test_q4_codes_are_within_half_a_step():
    W = workloads.gaussian_weight(40, 416, 3, outliers=True)
    for zeros in (False, True):
        codes, scales, points = q4.encode(W, zeros)
        s = np.repeat(scales.view(np.float16).astype(np.float64), 128, 1)[:, :416]
        err = np.abs(q4.values(codes, scales, points) - W)
        # half a step; the scale's rounding (2^-11 of up to 15 steps) can leave the ends outside the codes
        assert (err <= s * (0.5 + 15 * 2.0 ** -11 + (0.5 if zeros else 0))).all()
        assert codes.min() >= 0 and codes.max() <= 15
    assert np.array_equal(q4.unpack(q4.pack(codes)), codes)


def test_q4_of_planted_groups():
    """Codes, scale and zero point that a group was made from come back."""
    rng = np.random.default_rng(1)
    c = rng.integers(0, 16, (6, 128))
    c[:, 0], c[:, 1] = 0, 15
    z = np.array([0, 3, 8, 12, 15, 7])
    W = ((c - z[:, None]) * 0.25).astype(np.float32)
    codes, scales, points = q4.encode(W, True)
    assert np.array_equal(codes, c) and np.array_equal(points[:, 0], z)
    assert (scales.view(np.float16) == 0.25).all()
    sym = rng.integers(1, 16, (4, 128))
    sym[:, 5] = 15
    codes, scales, points = q4.encode(((sym - 8) * 0.5).astype(np.float32), False)
    assert np.array_equal(codes, sym) and (scales.view(np.float16) == 0.5).all() and (points == 8).all()
    codes, scales, points = q4.encode(np.zeros((1, 32), np.float32), True)
    assert (codes == 0).all() and scales.view(np.float16)[0, 0] == np.float16(2.0 ** -24)


def test_logits_oracle_against_autograd():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(4, 50)) * 3
    x[1, 7:20] = -np.inf
    targets = np.array([0, 49, -1, 30])
    a, b = rng.normal(size=4), rng.normal(size=4)
    T = 1.7
    xt = torch.from_numpy(x).requires_grad_()
    lp = torch.log_softmax(xt / T, 1)
    H = -(lp.exp() * torch.where(lp.exp() > 0, lp, 0.0)).sum(1)
    has = torch.from_numpy(targets >= 0)
    logp = torch.where(has, lp[torch.arange(4), torch.from_numpy(targets).clamp_min(0)], 0.0)
    r = logits.Rows(x, T)
    assert np.allclose(H.detach(), r.H) and np.allclose(np.where(r.p > 0, r.lp, 0), np.where(r.p > 0, lp.detach(), 0))
    (torch.from_numpy(a) * logp + torch.from_numpy(b) * H).sum().backward()
    g = logits.logprobs_grad(r, targets, a, b)
    assert np.allclose(np.nan_to_num(xt.grad.numpy()), g)


@pytest.mark.parametrize("tail", [False, True])
def test_distill_oracle_against_autograd(tail):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(5, 40)) * 2
    z = rng.normal(size=(5, 40)) * 2
    lp = z - np.log(np.exp(z).sum(1, keepdims=True))
    idx = np.argsort(-lp, 1)[:, :6]
    v = np.take_along_axis(lp, idx, 1)
    idx[0, 5], v[1, 2], idx[2, 1] = -1, -np.inf, idx[2, 0]
    T = 2.0
    if tail:
        v[2, 1] = v[2, 0] - 3
    xt = torch.from_numpy(x).requires_grad_()
    q = torch.softmax(xt / T, 1)
    total = 0.0
    for m in range(5):
        use = [j for j in range(6) if idx[m, j] >= 0 and v[m, j] > -np.inf]
        w = torch.tensor(v[m, use])
        p = w.exp() if tail else torch.softmax(w, 0)
        L = (p * (p.log() - q[m, idx[m, use]].log())).sum()
        if tail:
            others = [i for i in range(40) if i not in set(idx[m, use])]
            rest = 1 - p.sum()
            L = L + rest * (rest.log() - q[m, others].sum().log())
        total = total + L
        loss = logits.distill(logits.Rows(x[m:m + 1], T), idx[m:m + 1], v[m:m + 1], tail)[0]
        assert np.allclose(loss, L.item())
    total.backward()
    assert np.allclose(logits.distill(logits.Rows(x, T), idx, v, tail)[1], xt.grad.numpy())


def test_top_of_ties_and_masks():
    x = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0], [np.nan, 1, 2, 3, 4], [-np.inf] * 5])
    assert logits.top(x, 5).tolist() == [[1, 2, 4, 0, -1], [-1] * 5, [-1] * 5]


# ---- refusals -------------------------------------------------------------------

def each(call, args, changes, want):
    for k, v in changes:
        a = list(args)
        a[k] = v
        assert call(*a) == want, (k, v)


def test_q4_argument_errors():
    L = rbq.lib()
    enc = [OK, 8, 64, OK, OK, OK, None, None]
    each(L.rbq_encode_q4, enc, [(0, None), (3, None), (4, None), (1, -1), (2, 48), (2, -32)], BAD)
    each(L.rbq_encode_q4, enc, [(0, OK + 8), (3, OK + 4), (4, OK + 1), (6, OK + 2)], AL)
    each(L.rbq_encode_q4, enc, [(1, 2 ** 25 + 1), (2, 2 ** 25 + 32)], UN)
    assert L.rbq_encode_q4(OK, 2 ** 25, 2 ** 14, OK, OK, None, None, None) == UN       # 2^32 groups
    assert L.rbq_encode_q4(None, 0, 64, None, None, None, None, None) == rbq.RBQ_OK
    assert L.rbq_encode_q4(None, 8, 0, None, None, None, None, None) == rbq.RBQ_OK
    mul = [OK, OK, None, 8, 64, OK, 2, OK, 0, None, 0, None]
    each(L.rbq_gemm_q4, mul, [(0, None), (1, None), (5, None), (7, None), (3, -1), (4, 33), (6, -1), (8, 2), (10, 64)], BAD)
    each(L.rbq_gemm_q4, mul, [(0, OK + 8), (1, OK + 1), (5, OK + 8), (7, OK + 1), (9, OK + 8)], AL)
    each(L.rbq_gemm_q4, mul, [(3, 2 ** 25 + 1), (4, 2 ** 25 + 32)], UN)
    mul[8] = rbq.RBQ_Y_F32
    each(L.rbq_gemm_q4, mul, [(7, OK + 2)], AL)
    assert L.rbq_gemm_q4(None, None, None, 8, 64, None, 0, None, 0, None, 0, None) == rbq.RBQ_OK
    assert L.rbq_gemm_q4(None, None, None, 0, 64, None, 3, None, 0, None, 0, None) == rbq.RBQ_OK
    for a in ((-1, 64, 1, 0), (8, 33, 1, 0), (8, 64, 0, 0), (8, 64, 1, 2), (2 ** 25 + 1, 64, 9, 0)):
        assert L.rbq_gemm_q4_workspace_bytes(*a) == 0


ROW = [OK, 0, 4, 100, 100, 1.0]
ROW_BAD = [(0, None), (1, 3), (2, -1), (3, 0), (3, -5), (4, 99), (5, 0.0), (5, -1.0), (5, float("nan")), (5, float("inf")), (5, 0.9e-3), (5, 1.1e3)]


def test_logprobs_argument_errors():
    L = rbq.lib()
    a = ROW + [OK, OK, OK, 5, OK, OK, None, 0, None, None]
    each(L.rbq_token_logprobs, a, ROW_BAD + [(6, None), (9, -1), (10, None), (11, None), (13, 8)], BAD)
    each(L.rbq_token_logprobs, a, [(0, OK + 1), (6, OK + 4), (7, OK + 2), (8, OK + 2), (10, OK + 2), (11, OK + 2),
                                   (12, OK + 8), (14, OK + 2)], AL)
    each(L.rbq_token_logprobs, a, [(9, 129), (4, 2 ** 31 + 1)], UN)
    assert L.rbq_token_logprobs(OK, 0, 4, 2 ** 24 + 1, 2 ** 25, 1.0, *a[6:]) == UN
    assert L.rbq_token_logprobs(None, 0, 0, 100, 100, 1.0, None, None, None, 0, None, None, None, 0, None, None) == rbq.RBQ_OK
    # nothing asked for
    assert L.rbq_token_logprobs(OK, 0, 4, 100, 100, 1.0, None, None, None, 0, None, None, None, 0, None, None) == rbq.RBQ_OK
    g = ROW + [OK, OK, OK, OK + 0x100000, 100, OK, OK, None, 0, None, None]
    each(L.rbq_token_logprobs_backward, g, ROW_BAD + [(6, None), (9, None), (10, 99), (14, 8)], BAD)
    each(L.rbq_token_logprobs_backward, g, [(0, OK + 1), (6, OK + 4), (7, OK + 2), (8, OK + 2), (9, OK + 0x100001),
                                            (11, OK + 2), (12, OK + 2), (13, OK + 8), (15, OK + 2)], AL)
    assert L.rbq_token_logprobs_backward(*ROW, OK, None, None, OK + 0x100000, 100, None, None, None, 0, None, None) == BAD
    # the gradient half over the logits, or on them with another stride
    each(L.rbq_token_logprobs_backward, g, [(9, OK + 200), (9, OK + 700), (9, OK - 2)], BAD)
    assert L.rbq_token_logprobs_backward(*ROW, OK, OK, OK, OK, 101, OK, OK, None, 0, None, None) == BAD


def test_distill_argument_errors():
    L = rbq.lib()
    a = ROW + [OK, OK, 5, 1, OK, None, 0, None, None]
    each(L.rbq_distill_forward, a, ROW_BAD + [(6, None), (7, None), (8, -1), (9, 2), (10, None), (12, 8)], BAD)
    each(L.rbq_distill_forward, a, [(0, OK + 1), (6, OK + 2), (7, OK + 2), (10, OK + 2), (11, OK + 4), (13, OK + 1)], AL)
    each(L.rbq_distill_forward, a, [(8, 129)], UN)
    g = ROW + [OK, OK, 5, 1, OK, OK + 0x100000, 100, OK, None, 0, None, None]
    each(L.rbq_distill_backward, g, ROW_BAD + [(6, None), (7, None), (9, 4), (10, None), (11, None), (12, 50), (15, 8),
                                               (11, OK + 2)], BAD)
    each(L.rbq_distill_backward, g, [(10, OK + 2), (11, OK + 0x100001), (13, OK + 2), (14, OK + 8), (16, OK + 2)], AL)
    each(L.rbq_distill_backward, g, [(8, 129), (12, 2 ** 31 + 1)], UN)


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="only meaningful without a GPU")
def test_valid_calls_without_device():
    L = rbq.lib()
    assert L.rbq_encode_q4(OK, 8, 64, OK, OK, None, None, None) == rbq.RBQ_ERR_NO_DEVICE
    assert L.rbq_gemm_q4(OK, OK, None, 8, 64, OK, 2, OK, 0, None, 0, None) == rbq.RBQ_ERR_NO_DEVICE
    assert L.rbq_token_logprobs(*ROW, OK, OK, OK, 5, OK, OK, None, 0, None, None) == rbq.RBQ_ERR_NO_DEVICE
    assert L.rbq_distill_backward(*ROW, OK, OK, 5, 1, OK, OK, 100, OK, None, 0, None, None) == rbq.RBQ_ERR_NO_DEVICE


def test_binding_refusals():
    x = torch.zeros(4, 32)
    for call in (lambda: rbq.encode_q4(x), lambda: rbq.token_logprobs(x), lambda: rbq.token_logprobs_backward(x, None, None),
                 lambda: rbq.distill_forward(x, x, x), lambda: rbq.distill_backward(x, x, x, x),
                 lambda: rbq.gemm_q4(x, x, x)):
        with pytest.raises(TypeError, match="device tensor"):
            call()
    with pytest.raises(ValueError, match=r"x must be a tensor \[in\]"):
        rbq.gemv_q4(x, x, x)


def test_logits_workspaces():
    L = rbq.lib()
    for a in ((0, 100, 0), (-1, 100, 0), (4, 0, 0), (4, 2 ** 24 + 1, 0), (4, 100, 129), (4, 100, -1)):
        assert L.rbq_token_logprobs_workspace_bytes(*a) == 0 and L.rbq_distill_workspace_bytes(*a) == 0
    assert L.rbq_token_logprobs_workspace_bytes(4096, 128256, 128) == 0           # rows enough
    one = L.rbq_token_logprobs_workspace_bytes(1, 128256, 0)
    assert one > 0 and L.rbq_token_logprobs_workspace_bytes(1, 128256, 128) == one // 16 * (16 + 8 * 128)
    assert L.rbq_distill_workspace_bytes(1, 128256, 64) == one + 4 * 64
    assert _binding.RBQ_TOP_MAX == 128
