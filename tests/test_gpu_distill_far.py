"""Distillation with the tail where the student's mass on the unnamed tokens is tiny: the
rest's share of the gradient is finite however small the sum it is divided by.  Bounds as
in tests/test_gpu_logits.py: an unnamed token's part carries the errors of its exponent
(3 D + 1 steps, D up to 90) and of the unnamed tokens' sum (n + 60 + 3 D), together less
than the doubled share with its 3 (n + 60) + 4 D that check_distill allows from n = 24 on."""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
from test_gpu_logits import check_distill, dev, t

pytestmark = pytest.mark.gpu
INF = float("inf")


def sharp(M, V, k, seed, T):
    """Logits whose named tokens lie 80 to 86 T above the others, some of those masked;
    the teacher leaves them 0.3."""
    rng = np.random.default_rng(seed)
    x = -rng.uniform(80.0, 84.0, (M, V)) * T
    x[rng.random((M, V)) < 0.3] = -np.inf
    idx = np.stack([rng.permutation(V)[:k] for _ in range(M)]).astype(np.int32)
    np.put_along_axis(x, idx.astype(np.int64), rng.uniform(0.0, 2.0, (M, k)) * T, 1)
    p = rng.random((M, k)) + 0.1
    return x, idx, np.log(0.7 * p / p.sum(1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("scale", [1.0, 256.0, 65536.0, 2.0 ** 100])
@pytest.mark.parametrize("M,V", [(6, 3001), (600, 3001), (6, 9001), (520, 12001), (6, 30011), (3, 60007)])
def test_the_rest_far_below(M, V, scale):
    for dtype, T in ((torch.float32, 1.0), (torch.float32, 1e-3), (torch.float16, 1.0), (torch.bfloat16, 2.0)):
        if dtype == torch.float16 and scale > 65536 or dtype != torch.float32 and M > 6:
            continue
        x, idx, v = sharp(M, V, 5, M + V, T)
        d = np.full(M, scale, np.float32)
        d[M // 2] = -scale
        dx, loss = check_distill(t(x, torch.float64).to(dtype), idx, v, d, T, True)
        assert torch.isfinite(dx).all() and torch.isfinite(loss).all() and not dx[torch.from_numpy(x == -INF)].any()


@pytest.mark.parametrize("V", [3001, 30011, 60007])
def test_one_unnamed_token_is_left(V):
    """All others masked: the rest's whole gradient is its own."""
    M = 4
    x, idx, v = sharp(M, V, 5, V, 1.0)
    one = np.array([(set(range(6)) - set(row.tolist())).pop() for row in idx])
    keep = np.zeros((M, V), bool)
    np.put_along_axis(keep, idx.astype(np.int64), True, 1)
    x[~keep] = -np.inf
    x[np.arange(M), one] = -np.array([60.0, 80.0, 84.0, 86.0])
    # q is 0 from 87 below the row's largest logit on: e^-87 is the last that fp32 holds, 2^-126 = e^-87.3
    near = x.max(1) - x[np.arange(M), one] < 87.0
    d = np.full(M, 65536.0, np.float32)
    dx, _ = check_distill(t(x[near], torch.float32), idx[near], v[near], d[near], 1.0, True)
    got = dx[torch.arange(int(near.sum()), device=dev()), t(one[near], torch.int64)].double().cpu().numpy()
    rest = 1 - np.exp(v[near].astype(np.float64)).sum(1)
    assert (np.abs(got + 65536 * rest) <= 65536 * rest * 2.0 ** -23 * 1200).all()     # (as above: n up to 64)
    args = [t(x, torch.float32), t(idx, torch.int32), t(v, torch.float32)]
    dx, loss = rbq.distill_backward(*args, t(d, torch.float32), tail=True)
    assert torch.isfinite(dx).all() and torch.isfinite(loss[t(near, torch.bool)]).all() and not torch.isnan(loss).any()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V", [3001, 30011, 60007])
def test_named_tokens_far_below(V, tail):
    """ln q of a token that the teacher names is finite where its e^x is not held."""
    M = 4
    rng = np.random.default_rng(V)
    x = rng.normal(size=(M, V))
    idx = np.stack([rng.permutation(V)[:5] for _ in range(M)]).astype(np.int32)
    x[np.arange(M), idx[:, 1]] = [-80.0, -100.0, -1000.0, -30000.0]
    v = np.full((M, 5), np.log(0.1), np.float32)
    dx, loss = check_distill(t(x, torch.float32), idx, v, np.full(M, 2.0, np.float32), 1.0, tail)
    assert torch.isfinite(dx).all() and torch.isfinite(loss).all()


def test_rows_without_slots_are_not_looked_at():
    """Without the tail nothing depends on their logits, NaN or not; with it their sums do."""
    x = torch.zeros((3, 700), device=dev())
    x[1, 3], x[2] = float("nan"), -INF
    idx, v = torch.full((3, 2), -1, dtype=torch.int32, device=dev()), torch.zeros((3, 2), device=dev())
    one = torch.ones(3, device=dev())
    dx, loss = rbq.distill_backward(x, idx, v, one)
    assert not dx.any() and not loss.any()
    dx, loss = rbq.distill_backward(x, idx, v, one, tail=True)
    assert torch.isnan(dx[1]).all() and torch.isnan(loss[1]) and loss[2] == INF and not dx[2].any()
