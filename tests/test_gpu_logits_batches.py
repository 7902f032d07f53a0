"""Batches whose rows are held in LDS in part and walked many times around, and more
rows than one launch takes.  Bounds as in tests/test_gpu_logits.py."""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
from oracle import logits as oracle
from test_gpu_logits import TYPES, U, Bound, dev, half, near, np64, rows, t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,V", [(520, 50021), (515, 36863), (514, 12801)])
@pytest.mark.parametrize("dtype", TYPES)
def test_long_held_rows(M, V, dtype):
    """512 rows and more: the last turns of a walk from LDS, the others read again, four at a time and singly."""
    x = rows(M, V, M + V, dtype)
    rng = np.random.default_rng(V)
    targets = rng.integers(0, V, M)
    a, w = rng.normal(size=M).astype(np.float32), rng.normal(size=M).astype(np.float32)
    some = [0, 1, 255, 256, M - 2, M - 1]
    T = 0.7
    r = oracle.Rows(np64(x[some]), T)
    b = Bound(r, V)
    m = np.arange(len(some))
    lp = np.where(r.p > 0, np.abs(r.lp), 0.0)
    for both in (False, True):
        args = (t(targets, torch.int64), t(a, torch.float32), t(w, torch.float32) if both else None)
        dx, logp, H = rbq.token_logprobs_backward(x, *args, temperature=T)
        ww = w[some].astype(np.float64) if both else np.zeros(len(some))
        g = oracle.logprobs_grad(r, targets[some], a[some].astype(np.float64), ww)
        aa, wide = np.abs(a[some])[:, None], np.abs(ww)[:, None] * r.p
        tol = (aa * r.p * (b.rel + 4 * U) + aa * 4 * U * (g != 0)
               + wide * ((lp + r.H[:, None]) * (b.rel + 8 * U) + b.lp + b.H[:, None])) / T
        near(dx[some], g, tol + half(dtype, np.abs(g) + tol), f"gradient, both {both}")
        near(H[some], r.H, b.H, "entropy")
        near(logp[some], r.lp[m, targets[some]], b.lp[m, targets[some]], "logp")
        y = x.clone()
        got = rbq.token_logprobs_backward(y, *args, temperature=T, d_logits=y)
        assert torch.equal(got[0], dx) and torch.equal(got[1], logp) and torch.equal(got[2], H)


def test_more_rows_than_a_launch_takes():
    """2^22 workgroups a launch: the rows behind them are those of the rows alone."""
    M, V = 2 ** 22 + 37, 5
    x = torch.randn((M, V), device=dev(), generator=torch.Generator(dev()).manual_seed(1)).half()
    targets = torch.arange(M, device=dev()) % V
    end = slice(M - 70, M)
    a = torch.rand(M, device=dev()) + 0.5
    for got, ref in zip(rbq.token_logprobs(x, targets, top=3), rbq.token_logprobs(x[end], targets[end], top=3)):
        assert torch.equal(got[end], ref)
    for got, ref in zip(rbq.token_logprobs_backward(x, targets, a, a),
                        rbq.token_logprobs_backward(x[end], targets[end], a[end], a[end])):
        assert torch.equal(got[end], ref)
    *_, v, idx = rbq.token_logprobs(x * 0.5, top=2)
    for got, ref in zip(rbq.distill_backward(x, idx, v, a, tail=True),
                        rbq.distill_backward(x[end], idx[end], v[end], a[end], tail=True)):
        assert torch.equal(got[end], ref)
    assert torch.equal(rbq.distill_forward(x, idx, v, tail=True)[end], rbq.distill_forward(x[end], idx[end], v[end], tail=True))
