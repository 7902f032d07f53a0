"""GPU parity of token_logprobs, distill_forward and their gradients against
oracle/logits.py (float64).

The bounds.  u = 2^-23 (an operation rounds by at most half of it; the hardware's
exp2 and log2 by up to a whole one).  An exponent (x - m) c meets three roundings
of its size, and m lies at most 4 ln 2 / 1 (in nats) from the row's maximum, so
with D = distance to the maximum + 3 a term of the sum is off by (3 D + 1) u, and a
sum of n terms by n u more.  Where a thread adds n = 8 ceil(V / (8 threads)) terms (128
threads at least on up to 1200 vectors of 8, 256 on up to 12000, else 512; a cut row
has fewer), its wave 6, the workgroup 8 and the slices up to 10 joinings (two
roundings each):
  dS    = u (n + 60 + 3 (mean D))               relative, of a row's sum
  logp  : dS + u (4 D_target + 4 |logp| + 4 ln S + 4)
  H     : (mean D + 2)(dS) + u (4 mean D^2 + 4 mean D + 8 ln S + 8)
  p_v   : relative dS + u (4 D_v + 8)
and the gradients' parts carry the errors of p, ln p and H they are made of, and
one rounding to their type.
"""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
from oracle import logits as oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -23
TYPES = [torch.float16, torch.bfloat16, torch.float32]


def dev():
    return torch.device("cuda:0")


def t(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(dev())


def np64(x):
    return x.detach().cpu().double().numpy()


def rows(M, V, seed, dtype, masked=True, scale=3.0):
    """Normal logits with likely tokens and masked entries, rounded to the type."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(M, V)) * scale
    x[rng.random((M, V)) < 0.02] += 8
    if masked and V > 4:
        x[rng.random((M, V)) < 0.05] = -np.inf
    return t(x, torch.float64).to(dtype)


class Bound:
    def __init__(self, r, V):
        n = 8 * -(-V // (8 * (128 if V <= 9600 else 256 if V <= 96000 else 512)))
        self.D = r.far + 3.0
        mean, square = r.mean + 3.0, r.square + 6 * r.mean + 9.0
        self.dS = U * (n + 60 + 3 * mean)
        self.H = (mean + 2) * self.dS + U * (4 * square + 4 * mean + 8 * r.logS + 8)
        self.lp = self.dS[:, None] + U * (4 * self.D + 4 * np.where(np.isfinite(r.lp), -r.lp, 0) + 4 * r.logS[:, None] + 4)
        self.rel = self.dS[:, None] + U * (4 * self.D + 8)


def near(got, want, tol, what):
    got = np64(got) if isinstance(got, torch.Tensor) else got
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    err = np.where(same, 0.0, np.abs(got - want))
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}, " \
                          f"allowed {np.broadcast_to(tol, got.shape)[bad][0]}"


def half(dtype, v):
    """One rounding to the type, and half of its smallest step."""
    return torch.finfo(dtype).eps / 2 * np.abs(v) + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134)


SHAPES = [(1, 1), (3, 2), (2, 7), (1, 8), (5, 9), (2, 513), (4, 4099), (1, 32000), (2, 50257), (40, 8195), (1030, 1001)]
# ... and of rows cut into slices of every length, of which a few rows are compared
CUT_SHAPES = [(3, 9601), (5, 64009), (66, 60007), (60, 150_001), (60, 400_003), (400, 320_009), (2, 1_000_003), (400, 100_003)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V", SHAPES)
def test_logprobs(M, V, dtype):
    x = rows(M, V, M + V, dtype)
    rng = np.random.default_rng(1)
    targets = rng.integers(0, V, M)
    targets[M // 2] = -100 if M > 2 else targets[M // 2]
    T = 1.0 if V % 2 else 0.7
    k = min(128, max(1, V // 3)) if M % 2 else min(64, V)
    logp, H, top, idx = rbq.token_logprobs(x, t(targets, torch.int64), top=k, temperature=T)
    torch.cuda.synchronize()
    r = oracle.Rows(np64(x), T)
    b = Bound(r, V)
    m = np.arange(M)
    has = targets >= 0
    near(logp, np.where(has, r.lp[m, np.maximum(targets, 0)], 0.0), b.lp[m, np.maximum(targets, 0)], "logp")
    near(H, r.H, b.H, "entropy")
    want = oracle.top(np64(x), k)
    assert np.array_equal(idx.cpu().numpy(), want)
    at = np.maximum(want, 0)
    near(top, np.where(want >= 0, r.lp[m[:, None], at], -np.inf), b.lp[m[:, None], at], "top")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V", SHAPES)
def test_logprobs_gradient(M, V, dtype):
    x = rows(M, V, M + 2 * V, dtype)
    rng = np.random.default_rng(2)
    targets = rng.integers(0, V, M)
    if M > 2:
        targets[1] = -1
    a, w = rng.normal(size=M).astype(np.float32), rng.normal(size=M).astype(np.float32)
    if M > 4:
        a[3] = w[3] = 0.0
    T = 1.0 if V % 2 else 2.0
    for both in (False, True):
        dx, logp, H = rbq.token_logprobs_backward(x, t(targets, torch.int64), t(a, torch.float32),
                                                  t(w, torch.float32) if both else None, temperature=T)
        torch.cuda.synchronize()
        r = oracle.Rows(np64(x), T)
        b = Bound(r, V)
        ww = w.astype(np.float64) if both else np.zeros(M)
        g = oracle.logprobs_grad(r, targets, a.astype(np.float64), ww)
        aa = np.abs(np.where(targets >= 0, a, 0.0))[:, None]
        lp = np.where(r.p > 0, np.abs(r.lp), 0.0)
        wide = np.abs(ww)[:, None] * r.p
        tol = (aa * r.p * (b.rel + 4 * U) + aa * 4 * U * (g != 0)
               + wide * ((lp + r.H[:, None]) * (b.rel + 8 * U) + b.lp + b.H[:, None])) / T
        near(dx, g, tol + half(dtype, np.abs(g) + tol), f"gradient, both {both}")
        near(H, r.H, b.H, "entropy")
        m = np.arange(M)
        near(logp, np.where(targets >= 0, r.lp[m, np.maximum(targets, 0)], 0.0), b.lp[m, np.maximum(targets, 0)], "logp")


def teacher(M, V, k, seed, T, repeat=False):
    """Log probabilities of k tokens of each row; some slots unused."""
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(M, V)) * 3 / T
    lp = z - np.log(np.exp(z).sum(1, keepdims=True))
    idx = np.argsort(-lp, 1)[:, :k]
    v = np.take_along_axis(lp, idx, 1).astype(np.float32)
    idx = idx.astype(np.int32)
    if k > 3:
        idx[::3, k - 1] = -1
        v[1::3, 1] = -np.inf
        if repeat:
            idx[:, 2] = idx[:, 0]
            v[:, 2] = v[:, 0] - 1
    return idx, v


def check_distill(x, idx, v, d, T, tail, name="", **more):
    dtype = x.dtype
    M, V = x.shape
    r = oracle.Rows(np64(x), T)
    b = Bound(r, V)
    loss, grad, size = oracle.distill(r, idx, v, tail)
    with np.errstate(all="ignore"):
        used = (idx >= 0) & (v > -np.inf)
        far = np.where(used, np.take_along_axis(b.D, np.maximum(idx, 0).astype(np.int64), 1), 0.0).max(1, initial=0.0)
    tol = 4 * b.dS + U * (4 * far + np.abs(np.where(np.isfinite(loss), loss, 0)) + 4)
    L = rbq.distill_forward(x, t(idx, torch.int32), t(v, torch.float32), temperature=T, tail=tail, **more)
    near(L, loss, tol, name + "loss")
    kept = x.clone()
    dx, L2 = rbq.distill_backward(x, t(idx, torch.int32), t(v, torch.float32), t(d, torch.float32), temperature=T,
                                  tail=tail, **more)
    torch.cuda.synchronize()
    assert torch.equal(x.view(torch.uint8), kept.view(torch.uint8))
    near(L2, loss, tol, name + "loss of the backward")
    g = grad * d.astype(np.float64)[:, None]
    e = np.abs(d.astype(np.float64))[:, None] * (size * (b.rel + 2 * b.dS[:, None] + 8 * U) + 2.0 ** -40)
    near(dx, g, e + half(dtype, np.abs(g) + e), name + "gradient")
    return dx, L


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V", SHAPES)
def test_distill(M, V, dtype, tail):
    k = min(V, [1, 5, 64, 128][(M + V) % 4])
    T = 1.0 if V % 2 else 2.0
    idx, v = teacher(M, V, k, M * V, T, repeat=not tail)
    x = rows(M, V, M * V + 1, dtype, masked=False)
    d = np.random.default_rng(5).normal(size=M).astype(np.float32)
    if M > 2:
        d[1] = 0.0
    check_distill(x, idx, v, d, T, tail)


@pytest.mark.parametrize("M,V", CUT_SHAPES)
def test_cuts(M, V):
    T = 1.5
    x = (torch.randn((M, V), device=dev(), generator=torch.Generator(dev()).manual_seed(V)) * 3).half()
    some = sorted({0, 1, M // 2, M - 1})
    targets = torch.arange(M, device=dev()) * 7
    ones = torch.ones(M, device=dev())
    r = oracle.Rows(np64(x[some]), T)
    b = Bound(r, V)
    at = (np.arange(len(some)), targets[some].cpu().numpy())
    for k in (0, 20, 128):
        logp, H, top, idx = rbq.token_logprobs(x, targets, top=k, temperature=T)
        near(logp[some], r.lp[at], b.lp[at], "logp")
        near(H[some], r.H, b.H, "entropy")
        want = oracle.top(np64(x[some]), k)
        assert np.array_equal(idx[some].cpu().numpy(), want)
        m = np.arange(len(some))[:, None]
        near(top[some], r.lp[m, want], b.lp[m, want], "top")
    dx, logp, H = rbq.token_logprobs_backward(x, targets, ones, ones, temperature=T)
    g = oracle.logprobs_grad(r, at[1], np.ones(len(some)), np.ones(len(some)))
    lp = np.abs(r.lp)
    tol = (r.p * (b.rel + 4 * U) + 4 * U * (g != 0) + r.p * ((lp + r.H[:, None]) * (b.rel + 8 * U) + b.lp + b.H[:, None])) / T
    near(dx[some], g, tol + half(torch.float16, np.abs(g) + tol), "gradient")
    near(H[some], r.H, b.H, "entropy of the backward")
    tv, ti = top, idx
    loss, grad, size = oracle.distill(r, idx[some].cpu().numpy(), np64(tv[some]), True)
    L = rbq.distill_forward(x, ti, tv, temperature=T, tail=True)
    dx, L2 = rbq.distill_backward(x, ti, tv, ones, temperature=T, tail=True)
    tol = 4 * b.dS + U * (4 * b.D.max(1) + np.abs(loss) + 4)
    near(L[some], loss, tol, "loss")
    near(L2[some], loss, tol, "loss of the backward")
    e = size * (b.rel + 2 * b.dS[:, None] + 8 * U) + 2.0 ** -40
    near(dx[some], grad, e + half(torch.float16, np.abs(grad) + e), "gradient")
