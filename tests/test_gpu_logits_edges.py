"""Edges of the operators on logits: masks, values at the ends of the types,
NaN, ties, strides, buffers, streams, graphs, refused and broken inputs.  Bounds
as in tests/test_gpu_logits.py."""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
from oracle import logits as oracle
from test_gpu_logits import TYPES, Bound, check_distill, dev, near, np64, rows, t, teacher

pytestmark = pytest.mark.gpu
INF = float("inf")


def lowest(dtype):
    return torch.finfo(dtype).min


@pytest.mark.parametrize("M,V", [(2, 9001), (1100, 9001), (12, 60001)], ids=["two rows", "many rows", "slices"])
@pytest.mark.parametrize("dtype", TYPES)
def test_masks_and_extremes(dtype, M, V):
    x = rows(M, V, 3, dtype)
    x[0] = -INF                              # nothing left
    if M > 2:
        x[2] = lowest(dtype)                 # masked with the lowest value, all of it: uniform
        x[3, :V - 1] = lowest(dtype)         # ... but one entry
        x[3, V - 1] = 1.0
        x[4, 1:] = -INF                      # one token possible
        x[5] = 0.0                           # all equal
        x[6, 100] = INF
        x[7, 8999] = float("nan")
        x[8, :9] = torch.finfo(dtype).max    # far above the rest
        x[9] = -0.0
        x[9, 4::7] = 0.0
    targets = torch.full((M,), 77, dtype=torch.int64, device=dev())
    logp, H, top, idx = rbq.token_logprobs(x, targets, top=9)
    d = torch.ones(M, device=dev())
    dx, logp2, H2 = rbq.token_logprobs_backward(x, targets, d, d)
    torch.cuda.synchronize()
    r = oracle.Rows(np64(x), 1.0)
    b = Bound(r, V)
    nan = r.broken
    want = np.where(nan, np.nan, r.lp[:, 77])
    for got in (logp, logp2):
        near(got, want, b.lp[:, 77], "logp")
    for got in (H, H2):
        near(got, np.where(nan, np.nan, r.H), b.H, "entropy")
    assert np.array_equal(idx.cpu().numpy(), oracle.top(np64(x), 9))
    g = np64(dx)
    assert np.isnan(g[nan]).all() and not np.isnan(g[~nan]).any() and not g[0].any()
    ok = ~nan
    lp = np.where(r.p > 0, np.abs(r.lp), 0.0)
    w = oracle.logprobs_grad(r, np.full(M, 77), np.ones(M), np.ones(M))
    tol = (r.p * b.rel + 2.0 ** -20 * (w != 0) + r.p * ((lp + r.H[:, None]) * (b.rel + 2.0 ** -20) + b.lp + b.H[:, None]))
    near(g[ok], w[ok], (tol + torch.finfo(dtype).eps / 2 * (np.abs(w) + tol) + 2.0 ** -25)[ok], "gradient")


@pytest.mark.parametrize("V", [1000, 33000, 70001])
def test_ties_go_to_the_lowest_index(V):
    """Few different values: most alternatives are ties, also at the last place."""
    rng = np.random.default_rng(V)
    for M in (3, 1050):
        if M * V > 4_000_000:
            continue
        x = t(rng.integers(0, 3, (M, V)), torch.float16)
        x[0] = 1.0
        x[1, V // 2:] = -INF
        for k in (1, 7, 64, 65, 128):
            *_, top, idx = rbq.token_logprobs(x, top=k)
            assert np.array_equal(idx.cpu().numpy(), oracle.top(np64(x), k)), (M, k)


@pytest.mark.parametrize("M,V", [(2, 20000), (1025, 20000), (3, 64000)])
def test_unkind_orders(M, V):
    """Rows whose largest entries come last, first, or all from one thread's columns."""
    x = torch.arange(V, device=dev(), dtype=torch.float32).repeat(M, 1) / 1000
    x[1] = x[1].flip(0)
    if M > 2:
        x[2] = 0.0
        n = len(range(3, V // 8, 512))
        x[2].view(-1, 8)[3::512] = torch.arange(8 * n, device=dev(), dtype=torch.float32).view(n, 8) + 30
    for k in (5, 64, 128):
        *_, idx = rbq.token_logprobs(x, top=k)
        assert np.array_equal(idx.cpu().numpy()[:4], oracle.top(np64(x[:4]), k)), k


def test_fewer_entries_than_alternatives():
    x = rows(3, 50, 1, torch.float32, masked=False)
    x[1, 4:] = -INF
    x[2] = -INF
    *_, top, idx = rbq.token_logprobs(x, top=100)
    idx, top = idx.cpu().numpy(), np64(top)
    for m in range(3):
        n = [50, 4, 0][m]
        assert np.array_equal(idx[m, :n], oracle.top(np64(x), 50)[m, :n]) and (idx[m, n:] == -1).all()
        assert np.isfinite(top[m, :n]).all() and (top[m, n:] == -INF).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V", [(5, 5001), (1026, 777), (5, 60001)])
def test_rows_that_lie_apart(M, V, dtype):
    """Logits that are columns of a wider tensor, starting at an odd entry; what lies between gradients stays."""
    wide = rows(M, V + 13, 9, dtype)
    x = wide[:, 5:5 + V]
    targets = torch.randint(0, V, (M,), device=dev())
    d = torch.rand(M, device=dev()) + 0.5
    one = x.contiguous()
    for a, b in zip(rbq.token_logprobs(x, targets, top=3), rbq.token_logprobs(one, targets, top=3)):
        assert torch.equal(a, b)
    out = torch.full((M, V + 9), 7.0, dtype=dtype, device=dev())
    dx, *_ = rbq.token_logprobs_backward(x, targets, d, d_logits=out[:, 3:3 + V])
    ref, *_ = rbq.token_logprobs_backward(one, targets, d)
    assert torch.equal(dx, ref) and bool((out[:, :3] == 7).all()) and bool((out[:, 3 + V:] == 7).all())
    idx, v = teacher(M, V, 5, 4, 1.0)
    a = [t(idx, torch.int32), t(v, torch.float32)]
    out.fill_(7.0)
    dx, loss = rbq.distill_backward(x, *a, d, tail=True, d_logits=out[:, 3:3 + V])
    ref, loss2 = rbq.distill_backward(one, *a, d, tail=True)
    assert torch.equal(dx, ref) and torch.equal(loss, loss2)
    assert bool((out[:, :3] == 7).all()) and bool((out[:, 3 + V:] == 7).all())


@pytest.mark.parametrize("M,V", [(3, 8999), (1040, 8999), (3, 60007)])
def test_gradient_in_the_logits_place(M, V):
    x = rows(M, V, 11, torch.float16, masked=False)
    targets = torch.randint(0, V, (M,), device=dev())
    d = torch.rand(M, device=dev()) + 0.5
    ref = rbq.token_logprobs_backward(x, targets, d, d)
    y = x.clone()
    got = rbq.token_logprobs_backward(y, targets, d, d, d_logits=y)
    assert got[0] is y and all(torch.equal(a, b) for a, b in zip(ref, got))
    idx, v = teacher(M, V, 20, 4, 1.0, repeat=True)
    a = [t(idx, torch.int32), t(v, torch.float32)]
    for tail in (False, True):
        ref = rbq.distill_backward(x, *a, d, tail=tail)
        y = x.clone()
        got = rbq.distill_backward(y, *a, d, tail=tail, d_logits=y)
        assert all(torch.equal(p, q) for p, q in zip(ref, got))


@pytest.mark.parametrize("V", [900, 9000, 20007, 40001, 100003])
def test_without_a_workspace(V):
    """Rows not cut, by workgroups of every size: the same values within the bounds."""
    M = 3
    x = rows(M, V, 12, torch.float16)
    none = torch.empty(0, dtype=torch.uint8, device=dev())
    targets = torch.tensor([5, V - 1, 17], device=dev())
    r = oracle.Rows(np64(x), 1.0)
    b = Bound(r, 8 * V)                      # (a thread adds up to eight times the terms that one of 512 slices' does)
    at = (np.arange(3), targets.cpu().numpy())
    for k in (3, 64, 65):
        logp, H, top, idx = rbq.token_logprobs(x, targets, top=k, workspace=none)
        near(H, r.H, b.H, "entropy")
        near(logp, r.lp[at], b.lp[at], "logp")
        assert np.array_equal(idx.cpu().numpy(), oracle.top(np64(x), k))
    d = torch.rand(M, device=dev())
    dx, logp, _ = rbq.token_logprobs_backward(x, targets, d, d, workspace=none)
    g = oracle.logprobs_grad(r, at[1], d.cpu().double().numpy(), d.cpu().double().numpy())
    lp = np.where(r.p > 0, np.abs(r.lp), 0.0)
    tol = r.p * b.rel + 2.0 ** -20 * (g != 0) + r.p * ((lp + r.H[:, None]) * (b.rel + 2.0 ** -20) + b.lp + b.H[:, None])
    near(dx, g, tol + 2.0 ** -11 * (np.abs(g) + tol) + 2.0 ** -25, "gradient")
    for tail in (False, True):
        idx, v = teacher(M, V, 64, 4, 1.0)
        check_distill(rows(M, V, 13, torch.float32, masked=False), idx, v, np.ones(M, np.float32), 1.0, tail,
                      workspace=none)


@pytest.mark.parametrize("M,V", [(2, 1000), (1030, 1000), (1030, 130), (2, 128), (1030, 4003)])
def test_more_alternatives_than_threads_have(M, V):
    """As many alternatives as vectors, or nearly: every entry comes into question."""
    for seed in (0, 1):
        x = rows(M, V, seed, torch.float32) if seed else t(np.random.default_rng(2).integers(0, 40, (M, V)), torch.bfloat16)
        for k in (60, 100, 128):
            *_, idx = rbq.token_logprobs(x, top=k)
            assert np.array_equal(idx[:6].cpu().numpy(), oracle.top(np64(x[:6]), k)), k


def test_a_workspace_of_any_contents():
    M, V = 4, 60000
    x = rows(M, V, 14, torch.float32, masked=False)
    targets = torch.randint(0, V, (M,), device=dev())
    need = int(rbq.lib().rbq_token_logprobs_workspace_bytes(M, V, 128))
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev())
    ref = rbq.token_logprobs(x, targets, top=128)
    assert all(torch.equal(a, b) for a, b in zip(ref, rbq.token_logprobs(x, targets, top=128, workspace=ws)))
    idx, v = teacher(M, V, 64, 4, 1.0)
    a = [t(idx, torch.int32), t(v, torch.float32)]
    need = int(rbq.lib().rbq_distill_workspace_bytes(M, V, 64))
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=dev())
    d = torch.ones(M, device=dev())
    ref = rbq.distill_backward(x, *a, d, tail=True)
    got = rbq.distill_backward(x, *a, d, tail=True, workspace=ws[:need])
    assert all(torch.equal(p, q) for p, q in zip(ref, got)) and bool((ws[need:] == 255).all())


def test_broken_tokens():
    for M, V in ((4, 6000), (1030, 6000), (4, 64000)):
        x = rows(M, V, 15, torch.float16, masked=False)
        targets = torch.full((M,), 3, dtype=torch.int64, device=dev())
        targets[1], targets[2] = V, 2 ** 40
        targets[3] = -2 ** 40
        st = torch.zeros(1, dtype=torch.int32, device=dev())
        d = torch.ones(M, device=dev())
        logp, H, *_ = rbq.token_logprobs(x, targets, status=st)
        assert int(st.item()) == rbq.RBQ_STATUS_BAD_TOKEN
        dx, logp2, _ = rbq.token_logprobs_backward(x, targets, d, d)
        for lp in (logp, logp2):
            assert torch.isnan(lp[1:3]).all() and torch.isfinite(lp[4:]).all() and lp[3] == 0
        assert torch.isfinite(H).all()
        assert torch.isnan(dx[1:3]).all() and torch.isfinite(dx[3:]).all() and torch.isfinite(dx[0]).all()
        idx, v = teacher(M, V, 5, 4, 1.0)
        idx[1, 0] = V
        idx[2, 0] = 2 ** 31 - 1
        st.zero_()
        a = [t(idx, torch.int32), t(v, torch.float32)]
        dx, loss = rbq.distill_backward(x, *a, d, tail=True, status=st)
        assert int(st.item()) == rbq.RBQ_STATUS_BAD_TOKEN
        assert torch.isnan(loss[1:3]).all() and torch.isfinite(loss[3:]).all()
        assert torch.isnan(dx[1:3]).all() and torch.isfinite(dx[3:]).all()
        d[1:3] = 0.0                         # a row without weight takes no part
        dx, _ = rbq.distill_backward(x, *a, d, tail=True)
        assert torch.isfinite(dx).all() and not dx[1:3].any()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("M,V", [(6, 7000), (1030, 7000), (6, 60001)])
def test_distillation_edges(M, V, tail):
    x = rows(M, V, 16, torch.float32, masked=False)
    idx, v = teacher(M, V, 8, 17, 1.0)
    idx[0], v[0] = -1, 0.0                   # no slots
    v[1] = [0.0] + [-INF] * 7                # one token has all of the teacher's mass
    x[2] = -INF                              # the student has nothing
    x[3, 100] = float("nan")
    v[4, 0] = np.nan
    x[5, int(idx[5, 0])] = -INF              # the student rules out what the teacher likes
    d = np.ones(M, np.float32)
    loss = rbq.distill_forward(x, t(idx, torch.int32), t(v, torch.float32), tail=tail)
    dx, loss2 = rbq.distill_backward(x, t(idx, torch.int32), t(v, torch.float32), t(d, torch.float32), tail=tail)
    torch.cuda.synchronize()
    L, g = np64(loss), np64(dx)
    assert np.array_equal(np.isnan(L), np.isnan(np64(loss2))) and (L[np.isfinite(L)] >= -1e-5).all()
    assert abs(L[0]) < 1e-5 and np.abs(g[0]).max() < 1e-6
    assert L[2] == INF and not g[2].any()
    assert np.isnan(L[3]) and np.isnan(g[3]).all() and np.isnan(L[4]) and np.isnan(g[4]).all()
    assert L[5] == INF and np.isfinite(g[5]).all()
    rest = [m for m in range(M) if m not in (2, 3, 4, 5)]
    check_distill(x[rest].contiguous(), idx[rest], v[rest], d[rest], 1.0, tail)
    # the student masks all that the teacher does not name
    y = torch.full((2, V), -INF, device=dev())
    i2, v2 = teacher(2, V, 3, 18, 1.0)
    y.scatter_(1, t(i2, torch.int64), 1.0)
    dy, l2 = rbq.distill_backward(y, t(i2, torch.int32), t(v2, torch.float32), torch.ones(2, device=dev()), tail=tail)
    assert torch.isfinite(dy).all() and bool((torch.isinf(l2) if tail else torch.isfinite(l2)).all())


def test_no_slots_at_all():
    x = rows(3, 500, 1, torch.float16, masked=False)
    idx = torch.empty((3, 0), dtype=torch.int32, device=dev())
    v = torch.empty((3, 0), device=dev())
    for tail in (False, True):
        dx, loss = rbq.distill_backward(x, idx, v, torch.ones(3, device=dev()), tail=tail)
        assert float(loss.abs().max()) < 1e-6 and float(dx.abs().max()) < 1e-6


def test_gradients_against_differences():
    """Central differences of the calls themselves, in float32."""
    M, V = 2, 40
    x = rows(M, V, 19, torch.float32, masked=False, scale=1.0).clamp(-3, 3)
    targets = torch.tensor([3, 39], device=dev())
    a, b = torch.tensor([1.0, -2.0], device=dev()), torch.tensor([0.5, 1.5], device=dev())
    idx, v = teacher(M, V, 6, 20, 1.0)
    sl = [t(idx, torch.int32), t(v, torch.float32)]
    h = 2.0 ** -6                            # truncation ~ h^2 / 6 of third derivatives <= ~6; rounding ~ 2^-21 / h

    def value(y, which):
        if which == "logp":
            lp, H, *_ = rbq.token_logprobs(y, targets, temperature=1.5)
            return (a.double() * lp.double() + b.double() * H.double()).sum().item()
        return (a.double() * rbq.distill_forward(y, *sl, temperature=1.5, tail=which == "tail").double()).sum().item()

    for which in ("logp", "tail", "plain"):
        if which == "logp":
            g = rbq.token_logprobs_backward(x, targets, a, b, temperature=1.5)[0]
        else:
            g = rbq.distill_backward(x, *sl, a, temperature=1.5, tail=which == "tail")[0]
        for m in range(M):
            for j in range(0, V, 3):
                p, q = x.clone(), x.clone()
                p[m, j] += h
                q[m, j] -= h
                diff = (value(p, which) - value(q, which)) / (2 * h)
                assert abs(diff - g[m, j].item()) <= 4 * h * h + 2.0 ** -12, (which, m, j)


@pytest.mark.parametrize("M,V", [(3, 20001), (3, 60001)])
def test_streams_and_replayed_graphs(M, V):
    """Two graphs that share a workspace, replayed in turn with other work between, and a side stream."""
    xs = [rows(M, V, s, torch.float16, masked=False) for s in (31, 32)]
    targets = torch.randint(0, V, (M,), device=dev())
    d = torch.ones(M, device=dev())
    idx, v = teacher(M, V, 16, 33, 1.0)
    sl = [t(idx, torch.int32), t(v, torch.float32)]
    ref = [(rbq.token_logprobs(x, targets, top=20), rbq.distill_backward(x, *sl, d, tail=True)) for x in xs]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev())
    side = torch.cuda.Stream()
    graphs, outs = [], []
    torch.cuda.synchronize()
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((rbq.token_logprobs(x, targets, top=20, workspace=ws),
                         rbq.distill_backward(x, *sl, d, tail=True, workspace=ws)))
        graphs.append(g)
    for _ in range(3):
        for g, o, want in zip(graphs, outs, ref):
            for part in o:
                for y in part:
                    y.zero_()
            g.replay()
            torch.randn(100, 100, device=dev()).sum()
            torch.cuda.synchronize()
            for got, w in zip(o, want):
                assert all(torch.equal(p, q) for p, q in zip(got, w))
    side.wait_stream(torch.cuda.current_stream())
    got = rbq.token_logprobs(xs[0], targets, top=20, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, ref[0][0]))


def test_long_rows():
    """More entries than one map of named tokens covers, in one slice and in many."""
    V = 600_011
    x = rows(2, V, 40, torch.bfloat16)
    r = oracle.Rows(np64(x), 1.0)
    b = Bound(r, V)
    targets = torch.tensor([V - 1, 5], device=dev())
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=dev())):
        logp, H, top, idx = rbq.token_logprobs(x, targets, top=128, workspace=ws)
        near(H, r.H, b.H, "entropy")
        assert np.array_equal(idx.cpu().numpy(), oracle.top(np64(x), 128))
        y = torch.where(torch.isinf(x), torch.zeros_like(x), x)
        ti, tv = teacher(2, V, 128, 41, 1.0)
        ti[0, :2] = [V - 1, 262144]
        check_distill(y, ti, tv, np.ones(2, np.float32), 1.0, True, workspace=ws)


def test_rows_beyond_32_bit_offsets():
    """More than 2^31 entries: the last rows' results are those of the rows alone."""
    V, M = 131073, 16500
    x = torch.empty((M, V), dtype=torch.float16, device=dev())
    x[:100] = 0
    x[-3:] = rows(3, V, 42, torch.float16)
    targets = torch.zeros(M, dtype=torch.int64, device=dev())
    targets[:M - 3] = -1
    d = torch.zeros(M, device=dev())
    d[-3:] = 1.0
    x[100:-3] = 0.0
    none = torch.empty(0, dtype=torch.uint8, device=dev())
    logp, H, top, idx = rbq.token_logprobs(x, targets, top=4)
    ref = rbq.token_logprobs(x[-3:], targets[-3:], top=4, workspace=none)
    for a, c in zip((logp, H, top, idx), ref):
        assert torch.equal(a[-3:], c)
    dx, *_ = rbq.token_logprobs_backward(x, targets, d, d_logits=x)
    assert dx is x and not x[:-3].any() and bool(x[-3:].any())


def test_a_run_of_all(seed=50):
    """A teacher's head in 4 bits, its log probabilities and alternatives, and a step of a binarized student's head:
    the loss falls along the gradient that qat_backward takes from here."""
    torch.manual_seed(seed)
    M, inf, V = 48, 256, 2000
    W = torch.randn(V, inf, device=dev()) * 0.1
    X = torch.randn(M, inf, device=dev()).half()
    codes, scales, zeros = rbq.encode_q4(W, zeros=True)
    t_logits = rbq.gemm_q4(codes, scales, X, zeros, dtype=torch.float32)
    lp, H, top_logp, top_index = rbq.token_logprobs(t_logits, t_logits.argmax(1), top=32)
    assert torch.equal(top_index[:, 0].long(), t_logits.argmax(1)) and torch.equal(lp, top_logp[:, 0])
    planes, s = rbq.encode(W, 2)
    planes, Y = rbq.qat_forward(W, s, X)
    d = torch.full((M,), 64.0 / M, device=dev())
    dY, loss = rbq.distill_backward(Y, top_index, top_logp, d, tail=True)
    assert torch.equal(loss, rbq.distill_forward(Y, top_index, top_logp, tail=True))
    dX, dW, ds = rbq.qat_backward(planes, s, X, dY)
    # dY against float64 autograd of the same loss, dW as its product with X
    y = Y.double().requires_grad_()
    lq = torch.log_softmax(y, 1)
    p = top_logp.double().exp()
    rest = 1 - p.sum(1)
    named = torch.zeros_like(lq).scatter(1, top_index.long(), 1.0)
    q_rest = (lq.exp() * (1 - named)).sum(1)
    want = (p * (top_logp.double() - lq.gather(1, top_index.long()))).sum(1) + rest * (rest.log() - q_rest.log())
    assert torch.allclose(loss.double(), want, rtol=1e-5, atol=1e-5)
    (want * d.double()).sum().backward()
    size = y.grad.abs()
    assert bool(((dY.double() - y.grad).abs() <= 2.0 ** -11 * size + 2.0 ** -25 + 2.0 ** -14 * d[0] * lq.exp()).all())
    assert torch.allclose(dW, dY.float().t().contiguous() @ X.float(), rtol=1e-3, atol=1e-4)


@pytest.mark.parametrize("V", [500, 60001])
def test_refusals(V):
    """Types, sizes, strides and gradients that lie over what is read."""
    x = rows(4, V, 60, torch.float16)
    f, i = torch.zeros(4, device=dev()), torch.zeros(4, dtype=torch.int64, device=dev())
    ti, tv = torch.zeros((4, 3), dtype=torch.int32, device=dev()), torch.zeros((4, 3), device=dev())
    wrong = (TypeError, ValueError)
    for bad in (x.double(), x.int(), x[0], x.t(), x[:, ::2], x[:1].expand(4, V), x[:, :0], x.cpu()):
        for call in (lambda: rbq.token_logprobs(bad), lambda: rbq.token_logprobs_backward(bad, i, f),
                     lambda: rbq.distill_forward(bad, ti, tv), lambda: rbq.distill_backward(bad, ti, tv, f)):
            with pytest.raises(wrong):
                call()
    for call in (lambda: rbq.token_logprobs(x, i.int()), lambda: rbq.token_logprobs(x, i[:3]),
                 lambda: rbq.token_logprobs(x, top=129), lambda: rbq.token_logprobs(x, top=-1),
                 lambda: rbq.token_logprobs_backward(x, i, f.double()), lambda: rbq.token_logprobs_backward(x, i, f[:2]),
                 lambda: rbq.token_logprobs_backward(x, i, f, f.half()),
                 lambda: rbq.token_logprobs_backward(x, i, f, d_logits=x.float()),
                 lambda: rbq.token_logprobs_backward(x, i, f, d_logits=torch.empty_like(x)[:, :-1]),
                 lambda: rbq.distill_forward(x, ti.long(), tv), lambda: rbq.distill_forward(x, ti, tv.half()),
                 lambda: rbq.distill_forward(x, ti[:3], tv[:3]), lambda: rbq.distill_forward(x, ti, tv[:, :2]),
                 lambda: rbq.distill_forward(x, torch.zeros((4, 129), dtype=torch.int32, device=dev()),
                                             torch.zeros((4, 129), device=dev())),
                 lambda: rbq.distill_backward(x, ti, tv, f[:1])):
        with pytest.raises(wrong):
            call()
    for T in (0.0, -1.0, float("nan"), float("inf"), 1e-4, 1e4):
        with pytest.raises(rbq.RbqError):
            rbq.token_logprobs(x, temperature=T)
        with pytest.raises(rbq.RbqError):
            rbq.distill_forward(x, ti, tv, temperature=T)
    # a gradient half over the logits: another row's place, or another stride
    wide = torch.zeros(6, V, dtype=torch.float16, device=dev())
    with pytest.raises(rbq.RbqError):
        rbq.token_logprobs_backward(wide[:4], i, f, d_logits=wide[1:5])
    with pytest.raises(rbq.RbqError):
        rbq.distill_backward(wide[:4], ti, tv, f, d_logits=wide[2:6])
    # a gradient that is asked of a target needs targets
    with pytest.raises(rbq.RbqError):
        rbq.token_logprobs_backward(x, None, f)
    torch.cuda.synchronize()


def test_no_rows_and_one_entry():
    """No rows at all; a vocabulary of one, whose only token is certain."""
    e = torch.empty((0, 70), dtype=torch.bfloat16, device=dev())
    none = torch.empty(0, device=dev())
    logp, H, top, idx = rbq.token_logprobs(e, torch.empty(0, dtype=torch.int64, device=dev()), top=5)
    assert logp.shape == H.shape == (0,) and top.shape == idx.shape == (0, 5)
    assert rbq.distill_backward(e, idx, top, none)[0].shape == (0, 70)
    x = torch.tensor([[3.0], [-INF], [-7.0]], device=dev())
    i = torch.zeros(3, dtype=torch.int64, device=dev())
    logp, H, top, idx = rbq.token_logprobs(x, i, top=2)
    # (the bounds of tests/test_gpu_logits.py with n = 8, D = 3, nothing else: all of 4 (n + 60 + 3 D) + 4 D + 8 steps)
    tol = (4 * (8 + 60 + 9) + 4 * 3 + 8) * 2.0 ** -23
    near(logp[[0, 2]], np.zeros(2), tol, "logp")
    near(H[[0, 2]], np.zeros(2), tol, "entropy")
    assert idx[[0, 2]].tolist() == [[0, -1]] * 2 and idx[1].tolist() == [-1, -1]
    one = torch.ones(3, device=dev())
    d, *_ = rbq.token_logprobs_backward(x, i, one, one)
    near(d[[0, 2]], np.zeros((2, 1)), 2 * tol, "gradient")
    assert not d[1].any()
    d, loss = rbq.distill_backward(x[:1], idx[:1], top[:1], one[:1], tail=True)
    near(d, np.zeros((1, 1)), 2 * tol, "gradient")
    near(loss, np.zeros(1), 2 * tol, "loss")


@pytest.mark.parametrize("M,V", [(2, 100), (1030, 5000), (2, 60001)])
def test_a_rest_that_is_none(M, V):
    """Teacher and student mask the same tokens, or all are named: what the teacher's rounded log probabilities leave
    beside the named ones is no class of its own."""
    x, y = (rows(M, V, s, torch.float32, masked=False) for s in (70, 71))
    for mask in (-INF, lowest(torch.float32)):
        if V > 128:
            x[:, 100:] = mask
            y[:, 100:] = mask
        *_, v, idx = rbq.token_logprobs(y, top=128)
        dx, loss = rbq.distill_backward(x, idx, v, torch.ones(M, device=dev()), tail=True)
        assert torch.isfinite(loss).all() and torch.isfinite(dx).all()
        # of 100 tokens, all named: the full divergence
        lp, lq = (torch.log_softmax(z[:, :100].double(), 1) for z in (y, x))
        want = (lp.exp() * (lp - lq)).sum(1)
        # each side's sum off by dS = 2^-23 (n + 60 + 3 D), D and a term's distance up to 64 here, p by as much
        tol = 2.0 ** -23 * (8 * 64 + 60 + 3 * 64) * (2 + want)
        assert bool(((loss.double() - want).abs() <= tol).all())
