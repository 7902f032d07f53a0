"""GPU parity of 8-bit activation checkpoints (rbq_qat_checkpoint) and of the
backward that reads them (rbq_qat_backward_ckpt).

Checkpoint: codes and scale bits equal to oracle/f8.py's.  Gradients: the
bounds of the fp16 backward (test_gpu_qat.py) on the restored activations x^,
which are fp16 numbers, so the same arithmetic applies:
  dW   |err| <= 2 M 2^-24 sum_m |dY[m][r] x^[m][j]|
  da   sum_j tol_dW[r][j] + 2^-23 |da|, and the fp32 sums of at most 128
       entries of dW: 128 2^-24 sum_j |dW[r][j]|
  dX   sum_r |dY| (2^-21 |w| + 2^-25) + 4 out 2^-24 sum_r |dY w|
"""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
import workloads
from oracle import f8, qat

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def dev():
    return torch.device("cuda:0")


def t_f16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.float16)).to(dev())


def t_planes(p):
    return torch.from_numpy(p.view(np.int32)).to(dev())


@pytest.mark.parametrize("M,inf", [(1, 32), (1, 4096), (16, 128), (17, 160), (33, 4128), (5, 544)])
def test_checkpoint_equals_the_oracle(M, inf):
    X = workloads.gaussian_activations(M, inf, M + inf).copy()
    X[0, :4] = [0x0000, 0x8000, 0x0001, 0x8001]
    if M > 4:
        X[2] = 0
        X[3] &= 0x83FF                                     # subnormals
        X[4, 7] = 0x7BFF                                   # the largest maximum
        X[M - 1, inf - 1] = 0xFC00
        X[M - 1, 0] = 0x7E00
    codes, scales = rbq.qat_checkpoint(t_f16(X))
    torch.cuda.synchronize()
    c, s = f8.checkpoint(X)
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(scales.cpu().numpy().view(np.uint16), s)


def test_checkpoint_of_every_fp16_value():
    """Rows of neighbouring magnitudes (every scale, few codes each) and rows
    of mixed magnitudes (every code, ties among them)."""
    v = np.concatenate([np.arange(0x7C00), np.arange(0x8000, 0xFC00)]).astype(np.uint16)
    rows = v[np.argsort(v & 0x7FFF, kind="stable")].reshape(-1, 512)
    rng = np.random.default_rng(7)
    s = rng.integers(1, 0x5C00, (256, 1)).astype(np.uint16).view(np.float16).astype(np.float64)
    k = rng.integers(-254, 255, (256, 128)) / 2.0          # halves: ties wherever s k is an fp16 number
    k[:, 0] = 127
    ties = (s * k).astype(np.float16).view(np.uint16)
    for X in (rows, rng.permutation(v).reshape(-1, 512), ties):
        codes, scales = rbq.qat_checkpoint(t_f16(X))
        torch.cuda.synchronize()
        c, sb = f8.checkpoint(X)
        assert np.array_equal(codes.cpu().numpy(), c)
        assert np.array_equal(scales.cpu().numpy().view(np.uint16), sb)


def case(out, inf, K, group, M, seed):
    G = inf // group if group else 1
    planes = workloads.random_planes(K, out, inf, seed)
    s = workloads.random_scales(K, out, G, seed + 1)
    X = workloads.gaussian_activations(max(M, 1), inf, seed + 2)[:M].copy()
    X[:, ::37] = (X[:, ::37].view(np.float16) * np.float16(20)).view(np.uint16)
    dY = workloads.gaussian_activations(max(M, 1), out, seed + 3)[:M]
    return planes, s, X, dY


def check_grads(got, planes, s, x, dY, group):
    dX, dW, ds = got
    M, out = dY.shape
    K, inf = planes.shape[0], x.shape[1]
    rdX, rdW, rds = qat.backward(planes, s, x, dY, group)
    xa, da = np.abs(x.view(np.float16).astype(np.float64)), np.abs(dY.view(np.float16).astype(np.float64))
    if dW is not None:
        g = dW.cpu().numpy().astype(np.float64)
        t = 2.0 * max(M, 1) * U * (da.T @ xa) + 1e-300
        assert (np.abs(g - rdW) <= t).all(), f"dW {(np.abs(g - rdW) / t).max():.3f} of the bound"
        if ds is not None:
            n = group if group else inf
            sums = (t + 128 * U * np.abs(rdW)).reshape(out, inf // n, n).sum(2)
            e = np.abs(ds.cpu().numpy().astype(np.float64) - rds)
            assert (e <= sums + 2.0 ** -23 * np.abs(rds) + 1e-300).all(), "dscales"
    if dX is not None:
        wa = np.abs(qat.dequant(planes, s, group))
        t = da @ (2.0 ** -21 * wa + 2.0 ** -25) + 4.0 * out * U * (da @ wa) + 1e-300
        e = np.abs(dX.cpu().numpy().astype(np.float64) - rdX)
        assert (e <= t).all(), f"dX {(e / t).max():.3f} of the bound"


BACKWARD = [(256, 512, 2, 0, 5), (384, 1024, 4, 128, 130), (100, 4128, 3, 0, 33), (64, 96, 1, 0, 1),
            (1000, 2048, 2, 0, 16), (1024, 1280, 4, 128, 257), (33, 160, 2, 0, 70), (513, 288, 1, 0, 65),
            (8, 32, 2, 0, 3), (129, 128, 3, 128, 2), (264, 544, 2, 0, 511), (3, 64, 1, 0, 200), (1, 32, 2, 0, 129),
            (5, 96, 4, 0, 64), (600, 576, 2, 0, 1100), (601, 640, 4, 128, 1030), (1501, 384, 1, 0, 100),
            (4100, 96, 3, 0, 20)]


@pytest.mark.parametrize("out,inf,K,group,M", BACKWARD)
def test_backward_matches_the_oracle(out, inf, K, group, M):
    planes, s, X, dY = case(out, inf, K, group, M, 30 + out + M)
    codes, cs = rbq.qat_checkpoint(t_f16(X))
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    args = (t_planes(planes), t_f16(s), codes, cs, t_f16(dY), group)
    got = rbq.qat_backward_ckpt(*args, status=st)
    again = rbq.qat_backward_ckpt(*args)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_grads(got, planes, s, f8.restore(*f8.checkpoint(X)), dY, group)
    assert all(torch.equal(a, b) for a, b in zip(got, again))       # the same bits in every run
    less = rbq.qat_backward_ckpt(*args, workspace=torch.empty(0, dtype=torch.uint8, device=dev()))
    check_grads(less, planes, s, f8.restore(*f8.checkpoint(X)), dY, group)


LARGE = [(4101, 4128, 2, 0, 131), (3900, 4224, 4, 128, 65), (4096, 4096, 1, 0, 320), (700, 4096, 3, 0, 700),
         (8200, 1024, 2, 128, 257)]


@pytest.mark.parametrize("out,inf,K,group,M", LARGE)
def test_backward_of_large_layers_in_64_bits(out, inf, K, group, M):
    """The bounds above, with the sums in 64 bits on the device; once with the
    workspace and once without."""
    planes, s, X, dY = case(out, inf, K, group, M, out + M)
    codes, cs = rbq.qat_checkpoint(t_f16(X))
    a = (t_planes(planes), t_f16(s), codes, cs, t_f16(dY), group)
    x = t_f16(f8.restore(codes.cpu().numpy(), cs.cpu().numpy().view(np.uint16))).double()
    d = t_f16(dY).double()
    w = torch.from_numpy(qat.dequant(planes, s, group)).to(dev()).double()
    G = inf // group if group else 1
    dw = d.t().contiguous() @ x
    t_dw = 2.0 * M * U * (d.abs().t().contiguous() @ x.abs()) + 1e-300
    dx = d @ w
    t_dx = d.abs() @ (2.0 ** -21 * w.abs() + 2.0 ** -25) + 4.0 * out * U * (d.abs() @ w.abs()) + 1e-300
    sums = (t_dw + 128 * U * dw.abs()).view(out, G, -1).sum(2)
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=dev())):
        gdx, gdw, gds = rbq.qat_backward_ckpt(*a, workspace=ws)
        assert bool(((gdw.double() - dw).abs() <= t_dw).all()), "dW"
        assert bool(((gdx.double() - dx).abs() <= t_dx).all()), "dX"
        word = a[0].long() & 0xFFFFFFFF
        for k in range(K):
            sign = torch.stack([(word[k] >> b) & 1 for b in range(32)], -1).view(out, inf).double() * 2 - 1
            ds = (sign * dw).view(out, G, -1).sum(2)
            assert bool(((gds[k].double() - ds).abs() <= sums + 2.0 ** -23 * ds.abs() + 1e-300).all()), "dscales"


def test_backward_of_exact_activations_is_the_fp16_backwards():
    """Activations that a checkpoint holds exactly (multiples of a power of
    two up to 127): both backward passes compute the same sums."""
    out, inf, K, M = 200, 256, 2, 40
    planes, s, _, dY = case(out, inf, K, 0, M, 91)
    rng = np.random.default_rng(92)
    x = rng.integers(-127, 128, (M, inf)) * 2.0 ** -6
    x[:, ::128] = 127 * 2.0 ** -6
    X = x.astype(np.float16).view(np.uint16)
    codes, cs = rbq.qat_checkpoint(t_f16(X))
    got = rbq.qat_backward_ckpt(t_planes(planes), t_f16(s), codes, cs, t_f16(dY))
    fp16 = rbq.qat_backward(t_planes(planes), t_f16(s), t_f16(X), t_f16(dY))
    torch.cuda.synchronize()
    check_grads(got, planes, s, X, dY, 0)
    check_grads(fp16, planes, s, X, dY, 0)


def test_backward_against_differences():
    """L = sum dY (x^ What^T) is linear in every weight and scale: the change
    of L (in 64 bits) with a scale or a weight is the gradient."""
    out, inf, K, M = 40, 96, 2, 7
    planes, s, X, dY = case(out, inf, K, 0, M, 51)
    codes, cs = rbq.qat_checkpoint(t_f16(X))
    _, dW, ds = rbq.qat_backward_ckpt(t_planes(planes), t_f16(s), codes, cs, t_f16(dY), need_dx=False)
    torch.cuda.synchronize()
    x = f8.restore(*f8.checkpoint(X)).view(np.float16).astype(np.float64)
    d = dY.view(np.float16).astype(np.float64)
    w = qat.dequant(planes, s, 0)
    rng = np.random.default_rng(52)
    scale = 2.0 * M * U * (np.abs(d).T @ np.abs(x))

    def loss(v):
        return float((d * (x @ v.T)).sum())

    for _ in range(5):
        r, j, k = int(rng.integers(out)), int(rng.integers(inf)), int(rng.integers(K))
        v = w.copy()
        v[r, j] += 0.5
        diff = (loss(v) - loss(w)) / 0.5
        round_off = 2.0 ** -40 * (np.abs(d) * (np.abs(x) @ np.abs(v).T)).sum()
        assert abs(diff - float(dW[r, j])) <= scale[r, j] + round_off
        s2 = s.copy().view(np.float16)
        s2[k, r, 0] += np.float16(0.5)
        h = float(s2[k, r, 0]) - float(s.view(np.float16)[k, r, 0])
        diff = (loss(qat.dequant(planes, s2.view(np.uint16), 0)) - loss(w)) / h
        # the differenced layer is formed in fp32: one rounding of each weight of the row
        formed = 2.0 ** -22 / abs(h) * float((np.abs(d[:, r]) @ np.abs(x)).sum())
        assert abs(diff - float(ds[k, r, 0])) <= scale[r].sum() + 2.0 ** -22 * float(dW[r].abs().sum()) + formed \
            + round_off


def test_outputs_on_request_and_empty_batches():
    out, inf, K, M = 128, 256, 2, 8
    planes, s, X, dY = case(out, inf, K, 0, M, 44)
    codes, cs = rbq.qat_checkpoint(t_f16(X))
    a = (t_planes(planes), t_f16(s), codes, cs, t_f16(dY))
    full = rbq.qat_backward_ckpt(*a)
    dx = rbq.qat_backward_ckpt(*a, need_dw=False, need_dscales=False)
    dw = rbq.qat_backward_ckpt(*a, need_dx=False, need_dscales=False)
    ds = rbq.qat_backward_ckpt(*a, need_dx=False, need_dw=False)
    none = rbq.qat_backward_ckpt(*a, need_dx=False, need_dw=False, need_dscales=False)
    torch.cuda.synchronize()
    assert dx[1] is None and dx[2] is None and torch.equal(dx[0], full[0])
    assert dw[0] is None and dw[2] is None and torch.equal(dw[1], full[1])
    assert ds[0] is None and ds[1] is None and torch.equal(ds[2], full[2])
    assert none == (None, None, None)
    e = rbq.qat_backward_ckpt(*a[:2], *rbq.qat_checkpoint(t_f16(X[:0])), t_f16(dY[:0]))
    torch.cuda.synchronize()
    assert e[0].shape == (0, inf) and not e[1].any() and not e[2].any()


def test_non_finite_blocks_reach_their_columns_only():
    out, inf, M = 40, 416, 19
    planes, s, X, dY = case(out, inf, 1, 0, M, 61)
    X[18, 200] = 0x7C00
    codes, cs = rbq.qat_checkpoint(t_f16(X))
    _, dW, _ = rbq.qat_backward_ckpt(t_planes(planes), t_f16(s), codes, cs, t_f16(dY), need_dx=False)
    torch.cuda.synchronize()
    bad = ~np.isfinite(dW.cpu().numpy())
    assert bad[:, 128:256].all() and not bad[:, :128].any() and not bad[:, 256:].any()
    # an infinite gradient of the last token stays in its row, with the sign of x^
    dY = dY.copy()
    dY[18, 7] = 0x7C00
    X[18, 200] = 0
    X[18, 3] = 0
    codes, cs = rbq.qat_checkpoint(t_f16(X))
    _, dW, _ = rbq.qat_backward_ckpt(t_planes(planes), t_f16(s), codes, cs, t_f16(dY), need_dx=False)
    torch.cuda.synchronize()
    x = f8.restore(*f8.checkpoint(X)).view(np.float16)[18].astype(np.float64)
    with np.errstate(invalid="ignore"):
        want = np.inf * x
    g = dW.cpu().numpy()
    assert np.array_equal(np.isnan(g[7]), np.isnan(want)) and np.isnan(want).any()
    assert np.array_equal(g[7][~np.isnan(want)], want[~np.isnan(want)].astype(np.float32))
    assert np.isfinite(np.delete(g, 7, 0)).all()


@pytest.mark.parametrize("out", [200, 203])
def test_a_training_step_with_checkpoints(out):
    """The operators together: forward, checkpoint, backward, twice on a side
    stream, then captured and replayed with eager work between."""
    inf, K, M = 416, 2, 50
    W = workloads.gaussian_weight(out, inf, 71)
    s = workloads.random_scales(K, out, 1, 72, signed=False)
    Xs = [workloads.gaussian_activations(M, inf, 73 + i) for i in range(3)]
    dY = workloads.gaussian_activations(M, out, 79)
    Wt, st, dYt = torch.from_numpy(W).to(dev()), t_f16(s), t_f16(dY)

    def step(x, stream=None):
        planes, _ = rbq.qat_forward(Wt, st, x, stream=stream)
        return rbq.qat_backward_ckpt(planes, st, *rbq.qat_checkpoint(x, stream=stream), dYt, stream=stream)

    eager = [step(t_f16(x)) for x in Xs]
    torch.cuda.synchronize()
    p = qat.cascade(W, s, 0)
    for x, g in zip(Xs, eager):
        check_grads(g, p, s, f8.restore(*f8.checkpoint(x)), dY, 0)
    x_in = t_f16(Xs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = step(x_in)
    b = rbq.qat_backward_ckpt(t_planes(p), st, *rbq.qat_checkpoint(x_in, stream=side), dYt, stream=side)
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, eager[0]))
    assert all(torch.equal(u, v) for u, v in zip(b, eager[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(x_in)
    for rep in range(6):
        x_in.copy_(t_f16(Xs[rep % 3]))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(captured, eager[rep % 3]))
        assert all(torch.equal(u, v) for u, v in zip(step(t_f16(Xs[1])), eager[1]))


def test_workspace_and_refusals():
    out, inf, K, M = 4096, 1024, 2, 16
    planes, s, X, dY = case(out, inf, K, 0, M, 81)
    codes, cs = rbq.qat_checkpoint(t_f16(X))
    a = (t_planes(planes), t_f16(s), codes, cs, t_f16(dY))
    full = rbq.qat_backward_ckpt(*a)
    less = rbq.qat_backward_ckpt(*a, workspace=torch.empty(0, dtype=torch.uint8, device=dev()))
    torch.cuda.synchronize()
    x = f8.restore(*f8.checkpoint(X))
    check_grads(full, planes, s, x, dY, 0)
    check_grads(less, planes, s, x, dY, 0)
    with pytest.raises(ValueError):
        rbq.qat_backward_ckpt(*a[:4], a[4][:8].contiguous())
    with pytest.raises(ValueError):
        rbq.qat_backward_ckpt(*a[:3], cs[:, :4].contiguous(), a[4])
    with pytest.raises(TypeError):
        rbq.qat_backward_ckpt(*a[:2], codes.view(torch.uint8), *a[3:])
    with pytest.raises(ValueError):
        rbq.qat_checkpoint(t_f16(X).t())
    with pytest.raises(rbq.RbqError):
        rbq.qat_checkpoint(torch.empty(4, 40, dtype=torch.float16, device=dev()))
