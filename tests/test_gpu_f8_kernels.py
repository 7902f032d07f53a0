"""Every kernel that rbq_gemm_f8 and rbq_gemv_f8 can choose, at ragged sizes,
within the bounds of test_gpu_f8.py in their tight form (the cut of the 8-bit
matrix instruction by the largest product of each 8 columns, not by the sum of
all), and non-finite codes and scales on each.  test_f8_plans_cpu.py checks
that the sizes here and in the other tests reach every kernel."""
import numpy as np
import pytest
import torch

import gemm_rbq_encode_amd as rbq
import workloads
from oracle import f8
from test_gpu_f8 import dev, layer, t_f16, t_f32, t_f8, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def definition(w8, ws, x8, xs, cut):
    """(y, sum of magnitudes, sum over each 8 columns of the largest product, if `cut`) in 64 bits on the device."""
    (out, inf), M = w8.shape, x8.shape[0]
    cols = torch.arange(inf, device=dev()) // 128
    w = w8.double() * ws.double()[torch.arange(out, device=dev()) // 128][:, cols]
    x = x8.double() * xs.double().t()[:, cols]
    y = x @ w.t().contiguous()
    wa, xa = w.abs(), x.abs()
    S = xa @ wa.t().contiguous()
    total = torch.zeros_like(y) if cut else 0.0
    if cut:
        wt, xt = wa.t().contiguous(), xa.t().contiguous()
        top, one = torch.empty_like(y), torch.empty_like(y)
        for c in range(0, inf, 8):
            top.zero_()
            for j in range(c, c + 8):
                torch.maximum(top, torch.outer(xt[j], wt[j], out=one), out=top)
            total += top
    return y, S, total


def bound(S, y, inf, half, cut):
    """The tolerance of test_gpu_f8.py on device tensors."""
    t = (inf + 3 * (-(-inf // 128)) + 16) * 2.0 ** -23 * S + 7 * 2.0 ** -13 * cut
    return 2.0 ** -11 * (y.abs() + t) + 2.0 ** -25 + t if half else t


# (out, in, tokens, fp32 outputs)
TILES = [(8191, 288, 2047, 0), (8190, 672, 2047, 0), (7001, 288, 2041, 0), (7168, 672, 2041, 0), (6139, 672, 2001, 0),
         (6144, 416, 2000, 0), (28067, 288, 259, 0), (35631, 288, 35, 0),
         (18455, 288, 139, 0), (5003, 4128, 777, 0), (2693, 8352, 133, 0), (32949, 4896, 141, 0),
         (17617, 320, 35, 0), (3103, 2144, 33, 0), (33529, 1760, 43, 0), (11008, 4096, 300, 0),
         (1001, 672, 301, 0), (16479, 7104, 75, 0), (3, 1504, 33, 0),
         (8937, 2848, 129, 1), (34293, 672, 139, 1), (17951, 320, 131, 1), (2851, 2208, 33, 1), (33157, 672, 39, 1),
         (19935, 288, 33, 1), (16681, 4064, 67, 1), (3, 960, 35, 1), (1001, 672, 301, 1)]
FEW = [(12301, 160, 5, 0), (12301, 160, 5, 1), (12299, 416, 27, 0), (12299, 416, 27, 1), (500, 672, 16, 1),
       (500, 672, 17, 0)]


@pytest.mark.parametrize("out,inf,M,f32", TILES + FEW)
def test_gemm_kernels(out, inf, M, f32):
    a = layer(out, inf, M, out + M + inf)
    a = (t_f8(a[0]), t_f32(a[1]), t_f8(a[2]), t_f32(a[3]))
    kind = torch.float32 if f32 else torch.float16
    buf = torch.full((M * out + 4096,), float("nan"), dtype=kind, device=dev())
    Y = buf[:M * out].view(M, out)
    rbq.gemm_f8(*a, dtype=kind, Y=Y)
    again = rbq.gemm_f8(*a, dtype=kind)
    none = rbq.gemm_f8(*a, dtype=kind, workspace=torch.empty(0, dtype=torch.uint8, device=dev()))
    torch.cuda.synchronize()
    assert torch.equal(Y, again) and bool(torch.isnan(buf[M * out:]).all())
    y, S, cut = definition(*a, not f32 and M > 32)
    t = bound(S, y, inf, not f32, cut)
    for got in (Y, none):
        e = (got.double() - y).abs() / t
        assert bool((e <= 1).all()), f"{e.max():.3f} of the bound"


# (out, in): one, two and four blocks of columns in flight for each wave
@pytest.mark.parametrize("out,inf", [(300, 1024), (300, 1056), (41, 2048), (41, 2080), (1, 1120)])
def test_gemv_kernels(out, inf):
    w8, ws, _, _ = layer(out, inf, 1, out + inf)
    X = workloads.gaussian_activations(1, inf, 3)
    c, s = f8.quantize(X)
    y_ref, S = f8.gemm(w8, ws, c, s)
    y = rbq.gemv_f8(t_f8(w8), t_f32(ws), t_f16(X[0]))
    tol = tolerance(S, y_ref, inf, True)[0]
    assert (np.abs(y.cpu().numpy().astype(np.float64) - y_ref[0]) <= tol).all()


NON_FINITE = [(8191, 672, 2047, 0), (8191, 288, 2047, 0), (7001, 672, 2041, 0), (7001, 288, 2041, 0),
              (6139, 672, 2001, 0), (5003, 672, 777, 0), (3001, 672, 1100, 0), (1001, 672, 301, 0), (3103, 2144, 77, 0),
              (11008, 4096, 300, 0), (5003, 672, 777, 1), (3003, 1056, 777, 1), (1001, 672, 301, 1), (1001, 672, 20, 0),
              (1001, 672, 20, 1), (12301, 416, 27, 0), (1001, 288, 9, 0)]


@pytest.mark.parametrize("out,inf,M,f32", NON_FINITE)
def test_non_finite_codes_and_scales_reach_their_outputs_only(out, inf, M, f32):
    """NaN codes and NaN and infinite scales in the first, the last whole and
    the short last block: exactly the outputs that read them are non-finite,
    the others within their bounds."""
    w8, ws, x8, xs = layer(out, inf, M, out + M)
    full, T, R = inf // 128, -(-inf // 128), -(-out // 128)
    clean = [v.copy() for v in (w8, ws, x8, xs)]
    want = np.zeros((M, out), bool)
    for m, c in ((1, 5), (M // 2, 128 * full - 3), (M - 1, inf - 1)):      # NaN codes of tokens
        x8[m, c], clean[2][m, c] = 0x7F if m == 1 else 0xFF, 0
        want[m] = True
    for m, t, v in ((M // 3, full - 1, np.nan), (M // 4, 0, np.inf), (M // 5 + 2, T - 1, np.nan)):
        xs[t, m], clean[3][t, m] = v, 1.0
        want[m] = True
    for r, c in ((7, inf - 1), (95, 0), (111, 130), (127, 128 * full - 1), (223, inf - 2), (out - 1, 128)):
        w8[r, c], clean[0][r, c] = 0x7F, 0
        want[:, r] = True
    for b, t, v in ((2, 0, np.inf), (R // 2, full - 1, np.nan), (R - 2, T - 1, -np.inf)):
        ws[b, t], clean[1][b, t] = v, 1.0
        want[:, 128 * b:128 * b + 128] = True
    kind = torch.float32 if f32 else torch.float16
    Y = rbq.gemm_f8(t_f8(w8), t_f32(ws), t_f8(x8), t_f32(xs), dtype=kind)
    torch.cuda.synchronize()
    want = torch.from_numpy(want).to(dev())
    assert torch.equal(~torch.isfinite(Y), want)
    assert 0.05 < float(want.double().mean()) < 0.95
    y, S, cut = definition(t_f8(clean[0]), t_f32(clean[1]), t_f8(clean[2]), t_f32(clean[3]), not f32 and M > 32)
    t = bound(S, y, inf, not f32, cut)
    assert bool((((Y.double() - y).abs() <= t) | want).all())
